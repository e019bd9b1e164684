// The layer for the few tokens of a decoding step with experts in 4 bits, forward
// only (moe_mx4_decode in moe.h):
//   y_n = sum_k gates[n,k] FFN_{e_nk}(x_n) (+ FFN_s(x_n)).
//
// Reading the chosen experts' codes once is what bounds it (17 bytes for 32
// weights), so:
//  - A strip of 16 columns of a matrix is one contiguous piece of memory in the
//    order in which a wave takes it: a 16-byte load a lane is a tile of 128 rows,
//    lane (g, c) holding the 32 values from 32g on of column c.  A strip can be as
//    narrow as that without reading less than whole lines, so work is dealt to
//    workgroups in strips and not in parts of the contraction, and no partial sums
//    travel through memory between workgroups.
//  - The four waves of a workgroup (sixteen where one token leaves few strips)
//    split the contraction; their float32 sums meet in LDS in wave order.
//  - Eight values of a lane are one operand of a 16x16x32 bf16 matrix instruction:
//    four conversions give them exactly, scale included.  The other operand is 16
//    token rows, packed so that a load of it is contiguous over the lanes.
//  - float32 rows enter as the exact sum of three bf16 operands, activations of
//    bfloat16 layers as the sum of two.
// Weights are the row operand, so that a lane ends with four neighbouring columns
// of one token.
#include <algorithm>
#include <cmath>

#include "decode_rows.h"
#include "mx4.h"

namespace {
using namespace moe;

// Eight float32 values as the sum of P bf16 operands.  P = 3: their bits cut in
// three, exact.  P = 2: the nearest bf16 and the rest, rounded: 2^-16 of the value
// at most.  P = 1: they are bf16.  An infinite or NaN value is all in the first.
template <int P>
__device__ __forceinline__ void split(const float* v, words4_t (&out)[P]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (P == 1) {
      out[0][j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
    } else {
      uint32_t hi[2], lo[2], mid[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float f = v[2 * j + i];
        hi[i] = __float_as_uint(f) & 0xffff0000u;
        if (P == 2) {
          const uint32_t near = uint32_t(f32_to_bf16(f)) << 16;
          hi[i] = (near & 0x7f800000u) == 0x7f800000u ? hi[i] : near;  // not to infinity
        }
        const float r = isfinite(f) ? f - __uint_as_float(hi[i]) : 0.f;
        mid[i] = __float_as_uint(r);
        lo[i] = __float_as_uint(r - __uint_as_float(mid[i] & 0xffff0000u));
        if (f != f) hi[i] = 0x7fc00000u;
      }
      constexpr uint32_t upper = 0x07060302u;
      out[0][j] = __builtin_amdgcn_perm(hi[1], hi[0], upper);
      if constexpr (P == 2) {
        out[1][j] = pack_bf16x2(__uint_as_float(mid[0]), __uint_as_float(mid[1]));
      } else {
        out[1][j] = __builtin_amdgcn_perm(mid[1], mid[0], upper);
        out[2][j] = __builtin_amdgcn_perm(lo[1], lo[0], upper);
      }
    }
  }
}

// Where rows as operands lie: planes of [L/32 operands][rows][32 values].  Operand
// 4*kt + j of a row has, for g = 0..3, the values 128kt + 32g + 8j .. + 7: what lane
// group g multiplies with word j of its codes of tile kt.  The first of the eight
// values from l on (l a multiple of 4: four of them):
__device__ __forceinline__ int64_t operand_at(int64_t l, int64_t row, int64_t rows) {
  return ((l / 128 * 4 + l % 32 / 8) * rows + row) * 32 + l % 128 / 32 * 8 + l % 8;
}

// k_decode_logits: x as operands.
template <typename T, int P> struct PackOperands {
  bf16_t* xp;
  __device__ __forceinline__ void operator()(const T* from, int n, int h, int N, int H) const {
    float v[8];
    Vec16<T>::load(from, v);
    if (Vec16<T>::n == 4) Vec16<T>::load(from + 4, v + 4);
    words4_t o[P];
    split<P>(v, o);
#pragma unroll
    for (int p = 0; p < P; ++p)
      *reinterpret_cast<words4_t*>(xp + int64_t(p) * N * H + operand_at(h, n, N)) = o[p];
  }
};

// A lane's eight values of word `w` of codes.
__device__ __forceinline__ bf16x8_t values(uint32_t w, float scale) {
  words4_t b;
  b[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
  b[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
  b[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
  b[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  return __builtin_bit_cast(bf16x8_t, b);
}

// U tiles in a row of NM * CG strips (CG neighbours of NM matrices), and the rows
// that they are multiplied with.
struct Item {
  const words4_t* code[2];  // the lane's, of tile 0 of the first strip
  const uint32_t* scale[2];
  const bf16_t* x;  // first plane of operand 0
  int64_t plane;
  int64_t rows;  // in an operand
  int tiles, kt;  // of the strip; the first
};

// acc[m][matrix * CG + strip] += rows . strip for this item, 16*MT rows: row
// 16m + c of the operand is row at[m].
template <int MT, int NM, int CG, int U, int P>
__device__ __forceinline__ void multiply(const Item& t, const int (&at)[MT], f32x4_t (&acc)[MT][NM * CG]) {
  const int g = lane_id() / 16, groups = (t.tiles + 3) / 4;
  words4_t w[U][NM * CG], a[U][MT][4][P];
  uint32_t s[NM * CG];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int kt = min(t.kt + u, t.tiles - 1);
#pragma unroll
    for (int i = 0; i < NM * CG; ++i)
      w[u][i] = __builtin_nontemporal_load(t.code[i / CG] + (int64_t(i % CG) * t.tiles + kt) * kWave);
  }
#pragma unroll
  for (int i = 0; i < NM * CG; ++i) s[i] = t.scale[i / CG][(int64_t(i % CG) * groups + t.kt / 4) * kWave];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int kt = min(t.kt + u, t.tiles - 1);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int p = 0; p < P; ++p)
          a[u][m][j][p] = *reinterpret_cast<const words4_t*>(
              t.x + p * t.plane + (int64_t(4 * kt + j) * t.rows + at[m]) * 32 + 8 * g);
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (t.kt + u >= t.tiles) break;
    const int shift = (t.kt + u) % 4 * 8;
#pragma unroll
    for (int i = 0; i < NM * CG; ++i) {
      const uint32_t byte = s[i] >> shift & 255u;
      const float scale = __uint_as_float(byte == 255u ? 0x7fc00000u : byte << 23);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bf16x8_t b = values(w[u][i][j], scale);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int p = P - 1; p >= 0; --p)  // the smallest first
            acc[m][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                b, __builtin_bit_cast(bf16x8_t, a[u][m][j][p]), acc[m][i], 0, 0, 0);
      }
    }
  }
}

template <int MT, int NS>
__device__ __forceinline__ void clear(f32x4_t (&acc)[MT][NS]) {
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < NS; ++i) acc[m][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
}

// The waves' sums added in wave order; out(row tile, strip, lane, sums) with the
// lane's four columns 4g + r of the strip and row c, for NM matrices at a time
// (sums[matrix]).  red: NW * NS * 64 vectors.
template <int MT, int NM, int CG, int NW, typename F>
__device__ __forceinline__ void join(const f32x4_t (&acc)[MT][NM * CG], f32x4_t* red, F out) {
  constexpr int NS = NM * CG;
  const int wave = threadIdx.x / kWave;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (m > 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < NS; ++i) red[(wave * NS + i) * kWave + lane_id()] = acc[m][i];
    __syncthreads();
    for (int t = threadIdx.x; t < CG * kWave; t += NW * kWave) {
      f32x4_t v[NM];
#pragma unroll
      for (int n = 0; n < NM; ++n) {
        v[n] = red[n * CG * kWave + t];
#pragma unroll
        for (int w = 1; w < NW; ++w) v[n] += red[(w * NS + n * CG) * kWave + t];
      }
      out(m, t / kWave, t % kWave, v);
    }
  }
}

// What the kernels share.
struct Shape {
  int N, H, F, Fs, E, K, units;
};

// Weights of one form: codes and scales of all experts.
struct View {
  const words4_t* codes;
  const uint32_t* scales;
  __device__ __forceinline__ const words4_t* code(int64_t strip, int k) const {
    return codes + mx_strip_codes(strip, k) + lane_id();
  }
  __device__ __forceinline__ const uint32_t* scale(int64_t strip, int k) const {
    return scales + mx_strip_scales(strip, k) + lane_id();
  }
};

// gate * silu(G) * U of four columns.  The hardware's reciprocal is good to 1 ulp;
// below 2^-126 it gives 0, an activation of less than 1e-36 of the up product.
__device__ __forceinline__ void activate(const f32x4_t& g, const f32x4_t& u, float gate, float* v) {
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] = gate * (g[r] * __builtin_amdgcn_rcpf(1.0f + expf(-g[r])) * u[r]);
}

// Tiles under way at once.
template <int NS, int MT, int P>
constexpr int kUnroll = NS * 2 > 8 || MT * P > 2 ? 1 : NS * 4 > 8 || MT * P > 1 ? 2 : 4;

// Activations of CG strips of one expert's gate and up for the rows `rows` (row r:
// token rows[r] / div), as operands.
template <int MT, int CG, int PX, int PA>
__device__ __forceinline__ void gate_up_rows(const bf16_t* xp, int N, int H, const View& wg, const View& wu,
                                             int64_t strip, int64_t col0, int64_t F, const int* rows, int M, int div,
                                             const float* gates, bf16_t* act, int64_t R, f32x4_t* red) {
  constexpr int U = kUnroll<2 * CG, MT, PX>;
  const int c = lane_id() % 16, wave = threadIdx.x / kWave;
  f32x4_t acc[MT][2 * CG];
  clear(acc);
  int at[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) at[m] = rows[16 * m + c < M ? 16 * m + c : 0] / div;
  Item t{{wg.code(strip, H), wu.code(strip, H)}, {wg.scale(strip, H), wu.scale(strip, H)}, xp, int64_t(N) * H, N,
         H / kMxTile, 0};
  for (t.kt = wave * U; t.kt < t.tiles; t.kt += kWaves * U) multiply<MT, 2, CG, U, PX>(t, at, acc);
  join<MT, 2, CG, kWaves>(acc, red, [&](int m, int s, int lane, const f32x4_t* v) {
    const int r = 16 * m + lane % 16;
    if (r >= M) return;
    float f[8];
    activate(v[0], v[1], gates != nullptr ? gates[rows[r]] : 1.f, f);
#pragma unroll
    for (int i = 4; i < 8; ++i) f[i] = 0.f;
    words4_t o[PA];
    split<PA>(f, o);
    bf16_t* to = act + operand_at(col0 + 16 * s + 4 * (lane / 16), rows[r], R);
#pragma unroll
    for (int p = 0; p < PA; ++p) *reinterpret_cast<uint2*>(to + p * R * F) = make_uint2(o[p][0], o[p][1]);
  });
}

template <int MTMAX, int CG, int PX, int PA>
__global__ __launch_bounds__(kNT) void k_mx4_gate_up(const bf16_t* __restrict__ xp, View wg, View wu, View swg,
                                                     View swu, const int32_t* __restrict__ topk,
                                                     const float* __restrict__ gates, bf16_t* __restrict__ act,
                                                     bf16_t* __restrict__ sact, Shape q) {
  __shared__ Chosen chosen;
  __shared__ int rows[kTok];
  __shared__ f32x4_t red[kWaves * 2 * CG * kWave];
  const int chunks = q.F / (16 * CG), shared = q.Fs / (16 * CG);
  int b = int(blockIdx.x) - shared, e = 0, M = q.N;
  const bool routed = b >= 0;
  const int64_t F = routed ? q.F : q.Fs;
  int64_t col0;
  if (routed) {
    M = unit_rows(topk, q.N, q.K, b / chunks, &chosen, &e, rows);
    if (M == 0) return;
    col0 = int64_t(b % chunks) * 16 * CG;
  } else {
    if (threadIdx.x < kTok) rows[threadIdx.x] = threadIdx.x;
    __syncthreads();
    col0 = int64_t(b + shared) * 16 * CG;
  }
  const int64_t strip = e * (F / 16) + col0 / 16;
  auto run = [&](auto mt) {
    gate_up_rows<decltype(mt)::value, CG, PX, PA>(xp, q.N, q.H, routed ? wg : swg, routed ? wu : swu, strip, col0, F,
                                                  rows, M, routed ? q.K : 1, routed ? gates : nullptr,
                                                  routed ? act : sact, routed ? int64_t(q.N) * q.K : q.N, red);
  };
  if constexpr (MTMAX > 2)
    if (M > 32) return run(std::integral_constant<int, 4>());
  if constexpr (MTMAX > 1)
    if (M > 16) return run(std::integral_constant<int, 2>());
  run(std::integral_constant<int, 1>());
}

// CG strips of one expert's down product: sums to out[rows[r]][H].
template <int MT, int CG, int PA>
__device__ __forceinline__ void down_rows(const bf16_t* act, int64_t R, int F, const View& wd, int64_t strip,
                                          int64_t col0, int64_t H, const int* rows, int M, float* out, f32x4_t* red) {
  constexpr int U = kUnroll<CG, MT, PA>;
  const int c = lane_id() % 16, wave = threadIdx.x / kWave;
  f32x4_t acc[MT][CG];
  clear(acc);
  int at[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) at[m] = rows[16 * m + c < M ? 16 * m + c : 0];
  Item t{{wd.code(strip, F), nullptr}, {wd.scale(strip, F), nullptr}, act, R * F, R, F / kMxTile, 0};
  for (t.kt = wave * U; t.kt < t.tiles; t.kt += kWaves * U) multiply<MT, 1, CG, U, PA>(t, at, acc);
  join<MT, 1, CG, kWaves>(acc, red, [&](int m, int s, int lane, const f32x4_t* v) {
    const int r = 16 * m + lane % 16;
    if (r < M) *reinterpret_cast<f32x4_t*>(out + rows[r] * H + col0 + 16 * s + 4 * (lane / 16)) = v[0];
  });
}

// More than one token: ys [slot][H], then sys [token][H] of the shared expert.
template <int MTMAX, int CG, int PA>
__global__ __launch_bounds__(kNT) void k_mx4_down(const bf16_t* __restrict__ act, const bf16_t* __restrict__ sact,
                                                  View wd, View swd, const int32_t* __restrict__ topk,
                                                  float* __restrict__ ys, float* __restrict__ sys, Shape q) {
  __shared__ Chosen chosen;
  __shared__ int rows[kTok];
  __shared__ f32x4_t red[kWaves * CG * kWave];
  const int chunks = q.H / (16 * CG), shared = q.Fs > 0 ? chunks : 0;
  int b = int(blockIdx.x) - shared, e = 0, M = q.N;
  const bool routed = b >= 0;
  if (routed) {
    M = unit_rows(topk, q.N, q.K, b / chunks, &chosen, &e, rows);
    if (M == 0) return;
  } else {
    b += shared;
    if (threadIdx.x < kTok) rows[threadIdx.x] = threadIdx.x;
    __syncthreads();
  }
  const int64_t col0 = int64_t(b % chunks) * 16 * CG, strip = e * int64_t(q.H / 16) + col0 / 16;
  auto run = [&](auto mt) {
    down_rows<decltype(mt)::value, CG, PA>(routed ? act : sact, routed ? int64_t(q.N) * q.K : q.N,
                                           routed ? q.F : q.Fs, routed ? wd : swd, strip, col0, q.H, rows, M,
                                           routed ? ys : sys, red);
  };
  if constexpr (MTMAX > 2)
    if (M > 32) return run(std::integral_constant<int, 4>());
  if constexpr (MTMAX > 1)
    if (M > 16) return run(std::integral_constant<int, 2>());
  run(std::integral_constant<int, 1>());
}

// One token: the sum over its experts and the shared one is part of the
// contraction, dealt to sixteen waves, and y leaves rounded.
constexpr int kOneWaves = 16;
template <typename T, int CG, int PA>
__global__ __launch_bounds__(kOneWaves* kWave) void k_mx4_down_one(const bf16_t* __restrict__ act,
                                                                   const bf16_t* __restrict__ sact, View wd, View swd,
                                                                   const int32_t* __restrict__ topk,
                                                                   T* __restrict__ y, Shape q) {
  constexpr int U = kUnroll<CG, 1, PA>;
  __shared__ f32x4_t red[kOneWaves * CG * kWave];
  const int wave = threadIdx.x / kWave;
  const int64_t col0 = int64_t(blockIdx.x) * 16 * CG;
  f32x4_t acc[1][CG];
  clear(acc);
  const int per = (q.F / kMxTile + U - 1) / U, routed = q.K * per, all = routed + (q.Fs / kMxTile + U - 1) / U;
  for (int i = wave; i < all; i += kOneWaves) {
    const bool sh = i >= routed;
    const int k = sh ? 0 : i / per, F = sh ? q.Fs : q.F;
    const int64_t strip = (sh ? 0 : int64_t(topk[k]) * (q.H / 16)) + col0 / 16;
    const View& w = sh ? swd : wd;
    const int at[1] = {k};
    multiply<1, 1, CG, U, PA>(Item{{w.code(strip, F), nullptr}, {w.scale(strip, F), nullptr}, sh ? sact : act,
                                   int64_t(sh ? 1 : q.K) * F, sh ? 1 : q.K, F / kMxTile, (sh ? i - routed : i % per) * U},
                              at, acc);
  }
  join<1, 1, CG, kOneWaves>(acc, red, [&](int, int s, int lane, const f32x4_t* v) {
    if (lane % 16 != 0) return;
    T* to = y + col0 + 16 * s + 4 * (lane / 16);
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<f32x4_t*>(to) = v[0];
    else
      *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(v[0][0], v[0][1]), pack_bf16x2(v[0][2], v[0][3]));
  });
}

// ------------------------------------------------------------------- host

struct Plan {
  Shape q;
  int logit_parts;
  int gu_cg, dn_cg;  // strips of a workgroup
  size_t logits, xp, act, sact, ys, sys, bytes;
};

// Strips of a workgroup, of `strips` in all: with more of them the rows are read
// less often for the same weights, with fewer there are more workgroups.
int strips_of(double rows, int64_t strips) {
  int cg = rows > 6.0 ? 4 : rows > 2.0 ? 2 : 1;
  while (cg > 1 && strips / cg < 512) cg /= 2;
  return cg;
}

Plan plan(const moe_launch::Dims& d, int64_t Fs) {
  Plan p;
  p.q = Shape{int(d.N), int(d.H), int(d.F), int(Fs), int(d.E), int(d.K), int(std::min(d.NK(), d.E))};
  const bool bf = d.dtype == MOE_BF16;
  const int64_t NK = d.NK(), px = bf ? 1 : 3, pa = bf ? 2 : 3;
  const double used = double(d.E) * (1.0 - std::pow(1.0 - double(d.K) / double(d.E), double(d.N)));
  const double rows = double(NK) / used;
  p.logit_parts = int((d.H + kLogitRows - 1) / kLogitRows);
  p.gu_cg = strips_of(rows, int64_t(used) * (d.F / 16));
  p.dn_cg = strips_of(rows, int64_t(used) * (d.H / 16));
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += (n + 255) & ~size_t(255);
    return here;
  };
  p.logits = take(size_t(p.logit_parts) * d.N * d.E * sizeof(double));
  p.xp = take(size_t(px) * d.N * d.H * 2);
  p.act = take(size_t(pa) * NK * d.F * 2);
  p.sact = take(size_t(pa) * d.N * Fs * 2);
  p.ys = take(d.N == 1 ? 0 : size_t(NK) * d.H * 4);
  p.sys = take(d.N == 1 || Fs == 0 ? 0 : size_t(d.N) * d.H * 4);
  p.bytes = at;
  return p;
}

#define MOE_LAUNCHED()                 \
  {                                    \
    const hipError_t e = hipGetLastError(); \
    if (e != hipSuccess) return e;     \
  }

struct Args {
  View wg, wu, wd, swg, swu, swd;
  int32_t* topk;
  float* gates;
  char* ws;
};

template <typename T, int MTMAX, int CG>
hipError_t gate_up(const Plan& p, const Args& a, hipStream_t s) {
  constexpr int PX = sizeof(T) == 2 ? 1 : 3, PA = sizeof(T) == 2 ? 2 : 3;
  const Shape& q = p.q;
  const unsigned grid = unsigned(q.units) * (q.F / (16 * CG)) + q.Fs / (16 * CG);
  k_mx4_gate_up<MTMAX, CG, PX, PA><<<dim3(grid), dim3(kNT), 0, s>>>(
      reinterpret_cast<const bf16_t*>(a.ws + p.xp), a.wg, a.wu, a.swg, a.swu, a.topk, a.gates,
      reinterpret_cast<bf16_t*>(a.ws + p.act), reinterpret_cast<bf16_t*>(a.ws + p.sact), q);
  return hipGetLastError();
}

template <typename T, int MTMAX, int CG>
hipError_t down(const Plan& p, const Args& a, T* y, hipStream_t s) {
  constexpr int PA = sizeof(T) == 2 ? 2 : 3;
  const Shape& q = p.q;
  const bf16_t* act = reinterpret_cast<const bf16_t*>(a.ws + p.act);
  const bf16_t* sact = reinterpret_cast<const bf16_t*>(a.ws + p.sact);
  if (q.N == 1) {
    if constexpr (MTMAX == 1)
      k_mx4_down_one<T, CG, PA><<<dim3(q.H / (16 * CG)), dim3(kOneWaves * kWave), 0, s>>>(act, sact, a.wd, a.swd,
                                                                                         a.topk, y, q);
    return hipGetLastError();
  }
  float* ys = reinterpret_cast<float*>(a.ws + p.ys);
  float* sys = reinterpret_cast<float*>(a.ws + p.sys);
  const unsigned chunks = q.H / (16 * CG);
  k_mx4_down<MTMAX, CG, PA><<<dim3((q.units + (q.Fs > 0 ? 1 : 0)) * chunks), dim3(kNT), 0, s>>>(
      act, sact, a.wd, a.swd, a.topk, ys, sys, q);
  MOE_LAUNCHED()
  k_decode_combine<T><<<dim3(q.H / 64, q.N), dim3(256), 0, s>>>(ys, sys, y, q.N, q.H, q.K, 1, q.Fs > 0 ? 1 : 0);
  return hipGetLastError();
}

template <typename T, int MTMAX>
hipError_t experts(const Plan& p, const Args& a, T* y, hipStream_t s) {
  const hipError_t e = p.gu_cg == 4   ? gate_up<T, MTMAX, 4>(p, a, s)
                       : p.gu_cg == 2 ? gate_up<T, MTMAX, 2>(p, a, s)
                                      : gate_up<T, MTMAX, 1>(p, a, s);
  if (e != hipSuccess) return e;
  return p.dn_cg == 4   ? down<T, MTMAX, 4>(p, a, y, s)
         : p.dn_cg == 2 ? down<T, MTMAX, 2>(p, a, y, s)
                        : down<T, MTMAX, 1>(p, a, y, s);
}

template <typename T>
hipError_t decode_t(const moe_launch::Dims& d, int64_t Fs, const T* x, const T* w_r, const float* bias, const Args& a,
                    T* y, hipStream_t s) {
  constexpr int PX = sizeof(T) == 2 ? 1 : 3;
  const Plan p = plan(d, Fs);
  const Shape& q = p.q;
  double* logits = reinterpret_cast<double*>(a.ws + p.logits);
  k_decode_logits<T><<<dim3(p.logit_parts, (q.E + 15) / 16, (q.N + 15) / 16), dim3(kLogitWaves * kWave), 0, s>>>(
      x, w_r, logits, PackOperands<T, PX>{reinterpret_cast<bf16_t*>(a.ws + p.xp)}, q.N, q.H, q.E);
  MOE_LAUNCHED()
  k_decode_topk<<<dim3(q.N), dim3(256), 0, s>>>(logits, bias, a.topk, a.gates, q.N, q.E, q.K, p.logit_parts);
  MOE_LAUNCHED()
  if (q.N <= 16) return experts<T, 1>(p, a, y, s);
  if (q.N <= 32) return experts<T, 2>(p, a, y, s);
  return experts<T, 4>(p, a, y, s);
}

View view(const moe_launch::Mx4& q) {
  return View{static_cast<const words4_t*>(q.codes), static_cast<const uint32_t*>(q.scales)};
}

}  // namespace

namespace moe_launch {

size_t mx4_decode_ws(const Dims& d, int64_t Fs) { return plan(d, Fs).bytes; }

hipError_t mx4_decode(const Dims& d, const void* x, const void* w_r, const float* bias, const Mx4& wg, const Mx4& wu,
                      const Mx4& wd, int64_t Fs, const Mx4& swg, const Mx4& swu, const Mx4& swd, int32_t* topk,
                      float* gates, void* y, void* ws, hipStream_t s) {
  const Args a{view(wg), view(wu), view(wd), view(swg), view(swu), view(swd), topk, gates, static_cast<char*>(ws)};
  return d.dtype == MOE_BF16
             ? decode_t(d, Fs, static_cast<const bf16_t*>(x), static_cast<const bf16_t*>(w_r), bias, a,
                        static_cast<bf16_t*>(y), s)
             : decode_t(d, Fs, static_cast<const float*>(x), static_cast<const float*>(w_r), bias, a,
                        static_cast<float*>(y), s);
}

}  // namespace moe_launch
