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
//    workgroups in strips, and in parts of the contraction, whose sums travel through
//    memory, only for long down products of few experts.
//  - The four waves of a workgroup (sixteen where one token leaves few strips)
//    split the contraction; their float32 sums meet in LDS in wave order.
//  - Eight values of a lane are one operand of a 16x16x32 bf16 matrix instruction:
//    four conversions give them exactly, scale included.  The other operand is 16
//    token rows, packed so that a load of it is contiguous over the lanes.
//  - float32 rows, and the activations of either type, enter as the exact sum of
//    three bf16 operands.
// Weights are the row operand, so that a lane ends with four neighbouring columns
// of one token.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "decode_rows.h"
#include "mx4.h"

namespace {
using namespace moe;

// Eight float32 values as the sum of P bf16 operands.  P = 3: their bits cut in
// three, exact.  P = 1: they are bf16.  An infinite or NaN value is all in the first.
template <int P>
__device__ __forceinline__ void split(const float* v, words4_t (&out)[P]) {
  static_assert(P == 1 || P == 3, "exact");
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
        const float r = isfinite(f) ? f - __uint_as_float(hi[i]) : 0.f;
        mid[i] = __float_as_uint(r);
        lo[i] = __float_as_uint(r - __uint_as_float(mid[i] & 0xffff0000u));
        if (f != f) hi[i] = 0x7fc00000u;
      }
      constexpr uint32_t upper = 0x07060302u;
      out[0][j] = __builtin_amdgcn_perm(hi[1], hi[0], upper);
      out[1][j] = __builtin_amdgcn_perm(mid[1], mid[0], upper);
      out[2][j] = __builtin_amdgcn_perm(lo[1], lo[0], upper);
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

// Operands of an activation: all 24 bits of it, whatever the layer's type.
constexpr int kActParts = 3;

// Rows as operands: the eight values of operand 4*kt + j that lane (g, c) takes of row
// r start at p[kt * tile + j * word + r * row + g * group], plane by plane.
struct Operands {
  const bf16_t* p;
  int64_t plane, tile;
  int word, row, group;
};
// As PackOperands and the activations lie, R rows of L values.
__device__ __forceinline__ Operands packed(const bf16_t* p, int64_t R, int64_t L) {
  return Operands{p, R * L, R * kMxTile, int(R) * 32, 32, 8};
}
// bf16 rows as they are, [rows][L].
__device__ __forceinline__ Operands in_place(const bf16_t* p, int L) { return Operands{p, 0, kMxTile, 8, L, 32}; }

// CG neighbouring strips of each of NM matrices: their first words.  Addresses that
// are the same in all of a wave stay in scalar registers, with a lane's 32-bit offset
// beside them; with 64-bit ones for each lane the largest variants spill.
struct Strips {
  const words4_t* code[2];
  const uint32_t* scale[2];
  int tiles;
};

// What is the same in all lanes, as the compiler can know.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int wave_id() { return uniform(threadIdx.x / kWave); }

template <typename V>
__device__ __forceinline__ const V* at_lane(const V* p, uint32_t bytes) {
  return reinterpret_cast<const V*>(reinterpret_cast<const char*>(p) + bytes);
}

// acc[m][matrix * CG + strip] += rows . strip for U tiles from kt on, 16*MT rows: row
// 16m + c is row at[m].  All weights are asked for before the first product, the row
// operands AHEAD steps before theirs (a step is an operand, 8 of a lane's 32 values):
// the order is fixed, as the compiler left to itself asks for all of them at once and
// spills.
template <int MT, int NM, int CG, int U, int P>
__device__ __forceinline__ void multiply(const Strips& t, const Operands& x, int kt0, const int (&at)[MT],
                                         f32x4_t (&acc)[MT][NM * CG]) {
  constexpr int NS = NM * CG, AHEAD = MT * P == 1 ? 4 : MT * P == 2 ? 3 : MT * P <= 4 ? 2 : 1;
  const int g = lane_id() / 16, groups = (t.tiles + 3) / 4;
  words4_t w[U][NS], a[AHEAD + 1][MT][P];
  uint32_t s[NS];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (kt0 + u < t.tiles) {
#pragma unroll
      for (int i = 0; i < NS; ++i)
        w[u][i] = __builtin_nontemporal_load(
            at_lane(t.code[i / CG] + (int64_t(i % CG) * t.tiles + kt0 + u) * kWave, lane_id() * 16));
    }
#pragma unroll
  for (int i = 0; i < NS; ++i)
    s[i] = *at_lane(t.scale[i / CG] + (int64_t(i % CG) * groups + kt0 / 4) * kWave, lane_id() * 4);
  uint32_t px[MT];  // bytes: at most 512 rows of 2^20 values in place
#pragma unroll
  for (int m = 0; m < MT; ++m) px[m] = (uint32_t(at[m]) * uint32_t(x.row) + g * x.group) * 2;
  auto rows = [&](int n) {  // of step n
    const int64_t from = min(kt0 + n / 4, t.tiles - 1) * x.tile + n % 4 * x.word;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int p = 0; p < P; ++p)
        a[n % (AHEAD + 1)][m][p] =
            *reinterpret_cast<const words4_t*>(at_lane(x.p + from + p * x.plane, px[m]));
  };
#pragma unroll
  for (int n = 0; n < AHEAD; ++n) rows(n);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (kt0 + u >= t.tiles) break;
    float scale[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const uint32_t byte = s[i] >> (kt0 + u) % 4 * 8 & 255u;
      scale[i] = __uint_as_float(byte == 255u ? 0x7fc00000u : byte << 23);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = 4 * u + j;
      __builtin_amdgcn_sched_barrier(0);
      if (n + AHEAD < 4 * U) rows(n + AHEAD);
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const bf16x8_t b = values(w[u][i][j], scale[i]);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int p = P - 1; p >= 0; --p)  // the smallest first
            acc[m][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                b, __builtin_bit_cast(bf16x8_t, a[n % (AHEAD + 1)][m][p]), acc[m][i], 0, 0, 0);
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
    __syncthreads();  // what red held is read
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
  int parts;  // of the down contraction
};

// Weights of one form: codes and scales of all experts.
struct View {
  const words4_t* codes;
  const uint32_t* scales;
  __device__ __forceinline__ const words4_t* code(int64_t strip, int k) const {
    return codes + mx_strip_codes(strip, k);
  }
  __device__ __forceinline__ const uint32_t* scale(int64_t strip, int k) const {
    return scales + mx_strip_scales(strip, k);
  }
};

// gate * silu(G) * U of four columns, from exp(-|G|), which does not overflow.
__device__ __forceinline__ void activate(const f32x4_t& g, const f32x4_t& u, float gate, float* v) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float t = expf(-fabsf(g[r]));
    v[r] = gate * ((g[r] < 0.f ? g[r] * t : g[r]) / (1.0f + t) * u[r]);
  }
}

// Tiles a wave has under way: 16 KiB of weights at most, half of it where the rows
// take the registers.
template <int NS, int MT, int P>
constexpr int kUnroll = NS >= 8 ? (MT * P > 3 ? 1 : 2) : NS == 4 && MT > 2 ? 2 : MT * P >= 6 ? 2 : 4;

// The chosen experts, ascending, and their slots n*K + k: units number the experts,
// unit u's slots are slots[start[u] .. start[u+1]).  A workgroup builds it once for
// all its work.
struct Units {
  int16_t slots[kSlots];
  int count[MOE_MAX_EXPERTS], first[MOE_MAX_EXPERTS];
  int expert[MOE_MAX_EXPERTS], start[MOE_MAX_EXPERTS + 1];
  int sums[2][kWaves];
};

// All threads call it; returns the number of units.  Slots of an expert come in any
// order: a row's result does not depend on its place.
__device__ __forceinline__ int find_units(const int32_t* topk, int NK, Units* s) {
  static_assert(kNT == MOE_MAX_EXPERTS && kSlots <= 2 * kNT, "a thread per expert, two slots a thread");
  const int t = threadIdx.x, wave = t / kWave, lane = lane_id();
  s->count[t] = 0;
  __syncthreads();
  int id[2] = {-1, -1}, place[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int i = t + r * kNT;
    if (i < NK) {
      id[r] = topk[i];
      place[r] = atomicAdd(&s->count[id[r]], 1);
    }
  }
  __syncthreads();
  const int mine = s->count[t];
  const uint64_t mask = __ballot(mine > 0);
  int upto = mine;  // inclusive sum over the wave
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const int v = __shfl_up(upto, off, kWave);
    upto += lane >= off ? v : 0;
  }
  if (lane == kWave - 1) {
    s->sums[0][wave] = __popcll(mask);
    s->sums[1][wave] = upto;
  }
  __syncthreads();
  int unit = __popcll(mask & ((uint64_t(1) << lane) - 1)), first = upto - mine, units = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    unit += w < wave ? s->sums[0][w] : 0;
    first += w < wave ? s->sums[1][w] : 0;
    units += s->sums[0][w];
  }
  s->first[t] = first;
  if (mine > 0) {
    s->expert[unit] = t;
    s->start[unit] = first;
  }
  if (t == 0) s->start[units] = NK;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < 2; ++r)
    if (id[r] >= 0) s->slots[s->first[id[r]] + place[r]] = int16_t(t + r * kNT);
  __syncthreads();
  return units;
}

// f(row tiles, first row, rows) for M rows: all at once, or 32 at a time where the
// kernel has the registers of two row tiles only.
template <int MTMAX, typename F>
__device__ __forceinline__ void by_rows(int M, F f) {
  if constexpr (MTMAX == 1) {
    f(std::integral_constant<int, 1>(), 0, M);
  } else {
    if (M <= 16) return f(std::integral_constant<int, 1>(), 0, M);
    if constexpr (MTMAX > 2)
      if (M > 32) return f(std::integral_constant<int, 4>(), 0, M);
    for (int m0 = 0; m0 < M; m0 += 32) f(std::integral_constant<int, 2>(), m0, min(32, M - m0));
  }
}

// Activations of CG strips of one expert's gate and up for the M rows slot(0 ..), as
// operands.
template <int MT, int CG, int PX, typename Slot>
__device__ __forceinline__ void gate_up_rows(const Operands& x, const Strips& w, int64_t col0, int64_t F, Slot slot,
                                             int M, int div, const float* gates, bf16_t* act, int64_t R,
                                             f32x4_t* red) {
  constexpr int U = kUnroll<2 * CG, MT, PX>;
  const int c = lane_id() % 16, wave = wave_id();
  f32x4_t acc[MT][2 * CG];
  clear(acc);
  int at[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) at[m] = slot(16 * m + c < M ? 16 * m + c : 0) / div;
  for (int kt = wave * U; kt < w.tiles; kt += kWaves * U) multiply<MT, 2, CG, U, PX>(w, x, kt, at, acc);
  join<MT, 2, CG, kWaves>(acc, red, [&](int m, int s, int lane, const f32x4_t* v) {
    const int r = 16 * m + lane % 16;
    if (r >= M) return;
    const int row = slot(r);
    float f[8];
    activate(v[0], v[1], gates != nullptr ? gates[row] : 1.f, f);
#pragma unroll
    for (int i = 4; i < 8; ++i) f[i] = 0.f;
    words4_t o[kActParts];
    split<kActParts>(f, o);
    bf16_t* to = act + operand_at(col0 + 16 * s + 4 * (lane / 16), row, R);
#pragma unroll
    for (int p = 0; p < kActParts; ++p) *reinterpret_cast<uint2*>(to + p * R * F) = make_uint2(o[p][0], o[p][1]);
  });
}

// A workgroup takes every gridDim-th piece of CG strips (of both matrices): first the
// shared expert's, then those of the chosen experts.  ROUTE: it finds topk and gates
// itself, and the first one writes them.
template <typename T, int MTMAX, int CG, bool ROUTE>
__global__ __launch_bounds__(kNT, MTMAX > 2 ? 1 : 2) void k_mx4_gate_up(
    Operands x, View wg, View wu, View swg, View swu, int32_t* __restrict__ topk_out, float* __restrict__ gates_out,
    Route<T> route, bf16_t* __restrict__ act, bf16_t* __restrict__ sact, Shape q) {
  constexpr int PX = sizeof(T) == 2 ? 1 : 3;
  __shared__ Units units;
  __shared__ f32x4_t red[kWaves * 2 * CG * kWave];
  const int32_t* topk = topk_out;
  const float* gates = gates_out;
  if constexpr (ROUTE) {
    static_assert(sizeof(red) >= kWaves * 2048, "red holds the logits");
    __shared__ TopK routed;
    route_here(route, q.N, q.H, q.E, q.K, &routed, reinterpret_cast<double*>(red));
    topk = routed.ids;
    gates = routed.gates;
    if (blockIdx.x == 0 && int(threadIdx.x) < q.N * q.K) {
      topk_out[threadIdx.x] = routed.ids[threadIdx.x];
      gates_out[threadIdx.x] = routed.gates[threadIdx.x];
    }
  }
  const int found = uniform(find_units(topk, q.N * q.K, &units));
  const int chunks = q.F / (16 * CG), shared = q.Fs / (16 * CG), all = shared + found * chunks;
  for (int i = blockIdx.x; i < all; i += gridDim.x) {
    const int b = i - shared, u = b < 0 ? 0 : b / chunks;
    const bool routed = b >= 0;
    const int64_t F = routed ? q.F : q.Fs, col0 = int64_t(routed ? b % chunks : i) * 16 * CG;
    const int64_t strip = (routed ? uniform(units.expert[u]) * (F / 16) : 0) + col0 / 16;
    const View &g = routed ? wg : swg, &p = routed ? wu : swu;
    const Strips w{{g.code(strip, q.H), p.code(strip, q.H)}, {g.scale(strip, q.H), p.scale(strip, q.H)},
                   q.H / kMxTile};
    const int first = uniform(units.start[u]), M = routed ? uniform(units.start[u + 1]) - first : q.N;
    by_rows<MTMAX>(M, [&](auto mt, int m0, int m) {
      gate_up_rows<decltype(mt)::value, CG, PX>(
          x, w, col0, F, [&](int r) { return routed ? int(units.slots[first + m0 + r]) : m0 + r; }, m,
          routed ? q.K : 1, routed ? gates : nullptr, routed ? act : sact, routed ? int64_t(q.N) * q.K : q.N, red);
    });
  }
}

// CG strips of one expert's down product for the M rows slot(0 ..), the contraction's
// tiles from .. to (`from` a multiple of 4): sums to out[slot][H].
template <int MT, int CG, typename Slot>
__device__ __forceinline__ void down_rows(const Operands& a, const Strips& w, int64_t col0, int64_t H, Slot slot,
                                          int M, float* out, int from, int to, f32x4_t* red) {
  constexpr int U = kUnroll<CG, MT, kActParts>;
  const int c = lane_id() % 16, wave = wave_id();
  f32x4_t acc[MT][CG];
  clear(acc);
  int at[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) at[m] = slot(16 * m + c < M ? 16 * m + c : 0);
  for (int kt = from + wave * U; kt < to; kt += kWaves * U) multiply<MT, 1, CG, U, kActParts>(w, a, kt, at, acc);
  join<MT, 1, CG, kWaves>(acc, red, [&](int m, int s, int lane, const f32x4_t* v) {
    const int r = 16 * m + lane % 16;
    if (r < M) *reinterpret_cast<f32x4_t*>(out + slot(r) * H + col0 + 16 * s + 4 * (lane / 16)) = v[0];
  });
}

// More than one token: ys [part][slot][H], then sys [part][token][H] of the shared expert.  Pieces
// as in k_mx4_gate_up.
template <int MTMAX, int CG>
__global__ __launch_bounds__(kNT, MTMAX > 2 ? 1 : 2) void k_mx4_down(const bf16_t* __restrict__ act,
                                                                     const bf16_t* __restrict__ sact, View wd,
                                                                     View swd, const int32_t* __restrict__ topk,
                                                                     float* __restrict__ ys, float* __restrict__ sys,
                                                                     Shape q) {
  __shared__ Units units;
  __shared__ f32x4_t red[kWaves * CG * kWave];
  const int found = uniform(find_units(topk, q.N * q.K, &units));
  const int chunks = q.H / (16 * CG), each = chunks * q.parts, shared = q.Fs > 0 ? each : 0, all = shared + found * each;
  for (int i = blockIdx.x; i < all; i += gridDim.x) {
    const int b = i - shared, u = b < 0 ? 0 : b / each, F = b < 0 ? q.Fs : q.F, part = i % each / chunks;
    const bool routed = b >= 0;
    const int64_t col0 = int64_t(i % chunks) * 16 * CG;
    const int per = (F / kMxTile + 4 * q.parts - 1) / (4 * q.parts) * 4;  // tiles of a part
    const int64_t strip = (routed ? uniform(units.expert[u]) * int64_t(q.H / 16) : 0) + col0 / 16, R = routed ? q.N * q.K : q.N;
    const View& d = routed ? wd : swd;
    const Strips w{{d.code(strip, F), nullptr}, {d.scale(strip, F), nullptr}, F / kMxTile};
    const int first = uniform(units.start[u]), M = routed ? uniform(units.start[u + 1]) - first : q.N;
    by_rows<MTMAX>(M, [&](auto mt, int m0, int m) {
      down_rows<decltype(mt)::value, CG>(
          packed(routed ? act : sact, R, F), w, col0, q.H,
          [&](int r) { return routed ? int64_t(units.slots[first + m0 + r]) : int64_t(m0 + r); }, m,
          (routed ? ys : sys) + part * R * q.H, part * per, min((part + 1) * per, F / kMxTile), red);
    });
  }
}

// One token: the sum over its experts and the shared one is part of the
// contraction, dealt to sixteen waves, and y leaves rounded.
constexpr int kOneWaves = 16;
template <typename T>
__global__ __launch_bounds__(kOneWaves* kWave) void k_mx4_down_one(const bf16_t* __restrict__ act,
                                                                   const bf16_t* __restrict__ sact, View wd, View swd,
                                                                   const int32_t* __restrict__ topk,
                                                                   T* __restrict__ y, Shape q) {
  constexpr int U = kUnroll<1, 1, kActParts>;
  __shared__ f32x4_t red[kOneWaves * kWave];
  const int wave = wave_id();
  const int64_t col0 = int64_t(blockIdx.x) * 16;
  f32x4_t acc[1][1];
  clear(acc);
  const int per = (q.F / kMxTile + U - 1) / U, routed = q.K * per, all = routed + (q.Fs / kMxTile + U - 1) / U;
  for (int i = wave; i < all; i += kOneWaves) {
    const bool sh = i >= routed;
    const int k = sh ? 0 : i / per, F = sh ? q.Fs : q.F;
    const int64_t strip = (sh ? 0 : int64_t(uniform(topk[k])) * (q.H / 16)) + blockIdx.x;
    const View& d = sh ? swd : wd;
    const int at[1] = {k};
    multiply<1, 1, 1, U, kActParts>(Strips{{d.code(strip, F), nullptr}, {d.scale(strip, F), nullptr}, F / kMxTile},
                             packed(sh ? sact : act, sh ? 1 : q.K, F), (sh ? i - routed : i % per) * U, at, acc);
  }
  join<1, 1, 1, kOneWaves>(acc, red, [&](int, int, int lane, const f32x4_t* v) {
    if (lane % 16 != 0) return;
    T* to = y + col0 + 4 * (lane / 16);
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<f32x4_t*>(to) = v[0];
    else
      *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(v[0][0], v[0][1]), pack_bf16x2(v[0][2], v[0][3]));
  });
}

// ------------------------------------------------------------------- host

constexpr int64_t kCUs = 256;

struct Plan {
  Shape q;
  int logit_parts;   // 0: gate/up forms the logits itself
  bool route;        // gate/up ranks them itself
  int gu_cg, dn_cg;  // strips of a piece
  int row_tiles;     // that a kernel has registers for
  size_t logits, xp, act, sact, ys, sys, bytes;
};

// Strips of a piece, of `strips` in all: the rows are read again for each piece, so as many as
// leave every CU one (8 strips of both kinds of product at most: their sums take the registers).
// 64 tokens of 8 experts, H 4096, F 14336: gate/up 101 us with four strips of both matrices, 120 with
// two, 167 with one; down (whole contractions) 106 with eight, 115 with four, 181 with two.
int strips_of(int64_t strips, int most) {
  int cg = most;
  while (cg > 1 && strips / cg < kCUs) cg /= 2;
  return cg;
}

Plan plan(const moe_launch::Dims& d, int64_t Fs) {
  Plan p;
  p.q = Shape{int(d.N), int(d.H), int(d.F), int(Fs), int(d.E), int(d.K), int(std::min(d.NK(), d.E)), 1};
  const bool bf = d.dtype == MOE_BF16;
  const int64_t NK = d.NK(), px = bf ? 1 : 3;
  const double used = double(d.E) * (1.0 - std::pow(1.0 - double(d.K) / double(d.E), double(d.N)));
  const double rows = double(NK) / used;
  p.route = d.N <= 16 && d.N * d.E <= kPairs;
  const bool small_router = (d.E + 15) / 16 * (d.H / 32) <= 4 * kWaves;
  p.logit_parts = p.route && small_router && bf && d.N <= 4 ? 0 : int((d.H + kLogitRows - 1) / kLogitRows);
  p.gu_cg = strips_of(std::llround(used * double(d.F / 16)) + Fs / 16, 4);
  const int64_t strips = std::llround(used * double(d.H / 16));
  p.dn_cg = strips_of(strips, 8);
  // Where that leaves a CU few pieces, each takes a part of the contraction, 16 tiles or more: pieces of
  // experts with more rows take longer.  The parts' sums meet in the kernel that adds a token's.
  // 64 tokens of 8 experts, H 4096, F 14336: down and that kernel 94 us with four parts, 111 with one.
  p.q.parts = d.N == 1 ? 1 : int(std::max<int64_t>(1, std::min<int64_t>(d.F / kMxTile / 16, 4 * kCUs * p.dn_cg / strips)));
  p.row_tiles = d.N <= 16 ? 1 : std::max(rows, Fs > 0 ? double(d.N) : 0.0) > 24.0 ? 4 : 2;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += (n + 255) & ~size_t(255);
    return here;
  };
  p.logits = take(size_t(p.logit_parts) * d.N * d.E * sizeof(double));
  p.xp = take(p.logit_parts == 0 ? 0 : size_t(px) * d.N * d.H * 2);
  p.act = take(size_t(kActParts) * NK * d.F * 2);
  p.sact = take(size_t(kActParts) * d.N * Fs * 2);
  p.ys = take(d.N == 1 ? 0 : size_t(p.q.parts) * NK * d.H * 4);
  p.sys = take(d.N == 1 || Fs == 0 ? 0 : size_t(p.q.parts) * d.N * d.H * 4);
  p.bytes = at;
  return p;
}

#define MOE_LAUNCHED()                 \
  {                                    \
    const hipError_t e = hipGetLastError(); \
    if (e != hipSuccess) return e;     \
  }

template <typename T> struct Args {
  const T *x, *w_r;
  const float* bias;
  View wg, wu, wd, swg, swu, swd;
  int32_t* topk;
  float* gates;
  T* y;
  char* ws;
};

// Workgroups for `pieces` pieces at most.  Finding the units takes a workgroup about 3 us,
// so it does it for several pieces; two to three fit a CU, the others follow them where
// pieces run unevenly (32 tokens of 256 experts, gate/up: 428 us with two a CU in all, 424
// with four, 421 with eight; 13 of 64, down: 29.7, 27.6 and 28.1).
dim3 grid_of(int64_t pieces) { return dim3(unsigned(std::min(pieces, 4 * kCUs))); }

template <typename T, int MTMAX, int CG>
hipError_t gate_up(const Plan& p, const Args<T>& a, hipStream_t s) {
  const Shape& q = p.q;
  const dim3 grid = grid_of((int64_t(q.units) * q.F + q.Fs) / (16 * CG));
  bf16_t* act = reinterpret_cast<bf16_t*>(a.ws + p.act);
  bf16_t* sact = reinterpret_cast<bf16_t*>(a.ws + p.sact);
  const bf16_t* xp = reinterpret_cast<const bf16_t*>(a.ws + p.xp);
  const Operands x = p.logit_parts > 0
                         ? Operands{xp, int64_t(q.N) * q.H, int64_t(q.N) * kMxTile, q.N * 32, 32, 8}
                         : Operands{reinterpret_cast<const bf16_t*>(a.x), 0, kMxTile, 8, q.H, 32};
  const Route<T> route{a.x, a.w_r, p.logit_parts > 0 ? reinterpret_cast<const double*>(a.ws + p.logits) : nullptr,
                       a.bias, p.logit_parts};
  if constexpr (MTMAX == 1)
    if (p.route) {
      k_mx4_gate_up<T, MTMAX, CG, true><<<grid, dim3(kNT), 0, s>>>(x, a.wg, a.wu, a.swg, a.swu, a.topk, a.gates, route,
                                                                   act, sact, q);
      return hipGetLastError();
    }
  k_mx4_gate_up<T, MTMAX, CG, false><<<grid, dim3(kNT), 0, s>>>(x, a.wg, a.wu, a.swg, a.swu, a.topk, a.gates, route, act,
                                                                sact, q);
  return hipGetLastError();
}

template <typename T, int MTMAX, int CG>
hipError_t down(const Plan& p, const Args<T>& a, hipStream_t s) {
  const Shape& q = p.q;
  float* ys = reinterpret_cast<float*>(a.ws + p.ys);
  float* sys = reinterpret_cast<float*>(a.ws + p.sys);
  k_mx4_down<MTMAX, CG>
      <<<grid_of((int64_t(q.units) + (q.Fs > 0 ? 1 : 0)) * q.parts * q.H / (16 * CG)), dim3(kNT), 0, s>>>(
          reinterpret_cast<const bf16_t*>(a.ws + p.act), reinterpret_cast<const bf16_t*>(a.ws + p.sact), a.wd, a.swd,
          a.topk, ys, sys, q);
  MOE_LAUNCHED()
  k_decode_combine<T><<<dim3(q.H / 64, q.N), dim3(256), 0, s>>>(ys, sys, a.y, q.N, q.H, q.K, q.parts,
                                                                       q.Fs > 0 ? q.parts : 0);
  return hipGetLastError();
}

template <typename T, int MTMAX>
hipError_t experts(const Plan& p, const Args<T>& a, hipStream_t s) {
  const hipError_t e = p.gu_cg == 4   ? gate_up<T, MTMAX, 4>(p, a, s)
                       : p.gu_cg == 2 ? gate_up<T, MTMAX, 2>(p, a, s)
                                      : gate_up<T, MTMAX, 1>(p, a, s);
  if (e != hipSuccess) return e;
  if (p.q.N == 1) {
    k_mx4_down_one<T><<<dim3(p.q.H / 16), dim3(kOneWaves * kWave), 0, s>>>(
        reinterpret_cast<const bf16_t*>(a.ws + p.act), reinterpret_cast<const bf16_t*>(a.ws + p.sact), a.wd, a.swd,
        a.topk, a.y, p.q);
    return hipGetLastError();
  }
  return p.dn_cg == 8   ? down<T, MTMAX, 8>(p, a, s)
         : p.dn_cg == 4 ? down<T, MTMAX, 4>(p, a, s)
         : p.dn_cg == 2 ? down<T, MTMAX, 2>(p, a, s)
                        : down<T, MTMAX, 1>(p, a, s);
}

template <typename T>
hipError_t decode_t(const moe_launch::Dims& d, int64_t Fs, const Args<T>& a, hipStream_t s) {
  constexpr int PX = sizeof(T) == 2 ? 1 : 3;
  const Plan p = plan(d, Fs);
  const Shape& q = p.q;
  double* logits = reinterpret_cast<double*>(a.ws + p.logits);
  if (p.logit_parts > 0) {
    k_decode_logits<T><<<dim3(p.logit_parts, (q.E + 15) / 16, (q.N + 15) / 16), dim3(kLogitWaves * kWave), 0, s>>>(
        a.x, a.w_r, logits, PackOperands<T, PX>{reinterpret_cast<bf16_t*>(a.ws + p.xp)}, q.N, q.H, q.E);
    MOE_LAUNCHED()
  }
  if (!p.route) {
    k_decode_topk<<<dim3(q.N), dim3(256), 0, s>>>(logits, a.bias, a.topk, a.gates, q.N, q.E, q.K, p.logit_parts);
    MOE_LAUNCHED()
  }
  return p.row_tiles == 1   ? experts<T, 1>(p, a, s)
         : p.row_tiles == 2 ? experts<T, 2>(p, a, s)
                            : experts<T, 4>(p, a, s);
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
#define MOE_DECODE(T)                                                                                               \
  decode_t<T>(d, Fs, Args<T>{static_cast<const T*>(x), static_cast<const T*>(w_r), bias, view(wg), view(wu), view(wd), \
                             view(swg), view(swu), view(swd), topk, gates, static_cast<T*>(y),                      \
                             static_cast<char*>(ws)}, s)
  return d.dtype == MOE_BF16 ? MOE_DECODE(bf16_t) : MOE_DECODE(float);
#undef MOE_DECODE
}

}  // namespace moe_launch
