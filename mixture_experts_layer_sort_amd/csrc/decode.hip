// The whole layer for the few tokens of a decoding step (at most
// MOE_DECODE_MAX_TOKENS), forward only.
//
//   l = x.W_r (+ bias), top-K by (l desc, id asc), gates = softmax over the K;
//   y_n = sum_k gates[n,k] FFN_{e_nk}(x_n) (+ FFN_s(x_n)),
//   FFN(v) = (silu(v.W_gate) * (v.W_up)).W_down.
//
// With few rows per expert the weights of the chosen experts are all that
// matters: they are read once, and HBM bounds the call.  So there is no sort,
// no row tile list and no staging of weights through LDS:
//  - A wave reads 32 rows of a weight matrix times 16 * CW columns straight
//    into registers: lane (g, c) = (lane / 16, lane % 16) takes the CW columns
//    CW*c .. of rows 8g .. 8g+7, so each row is read as one contiguous segment.
//    Those eight rows of one column are exactly a lane's share of a 16x16x32
//    bf16 matrix operand with column index c, so column i of every lane forms
//    one operand after packing row pairs (4 byte permutes for 8 values): CW
//    matrix instructions use up the 32 x 16*CW panel.  float32 needs no packing:
//    row j of the eight is one operand of a 16x16x4 instruction.
//  - The other operand holds up to 16 token rows; rows past the expert's last
//    repeat row 0 and their results are dropped.
//  - The waves of a workgroup split the contraction; their float32 sums meet
//    in LDS in a fixed order.
// The activation silu(g)*u keeps float32 accuracy on its way to the second
// product: for bf16 it is stored as the sum of two bf16 values (hi + lo).  y is
// rounded once.  Router logits are summed in float64, so the choice of experts
// does not depend on the order of the sum.
#include <algorithm>

#include "common.h"

namespace {
using namespace moe;

constexpr int kTok = MOE_DECODE_MAX_TOKENS;
constexpr int kSlots = kTok * MOE_MAX_TOPK;
constexpr int kWaves = 8;
constexpr int kNT = kWaves * kWave;
static_assert(kSlots <= kNT, "one thread per (token, k) slot builds the row lists");

// ------------------------------------------------------------------ router

constexpr int kLogitRows = 128;  // rows of W_r per workgroup
constexpr int kLogitTok = 8;     // tokens per thread

// Partial logits part[s][n][e] over rows s*128 .. of W_r.  Thread (e, token
// group, h slice); the h slices meet in LDS.
template <typename T>
__global__ __launch_bounds__(256) void k_decode_logits(const T* __restrict__ x, const T* __restrict__ w_r,
                                                       double* __restrict__ part, int N, int H, int E) {
  __shared__ float xs[kTok][kLogitRows];
  __shared__ double red[256 * kLogitTok];
  const int h0 = blockIdx.x * kLogitRows;
  const int tid = threadIdx.x;
  for (int i = tid; i < N * kLogitRows; i += 256)
    xs[i / kLogitRows][i % kLogitRows] = Elt<T>::load(x + int64_t(i / kLogitRows) * H + h0 + i % kLogitRows);
  __syncthreads();
  const int groups = (N + kLogitTok - 1) / kLogitTok;
  int slices = 1;  // h slices per (expert, group): fill the workgroup
  while (slices < 32 && 2 * slices * E <= 256) slices *= 2;
  const int e = tid % E, q = tid / E;  // q: slice
  for (int g = 0; g < groups; ++g) {
    double acc[kLogitTok];
#pragma unroll
    for (int j = 0; j < kLogitTok; ++j) acc[j] = 0.0;
    if (q < slices) {
      const int len = kLogitRows / slices;
      for (int h = q * len; h < (q + 1) * len; ++h) {
        const double w = Elt<T>::load(w_r + int64_t(h0 + h) * E + e);
#pragma unroll
        for (int j = 0; j < kLogitTok; ++j) acc[j] = fma(double(xs[min(g * kLogitTok + j, N - 1)][h]), w, acc[j]);
      }
#pragma unroll
      for (int j = 0; j < kLogitTok; ++j) red[(q * kLogitTok + j) * E + e] = acc[j];
    }
    __syncthreads();
    for (int i = tid; i < kLogitTok * E; i += 256) {
      const int n = g * kLogitTok + i / E;
      if (n < N) {
        double v = 0.0;
        for (int s = 0; s < slices; ++s) v += red[s * kLogitTok * E + i];
        part[(int64_t(blockIdx.x) * N + n) * E + i % E] = v;
      }
    }
    __syncthreads();
  }
}

// Top-K and gates of token blockIdx.x: expert e's place is the number of
// experts before it in the order (logit desc, id asc); NaN logits come last.
__global__ __launch_bounds__(256) void k_decode_topk(const double* __restrict__ part, const float* __restrict__ bias,
                                                     int32_t* __restrict__ topk, float* __restrict__ gates, int N,
                                                     int E, int K, int S) {
  __shared__ double l[MOE_MAX_EXPERTS];
  __shared__ double sel[MOE_MAX_TOPK];
  const int n = blockIdx.x, e = threadIdx.x;
  double v = 0.0;
  if (e < E) {
    for (int s = 0; s < S; ++s) v += part[(int64_t(s) * N + n) * E + e];
    if (bias != nullptr) v += double(bias[e]);
    if (v != v) v = -INFINITY;
    l[e] = v;
  }
  __syncthreads();
  if (e < E) {
    int before = 0;
    for (int i = 0; i < E; ++i) before += l[i] > v || (l[i] == v && i < e);
    if (before < K) {
      topk[n * K + before] = e;
      sel[before] = v;
    }
  }
  __syncthreads();
  if (e < K) {
    float sum = 0.f, mine = 0.f;
    for (int k = 0; k < K; ++k) {
      const float z = expf(float(sel[k] - sel[0]));
      sum += z;
      if (k == e) mine = z;
    }
    gates[n * K + e] = mine / sum;
  }
}

// ------------------------------------------------------- rows of an expert

// Slots n*K + k of expert e in ascending order to rows[0, count); the count.
// All threads of the workgroup call it.
__device__ __forceinline__ int expert_slots(const int32_t* __restrict__ topk, int NK, int e, int* rows) {
  __shared__ int wave_count[kWaves];
  const int t = threadIdx.x, w = t / kWave;
  const bool mine = t < NK && topk[t] == e;
  const uint64_t mask = __ballot(mine);
  if (lane_id() == 0) wave_count[w] = __popcll(mask);
  __syncthreads();
  int base = 0, count = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    if (i < w) base += wave_count[i];
    count += wave_count[i];
  }
  // one token names an expert once, so count <= N <= kTok for any legal topk
  const int at = base + __popcll(mask & ((uint64_t(1) << lane_id()) - 1));
  if (mine && at < kTok) rows[at] = t;
  __syncthreads();
  return min(count, kTok);
}

// Unit u of the grid's expert axis: with at most E slots it is a slot, whose
// expert is worked on by the first slot that names it, else expert u.  Builds
// the expert's rows; returns their number, 0 when there is nothing to do.
__device__ __forceinline__ int unit_rows(const int32_t* __restrict__ topk, int NK, int E, int u, int* e, int* rows) {
  *e = NK <= E ? topk[u] : u;
  const int M = expert_slots(topk, NK, *e, rows);
  return NK <= E && rows[0] != u ? 0 : M;
}

// --------------------------------------------------------------- the panels

template <int BYTES> struct Raw;
template <> struct Raw<16> { typedef uint32_t type __attribute__((ext_vector_type(4))); };
template <> struct Raw<8> { typedef uint32_t type __attribute__((ext_vector_type(2))); };

// A wave's share of 32 rows x 16*CW columns of a weight matrix, and of the
// same 32 columns of the row operand.  NA: row operands added up (bf16
// activations are hi + lo).
template <typename T, int CW, int NA> struct Panel;

template <int CW, int NA> struct Panel<bf16_t, CW, NA> {
  typedef typename Raw<CW * 2>::type raw_t;
  typedef uint32_t words4 __attribute__((ext_vector_type(4)));
  raw_t w[8];
  // row operand of one tile of 16 rows: 8 consecutive bf16 of row lane%16
  struct A {
    words4 a[NA];
    __device__ __forceinline__ void load(const bf16_t* const* p, int64_t off) {
#pragma unroll
      for (int i = 0; i < NA; ++i) a[i] = *reinterpret_cast<const words4*>(p[i] + off);
    }
  };
  __device__ __forceinline__ void load(const bf16_t* p, int64_t ld) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = __builtin_nontemporal_load(reinterpret_cast<const raw_t*>(p + j * ld));
  }
  template <int MT>
  __device__ __forceinline__ void multiply(const A (&a)[MT], f32x4_t (&acc)[MT][CW]) const {
#pragma unroll
    for (int i = 0; i < CW; ++i) {
      words4 b;
#pragma unroll
      for (int d = 0; d < 4; ++d)
        b[d] = __builtin_amdgcn_perm(w[2 * d + 1][i / 2], w[2 * d][i / 2], i % 2 ? 0x07060302u : 0x05040100u);
      const bf16x8_t bv = __builtin_bit_cast(bf16x8_t, b);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int q = 0; q < NA; ++q)
          acc[m][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a[m].a[q]), bv, acc[m][i],
                                                              0, 0, 0);
    }
  }
};

template <int CW> struct Panel<float, CW, 1> {
  typedef float raw_t __attribute__((ext_vector_type(CW)));
  raw_t w[8];
  struct A {
    float a[8];
    __device__ __forceinline__ void load(const float* const* p, int64_t off) {
      Vec16<float>::load(p[0] + off, a);
      Vec16<float>::load(p[0] + off + 4, a + 4);
    }
  };
  __device__ __forceinline__ void load(const float* p, int64_t ld) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = __builtin_nontemporal_load(reinterpret_cast<const raw_t*>(p + j * ld));
  }
  template <int MT>
  __device__ __forceinline__ void multiply(const A (&a)[MT], f32x4_t (&acc)[MT][CW]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < CW; ++i)
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[m][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[m].a[j], w[j][i], acc[m][i], 0, 0, 0);
  }
};

// acc[m] += rows of tile m (pa[m], NA pointers at this lane's row and first
// column) . W over the panels first, first + stride, ... below `panels`.
// wp: this lane's first element of panel 0.  The next panel's loads are issued
// before this one's products.
template <typename T, int CW, int NA, int MT>
__device__ __forceinline__ void stream(const T* wp, int64_t ld, const T* const (&pa)[MT][NA], int first, int stride,
                                       int panels, f32x4_t (&acc)[MT][CW]) {
  typedef Panel<T, CW, NA> P;
  P p[2];
  typename P::A a[2][MT];
  auto fetch = [&](P& q, typename P::A (&b)[MT], int i) {
    q.load(wp + int64_t(i) * 32 * ld, ld);
#pragma unroll
    for (int m = 0; m < MT; ++m) b[m].load(pa[m], int64_t(i) * 32);
  };
  if (first >= panels) return;
  fetch(p[0], a[0], first);
  int i = first;
  while (true) {
    const int i1 = i + stride, i2 = i + 2 * stride;
    if (i1 < panels) fetch(p[1], a[1], i1);
    p[0].template multiply<MT>(a[0], acc);
    if (i1 >= panels) break;
    if (i2 < panels) fetch(p[0], a[0], i2);
    p[1].template multiply<MT>(a[1], acc);
    if (i2 >= panels) break;
    i = i2;
  }
}

// Writes a wave's 16 x 16*CW sums to red [16][16*CW] (the matrix instruction
// leaves row 4*(lane/16) + r, operand column lane%16 in element r).
template <int CW>
__device__ __forceinline__ void park(const f32x4_t (&acc)[CW], float* red) {
  const int g = lane_id() / 16, c = lane_id() % 16;
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int i = 0; i < CW; ++i) red[(4 * g + r) * 16 * CW + c * CW + i] = acc[i][r];
}

// ------------------------------------------------------------ gate and up

template <typename T> struct ActStore;
template <> struct ActStore<bf16_t> {
  static constexpr int n = 2;  // hi and lo
  static __device__ __forceinline__ void put(bf16_t* act, int64_t plane, int64_t at, float v) {
    const bf16_t hi = f32_to_bf16(v);
    const float rest = v - bf16_to_f32(hi);
    act[at] = hi;
    act[plane + at] = isfinite(rest) ? f32_to_bf16(rest) : bf16_t(0);  // infinite or NaN activations: hi says it all
  }
};
template <> struct ActStore<float> {
  static constexpr int n = 1;
  static __device__ __forceinline__ void put(float* act, int64_t, int64_t at, float v) { act[at] = v; }
};

// Rows rows[0, M) (token = row / div) of one expert: silu(x.wg) * (x.wu) for
// the 16*CW columns from col0, to act[row][ld].  Waves 2s and 2s+1 take every
// fourth panel from s of W_gate and W_up.
template <typename T, int CW, int MT>
__device__ __forceinline__ void gate_up_rows(const T* __restrict__ x, const T* wg, const T* wu, int H, int64_t ld,
                                             int64_t col0, const int* rows, int M, int div, T* act, int64_t plane,
                                             float* red) {
  const int wave = threadIdx.x / kWave, g = lane_id() / 16, c = lane_id() % 16;
  f32x4_t acc[MT][CW];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < CW; ++i) acc[m][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const T* pa[MT][1];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = 16 * m + c;
    pa[m][0] = x + int64_t(rows[r < M ? r : 0] / div) * H + 8 * g;
  }
  stream<T, CW, 1, MT>((wave & 1 ? wu : wg) + 8 * g * ld + col0 + CW * c, ld, pa, wave / 2, kWaves / 2, H / 32, acc);
  constexpr int TILE = 16 * 16 * CW;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    __syncthreads();
    park<CW>(acc[m], red + wave * TILE);
    __syncthreads();
    for (int i = threadIdx.x; i < TILE; i += kNT) {
      const int r = 16 * m + i / (16 * CW);
      if (r >= M) break;
      float gv = 0.f, uv = 0.f;
#pragma unroll
      for (int s = 0; s < kWaves / 2; ++s) {
        gv += red[2 * s * TILE + i];
        uv += red[(2 * s + 1) * TILE + i];
      }
      ActStore<T>::put(act, plane, rows[r] * ld + col0 + i % (16 * CW), gv / (1.0f + expf(-gv)) * uv);
    }
  }
}

template <typename T, int CW, int MT>
__global__ __launch_bounds__(kNT) void k_decode_gate_up(const T* __restrict__ x, const T* __restrict__ wg,
                                                        const T* __restrict__ wu, const T* __restrict__ swg,
                                                        const T* __restrict__ swu, const int32_t* __restrict__ topk,
                                                        T* __restrict__ act, T* __restrict__ sact, int N, int H,
                                                        int F, int Fs, int E, int K, int units) {
  __shared__ int rows[kTok];
  __shared__ __attribute__((aligned(16))) float red[kWaves * 16 * 16 * CW];
  const int chunks = F / (16 * CW);
  const int b = blockIdx.x;
  int M, div;
  const T *mg, *mu;
  T* out;
  int64_t ld, col0, plane;
  if (b < units * chunks) {
    int e;
    M = unit_rows(topk, N * K, E, b / chunks, &e, rows);
    div = K;
    ld = F;
    col0 = int64_t(b % chunks) * 16 * CW;
    mg = wg + int64_t(e) * H * F;
    mu = wu + int64_t(e) * H * F;
    out = act;
    plane = int64_t(N) * K * F;
  } else {
    if (threadIdx.x < kTok) rows[threadIdx.x] = threadIdx.x;
    __syncthreads();
    M = N;
    div = 1;
    ld = Fs;
    col0 = int64_t(b - units * chunks) * 16 * CW;
    mg = swg;
    mu = swu;
    out = sact;
    plane = int64_t(N) * Fs;
  }
  for (int m0 = 0; m0 < M; m0 += 16 * MT)
    gate_up_rows<T, CW, MT>(x, mg, mu, H, ld, col0, rows + m0, min(M - m0, 16 * MT), div, out, plane, red);
}

// ------------------------------------------------------------------- down

// Rows of one expert: act.wd over this split's panels, for the 16*CW columns
// from col0, to ysp[row][H].
template <typename T, int CW, int MT>
__device__ __forceinline__ void down_rows(const T* act, int64_t plane, const T* wd, int F, int64_t H, int64_t col0,
                                          const int* rows, int M, int split, int splits, float* ysp, float* red) {
  constexpr int NA = ActStore<T>::n;
  const int wave = threadIdx.x / kWave, g = lane_id() / 16, c = lane_id() % 16;
  f32x4_t acc[MT][CW];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < CW; ++i) acc[m][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const T* pa[MT][NA];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int q = 0; q < NA; ++q) {
      const int r = 16 * m + c;
      pa[m][q] = act + q * plane + int64_t(rows[r < M ? r : 0]) * F + 8 * g;
    }
  stream<T, CW, NA, MT>(wd + 8 * g * H + col0 + CW * c, H, pa, split * kWaves + wave, splits * kWaves, F / 32, acc);
  constexpr int TILE = 16 * 16 * CW;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    __syncthreads();
    park<CW>(acc[m], red + wave * TILE);
    __syncthreads();
    for (int i = threadIdx.x; i < TILE; i += kNT) {
      const int r = 16 * m + i / (16 * CW);
      if (r >= M) break;
      float v = 0.f;
#pragma unroll
      for (int s = 0; s < kWaves; ++s) v += red[s * TILE + i];
      ysp[rows[r] * H + col0 + i % (16 * CW)] = v;
    }
  }
}

template <typename T, int CW, int MT>
__global__ __launch_bounds__(kNT) void k_decode_down(const T* __restrict__ act, const T* __restrict__ sact,
                                                     const T* __restrict__ wd, const T* __restrict__ swd,
                                                     const int32_t* __restrict__ topk, float* __restrict__ ysp,
                                                     float* __restrict__ sysp, int N, int H, int F, int Fs, int E,
                                                     int K, int units, int splits, int ssplits) {
  __shared__ int rows[kTok];
  __shared__ __attribute__((aligned(16))) float red[kWaves * 16 * 16 * CW];
  const int chunks = H / (16 * CW);
  int b = blockIdx.x;
  const int64_t col0 = int64_t(b % chunks) * 16 * CW;
  b /= chunks;
  if (b < units * splits) {
    int e;
    const int M = unit_rows(topk, N * K, E, b / splits, &e, rows);
    const int sp = b % splits;
    for (int m0 = 0; m0 < M; m0 += 16 * MT)
      down_rows<T, CW, MT>(act, int64_t(N) * K * F, wd + int64_t(e) * F * H, F, H, col0, rows + m0,
                           min(M - m0, 16 * MT), sp, splits, ysp + int64_t(sp) * N * K * H, red);
  } else {
    if (threadIdx.x < kTok) rows[threadIdx.x] = threadIdx.x;
    __syncthreads();
    const int sp = b - units * splits;
    for (int m0 = 0; m0 < N; m0 += 16 * MT)
      down_rows<T, CW, MT>(sact, int64_t(N) * Fs, swd, Fs, H, col0, rows + m0, min(N - m0, 16 * MT), sp, ssplits,
                           sysp + int64_t(sp) * N * H, red);
  }
}

// y[n] = sum_k gates[n,k] * (sum over the splits) (+ the shared expert's sum),
// k and splits ascending, float32, one rounding.
template <typename T>
__global__ __launch_bounds__(256) void k_decode_combine(const float* __restrict__ ysp, const float* __restrict__ sysp,
                                                        const float* __restrict__ gates, T* __restrict__ y, int N,
                                                        int H, int K, int splits, int ssplits) {
  const int h = blockIdx.x * 256 + threadIdx.x;
  const int n = blockIdx.y;
  if (h >= H) return;
  float v = 0.f;
  for (int k = 0; k < K; ++k) {
    float a = 0.f;
    for (int s = 0; s < splits; ++s) a += ysp[(int64_t(s) * N * K + n * K + k) * H + h];
    v = fmaf(gates[n * K + k], a, v);
  }
  for (int s = 0; s < ssplits; ++s) v += sysp[(int64_t(s) * N + n) * H + h];
  y[int64_t(n) * H + h] = Elt<T>::from_f32(v);
}

// ------------------------------------------------------------------- host

// How the call is cut up, and where its scratch lies.
struct Plan {
  int logit_parts, units, splits, ssplits;
  size_t logits, act, sact, ysp, sysp, bytes;
};

int splits_of(int64_t f, int64_t blocks) {
  // enough workgroups for two on each of 256 CUs, with two panels per wave at least
  int s = 1;
  while (s * blocks < 512 && f / 32 >= int64_t(4) * s * kWaves) s *= 2;
  return s;
}

Plan plan_of(const moe_launch::Dims& d, int64_t Fs) {
  Plan p;
  const int cw = d.dtype == MOE_BF16 ? 8 : 4;
  const int64_t chunks = d.H / (16 * cw), NK = d.NK();
  p.logit_parts = int(d.H / kLogitRows);
  p.units = int(std::min(NK, d.E));
  p.splits = splits_of(d.F, chunks * p.units);
  p.ssplits = Fs > 0 ? splits_of(Fs, chunks) : 0;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += (n + 255) & ~size_t(255);
    return here;
  };
  p.logits = take(size_t(p.logit_parts) * d.N * d.E * sizeof(double));
  p.act = take(size_t(NK) * d.F * 4);  // bf16: hi and lo planes; float32: one plane
  p.sact = take(size_t(d.N) * Fs * 4);
  p.ysp = take(size_t(p.splits) * NK * d.H * 4);
  p.sysp = take(size_t(p.ssplits) * d.N * d.H * 4);
  p.bytes = at;
  return p;
}

template <typename T, int CW, int MT>
hipError_t decode_experts(const moe_launch::Dims& d, const Plan& p, const T* x, const T* wg, const T* wu, const T* wd,
                          int64_t Fs, const T* swg, const T* swu, const T* swd, const int32_t* topk, char* ws,
                          hipStream_t s) {
  const int N = int(d.N), H = int(d.H), F = int(d.F), E = int(d.E), K = int(d.K);
  T* act = reinterpret_cast<T*>(ws + p.act);
  T* sact = reinterpret_cast<T*>(ws + p.sact);
  const unsigned gu = unsigned(p.units * (F / (16 * CW)) + Fs / (16 * CW));
  k_decode_gate_up<T, CW, MT><<<dim3(gu), dim3(kNT), 0, s>>>(x, wg, wu, swg, swu, topk, act, sact, N, H, F, int(Fs), E,
                                                             K, p.units);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const unsigned dn = unsigned((p.units * p.splits + p.ssplits) * (H / (16 * CW)));
  k_decode_down<T, CW, MT><<<dim3(dn), dim3(kNT), 0, s>>>(act, sact, wd, swd, topk, reinterpret_cast<float*>(ws + p.ysp),
                                                          reinterpret_cast<float*>(ws + p.sysp), N, H, F, int(Fs), E,
                                                          K, p.units, p.splits, p.ssplits);
  return hipGetLastError();
}

template <typename T, int CW>
hipError_t decode_t(const moe_launch::Dims& d, const T* x, const T* w_r, const float* bias, const T* wg, const T* wu,
                    const T* wd, int64_t Fs, const T* swg, const T* swu, const T* swd, int32_t* topk, float* gates,
                    T* y, char* ws, hipStream_t s) {
  const Plan p = plan_of(d, Fs);
  const int N = int(d.N), H = int(d.H), E = int(d.E), K = int(d.K);
  double* logits = reinterpret_cast<double*>(ws + p.logits);
  k_decode_logits<T><<<dim3(p.logit_parts), dim3(256), 0, s>>>(x, w_r, logits, N, H, E);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_decode_topk<<<dim3(N), dim3(256), 0, s>>>(logits, bias, topk, gates, N, E, K, p.logit_parts);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (N <= 16)
    e = decode_experts<T, CW, 1>(d, p, x, wg, wu, wd, Fs, swg, swu, swd, topk, ws, s);
  else
    e = decode_experts<T, CW, 2>(d, p, x, wg, wu, wd, Fs, swg, swu, swd, topk, ws, s);
  if (e != hipSuccess) return e;
  k_decode_combine<T><<<dim3((H + 255) / 256, N), dim3(256), 0, s>>>(
      reinterpret_cast<const float*>(ws + p.ysp), reinterpret_cast<const float*>(ws + p.sysp), gates, y, N, H, K,
      p.splits, p.ssplits);
  return hipGetLastError();
}

}  // namespace

namespace moe_launch {

size_t decode_ws(const Dims& d, int64_t Fs) { return plan_of(d, Fs).bytes; }

hipError_t decode(const Dims& d, const void* x, const void* w_r, const float* bias, const void* wg, const void* wu,
                  const void* wd, int64_t Fs, const void* swg, const void* swu, const void* swd, int32_t* topk,
                  float* gates, void* y, void* ws, hipStream_t s) {
  char* w = static_cast<char*>(ws);
#define MOE_DECODE(T, CW)                                                                                          \
  decode_t<T, CW>(d, static_cast<const T*>(x), static_cast<const T*>(w_r), bias, static_cast<const T*>(wg),        \
                  static_cast<const T*>(wu), static_cast<const T*>(wd), Fs, static_cast<const T*>(swg),            \
                  static_cast<const T*>(swu), static_cast<const T*>(swd), topk, gates, static_cast<T*>(y), w, s)
  return d.dtype == MOE_BF16 ? MOE_DECODE(bf16_t, 8) : MOE_DECODE(float, 4);
#undef MOE_DECODE
}

}  // namespace moe_launch
