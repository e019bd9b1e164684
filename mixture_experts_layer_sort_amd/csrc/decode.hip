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
//  - A wave reads a panel of 32 rows of a weight matrix straight into
//    registers: lane (g, c) = (lane / 16, lane % 16) takes, of rows 8g .. 8g+7,
//    16 bytes at c*16 of each of S segments of 256 bytes.  S = 2 puts 512
//    contiguous bytes of a row on their way at once: reading a matrix in
//    column strips ran at 6.5 TB/s with 256-byte segments and 7.0 with 512
//    (1024: 7.0, but half the workgroups), without the streaming hint at 6.
//  - Those eight rows of one column are exactly a lane's share of a 16x16x32
//    bf16 matrix operand with column index c, so column i of every lane forms
//    one operand after packing row pairs (4 byte permutes for 8 values).
//    float32 needs no packing: row j of the eight is one operand of a 16x16x4
//    instruction.
//  - All of a panel's loads are issued before its first product: left to itself
//    the compiler spreads a float32 panel's loads over its products to save
//    registers (64 tokens of a 16-expert float32 layer: 135 us so, 92 in order).
//  - The other operand holds up to 16 token rows; rows past the last repeat
//    row 0 and their results are dropped.
//  - The waves of a workgroup split the contraction; their float32 sums meet
//    in LDS in a fixed order, those of several workgroups in the next kernel.
// gate/up leaves float32 sums; the down kernel forms gate * silu(G) * U as it
// loads them, for bf16 as the exact sum of three bf16 values of eight significant
// bits each, so the activation keeps its 24.  y is rounded once.  Router logits are
// summed in float64, so the choice of experts does not depend on the order of
// the sum.
#include <algorithm>
#include <cmath>

#include "common.h"

namespace {
using namespace moe;

constexpr int kTok = MOE_DECODE_MAX_TOKENS;
constexpr int kSlots = kTok * MOE_MAX_TOPK;
constexpr int kWaves = 4;
constexpr int kNT = kWaves * kWave;

typedef uint32_t words4_t __attribute__((ext_vector_type(4)));
typedef double f64x4_t __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ router

constexpr int kLogitWaves = 16;
constexpr int kLogitRows = 32 * kLogitWaves;  // rows of W_r per workgroup

// 8 consecutive elements as double.
template <typename T>
__device__ __forceinline__ void load8_f64(const T* p, double* out) {
  float v[8];
  Vec16<T>::load(p, v);
  if (Vec16<T>::n == 4) Vec16<T>::load(p + 4, v + 4);
#pragma unroll
  for (int j = 0; j < 8; ++j) out[j] = double(v[j]);
}

// acc += x.W_r for 16 tokens (rows of x) and 16 experts over the 32 rows of W_r
// from h, on the float64 matrix instruction (16 x 16 x 4): lane (g, c) holds row
// 8g + j of step j, for token c and for expert e.
template <typename T>
__device__ __forceinline__ void logit_panel(const T* __restrict__ px, const T* __restrict__ w_r, int h, int E, int e,
                                            f64x4_t& acc) {
  const int g = lane_id() / 16;
  T w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = w_r[int64_t(h + 8 * g + j) * E + e];
  double a[8];
  load8_f64(px + h + 8 * g, a);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    acc = __builtin_amdgcn_mfma_f64_16x16x4f64(a[j], double(Elt<T>::to_f32(w[j])), acc, 0, 0, 0);
}

// A wave's 16 x 16 sums to red [token][expert]: element r is token 4r + g, expert c.
__device__ __forceinline__ void park_logits(const f64x4_t& acc, double* red) {
#pragma unroll
  for (int r = 0; r < 4; ++r) red[(4 * r + lane_id() / 16) * 16 + lane_id() % 16] = acc[r];
}

// Partial logits part[s][n][e] over rows s*512 .. of W_r for 16 experts and 16
// tokens.  A wave has 32 rows; the waves' sums meet in LDS in wave order.  The
// first workgroup of each row range and token tile also packs x as xp
// [H/32][N][32], so that the row operand of a panel is one contiguous piece.  The
// token tiles are workgroups of their own: 64 tokens take 5 us so, 9 in a loop.
template <typename T>
__global__ __launch_bounds__(kLogitWaves * kWave) void k_decode_logits(const T* __restrict__ x,
                                                                      const T* __restrict__ w_r,
                                                                      double* __restrict__ part, T* __restrict__ xp,
                                                                      int N, int H, int E) {
  __shared__ double red[kLogitWaves][256];
  const int wave = threadIdx.x / kWave, g = lane_id() / 16, c = lane_id() % 16;
  const int e0 = blockIdx.y * 16, n0 = blockIdx.z * 16;
  const int h = blockIdx.x * kLogitRows + wave * 32;
  f64x4_t acc = {0.0, 0.0, 0.0, 0.0};
  const int n = min(n0 + c, N - 1);
  if (h < H) {  // the same in the whole wave: H is a multiple of 128
    const T* px = x + int64_t(n) * H;
    logit_panel(px, w_r, h, E, min(e0 + c, E - 1), acc);
    if (blockIdx.y == 0 && n == n0 + c) {
      const uint4* from = reinterpret_cast<const uint4*>(px + h + 8 * g);
      uint4* to = reinterpret_cast<uint4*>(xp + (int64_t(h / 32) * N + n) * 32 + 8 * g);
#pragma unroll
      for (int j = 0; j < 8 * int(sizeof(T)) / 16; ++j) to[j] = from[j];
    }
  }
  park_logits(acc, red[wave]);
  __syncthreads();
  const int tok = n0 + threadIdx.x / 16, ex = e0 + threadIdx.x % 16;
  if (threadIdx.x < 256 && tok < N && ex < E) {
    double v = 0.0;
#pragma unroll
    for (int i = 0; i < kLogitWaves; ++i) v += red[i][threadIdx.x];
    part[(int64_t(blockIdx.x) * N + tok) * E + ex] = v;
  }
}

// Scratch and results of rank_pairs.
constexpr int kPairs = 256;  // (token, expert): one a thread
struct TopK {
  double l[kPairs], sel[16 * MOE_MAX_TOPK];
  int32_t ids[16 * MOE_MAX_TOPK];
  float gates[16 * MOE_MAX_TOPK];
};

// This thread's pair of the tokens from n0 on: its logit from S partial sums.
__device__ __forceinline__ double sum_parts(const double* __restrict__ part, int n0, int N, int E, int S) {
  double v = 0.0;
  for (int s0 = 0; s0 < S; s0 += 16) {
    double t[16];  // loads of one round trip
#pragma unroll
    for (int s = 0; s < 16; ++s) t[s] = s0 + s < S ? part[(int64_t(s0 + s) * N + n0) * E + threadIdx.x] : 0.0;
#pragma unroll
    for (int s = 0; s < 16; ++s) v += t[s];
  }
  return v;
}

// Top-K and gates of `count` tokens (at most 16, count * E <= kPairs) by 256
// threads, thread n*E + e with that pair's logit v: the expert's place is the
// number of experts before it in the order (logit desc, id asc); NaN logits come
// last.  ids and gates [count][K] to *out, thread p's own p behind it, the others'
// after a barrier.
__device__ __forceinline__ void rank_pairs(double v, const float* __restrict__ bias, int count, int E, int K,
                                           TopK* out) {
  const int p = threadIdx.x, n = p / E, e = p % E;
  const bool live = n < count;
  if (live) {
    if (bias != nullptr) v += double(bias[e]);
    if (v != v) v = -INFINITY;
    out->l[p] = v;
  }
  __syncthreads();
  if (live) {
    const double* l = out->l + n * E;
    // one comparison each for the experts below and above all of the wave's own
    const int first = __builtin_amdgcn_readfirstlane(e), lo = first + kWave <= E ? first : 0;
    const int hi = first + kWave <= E ? first + kWave : E;
    int before = 0;
#pragma unroll 8
    for (int i = 0; i < lo; ++i) before += l[i] >= v;
#pragma unroll 8
    for (int i = lo; i < hi; ++i) before += l[i] > v || (l[i] == v && i < e);
#pragma unroll 8
    for (int i = hi; i < E; ++i) before += l[i] > v;
    if (before < K) {
      out->ids[n * K + before] = e;
      out->sel[n * K + before] = v;
    }
  }
  __syncthreads();
  if (p < count * K) {
    const double* sel = out->sel + p / K * K;
    float sum = 0.f, mine = 0.f;
    for (int k = 0; k < K; ++k) {
      // the difference of two float64 logits d, rounded to float32 once: 2^-24 |d| of the gate, about
      // what expf (1 ulp) and the quotient add; the gate itself is a float32
      const float z = expf(float(sel[k] - sel[0]));
      sum += z;
      if (k == p % K) mine = z;
    }
    out->gates[p] = mine / sum;
  }
}

// A token a workgroup.
__global__ __launch_bounds__(kPairs) void k_decode_topk(const double* __restrict__ part,
                                                        const float* __restrict__ bias, int32_t* __restrict__ topk,
                                                        float* __restrict__ gates, int N, int E, int K, int S) {
  __shared__ TopK s;
  const int n = blockIdx.x, t = threadIdx.x;
  rank_pairs(t < E ? sum_parts(part, n, N, E, S) : 0.0, bias, 1, E, K, &s);
  if (t < K) {
    topk[n * K + t] = s.ids[t];
    gates[n * K + t] = s.gates[t];
  }
}

// Routing of all tokens by every workgroup of gate/up for itself.
template <typename T> struct Route {
  const T *x, *w_r;
  const double* part;  // null: the workgroup forms the logits as well
  const float* bias;
  int S;
};

// red: 2 KiB per wave.
template <typename T>
__device__ __forceinline__ void route_here(const Route<T>& r, int N, int H, int E, int K, TopK* out, double* red) {
  static_assert(kNT == kPairs, "a thread per pair");
  const int t = threadIdx.x, wave = t / kWave, c = lane_id() % 16;
  double v = 0.0;
  if (r.part == nullptr) {
    const T* px = r.x + int64_t(min(c, N - 1)) * H;
    for (int e0 = 0; e0 < E; e0 += 16) {
      f64x4_t acc = {0.0, 0.0, 0.0, 0.0};
      for (int h = wave * 32; h < H; h += kWaves * 32) logit_panel(px, r.w_r, h, E, min(e0 + c, E - 1), acc);
      __syncthreads();
      park_logits(acc, red + wave * 256);
      __syncthreads();
      const int n = t / E, e = t % E - e0;
      if (n < N && e >= 0 && e < 16) {
#pragma unroll
        for (int i = 0; i < kWaves; ++i) v += red[i * 256 + n * 16 + e];
      }
    }
  } else if (t < N * E) {
    v = sum_parts(r.part, 0, N, E, r.S);
  }
  rank_pairs(v, r.bias, N, E, K, out);
  __syncthreads();
}

// ------------------------------------------------------- rows of an expert

// The chosen experts, ascending, and the slots' experts, in LDS.  Workgroups are
// numbered over the chosen experts only: they go to the XCDs in turn by their
// number, so numbers that had nothing to do would leave some XCDs with more
// weights to read than others.
struct Chosen {
  int ids[kSlots];
  int expert[MOE_MAX_EXPERTS];
  int counts[2 * kSlots / kWave];
};

// Builds it; returns the number of chosen experts.  All threads call it.
__device__ __forceinline__ int chosen_experts(const int32_t* __restrict__ topk, int NK, Chosen* c) {
  static_assert(kNT == MOE_MAX_EXPERTS, "a thread per expert");
  const int t = threadIdx.x;
  c->expert[t] = 0;
  __syncthreads();
  for (int i = t; i < NK; i += kNT) {
    const int e = topk[i];
    c->ids[i] = e;
    c->expert[e] = 1;
  }
  __syncthreads();
  const bool mine = c->expert[t] != 0;
  const uint64_t mask = __ballot(mine);
  if (lane_id() == 0) c->counts[t / kWave] = __popcll(mask);
  __syncthreads();
  int active = 0, at = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w == t / kWave) at = active + __popcll(mask & ((uint64_t(1) << lane_id()) - 1));
    active += c->counts[w];
  }
  if (mine) c->expert[at] = t;  // every thread has read its own flag
  __syncthreads();
  return active;
}

// Slots n*K + k of expert e in ascending order to rows[0, count); the count.
// All threads of the workgroup call it.
__device__ __forceinline__ int expert_slots(Chosen* c, int NK, int e, int* rows) {
  constexpr int R = kSlots / kNT;
  const int w = threadIdx.x / kWave;
  bool mine[R];
  uint64_t mask[R];
  __syncthreads();  // rows and counts are free
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int t = r * kNT + threadIdx.x;
    mine[r] = t < NK && c->ids[t] == e;
    mask[r] = __ballot(mine[r]);
    if (lane_id() == 0) c->counts[r * kWaves + w] = __popcll(mask[r]);
  }
  __syncthreads();
  int count = 0;
#pragma unroll
  for (int i = 0; i < R * kWaves; ++i) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (i == r * kWaves + w && mine[r]) {
        // one token names an expert once, so there are at most N <= kTok slots
        const int at = count + __popcll(mask[r] & ((uint64_t(1) << lane_id()) - 1));
        if (at < kTok) rows[at] = r * kNT + threadIdx.x;
      }
    count += c->counts[i];
  }
  __syncthreads();
  return min(count, kTok);
}

// The rows of unit u: the u-th chosen expert's slots; their number, 0 when there
// is no such unit.  One token's experts are its slots as they stand.
__device__ __forceinline__ int unit_rows(const int32_t* __restrict__ topk, int N, int K, int u, Chosen* c, int* e,
                                         int* rows) {
  if (N == 1) {
    if (u >= K) return 0;
    *e = topk[u];
    if (threadIdx.x == 0) rows[0] = u;
    __syncthreads();
    return 1;
  }
  if (u >= chosen_experts(topk, N * K, c)) return 0;
  *e = c->expert[u];
  return expert_slots(c, N * K, *e, rows);
}

// --------------------------------------------------------------- the panels

// A wave's share of a panel: 32 rows x S segments of 16 lanes x 16 bytes, and
// the row operand of 16 rows over the same 32 contraction indices.
template <typename T, int S> struct Panel;

template <int S> struct Panel<bf16_t, S> {
  static constexpr int CW = 8;  // columns per lane and segment
  words4_t w[S][8];
  struct A {
    words4_t a;
    __device__ __forceinline__ void load(const bf16_t* p) { a = *reinterpret_cast<const words4_t*>(p); }
  };
  // float32 values as the sum of three bf16 operands, the bits of a value cut in
  // three, so that the sum is exact and a finite value's parts are finite; stored,
  // each operand lies a plane behind the one before
  struct A2 {
    words4_t hi, mid, lo;
    __device__ __forceinline__ void load(const bf16_t* p, int64_t plane) {
      hi = *reinterpret_cast<const words4_t*>(p);
      mid = *reinterpret_cast<const words4_t*>(p + plane);
      lo = *reinterpret_cast<const words4_t*>(p + 2 * plane);
    }
    __device__ __forceinline__ void store(bf16_t* p, int64_t plane) const {
      *reinterpret_cast<words4_t*>(p) = hi;
      *reinterpret_cast<words4_t*>(p + plane) = mid;
      *reinterpret_cast<words4_t*>(p + 2 * plane) = lo;
    }
    // the upper halves of two floats in one word
    static __device__ __forceinline__ uint32_t upper(const float* r) {
      return __builtin_amdgcn_perm(__float_as_uint(r[1]), __float_as_uint(r[0]), 0x07060302u);
    }
    static __device__ __forceinline__ float rest(float r) { return r - __uint_as_float(__float_as_uint(r) & 0xffff0000u); }
    __device__ __forceinline__ void set(const float* v) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float r[2] = {v[2 * j], v[2 * j + 1]};
        hi[j] = upper(r);
#pragma unroll
        for (int i = 0; i < 2; ++i) r[i] = isfinite(r[i]) ? rest(r[i]) : 0.f;  // an infinite or NaN value is all in hi
        mid[j] = upper(r);
#pragma unroll
        for (int i = 0; i < 2; ++i) r[i] = rest(r[i]);
        lo[j] = upper(r);
      }
    }
  };
  __device__ __forceinline__ void load(const bf16_t* p, int64_t ld) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int s = 0; s < S; ++s)
        w[s][j] = __builtin_nontemporal_load(reinterpret_cast<const words4_t*>(p + j * ld + s * 16 * CW));
  }
  __device__ __forceinline__ bf16x8_t column(int s, int i) const {
    words4_t b;
#pragma unroll
    for (int d = 0; d < 4; ++d)
      b[d] = __builtin_amdgcn_perm(w[s][2 * d + 1][i / 2], w[s][2 * d][i / 2], i % 2 ? 0x07060302u : 0x05040100u);
    return __builtin_bit_cast(bf16x8_t, b);
  }
  static __device__ __forceinline__ void fma(words4_t a, bf16x8_t b, f32x4_t& acc) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), b, acc, 0, 0, 0);
  }
  static __device__ __forceinline__ void fma(const A& a, bf16x8_t b, f32x4_t& acc) { fma(a.a, b, acc); }
  static __device__ __forceinline__ void fma(const A2& a, bf16x8_t b, f32x4_t& acc) {
    fma(a.lo, b, acc);
    fma(a.mid, b, acc);
    fma(a.hi, b, acc);
  }
  template <int MT, typename Op>
  __device__ __forceinline__ void multiply(const Op (&a)[MT], f32x4_t (&acc)[MT][S][CW]) const {
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int i = 0; i < CW; ++i) {
        const bf16x8_t b = column(s, i);
#pragma unroll
        for (int m = 0; m < MT; ++m) fma(a[m], b, acc[m][s][i]);
      }
  }
  // The same for one row tile, rows 4g + r of the sums changing only where
  // keep[r]: a zero row times an infinite or NaN weight is not zero.
  __device__ __forceinline__ void multiply_kept(const A2& a, const bool (&keep)[4], f32x4_t (&acc)[S][CW]) const {
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int i = 0; i < CW; ++i) {
        f32x4_t t = {0.f, 0.f, 0.f, 0.f};
        fma(a, column(s, i), t);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[s][i][r] += keep[r] ? t[r] : 0.f;
      }
  }
};

template <int S> struct Panel<float, S> {
  static constexpr int CW = 4;
  f32x4_t w[S][8];
  struct A {
    float a[8];
    __device__ __forceinline__ void load(const float* p) {
      Vec16<float>::load(p, a);
      Vec16<float>::load(p + 4, a + 4);
    }
    __device__ __forceinline__ void load(const float* p, int64_t) { load(p); }
    __device__ __forceinline__ void store(float* p, int64_t) const {
      Vec16<float>::store(p, a);
      Vec16<float>::store(p + 4, a + 4);
    }
    __device__ __forceinline__ void set(const float* v) {
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = v[j];
    }
  };
  typedef A A2;
  __device__ __forceinline__ void load(const float* p, int64_t ld) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int s = 0; s < S; ++s)
        w[s][j] = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(p + j * ld + s * 16 * CW));
  }
  template <int MT>
  __device__ __forceinline__ void multiply(const A (&a)[MT], f32x4_t (&acc)[MT][S][CW]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < CW; ++i)
#pragma unroll
          for (int m = 0; m < MT; ++m)
            acc[m][s][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[m].a[j], w[s][j][i], acc[m][s][i], 0, 0, 0);
  }
  __device__ __forceinline__ void multiply_kept(const A2& a, const bool (&keep)[4], f32x4_t (&acc)[S][CW]) const {
    f32x4_t t[S][CW];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < CW; ++i)
          t[s][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(a.a[j], w[s][j][i], j == 0 ? f32x4_t{0.f, 0.f, 0.f, 0.f} : t[s][i],
                                                         0, 0, 0);
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int i = 0; i < CW; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[s][i][r] += keep[r] ? t[s][i][r] : 0.f;
  }
};

// Columns of one workgroup: two segments.
template <typename T>
constexpr int kCols = 2 * 16 * Panel<T, 1>::CW;
constexpr int kAlign = 128;  // every dimension but N, E and K is a multiple of it

template <int MT, int S, int CW>
__device__ __forceinline__ void clear(f32x4_t (&acc)[MT][S][CW]) {
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int i = 0; i < CW; ++i) acc[m][s][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
}

// A wave's 16 x 16*CW sums to mine [16][16*CW]: the matrix instruction leaves
// row 4g + r, operand column c in element r.
template <int CW>
__device__ __forceinline__ void park(const f32x4_t (&acc)[CW], float* mine) {
  const int g = lane_id() / 16, c = lane_id() % 16;
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int i = 0; i < CW; i += 4)
      *reinterpret_cast<f32x4_t*>(mine + (4 * g + r) * 16 * CW + c * CW + i) =
          f32x4_t{acc[i][r], acc[i + 1][r], acc[i + 2][r], acc[i + 3][r]};
}

// How the four waves of a workgroup share its columns and its contraction:
//   all split the contraction (the sums of a piece are all waves');
//   JOINT: even waves have W_gate, odd ones W_up;
//   HALVES: the first two waves have the first segment, the others the second,
//   so that twice the row tiles fit the registers and a row's 512 bytes are
//   still read together.
template <bool JOINT, bool HALVES>
struct Role {
  static constexpr int KW = kWaves / (JOINT ? 2 : 1) / (HALVES ? 2 : 1);  // waves along the contraction
  int mat, seg, k;
  __device__ __forceinline__ Role() {
    const int w = threadIdx.x / kWave;
    mat = JOINT ? w % 2 : 0;
    seg = HALVES ? w / 2 : 0;
    k = HALVES ? (JOINT ? 0 : w % 2) : JOINT ? w / 2 : w;
  }
  // wave of a role
  static __device__ __forceinline__ int wave(int mat, int seg, int k) {
    return HALVES ? 2 * seg + (JOINT ? mat : k) : JOINT ? 2 * k + mat : k;
  }
};

// The waves' sums of each 16 x 16*CW piece added in wave order; out(row tile,
// segment, row, first of 4 columns, their sums), with JOINT out(..., first of 8
// columns, their G and U sums as 4 vectors), for all of it.  red: 16 * 16 * CW
// floats per wave.
template <bool JOINT, bool HALVES, int MT, int S, int CW, typename F>
__device__ __forceinline__ void join(const f32x4_t (&acc)[MT][S][CW], float* red, F out) {
  typedef Role<JOINT, HALVES> R;
  constexpr int W = 16 * CW, PIECE = 16 * W, C = JOINT ? 8 : 4;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int s = 0; s < S; ++s) {
      __syncthreads();
      park(acc[m][s], red + threadIdx.x / kWave * PIECE);
      __syncthreads();
      for (int j = C * threadIdx.x; j < (HALVES ? 2 : 1) * PIECE; j += C * kNT) {
        const int h = j / PIECE, i = j % PIECE;
        f32x4_t v[JOINT ? 4 : 1];
#pragma unroll
        for (int n = 0; n < (JOINT ? 4 : 1); ++n) {  // G, U of the first four columns, then of the others
          const float* p = red + i + n / 2 * 4;
          v[n] = *reinterpret_cast<const f32x4_t*>(p + R::wave(n % 2, h, 0) * PIECE);
#pragma unroll
          for (int k = 1; k < R::KW; ++k) v[n] += *reinterpret_cast<const f32x4_t*>(p + R::wave(n % 2, h, k) * PIECE);
        }
        out(m, s + h, i / W, i % W, v);
      }
    }
}

// ------------------------------------------------------------ gate and up

// gate * silu(G) * U of 8 consecutive columns from the parts' sums: part p's G
// at gu + 2*p*stride, its U behind at + stride.  load() before the panel's
// weights are asked for, so that finish() runs while they are on their way.
struct Act {
  float gs[8], us[8];
  __device__ __forceinline__ void load(const float* __restrict__ gu, int64_t stride, int parts) {
    Vec16<float>::load(gu, gs);
    Vec16<float>::load(gu + 4, gs + 4);
    Vec16<float>::load(gu + stride, us);
    Vec16<float>::load(gu + stride + 4, us + 4);
    for (int p = 1; p < parts; ++p) {
      gu += 2 * stride;
      float t[16];
      Vec16<float>::load(gu, t);
      Vec16<float>::load(gu + 4, t + 4);
      Vec16<float>::load(gu + stride, t + 8);
      Vec16<float>::load(gu + stride + 4, t + 12);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        gs[j] += t[j];
        us[j] += t[j + 8];
      }
    }
  }
  // four consecutive ones from sums at hand
  __device__ __forceinline__ void take(int j, f32x4_t g, f32x4_t u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      gs[j + i] = g[i];
      us[j + i] = u[i];
    }
  }
  // The hardware's reciprocal is good to 1 ulp; below 2^-126 it gives 0, an activation
  // of less than 1e-36 of the up product.
  __device__ __forceinline__ void finish(float gate, float* v) const {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = gate * (gs[j] * __builtin_amdgcn_rcpf(1.0f + expf(-gs[j])) * us[j]);
  }
};


// Where the sums of gate and up go.
template <typename T, bool JOINT> struct GuOut;
// One matrix: its sums, [row][ld].
template <typename T> struct GuOut<T, false> {
  float* sums;
};
// Both: the activations, as the down kernels load them ([ld/32][R][32], planes);
// gates null: 1.
template <typename T> struct GuOut<T, true> {
  T* act;
  const float* gates;
  int R;
};

// The token rows: element (row, k) at p[row * row_step + k / 32 * panel_step + k % 32].
template <typename T> struct XRows {
  const T* p;
  int row_step, panel_step;
};

// x times W for up to 16*MT rows (row r: token rows[r] / div) and the columns
// from col0 (S segments, or two with HALVES), part `part` of `parts` of the
// contraction.
template <typename T, int S, int MT, bool JOINT, bool HALVES>
__device__ __forceinline__ void gate_up_rows(const XRows<T>& x, const T* wg, const T* wu, int H, int64_t ld,
                                             int64_t col0, const int* rows, int M, int div, int part, int parts,
                                             const GuOut<T, JOINT>& out, float* red) {
  typedef Panel<T, S> P;
  constexpr int SEG = 16 * P::CW;
  const Role<JOINT, HALVES> role;
  const int g = lane_id() / 16, c = lane_id() % 16;
  f32x4_t acc[MT][S][P::CW];
  clear(acc);
  const T* px[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = 16 * m + c;
    px[m] = x.p + int64_t(rows[r < M ? r : 0] / div) * x.row_step + 8 * g;
  }
  const T* pw = (JOINT && role.mat ? wu : wg) + 8 * g * ld + col0 + role.seg * SEG + P::CW * c;
  if (!HALVES || col0 + role.seg * SEG < ld)
    for (int i = part * role.KW + role.k; i < H / 32; i += parts * role.KW) {
      P p;
      typename P::A a[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) a[m].load(px[m] + int64_t(i) * x.panel_step);
      p.load(pw + int64_t(i) * 32 * ld, ld);
      __builtin_amdgcn_sched_barrier(0);
      p.template multiply<MT>(a, acc);
    }
  join<JOINT, HALVES>(acc, red, [&](int m, int s, int row, int col, const f32x4_t* v) {
    const int r = 16 * m + row;
    const int64_t at = col0 + s * SEG + col;
    if (r >= M || (HALVES && at >= ld)) return;
    if constexpr (JOINT) {
      Act act;
      act.take(0, v[0], v[1]);
      act.take(4, v[2], v[3]);
      float f[8];
      act.finish(out.gates != nullptr ? out.gates[rows[r]] : 1.f, f);
      typename P::A2 o;
      o.set(f);
      o.store(out.act + (at / 32 * out.R + rows[r]) * 32 + at % 32, ld * out.R);
    } else {
      *reinterpret_cast<f32x4_t*>(out.sums + rows[r] * ld + at) = v[0];
    }
  });
}

// All M rows of one expert and the workgroup's columns.
template <typename T, int MTMAX, bool JOINT>
__device__ __forceinline__ void gate_up(const XRows<T>& x, const T* wg, const T* wu, int H, int64_t ld, int64_t col0,
                                        const int* rows, int M, int div, int part, int parts,
                                        const GuOut<T, JOINT>& out, float* red) {
  const bool wide = kCols<T> == kAlign || col0 + kCols<T> <= ld;  // else a last single segment
  if constexpr (MTMAX > 2)
    if (M > 32)
      return M > 48 ? gate_up_rows<T, 1, 4, JOINT, true>(x, wg, wu, H, ld, col0, rows, M, div, part, parts, out, red)
                    : gate_up_rows<T, 1, 3, JOINT, true>(x, wg, wu, H, ld, col0, rows, M, div, part, parts, out, red);
  if constexpr (MTMAX > 1)
    if (M > 16)
      return wide ? gate_up_rows<T, 2, 2, JOINT, false>(x, wg, wu, H, ld, col0, rows, M, div, part, parts, out, red)
                  : gate_up_rows<T, 1, 2, JOINT, false>(x, wg, wu, H, ld, col0, rows, M, div, part, parts, out, red);
  if (wide)
    gate_up_rows<T, 2, 1, JOINT, false>(x, wg, wu, H, ld, col0, rows, M, div, part, parts, out, red);
  else
    gate_up_rows<T, 1, 1, JOINT, false>(x, wg, wu, H, ld, col0, rows, M, div, part, parts, out, red);
}

// What the experts' kernels share.
struct Shape {
  int N, H, F, Fs, E, K;
  int units;     // experts that can be chosen at most
  int gu_parts;  // workgroups that share the contraction over H
  int dn_parts;  // ... over F (N > 16), or over all experts' F (N <= 16)
  int sdn_parts;  // ... over Fs (N > 16)
};

// G and U sums, a workgroup having one matrix's columns and part of its
// contraction: gu [part][2][slot][F], sgu [part][2][token][Fs].  ROUTE: the
// workgroup finds topk and gates itself (one of the shared expert needs none), the
// first of the routed experts writes them.
template <typename T, int MTMAX, bool ROUTE>
__global__ __launch_bounds__(kNT, 2) void k_decode_gate_up(XRows<T> x, const T* __restrict__ wg,
                                                           const T* __restrict__ wu, const T* __restrict__ swg,
                                                           const T* __restrict__ swu, int32_t* __restrict__ topk_out,
                                                           float* __restrict__ gates, Route<T> route,
                                                           float* __restrict__ gu, float* __restrict__ sgu, Shape q) {
  __shared__ Chosen chosen;
  __shared__ int rows[kTok];
  __shared__ __attribute__((aligned(16))) float red[kWaves * 16 * kCols<T> / 2];
  const int32_t* topk = topk_out;
  const int chunks = (q.F + kCols<T> - 1) / kCols<T>;
  const int schunks = (q.Fs + kCols<T> - 1) / kCols<T>, shared = 2 * q.gu_parts * schunks;
  if constexpr (ROUTE) {
    __shared__ TopK routed;
    if (int(blockIdx.x) >= shared) {  // the shared expert needs no choice
      route_here(route, q.N, q.H, q.E, q.K, &routed, reinterpret_cast<double*>(red));
      topk = routed.ids;
      if (int(blockIdx.x) == shared && int(threadIdx.x) < q.N * q.K) {
        topk_out[threadIdx.x] = routed.ids[threadIdx.x];
        gates[threadIdx.x] = routed.gates[threadIdx.x];
      }
    }
  }
  int b = int(blockIdx.x) - shared;
  if (b >= 0) {
    const int chunk = b % chunks;
    b /= chunks;
    const int mat = b % 2, part = b / 2 % q.gu_parts;
    int e = 0;
    const int M = unit_rows(topk, q.N, q.K, b / 2 / q.gu_parts, &chosen, &e, rows);
    if (M == 0) return;
    gate_up<T, MTMAX, false>(x, (mat ? wu : wg) + int64_t(e) * q.H * q.F, nullptr, q.H, q.F,
                             int64_t(chunk) * kCols<T>, rows, M, q.K, part, q.gu_parts,
                             GuOut<T, false>{gu + int64_t(part * 2 + mat) * q.N * q.K * q.F}, red);
  } else {
    b += shared;
    const int chunk = b % schunks;
    b /= schunks;
    const int mat = b % 2, part = b / 2;
    if (threadIdx.x < kTok) rows[threadIdx.x] = threadIdx.x;
    __syncthreads();
    gate_up<T, MTMAX, false>(x, mat ? swu : swg, nullptr, q.H, q.Fs, int64_t(chunk) * kCols<T>, rows, q.N, 1, part,
                             q.gu_parts,
                             GuOut<T, false>{sgu + int64_t(part * 2 + mat) * q.N * q.Fs}, red);
  }
}

// Activations, a workgroup having the same columns of both matrices (two waves
// each) and the whole contraction.
template <typename T, int MTMAX>
__global__ __launch_bounds__(kNT, 2) void k_decode_gate_up_act(XRows<T> x, const T* __restrict__ wg,
                                                               const T* __restrict__ wu, const T* __restrict__ swg,
                                                               const T* __restrict__ swu,
                                                               const int32_t* __restrict__ topk,
                                                               const float* __restrict__ gates,
                                                               T* __restrict__ act, T* __restrict__ sact, Shape q) {
  __shared__ Chosen chosen;
  __shared__ int rows[kTok];
  __shared__ __attribute__((aligned(16))) float red[kWaves * 16 * kCols<T> / 2];
  const int chunks = (q.F + kCols<T> - 1) / kCols<T>;
  const int shared = (q.Fs + kCols<T> - 1) / kCols<T>;
  int b = int(blockIdx.x) - shared;
  if (b >= 0) {
    int e = 0;
    const int M = unit_rows(topk, q.N, q.K, b / chunks, &chosen, &e, rows);
    if (M == 0) return;
    const int64_t at = int64_t(e) * q.H * q.F;
    gate_up<T, MTMAX, true>(x, wg + at, wu + at, q.H, q.F, int64_t(b % chunks) * kCols<T>, rows, M, q.K, 0, 1,
                            GuOut<T, true>{act, gates, q.N * q.K}, red);
  } else {
    b += shared;
    if (threadIdx.x < kTok) rows[threadIdx.x] = threadIdx.x;
    __syncthreads();
    gate_up<T, MTMAX, true>(x, swg, swu, q.H, q.Fs, int64_t(b) * kCols<T>, rows, q.N, 1, 0, 1,
                            GuOut<T, true>{sact, nullptr, q.N}, red);
  }
}

// ------------------------------------------------------------------- down

// The activations of all slots, then of the shared expert's tokens, in the form
// that the down kernels load: act [F/32][slot][32] and sact [Fs/32][token][32],
// three planes for bf16.  A thread has 8 columns.
template <typename T>
__global__ __launch_bounds__(256) void k_decode_act(const float* __restrict__ gu, const float* __restrict__ sgu,
                                                    const float* __restrict__ gates, T* __restrict__ act,
                                                    T* __restrict__ sact, Shape q) {
  const int64_t NK = int64_t(q.N) * q.K, routed = NK * (q.F / 8), all = routed + int64_t(q.N) * (q.Fs / 8);
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < all; i += int64_t(gridDim.x) * 256) {
    const bool sh = i >= routed;
    const int64_t at = (sh ? i - routed : i) * 8, R = sh ? q.N : NK, F = sh ? q.Fs : q.F;
    const int64_t panel = at / (32 * R);
    const int row = int(at % (32 * R)) / 32;
    Act a;
    float v[8];
    a.load((sh ? sgu : gu) + row * F + panel * 32 + at % 32, R * F, q.gu_parts);
    a.finish(sh ? 1.f : gates[row], v);
    typename Panel<T, 1>::A2 o;
    o.set(v);
    o.store((sh ? sact : act) + at, R * F);
  }
}

// One expert's rows (slots rows[0, M)) times its W_down, part `part` of `parts` of
// the contraction: sums to out[rows[r]][H].
template <typename T, int S, int MT, bool HALVES>
__device__ __forceinline__ void down_rows(const T* __restrict__ act, int64_t plane, const T* wd, int F, int64_t H,
                                          int64_t col0, const int* rows, int M, int part, int parts, float* out,
                                          float* red) {
  typedef Panel<T, S> P;
  constexpr int SEG = 16 * P::CW;
  const Role<false, HALVES> role;
  const int g = lane_id() / 16, c = lane_id() % 16;
  f32x4_t acc[MT][S][P::CW];
  clear(acc);
  const T* pa[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) pa[m] = act + rows[16 * m + c < M ? 16 * m + c : 0] * 32 + 8 * g;
  const T* pw = wd + 8 * g * H + col0 + role.seg * SEG + P::CW * c;
  if (!HALVES || col0 + role.seg * SEG < H)
    for (int i = part * role.KW + role.k; i < F / 32; i += parts * role.KW) {
      P p;
      typename P::A2 a[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) a[m].load(pa[m] + int64_t(i) * 32 * (plane / F), plane);
      p.load(pw + int64_t(i) * 32 * H, H);
      __builtin_amdgcn_sched_barrier(0);
      p.template multiply<MT>(a, acc);
    }
  join<false, HALVES>(acc, red, [&](int m, int s, int row, int col, const f32x4_t* v) {
    const int r = 16 * m + row;
    const int64_t at = col0 + s * SEG + col;
    if (r < M && (!HALVES || at < H)) *reinterpret_cast<f32x4_t*>(out + rows[r] * H + at) = v[0];
  });
}

template <typename T, int MTMAX>
__device__ __forceinline__ void down(const T* __restrict__ act, int64_t plane, const T* wd, int F, int64_t H,
                                     int64_t col0, const int* rows, int M, int part, int parts, float* out,
                                     float* red) {
  const bool wide = kCols<T> == kAlign || col0 + kCols<T> <= H;
  if constexpr (MTMAX > 2)
    if (M > 32)
      return M > 48 ? down_rows<T, 1, 4, true>(act, plane, wd, F, H, col0, rows, M, part, parts, out, red)
                    : down_rows<T, 1, 3, true>(act, plane, wd, F, H, col0, rows, M, part, parts, out, red);
  if (M > 16)
    return wide ? down_rows<T, 2, 2, false>(act, plane, wd, F, H, col0, rows, M, part, parts, out, red)
                : down_rows<T, 1, 2, false>(act, plane, wd, F, H, col0, rows, M, part, parts, out, red);
  if (wide)
    down_rows<T, 2, 1, false>(act, plane, wd, F, H, col0, rows, M, part, parts, out, red);
  else
    down_rows<T, 1, 1, false>(act, plane, wd, F, H, col0, rows, M, part, parts, out, red);
}

// More than 16 tokens: a workgroup has one expert's columns and part of its
// contraction; ysp [part][slot][H], then sysp [part][token][H].
template <typename T, int MTMAX>
__global__ __launch_bounds__(kNT, 2) void k_decode_down(const T* __restrict__ act, const T* __restrict__ sact,
                                                        const T* __restrict__ wd, const T* __restrict__ swd,
                                                        const int32_t* __restrict__ topk, float* __restrict__ ysp,
                                                        float* __restrict__ sysp, Shape q) {
  __shared__ Chosen chosen;
  __shared__ int rows[kTok];
  __shared__ __attribute__((aligned(16))) float red[kWaves * 16 * kCols<T> / 2];
  const int chunks = (q.H + kCols<T> - 1) / kCols<T>;
  int b = blockIdx.x;
  const int64_t col0 = int64_t(b % chunks) * kCols<T>;
  b /= chunks;
  b -= q.sdn_parts;
  if (b >= 0) {
    const int part = b % q.dn_parts, u = b / q.dn_parts;
    int e = 0;
    const int M = unit_rows(topk, q.N, q.K, u, &chosen, &e, rows);
    if (M == 0) return;
    down<T, MTMAX>(act, int64_t(q.N) * q.K * q.F, wd + int64_t(e) * q.F * q.H, q.F, q.H, col0, rows, M, part, q.dn_parts,
                   ysp + int64_t(part) * q.N * q.K * q.H, red);
  } else {
    const int part = b + q.sdn_parts;
    if (threadIdx.x < kTok) rows[threadIdx.x] = threadIdx.x;
    __syncthreads();
    down<T, MTMAX>(sact, int64_t(q.N) * q.Fs, swd, q.Fs, q.H, col0, rows, q.N, part, q.sdn_parts,
                   sysp + int64_t(part) * q.N * q.H, red);
  }
}

// Where k_decode_down_all finds the activations: FUSED, in the sums of gate and
// up (formed here, once per workgroup that needs them: for few tokens cheaper
// than a launch), else as k_decode_act left them.
template <typename T, bool FUSED> struct Rows;
template <typename T> struct Rows<T, true> {
  const float *gu, *sgu;
};
template <typename T> struct Rows<T, false> {
  const T *act, *sact;
};

// At most 16 tokens: the row operand's rows are the tokens themselves, zero
// where a token did not choose the panel's expert, so that the sum over the
// experts is part of the contraction.  All panels of the chosen experts (and of
// the shared one) are dealt evenly to the waves of dn_parts workgroups; yp
// [part][token][H], added up by a launch of its own: the strip's last workgroup
// could do it, but the fence that each of its waves needs first costs more (one
// token, H 512, F 1024, 8 experts: 18.5 us so, 17.9 with the launch; float32 20.7
// and 18.4).
template <typename T, int S, bool FUSED>
__device__ __forceinline__ void down_all(const Rows<T, FUSED>& in, const T* __restrict__ wd,
                                         const T* __restrict__ swd, const Shape& q, int64_t col0, const int* expert,
                                         const int16_t (*slot)[16], const float* gate, int active, int part,
                                         float* yp, float* red) {
  typedef Panel<T, S> P;
  const int wave = threadIdx.x / kWave, g = lane_id() / 16, c = lane_id() % 16;
  const int64_t H = q.H, plane = int64_t(q.N) * q.K * q.F, splane = int64_t(q.N) * q.Fs;
  f32x4_t acc[1][S][P::CW];
  clear(acc);
  const int per = q.F / 32, routed = active * per, all = routed + q.Fs / 32;
  const int64_t lane0 = 8 * g * H + col0 + P::CW * c;
  for (int i = part * kWaves + wave; i < all; i += q.dn_parts * kWaves) {
    const bool sh = i >= routed;
    const int u = sh ? 0 : i / per, f = (sh ? i - routed : i % per) * 32;
    const int row = sh ? (c < q.N ? c : -1) : slot[u][c];  // -1: no such row
    const int64_t at = FUSED ? int64_t(row < 0 ? 0 : row) * (sh ? q.Fs : q.F) + f + 8 * g
                             : int64_t(f) * (sh ? q.N : q.N * q.K) + (row < 0 ? 0 : row) * 32 + 8 * g;
    P p;
    typename P::A2 a[1];
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    a[0].set(v);
    const T* pw = (sh ? swd + int64_t(f) * H : wd + (int64_t(expert[u]) * q.F + f) * H) + lane0;
    if constexpr (FUSED) {
      Act act;
      if (row >= 0) act.load((sh ? in.sgu : in.gu) + at, sh ? splane : plane, q.gu_parts);
      p.load(pw, H);
      __builtin_amdgcn_sched_barrier(0);
      if (row >= 0) {
        act.finish(sh ? 1.f : gate[row], v);
        a[0].set(v);
      }
    } else {
      if (row >= 0) a[0].load((sh ? in.sact : in.act) + at, sh ? splane : plane);
      p.load(pw, H);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (q.N == 1 || sh) {  // every row that counts has this expert
      p.template multiply<1>(a, acc);
    } else {
      bool keep[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) keep[r] = slot[u][4 * g + r] >= 0;
      p.multiply_kept(a[0], keep, acc[0]);
    }
  }
  join<false, false>(acc, red, [&](int, int s, int row, int col, const f32x4_t* v) {
    if (row < q.N)
      *reinterpret_cast<f32x4_t*>(yp + (int64_t(part) * q.N + row) * H + col0 + s * 16 * P::CW + col) = v[0];
  });
}

template <typename T, bool FUSED>
__global__ __launch_bounds__(kNT, 2) void k_decode_down_all(Rows<T, FUSED> in, const T* __restrict__ wd,
                                                            const T* __restrict__ swd,
                                                            const int32_t* __restrict__ topk,
                                                            const float* __restrict__ gates, float* __restrict__ yp,
                                                            Shape q) {
  constexpr int SL = 16 * MOE_MAX_TOPK;
  __shared__ int expert[SL];
  __shared__ int16_t slot[SL][16];
  __shared__ float gate[SL];
  __shared__ int ids[SL], unit[SL], counts[kWaves];
  __shared__ __attribute__((aligned(16))) float red[kWaves * 16 * kCols<T> / 2];
  const int NK = q.N * q.K, t = threadIdx.x;
  static_assert(SL <= kNT, "a thread per slot");
  if (t < NK) {
    ids[t] = topk[t];
    gate[t] = gates[t];
  }
  for (int i = t; i < NK * 16; i += kNT) slot[i / 16][i % 16] = -1;
  __syncthreads();
  int active = NK;
  if (q.N == 1) {  // its slots are its experts
    if (t < NK) {
      expert[t] = ids[t];
      slot[t][0] = int16_t(t);
    }
  } else {
    // a slot's unit: how many experts' first slots come before its expert's first slot
    int first = t;
    if (t < NK)
      for (first = 0; ids[first] != ids[t]; ++first) {}
    const bool head = t < NK && first == t;
    const uint64_t heads = __ballot(head);
    if (lane_id() == 0) counts[t / kWave] = __popcll(heads);
    __syncthreads();
    active = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w == t / kWave && head) unit[t] = active + __popcll(heads & ((uint64_t(1) << lane_id()) - 1));
      active += counts[w];
    }
    __syncthreads();
    if (t < NK) {
      expert[unit[first]] = ids[t];  // the same value from all of the expert's slots
      slot[unit[first]][t / q.K] = int16_t(t);
    }
  }
  __syncthreads();
  const int chunks = (q.H + kCols<T> - 1) / kCols<T>;
  const int64_t col0 = int64_t(blockIdx.x % chunks) * kCols<T>;
  const int part = blockIdx.x / chunks;
  if (kCols<T> == kAlign || col0 + kCols<T> <= q.H)
    down_all<T, 2, FUSED>(in, wd, swd, q, col0, expert, slot, gate, active, part, yp, red);
  else
    down_all<T, 1, FUSED>(in, wd, swd, q, col0, expert, slot, gate, active, part, yp, red);
}

// y[n] = sum over the parts of a token's `per` rows (+ the shared expert's
// parts), float32, one rounding.  64 columns a workgroup; thread (slice, column)
// sums every fourth row, eight loads in flight, and the slices meet in order.
template <typename T>
__global__ __launch_bounds__(256) void k_decode_combine(const float* __restrict__ ysp, const float* __restrict__ sysp,
                                                        T* __restrict__ y, int N, int H, int per, int parts,
                                                        int sparts) {
  __shared__ float s[4][64];
  const int col = threadIdx.x % 64, slice = threadIdx.x / 64;
  const int h = blockIdx.x * 64 + col, n = blockIdx.y;
  const int routed = per * parts, all = routed + sparts;
  float v = 0.f;
  for (int i0 = slice; i0 < all; i0 += 32) {
    float t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + 4 * j;
      const float* p = i < routed ? ysp + (int64_t(i / per) * N + n) * per * H + int64_t(i % per) * H
                                  : sysp + (int64_t(i - routed) * N + n) * H;
      t[j] = i < all ? p[h] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v += t[j];
  }
  s[slice][col] = v;
  __syncthreads();
  if (slice == 0) y[int64_t(n) * H + h] = Elt<T>::from_f32(((s[0][col] + s[1][col]) + s[2][col]) + s[3][col]);
}

// ------------------------------------------------------------------- host

// How the call is cut up, and where its scratch lies.
struct Plan {
  Shape q;
  int logit_parts;
  bool few;    // at most 16 tokens: k_decode_down_all
  bool joint;  // k_decode_gate_up_act; else k_decode_gate_up, and then
  bool route;  // ... which finds topk itself, and with logit_parts == 0 the logits too
  bool fused;  // k_decode_down_all forms the activations itself, else k_decode_act does
  size_t logits, xp, gu, sgu, act, sact, ysp, sysp, bytes;
};

constexpr int64_t kCUs = 256;

// The number of experts that N tokens choose.
struct Used {
  double mean;  // if they choose evenly
  double most;
};

// Workgroups (max_parts at most) that share a strip of `panels` panels when an
// expert has `per` strips and the shared one `shared`, by the time that this
// would take in us:
//  - A CU reads its workgroups' panels at about 31 bytes a nanosecond (0.5 us for
//    the 16 KiB of a panel), and the CU with most of them sets the time; all
//    together read no faster than HBM (0.56 us).  Nothing covers a workgroup's
//    start and end when it is alone on its CU (2%).
//  - 1.2 us of latency for each of a wave's first panels, 1 us when workgroups
//    follow those that a CU holds at a time (`fit`).
//  - part_cost for writing and adding up one part more.
// It is the mean over the expected number of experts and a tenth more and less, as
// the fullest CU's count jumps.  Over 54 sizes the cut so found cost 0.5 % more than
// the best one of each on average, 5 % at most; the fullest CU alone, without the
// other terms, 2 % and 15 %.  Strips of other widths would even the CUs out better,
// but a row segment that is not 256 bytes, aligned, reads a third slower.
struct Cut {
  int parts;
  double us;
};
Cut cut(const Used& used, double per, double shared, int64_t panels, int max_parts, double fit, double part_cost) {
  Cut best = {1, 0.0};
  for (int p = 1; p <= max_parts && (p == 1 || kWaves * p <= panels); ++p) {
    const int64_t longest = (panels + kWaves * p - 1) / (kWaves * p);  // panels of a workgroup's busiest wave
    double t = 0.0;
    for (const double u : {std::max(1.0, 0.9 * used.mean), used.mean, std::min(used.most, 1.1 * used.mean)}) {
      const double per_cu = (u * per + shared) * p / double(kCUs);
      const double turns = std::ceil(per_cu) * (per_cu <= 1.0 ? 1.02 : 1.0);
      t += std::max(0.5 * turns * double(kWaves * longest), 0.56 * per_cu * double(panels) / p) + std::ceil(per_cu / fit);
    }
    t = t / 3.0 + 1.2 * double(std::min<int64_t>(4, longest)) + part_cost * (p - 1);
    if (p == 1 || t < best.us) best = {p, t};
  }
  return best;
}

template <typename T>
Plan plan_t(const moe_launch::Dims& d, int64_t Fs) {
  constexpr int cols = kCols<T>;
  Plan p;
  Shape& q = p.q;
  q = Shape{};
  q.N = int(d.N); q.H = int(d.H); q.F = int(d.F); q.Fs = int(Fs); q.E = int(d.E); q.K = int(d.K);
  const int64_t NK = d.NK();
  const int64_t fchunks = (d.F + cols - 1) / cols, schunks = (Fs + cols - 1) / cols, chunks = (d.H + cols - 1) / cols;
  q.units = int(std::min(NK, d.E));
  const Used used{double(d.E) * (1.0 - std::pow(1.0 - double(d.K) / double(d.E), double(d.N))), double(q.units)};
  p.few = d.N <= 16;
  // Up to 16 tokens every strip of the down product reads all parts of its rows' sums; beyond, one
  // kernel does, once.
  const double row_elements = 1e-5 * double(NK * d.F + d.N * Fs);
  const double fit = p.few ? 3.0 : 2.0;
  const Cut apart = cut(used, 2.0 * double(fchunks), 2.0 * double(schunks), d.H / 32, 4, fit,
                        p.few ? 3.0 + 3.0 * row_elements : 0.5 + 0.5 * row_elements);
  // Both matrices in one workgroup spare the sums of G and U their way through memory, and the
  // workgroups that load them the activations, but leave half as many strips to spread.  20 tokens
  // of 8 experts (H 4096, F 14336): 431 us so, 440 apart; 64 of them 483 and 509; 16 tokens of 16
  // experts (H 2048, F 6400): 222 and 228; 64 tokens of 64 experts (H 2048, F 1408): 209 and 207;
  // with two rows an expert (8 tokens of 8 experts) 424 and 416; 12 tokens of 10 experts (H 640,
  // F 7168, K 8) 85 and 78.
  const Cut both = cut(used, double(fchunks), double(schunks), d.H / 16, 1, fit, 0.0);
  p.joint = NK >= 4 * q.units && both.us <= (p.few ? 1.08 * apart.us : 1.05 * apart.us + 0.9 * row_elements);
  q.gu_parts = p.joint ? 1 : apart.parts;
  p.fused = p.few && !p.joint && d.N * q.gu_parts <= 32;
  // Each workgroup of gate/up ranks the pairs (token, expert) for itself while there is one a
  // thread at most: 1 to 4 us less than with a launch for it (4 tokens, 16 experts: 27.2
  // against 28.9; 4 tokens, 64 experts: 76 against 78), but with two pairs a thread 123 against
  // 122 (8 tokens, 64 experts), with four 164 against 160.
  p.route = p.few && !p.joint && d.N * d.E <= kPairs;
  // The logits too where the router is a few panels (18.3 us against 20.3 with the logits'
  // launch at one token, H 512 and 8 experts, 23.4 against 25.0 at three; 27.4 against 27.1 at
  // four tokens, H 1024 and 16 experts).
  const bool small_router = (d.E + 15) / 16 * (d.H / 32) <= 4 * kWaves;
  p.logit_parts = p.route && small_router ? 0 : int((d.H + kLogitRows - 1) / kLogitRows);
  if (p.few) {
    const double panels = used.mean * double(d.F / 32) + double(Fs / 32);
    const int64_t want = std::max(kCUs / chunks, int64_t(panels / (4 * kWaves)));
    q.dn_parts = int(std::max<int64_t>(1, std::min({int64_t(panels / kWaves), 2 * kCUs / chunks, want})));
  } else {
    // Two workgroups fit a CU (row tiles take the registers).  A longer shared strip is cut
    // more often, but all of them into no more pieces than CUs (64 tokens, H 2048, F 128,
    // Fs 32768: 127 us so, 177 without the bound).
    q.dn_parts = cut(used, double(chunks), double(chunks) * double(Fs) / double(d.F), d.F / 32, 16, 2.0,
                     0.1 + 7.5e-6 * double(NK * d.H)).parts;
    const int64_t longer = q.dn_parts * ((Fs + d.F - 1) / d.F), most = std::max<int64_t>(kCUs / chunks, 1);
    q.sdn_parts = int(std::min({Fs / (32 * kWaves), longer, most}));
  }
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += (n + 255) & ~size_t(255);
    return here;
  };
  p.logits = take(size_t(p.logit_parts) * d.N * d.E * sizeof(double));
  p.xp = take(size_t(d.N) * d.H * sizeof(T));
  p.gu = take(p.joint ? 0 : size_t(q.gu_parts) * 2 * NK * d.F * 4);
  p.sgu = take(p.joint ? 0 : size_t(q.gu_parts) * 2 * d.N * Fs * 4);
  constexpr size_t act = sizeof(T) == 2 ? 3 * sizeof(T) : sizeof(T);  // bytes of an activation: Panel<T, S>::A2
  p.act = take(p.fused ? 0 : size_t(NK) * d.F * act);
  p.sact = take(p.fused ? 0 : size_t(d.N) * Fs * act);
  p.ysp = take(size_t(q.dn_parts) * (p.few ? d.N : NK) * d.H * 4);
  p.sysp = take(p.few ? 0 : size_t(q.sdn_parts) * d.N * d.H * 4);
  p.bytes = at;
  return p;
}

// Pointers of one call.
template <typename T> struct Args {
  const T *x, *w_r;
  const float* bias;
  const T *wg, *wu, *wd, *swg, *swu, *swd;
  int32_t* topk;
  float* gates;
  T* y;
  char* ws;
};

#define MOE_LAUNCHED()                 \
  {                                    \
    const hipError_t e = hipGetLastError(); \
    if (e != hipSuccess) return e;     \
  }

template <typename T, int MTMAX>
hipError_t decode_experts(const Plan& p, const Args<T>& a, hipStream_t s) {
  const Shape& q = p.q;
  constexpr int cols = kCols<T>;
  const unsigned chunks = (q.H + cols - 1) / cols;
  float* gu = reinterpret_cast<float*>(a.ws + p.gu);
  float* sgu = reinterpret_cast<float*>(a.ws + p.sgu);
  T* act = reinterpret_cast<T*>(a.ws + p.act);
  T* sact = reinterpret_cast<T*>(a.ws + p.sact);
  float* ysp = reinterpret_cast<float*>(a.ws + p.ysp);
  float* sysp = reinterpret_cast<float*>(a.ws + p.sysp);
  const T* xp = reinterpret_cast<const T*>(a.ws + p.xp);
  const XRows<T> x = p.logit_parts > 0 ? XRows<T>{xp, 32, 32 * q.N} : XRows<T>{a.x, q.H, 32};
  const Route<T> route{a.x, a.w_r, p.logit_parts > 0 ? reinterpret_cast<const double*>(a.ws + p.logits) : nullptr,
                       a.bias, p.logit_parts};
  const unsigned strips = 2 * (unsigned(q.units) * ((q.F + cols - 1) / cols) + (q.Fs + cols - 1) / cols) * q.gu_parts;
  if (p.joint) {
    k_decode_gate_up_act<T, MTMAX><<<dim3(strips / 2), dim3(kNT), 0, s>>>(x, a.wg, a.wu, a.swg, a.swu, a.topk, a.gates,
                                                                          act, sact, q);
  } else {
    bool done = false;
    if constexpr (MTMAX == 1)
      if (p.route) {
        k_decode_gate_up<T, 1, true><<<dim3(strips), dim3(kNT), 0, s>>>(x, a.wg, a.wu, a.swg, a.swu, a.topk, a.gates,
                                                                        route, gu, sgu, q);
        done = true;
      }
    if (!done)
      k_decode_gate_up<T, MTMAX, false><<<dim3(strips), dim3(kNT), 0, s>>>(
          x, a.wg, a.wu, a.swg, a.swu, a.topk, a.gates, route, gu, sgu, q);
    MOE_LAUNCHED()
    if (!p.fused) {
      const int64_t groups = (int64_t(q.N) * q.K * q.F + int64_t(q.N) * q.Fs) / 8;
      k_decode_act<T><<<dim3(unsigned(std::min<int64_t>((groups + 255) / 256, 1 << 16))), dim3(256), 0, s>>>(
          gu, sgu, a.gates, act, sact, q);
    }
  }
  MOE_LAUNCHED()
  if constexpr (MTMAX == 1) {
    const dim3 grid(chunks * q.dn_parts);
    if (p.fused)
      k_decode_down_all<T, true><<<grid, dim3(kNT), 0, s>>>(Rows<T, true>{gu, sgu}, a.wd, a.swd, a.topk, a.gates, ysp,
                                                            q);
    else
      k_decode_down_all<T, false><<<grid, dim3(kNT), 0, s>>>(Rows<T, false>{act, sact}, a.wd, a.swd, a.topk, a.gates,
                                                             ysp, q);
  } else {
    k_decode_down<T, MTMAX><<<dim3((q.units * q.dn_parts + q.sdn_parts) * chunks), dim3(kNT), 0, s>>>(
        act, sact, a.wd, a.swd, a.topk, ysp, sysp, q);
  }
  MOE_LAUNCHED()
  k_decode_combine<T><<<dim3(q.H / 64, q.N), dim3(256), 0, s>>>(ysp, sysp, a.y, q.N, q.H, MTMAX == 1 ? 1 : q.K,
                                                                q.dn_parts, MTMAX == 1 ? 0 : q.sdn_parts);
  return hipGetLastError();
}

template <typename T>
hipError_t decode_t(const moe_launch::Dims& d, int64_t Fs, const Args<T>& a, hipStream_t s) {
  const Plan p = plan_t<T>(d, Fs);
  const Shape& q = p.q;
  double* logits = reinterpret_cast<double*>(a.ws + p.logits);
  if (p.logit_parts > 0) {
    k_decode_logits<T><<<dim3(p.logit_parts, (q.E + 15) / 16, (q.N + 15) / 16), dim3(kLogitWaves * kWave), 0, s>>>(
        a.x, a.w_r, logits, reinterpret_cast<T*>(a.ws + p.xp), q.N, q.H, q.E);
    MOE_LAUNCHED()
  }
  if (!p.route) {
    k_decode_topk<<<dim3(q.N), dim3(256), 0, s>>>(logits, a.bias, a.topk, a.gates, q.N, q.E, q.K, p.logit_parts);
    MOE_LAUNCHED()
  }
  if (q.N <= 16) return decode_experts<T, 1>(p, a, s);
  if (q.N <= 32) return decode_experts<T, 2>(p, a, s);
  return decode_experts<T, 4>(p, a, s);
}

}  // namespace

namespace moe_launch {

size_t decode_ws(const Dims& d, int64_t Fs) {
  return d.dtype == MOE_BF16 ? plan_t<bf16_t>(d, Fs).bytes : plan_t<float>(d, Fs).bytes;
}

hipError_t decode(const Dims& d, const void* x, const void* w_r, const float* bias, const void* wg, const void* wu,
                  const void* wd, int64_t Fs, const void* swg, const void* swu, const void* swd, int32_t* topk,
                  float* gates, void* y, void* ws, hipStream_t s) {
#define MOE_DECODE(T)                                                                                              \
  decode_t<T>(d, Fs, Args<T>{static_cast<const T*>(x), static_cast<const T*>(w_r), bias, static_cast<const T*>(wg),  \
                             static_cast<const T*>(wu), static_cast<const T*>(wd), static_cast<const T*>(swg),     \
                             static_cast<const T*>(swu), static_cast<const T*>(swd), topk, gates,                  \
                             static_cast<T*>(y), static_cast<char*>(ws)}, s)
  return d.dtype == MOE_BF16 ? MOE_DECODE(bf16_t) : MOE_DECODE(float);
#undef MOE_DECODE
}

}  // namespace moe_launch
