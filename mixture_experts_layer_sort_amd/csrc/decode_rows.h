// What the layer for few tokens does whatever the form of its experts' weights:
// router logits in float64, top-K and gates, the sum of a token's rows.
#pragma once

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
// first workgroup of each row range and token tile also packs x as the products
// want it (Pack).  The token tiles are workgroups of their own: 64 tokens take
// 5 us so, 9 in a loop.
template <typename T, typename Pack>
__global__ __launch_bounds__(kLogitWaves * kWave) void k_decode_logits(const T* __restrict__ x,
                                                                      const T* __restrict__ w_r,
                                                                      double* __restrict__ part, Pack pack,
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
    if (blockIdx.y == 0 && n == n0 + c) pack(px + h + 8 * g, n, h + 8 * g, N, H);
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

// ---------------------------------------------------------------- combine

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

}  // namespace
