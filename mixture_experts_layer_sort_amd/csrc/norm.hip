// Root-mean-square norm of the token rows with the residual's addition, the
// step in front of the layer, and its backward.
//
// Forward, row n:
//   h = x (+ residual), stored rounded to the element type;
//   rstd = 1 / sqrt(mean(h^2) + eps), y = h * rstd * weight   (from the stored h).
// Backward, with dh the gradient that reaches h along the residual stream:
//   t = dy * weight, xhat = h * rstd,
//   dx = rstd * (t - xhat * mean(t * xhat)) (+ dh)     (also the residual's gradient),
//   dweight = sum_n dy * xhat.
// Every sum is float32 or wider; h, y and dx are rounded once each.
//
// A row stays in registers between its one read and its write, so memory
// traffic is the inputs and outputs alone and HBM bounds both directions.  A
// row belongs to one wave, or 16 or 32 lanes of one, while it has at most 256
// 16-byte vectors (no LDS, no barrier), else to a workgroup.  In the backward a workgroup walks over many
// rows and keeps its share of dweight in registers; the workgroups' partial
// sums are added in a fixed order by a second kernel, so results do not depend
// on timing.
#include <algorithm>

#include "common.h"

namespace {
using namespace moe;

// Workgroups of the backward: each leaves a row of H float32 partial sums.  Three
// per CU: 108 us for a training step of 16383 x 2048 bf16 rows (512: 109, 896:
// 115, 1024: 116).
constexpr int kNormBwdBlocks = 768;
// Workgroups of the forward at most (threads in a grid are counted in 32 bits).
constexpr int64_t kNormMaxBlocks = 1 << 20;

// Sum over the threads that share a row (NT up to 64: lanes of a wave), the same
// in each of them.  s: one float per wave.
template <int NT>
__device__ __forceinline__ float row_sum(float v, float* s) {
  if constexpr (NT < kWave) {
#pragma unroll
    for (int off = NT / 2; off > 0; off >>= 1) v += __shfl_xor(v, off, NT);
    return v;
  }
  v = wave_sum(v);
  if constexpr (NT > kWave) {
    __syncthreads();  // s is free again
    if (lane_id() == 0) s[threadIdx.x / kWave] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < NT / kWave; ++i) v += s[i];
  }
  return v;
}

typedef uint32_t raw_t __attribute__((ext_vector_type(4)));

// 16 bytes of a row.  STREAM: past the caches, for tensors that the last-level
// cache (256 MB) would not keep until their next use anyway.  Measured both ways
// at 8192 x 7168 bf16: 82 us with the hint on x, residual, h and y, 92 without;
// smaller calls leave h and y in the cache for the layer that reads them next.
template <bool STREAM, typename T>
__device__ __forceinline__ void load_row(const T* p, float* v) {
  const raw_t* q = reinterpret_cast<const raw_t*>(p);
  const raw_t r = STREAM ? __builtin_nontemporal_load(q) : *q;
  Vec16<T>::load(reinterpret_cast<const T*>(&r), v);
}
template <bool STREAM, typename T>
__device__ __forceinline__ void store_row(T* p, const float* v) {
  raw_t r;
  Vec16<T>::store(reinterpret_cast<T*>(&r), v);
  if (STREAM)
    __builtin_nontemporal_store(r, reinterpret_cast<raw_t*>(p));
  else
    *reinterpret_cast<raw_t*>(p) = r;
}
constexpr int64_t kStreamBytes = 32 << 20;  // of one tensor

// h may be x or residual itself (each element is read before it is written).
template <typename T, int NT, int VPT, bool STREAM>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void k_norm(const T* x, const T* residual,
                                                             const T* __restrict__ weight, T* h,
                                                             T* __restrict__ y, float* __restrict__ rstd, int64_t N,
                                                             int H, float eps) {
  constexpr int V = Vec16<T>::n;
  constexpr int RPB = NT < 256 ? 256 / NT : 1;  // rows per workgroup
  __shared__ float s[NT > kWave ? NT / kWave : 1];
  const int t = threadIdx.x % NT;
  const int nv = H / V;
  // waves of one workgroup may end at different rows: they share no barrier then
  for (int64_t n = (int64_t)blockIdx.x * RPB + threadIdx.x / NT; n < N; n += (int64_t)gridDim.x * RPB) {
    const int64_t base = n * H;
    float v[VPT][V];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * NT;
      if (c < nv) load_row<STREAM>(x + base + c * V, v[i]);
    }
    if (residual != nullptr) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = t + i * NT;
        if (c < nv) {
          float r[V];
          load_row<STREAM>(residual + base + c * V, r);
#pragma unroll
          for (int j = 0; j < V; ++j) v[i][j] = Elt<T>::to_f32(Elt<T>::from_f32(v[i][j] + r[j]));
          store_row<STREAM>(h + base + c * V, v[i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (t + i * NT < nv)
#pragma unroll
        for (int j = 0; j < V; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    ss = row_sum<NT>(ss, s);
    const float r = 1.0f / sqrtf(ss / float(H) + eps);
    if (t == 0 && rstd != nullptr) rstd[n] = r;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * NT;
      if (c < nv) {
        float w[V];
        Vec16<T>::load(weight + c * V, w);
#pragma unroll
        for (int j = 0; j < V; ++j) w[j] *= v[i][j] * r;
        store_row<STREAM>(y + base + c * V, w);
      }
    }
  }
}

// dx may be dy or dh itself.  part [gridDim.x][H].
template <typename T, int NT, int VPT, bool STREAM>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void k_norm_bwd(const T* dy, const T* __restrict__ h,
                                                                 const T* __restrict__ weight,
                                                                 const float* __restrict__ rstd, const T* dh, T* dx,
                                                                 float* __restrict__ part, int64_t N, int H) {
  constexpr int V = Vec16<T>::n;
  constexpr int RPB = NT < 256 ? 256 / NT : 1;
  __shared__ float s[NT > kWave ? NT / kWave : 1];
  const int t = threadIdx.x % NT;
  const int nv = H / V;
  float dw[VPT][V];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) dw[i][j] = 0.f;
  for (int64_t n = (int64_t)blockIdx.x * RPB + threadIdx.x / NT; n < N; n += (int64_t)gridDim.x * RPB) {
    const int64_t base = n * H;
    const float r = rstd[n];
    float g[VPT][V], xh[VPT][V];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * NT;
      if (c < nv) {
        load_row<STREAM>(dy + base + c * V, g[i]);
        load_row<STREAM>(h + base + c * V, xh[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * NT;
      if (c < nv) {
        float w[V];
        Vec16<T>::load(weight + c * V, w);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          xh[i][j] *= r;
          dw[i][j] = fmaf(g[i][j], xh[i][j], dw[i][j]);
          g[i][j] *= w[j];
          dot = fmaf(g[i][j], xh[i][j], dot);
        }
      }
    }
    dot = row_sum<NT>(dot, s) / float(H);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * NT;
      if (c < nv) {
        float a[V];
#pragma unroll
        for (int j = 0; j < V; ++j) a[j] = 0.f;
        if (dh != nullptr) Vec16<T>::load(dh + base + c * V, a);  // without the hint: 52 us, with it 56 (16383 x 2048 bf16)
#pragma unroll
        for (int j = 0; j < V; ++j) a[j] = fmaf(r, g[i][j] - xh[i][j] * dot, a[j]);
        store_row<STREAM>(dx + base + c * V, a);
      }
    }
  }
  if constexpr (RPB > 1) {
    // the waves' sums, added in wave order
    __shared__ float sw[VPT * NT * V];
    for (int q = 0; q < RPB; ++q) {
      if ((int)threadIdx.x / NT == q)
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j) {
            float* p = sw + (i * NT + t) * V + j;
            dw[i][j] += q == 0 ? 0.f : *p;
            *p = dw[i][j];
          }
      __syncthreads();
    }
    if ((int)threadIdx.x / NT != RPB - 1) return;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = t + i * NT;
    if (c < nv)
#pragma unroll
      for (int j = 0; j < V; ++j) part[(int64_t)blockIdx.x * H + c * V + j] = dw[i][j];
  }
}

// dweight[c] = sum_b part[b][c] in float64: 16 columns a workgroup, 64 threads a
// column, each adding every 64th partial sum (eight loads in flight), then a tree.
__global__ __launch_bounds__(1024) void k_norm_dw(const float* __restrict__ part, float* __restrict__ dw, int B,
                                                  int H) {
  constexpr int C = 16, R = 1024 / C;
  __shared__ double s[R][C + 1];
  const int c = threadIdx.x % C, r = threadIdx.x / C;
  const float* p = part + blockIdx.x * C + c;
  double acc = 0.0;
  for (int b0 = r; b0 < B; b0 += 8 * R) {
    float t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = b0 + j * R < B ? p[int64_t(b0 + j * R) * H] : 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) acc += double(t[j]);
  }
  s[r][c] = acc;
  for (int n = R / 2; n > 0; n /= 2) {
    __syncthreads();
    if (r < n) s[r][c] += s[r + n][c];
  }
  if (r == 0) dw[blockIdx.x * C + c] = float(s[0][c]);
}

// Threads per row and vectors per thread for a row of nv 16-byte vectors, as
// F<NT, VPT>().  A short row has no more lanes than vectors: a training step of
// 65536 x 128 bf16 rows takes 32 us so, 55 with a wave a row; of 16384 x 256, 20
// and 23.5.
template <typename T, typename F>
hipError_t by_row(int nv, F f) {
  constexpr int most = MOE_NORM_MAX_H / Vec16<T>::n;  // 4096 in bf16, 8192 in float32
  static_assert(most <= 8192, "the last case has all longer rows");
  if (nv <= 16) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 1>());
  if (nv <= 32) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 1>());
  if (nv <= 64) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
  if (nv <= 128) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 2>());
  if (nv <= 256) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 4>());
  if (nv <= 512) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 2>());
  if (nv <= 1024) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 4>());
  if (nv <= 2048) return f(std::integral_constant<int, 512>(), std::integral_constant<int, 4>());
  if constexpr (most > 4096)
    if (nv > 4096) return f(std::integral_constant<int, 1024>(), std::integral_constant<int, 8>());
  return f(std::integral_constant<int, 1024>(), std::integral_constant<int, 4>());
}

template <typename T>
bool streams(const moe_launch::Dims& d) {
  return d.N * d.H * int64_t(sizeof(T)) >= kStreamBytes;
}

template <typename T>
hipError_t norm_t(const moe_launch::Dims& d, const void* x, const void* residual, const void* weight, float eps,
                  void* h, void* y, float* rstd, hipStream_t s) {
  return by_row<T>(int(d.H / Vec16<T>::n), [&](auto nt, auto vpt) {
    constexpr int NT = decltype(nt)::value, VPT = decltype(vpt)::value;
    constexpr int RPB = NT < 256 ? 256 / NT : 1;
    const int64_t blocks = std::min<int64_t>((d.N + RPB - 1) / RPB, kNormMaxBlocks);
    auto* const kernel = streams<T>(d) ? k_norm<T, NT, VPT, true> : k_norm<T, NT, VPT, false>;
    kernel<<<dim3(unsigned(blocks)), dim3(NT < 256 ? 256 : NT), 0, s>>>(
        static_cast<const T*>(x), static_cast<const T*>(residual), static_cast<const T*>(weight), static_cast<T*>(h),
        static_cast<T*>(y), rstd, d.N, int(d.H), eps);
    return hipGetLastError();
  });
}

template <typename T>
int norm_bwd_blocks(const moe_launch::Dims& d) {
  const int64_t nv = d.H / Vec16<T>::n;
  const int64_t rpb = nv <= 16 ? 16 : nv <= 32 ? 8 : nv <= 256 ? 4 : 1;  // as by_row
  return int(std::min<int64_t>(kNormBwdBlocks, (d.N + rpb - 1) / rpb));
}

template <typename T>
hipError_t norm_bwd_t(const moe_launch::Dims& d, const void* dy, const void* h, const void* weight, const float* rstd,
                      const void* dh, void* dx, float* dw, void* ws, hipStream_t s) {
  const int B = norm_bwd_blocks<T>(d);
  float* part = B == 1 ? dw : static_cast<float*>(ws);  // one workgroup's sums are the result
  hipError_t e = by_row<T>(int(d.H / Vec16<T>::n), [&](auto nt, auto vpt) {
    constexpr int NT = decltype(nt)::value, VPT = decltype(vpt)::value;
    auto* const kernel = streams<T>(d) ? k_norm_bwd<T, NT, VPT, true> : k_norm_bwd<T, NT, VPT, false>;
    kernel<<<dim3(B), dim3(NT < 256 ? 256 : NT), 0, s>>>(
        static_cast<const T*>(dy), static_cast<const T*>(h), static_cast<const T*>(weight), rstd,
        static_cast<const T*>(dh), static_cast<T*>(dx), part, d.N, int(d.H));
    return hipGetLastError();
  });
  if (e != hipSuccess || B == 1) return e;
  k_norm_dw<<<dim3(unsigned(d.H / 16)), dim3(1024), 0, s>>>(part, dw, B, int(d.H));
  return hipGetLastError();
}

}  // namespace

namespace moe_launch {

size_t rms_norm_bwd_ws(const Dims& d) {
  const int B = d.dtype == MOE_BF16 ? norm_bwd_blocks<bf16_t>(d) : norm_bwd_blocks<float>(d);
  return size_t(B) * size_t(d.H) * sizeof(float);
}

hipError_t rms_norm(const Dims& d, const void* x, const void* residual, const void* weight, float eps, void* h,
                    void* y, float* rstd, hipStream_t s) {
  return d.dtype == MOE_BF16 ? norm_t<bf16_t>(d, x, residual, weight, eps, h, y, rstd, s)
                             : norm_t<float>(d, x, residual, weight, eps, h, y, rstd, s);
}

hipError_t rms_norm_bwd(const Dims& d, const void* dy, const void* h, const void* weight, const float* rstd,
                        const void* dh, void* dx, float* dw, void* ws, hipStream_t s) {
  return d.dtype == MOE_BF16 ? norm_bwd_t<bf16_t>(d, dy, h, weight, rstd, dh, dx, dw, ws, s)
                             : norm_bwd_t<float>(d, dy, h, weight, rstd, dh, dx, dw, ws, s);
}

}  // namespace moe_launch
