// 2-norm over a list of gradients, and the gradients scaled so that it is at
// most max_norm:
//   norm = sqrt(sum_t sum_i g_t[i]^2), coef = min(1, max_norm / (norm + 1e-6)),
//   out_t[i] = coef * g_t[i], rounded once to the output's type.
//
// Squares are summed in float64 from the first element on: the vector unit
// runs float64 multiply-adds at the float32 rate, HBM is the bound either way,
// and no gradient's square can overflow or vanish.  The list travels in kernel
// arguments (kTable tensors a launch), so a captured graph holds its own copy.
// Each launch cuts its tensors into chunks of kChunk elements that the
// workgroups take in turn; workgroup b leaves one partial sum in ws[b] (later
// launches of a long list add to it).  The scaling kernel needs no launch
// between: every workgroup adds the same partial sums in the same order.
#include <algorithm>

#include "common.h"

namespace {
using namespace moe;

constexpr int kTable = 64;                    // tensors in one launch
constexpr int kThreads = 256;
constexpr int kGroup = 8;                     // elements a thread handles at once
constexpr int kUnroll = 4;
constexpr int64_t kChunk = kThreads * kGroup * kUnroll;
constexpr int kMaxPart = 1024;                // partial sums (workgroups of the norm)
static_assert(kMaxPart * sizeof(double) == MOE_GRAD_WS_BYTES, "the header states the workspace");

struct Table {
  const void* in[kTable];
  void* out[kTable];
  int64_t n[kTable];
  uint32_t first[kTable + 1];  // first chunk of each tensor; first[count]: all chunks
  uint8_t in_dtype[kTable], out_dtype[kTable], vec[kTable];
  int count;
};

// Elements [i, i + 8) of a 16-byte aligned tensor, i a multiple of 8.
__device__ __forceinline__ void load8(const void* p, int dtype, int64_t i, float* v) {
  if (dtype == MOE_BF16) {
    Vec16<bf16_t>::load(static_cast<const bf16_t*>(p) + i, v);
  } else {
    Vec16<float>::load(static_cast<const float*>(p) + i, v);
    Vec16<float>::load(static_cast<const float*>(p) + i + 4, v + 4);
  }
}
__device__ __forceinline__ void store8(void* p, int dtype, int64_t i, const float* v) {
  if (dtype == MOE_BF16) {
    Vec16<bf16_t>::store(static_cast<bf16_t*>(p) + i, v);
  } else {
    Vec16<float>::store(static_cast<float*>(p) + i, v);
    Vec16<float>::store(static_cast<float*>(p) + i + 4, v + 4);
  }
}
__device__ __forceinline__ float load1(const void* p, int dtype, int64_t i) {
  return dtype == MOE_BF16 ? bf16_to_f32(static_cast<const bf16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store1(void* p, int dtype, int64_t i, float v) {
  if (dtype == MOE_BF16)
    static_cast<bf16_t*>(p)[i] = f32_to_bf16(v);
  else
    static_cast<float*>(p)[i] = v;
}

// Calls f8(tensor, i) for the whole groups of 8 elements and f1(tensor, i) for
// the single ones (tails, tensors that are not 16-byte aligned) of the chunks
// that this workgroup takes.
template <typename F8, typename F1>
__device__ __forceinline__ void for_chunks(const Table& tab, F8 f8, F1 f1) {
  int t = 0;
  const uint32_t total = tab.first[tab.count];
  for (uint32_t c = blockIdx.x; c < total; c += gridDim.x) {
    while (c >= tab.first[t + 1]) ++t;
    const int64_t lo = int64_t(c - tab.first[t]) * kChunk;
    const int64_t n = tab.n[t];
    if (tab.vec[t]) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = lo + (int64_t(u) * kThreads + threadIdx.x) * kGroup;
        if (i + kGroup <= n)
          f8(t, i);
        else
          for (int64_t j = i; j < n; ++j) f1(t, j);
      }
    } else {
      const int64_t hi = min(n, lo + kChunk);
      for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) f1(t, i);
    }
  }
}

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
  return v;
}
// The sum over the workgroup, in every thread.
__device__ __forceinline__ double block_sum64(double v) {
  __shared__ double s[kThreads / kWave];
  v = wave_sum64(v);
  if (lane_id() == 0) s[threadIdx.x / kWave] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int i = 0; i < kThreads / kWave; ++i) v += s[i];
  return v;
}

__global__ __launch_bounds__(kThreads) void k_grad_squares(Table tab, double* __restrict__ part, int add) {
  double acc = 0.0;
  for_chunks(
      tab,
      [&](int t, int64_t i) {
        float v[kGroup];
        load8(tab.in[t], tab.in_dtype[t], i, v);
#pragma unroll
        for (int j = 0; j < kGroup; ++j) acc = fma(double(v[j]), double(v[j]), acc);
      },
      [&](int t, int64_t i) {
        const double v = load1(tab.in[t], tab.in_dtype[t], i);
        acc = fma(v, v, acc);
      });
  acc = block_sum64(acc);
  if (threadIdx.x == 0) part[blockIdx.x] = add ? part[blockIdx.x] + acc : acc;
}

__device__ __forceinline__ double norm_of(const double* __restrict__ part, int P) {
  double acc = 0.0;
  for (int i = threadIdx.x; i < P; i += kThreads) acc += part[i];
  return sqrt(block_sum64(acc));
}

__global__ __launch_bounds__(kThreads) void k_grad_norm(const double* __restrict__ part, int P,
                                                        float* __restrict__ norm) {
  const double v = norm_of(part, P);
  if (threadIdx.x == 0) *norm = float(v);
}

__global__ __launch_bounds__(kThreads) void k_grad_scale(Table tab, const double* __restrict__ part, int P,
                                                         float max_norm, float* __restrict__ norm) {
  const double v = norm_of(part, P);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = float(v);
  const double c = double(max_norm) / (v + 1e-6);
  const float coef = float(c > 1.0 ? 1.0 : c);  // NaN stays NaN
  for_chunks(
      tab,
      [&](int t, int64_t i) {
        float a[kGroup];
        load8(tab.in[t], tab.in_dtype[t], i, a);
#pragma unroll
        for (int j = 0; j < kGroup; ++j) a[j] *= coef;
        store8(tab.out[t], tab.out_dtype[t], i, a);
      },
      [&](int t, int64_t i) { store1(tab.out[t], tab.out_dtype[t], i, coef * load1(tab.in[t], tab.in_dtype[t], i)); });
}

// Tensors [from, ...) of the list that fit one launch; returns the next one.
int fill(const moe_grad* g, int count, int from, bool scaled, Table* tab) {
  tab->count = 0;
  tab->first[0] = 0;
  for (; from < count && tab->count < kTable; ++from) {
    if (g[from].n == 0) continue;
    const int t = tab->count++;
    tab->in[t] = g[from].in;
    tab->out[t] = scaled ? g[from].out : nullptr;
    tab->n[t] = g[from].n;
    tab->in_dtype[t] = uint8_t(g[from].in_dtype);
    tab->out_dtype[t] = uint8_t(scaled ? g[from].out_dtype : g[from].in_dtype);
    const uintptr_t at = reinterpret_cast<uintptr_t>(g[from].in) | (scaled ? reinterpret_cast<uintptr_t>(g[from].out) : 0);
    tab->vec[t] = (at & 15u) == 0;
    tab->first[t + 1] = tab->first[t] + uint32_t((g[from].n + kChunk - 1) / kChunk);
  }
  return from;
}

// Partial sums of squares of the whole list; returns how many there are (at
// least one), or -1 with *e set.
int squares(const moe_grad* g, int count, double* part, hipStream_t s, hipError_t* e) {
  // as many workgroups as the longest launch can use; the first launch writes every partial sum
  Table tab;
  uint32_t most = 1;
  for (int from = 0; from < count;) {
    from = fill(g, count, from, false, &tab);
    most = std::max(most, tab.first[tab.count]);
  }
  const int P = int(std::min<uint32_t>(most, kMaxPart));
  int add = 0;
  int from = 0;
  do {
    from = fill(g, count, from, false, &tab);
    k_grad_squares<<<dim3(P), dim3(kThreads), 0, s>>>(tab, part, add);
    *e = hipGetLastError();
    if (*e != hipSuccess) return -1;
    add = 1;
  } while (from < count);
  return P;
}

}  // namespace

namespace moe_launch {

int64_t grad_chunk() { return kChunk; }

hipError_t grad_norm(const moe_grad* g, int count, float* norm, void* ws, hipStream_t s) {
  hipError_t e = hipSuccess;
  double* part = static_cast<double*>(ws);
  const int P = squares(g, count, part, s, &e);
  if (P < 0) return e;
  k_grad_norm<<<dim3(1), dim3(kThreads), 0, s>>>(part, P, norm);
  return hipGetLastError();
}

hipError_t grad_clip(const moe_grad* g, int count, float max_norm, float* norm, void* ws, hipStream_t s) {
  hipError_t e = hipSuccess;
  double* part = static_cast<double*>(ws);
  const int P = squares(g, count, part, s, &e);
  if (P < 0) return e;
  Table tab;
  int from = 0;
  do {
    from = fill(g, count, from, true, &tab);
    const uint32_t blocks = std::max(1u, std::min(tab.first[tab.count], 2048u));
    k_grad_scale<<<dim3(blocks), dim3(kThreads), 0, s>>>(tab, part, P, max_norm, norm);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  } while (from < count);
  return hipSuccess;
}

}  // namespace moe_launch
