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

constexpr int kTable = 64;      // tensors in one launch
constexpr int kThreads = 256;
constexpr int kChunk = 4096;    // elements
constexpr uint32_t kMaxBlocks = 1 << 20;  // workgroups of a scaling launch
constexpr int kMaxPart = 1024;  // partial sums (workgroups of the norm)
static_assert(kMaxPart * sizeof(double) == MOE_GRAD_WS_BYTES, "the header states the workspace");

struct Table {
  const void* in[kTable];
  void* out[kTable];
  int64_t n[kTable];
  uint32_t first[kTable + 1];  // first chunk of each tensor; first[count]: all chunks
  uint8_t in_dtype[kTable], out_dtype[kTable], vec[kTable];
  int count;
};

__device__ __forceinline__ float load1(const void* p, int dtype, int64_t i) {
  return dtype == MOE_BF16 ? bf16_to_f32(static_cast<const bf16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store1(void* p, int dtype, int64_t i, float v) {
  if (dtype == MOE_BF16)
    static_cast<bf16_t*>(p)[i] = f32_to_bf16(v);
  else
    static_cast<float*>(p)[i] = v;
}

// V consecutive elements in one access of 8 or 16 bytes.
template <typename T, int V> struct Group {
  typedef T vec_t __attribute__((ext_vector_type(V)));
  vec_t v;
  __device__ __forceinline__ void load(const T* p) { v = __builtin_nontemporal_load(reinterpret_cast<const vec_t*>(p)); }
  __device__ __forceinline__ float get(int i) const { return Elt<T>::to_f32(v[i]); }
  __device__ __forceinline__ void set(int i, float f) { v[i] = Elt<T>::from_f32(f); }
  __device__ __forceinline__ void store(T* p) const {
    __builtin_nontemporal_store(v, reinterpret_cast<vec_t*>(p));
  }
};

// acc += squares of a whole chunk.
template <typename T>
__device__ __forceinline__ void chunk_squares(const void* in, int64_t lo, double& acc) {
  constexpr int V = Vec16<T>::n, U = kChunk / (kThreads * V);
  const T* p = static_cast<const T*>(in) + lo + threadIdx.x * V;
  Group<T, V> g[U];
#pragma unroll
  for (int u = 0; u < U; ++u) g[u].load(p + u * kThreads * V);
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const double f = g[u].get(i);
      acc = fma(f, f, acc);
    }
}

// A whole chunk, scaled by factor(), which is asked for once the loads are on
// their way.
template <typename I, typename O, typename F>
__device__ __forceinline__ void chunk_scale(const void* in, void* out, int64_t lo, F factor) {
  constexpr int V = sizeof(I) == 2 && sizeof(O) == 2 ? 8 : 4, U = kChunk / (kThreads * V);
  const I* p = static_cast<const I*>(in) + lo + threadIdx.x * V;
  O* q = static_cast<O*>(out) + lo + threadIdx.x * V;
  Group<I, V> g[U];
#pragma unroll
  for (int u = 0; u < U; ++u) g[u].load(p + u * kThreads * V);
  const float coef = factor();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    Group<O, V> o;
#pragma unroll
    for (int i = 0; i < V; ++i) o.set(i, coef * g[u].get(i));
    o.store(q + u * kThreads * V);
  }
}

// Calls whole(tensor, first element) for the whole chunks of 16-byte aligned
// tensors and rest(tensor, first, end) for the other chunks, among those that
// this workgroup takes.  REVERSE: from the last chunk on.
template <bool REVERSE, typename W, typename R>
__device__ __forceinline__ void for_chunks(const Table& tab, W whole, R rest) {
  const uint32_t total = tab.first[tab.count];
  int t = REVERSE ? tab.count - 1 : 0;
  for (uint32_t b = blockIdx.x; b < total; b += gridDim.x) {
    const uint32_t c = REVERSE ? total - 1 - b : b;
    if (REVERSE)
      while (c < tab.first[t]) --t;
    else
      while (c >= tab.first[t + 1]) ++t;
    const int64_t lo = int64_t(c - tab.first[t]) * kChunk;
    const int64_t n = tab.n[t];
    if (tab.vec[t] && lo + kChunk <= n)
      whole(t, lo);
    else
      rest(t, lo, min(n, lo + kChunk));
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
  for_chunks<false>(
      tab,
      [&](int t, int64_t lo) {
        if (tab.in_dtype[t] == MOE_BF16)
          chunk_squares<bf16_t>(tab.in[t], lo, acc);
        else
          chunk_squares<float>(tab.in[t], lo, acc);
      },
      [&](int t, int64_t lo, int64_t hi) {
        for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) {
          const double v = load1(tab.in[t], tab.in_dtype[t], i);
          acc = fma(v, v, acc);
        }
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
  // The same factor in every workgroup, found while its first chunk is loading
  // (all threads ask for it together: it holds a barrier).
  float coef = 0.f;
  bool known = false;
  auto factor = [&]() {
    if (!known) {
      const double v = norm_of(part, P);
      if (blockIdx.x == 0 && threadIdx.x == 0) *norm = float(v);
      const double c = double(max_norm) / (v + 1e-6);
      coef = float(c > 1.0 ? 1.0 : c);  // NaN stays NaN
      known = true;
    }
    return coef;
  };
  for_chunks<true>(
      tab,
      [&](int t, int64_t lo) {
        const bool bi = tab.in_dtype[t] == MOE_BF16, bo = tab.out_dtype[t] == MOE_BF16;
        if (bi && bo)
          chunk_scale<bf16_t, bf16_t>(tab.in[t], tab.out[t], lo, factor);
        else if (bi)
          chunk_scale<bf16_t, float>(tab.in[t], tab.out[t], lo, factor);
        else if (bo)
          chunk_scale<float, bf16_t>(tab.in[t], tab.out[t], lo, factor);
        else
          chunk_scale<float, float>(tab.in[t], tab.out[t], lo, factor);
      },
      [&](int t, int64_t lo, int64_t hi) {
        const float f = factor();
        for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads)
          store1(tab.out[t], tab.out_dtype[t], i, f * load1(tab.in[t], tab.in_dtype[t], i));
      });
  factor();  // a workgroup without a chunk: norm is written all the same
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
    const uint32_t blocks = std::max(1u, std::min(tab.first[tab.count], kMaxBlocks));
    k_grad_scale<<<dim3(blocks), dim3(kThreads), 0, s>>>(tab, part, P, max_norm, norm);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  } while (from < count);
  return hipSuccess;
}

}  // namespace moe_launch
