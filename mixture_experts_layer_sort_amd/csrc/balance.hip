// Balance and z loss of router logits, per sequence, padding left out, and the
// gradient of the logits (moe_balance in moe.h).
//
//   p_t = softmax(l_t) or sigmoid(l_t) / sum sigmoid(l_t),   lse_t = log sum exp(l_t),
//   f_s,e = E c_s,e / (K n_s),  P_s,e = mean_t p_t,e,
//   loss = alpha / B' sum_s f_s.P_s + z / n sum_t lse_t^2,
//   dl_t,e = alpha / (B' n_s) p_e (f_s,e - f_s.p_t) [1 - sigmoid(l_e)] + 2 z / n lse_t softmax_e.
//
// Sixteen lanes have a token, so that every sum over its experts stays within a
// row of lanes (DPP moves, no LDS).  The logits are read twice: f, which the
// gradient needs, is known only after all of a sequence's tokens.  Probabilities
// are formed again in the backward pass, which costs less than 4 bytes of them
// written and read for each logit.  Chunks of a sequence leave partial sums; the
// next launch adds them up in float64 in their order.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.h"

namespace {
using namespace moe;

constexpr int kLanes = 16;       // of a token
constexpr int kRows = 256 / kLanes;  // tokens a workgroup has under way
constexpr int kOneRows = 1024 / kLanes;  // where one workgroup does all
// Three workgroups a CU, what the registers of 256 experts allow. Kernels of fewer experts could have more, but
// the next launch reads each chunk's sums: 131072 tokens of 64 experts as one sequence take 61 us with 768 chunks,
// 69 with 1280, 86 with 2048; as 32 sequences 51, 50 and 48.
constexpr int64_t kMostChunks = 768;

// Over the sixteen lanes of a token, all of them getting the result: each step
// takes the value of a lane with the lowest 1, 2, 3, 4 bits of its number mirrored.
#define MOE_DPP(v, ctrl) __builtin_amdgcn_update_dpp(0, v, ctrl, 0xf, 0xf, true)
template <typename F>
__device__ __forceinline__ float over_lanes(float v, F f) {
  v = f(v, __int_as_float(MOE_DPP(__float_as_int(v), 0xb1)));   // quad_perm 1 0 3 2
  v = f(v, __int_as_float(MOE_DPP(__float_as_int(v), 0x4e)));   // quad_perm 2 3 0 1
  v = f(v, __int_as_float(MOE_DPP(__float_as_int(v), 0x141)));  // row_half_mirror
  return f(v, __int_as_float(MOE_DPP(__float_as_int(v), 0x140)));  // row_mirror
}
__device__ __forceinline__ float lanes_sum(float v) {
  return over_lanes(v, [](float a, float b) { return a + b; });
}
// The larger one; of a number and NaN the number.  (fmaxf makes its operands quiet
// first, an instruction for each.)
__device__ __forceinline__ float max_of(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, INFINITY); }
__device__ __forceinline__ float lanes_max(float v) { return over_lanes(v, max_of); }

// A token's NV * 16 >= E values over its lanes: VEC, four neighbours at a time
// (E a multiple of 4), else every sixteenth.
template <int NV, bool VEC> struct Place {
  static __device__ __forceinline__ int expert(int sub, int v) {
    return VEC ? v / 4 * 64 + sub * 4 + v % 4 : v * kLanes + sub;
  }
};

template <typename T, int NV, bool VEC>
__device__ __forceinline__ void load_row(const T* p, int sub, int E, float (&l)[NV]) {
  if constexpr (VEC) {
#pragma unroll
    for (int v = 0; v < NV; v += 4) {
      const int e = Place<NV, VEC>::expert(sub, v);
      if (e < E) {
        if constexpr (sizeof(T) == 4) {
          const float4 q = *reinterpret_cast<const float4*>(p + e);
          l[v] = q.x; l[v + 1] = q.y; l[v + 2] = q.z; l[v + 3] = q.w;
        } else {
          const uint2 q = *reinterpret_cast<const uint2*>(p + e);
          l[v] = __uint_as_float(q.x << 16);
          l[v + 1] = __uint_as_float(q.x & 0xffff0000u);
          l[v + 2] = __uint_as_float(q.y << 16);
          l[v + 3] = __uint_as_float(q.y & 0xffff0000u);
        }
      } else {
        l[v] = l[v + 1] = l[v + 2] = l[v + 3] = -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = Place<NV, VEC>::expert(sub, v);
      l[v] = e < E ? Elt<T>::load(p + e) : -INFINITY;
    }
  }
}

__device__ __forceinline__ int lanes_sum(int v) {
  v += MOE_DPP(v, 0xb1);
  v += MOE_DPP(v, 0x4e);
  v += MOE_DPP(v, 0x141);
  return v + MOE_DPP(v, 0x140);
}
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  v = max(v, uint32_t(MOE_DPP(int(v), 0xb1)));
  v = max(v, uint32_t(MOE_DPP(int(v), 0x4e)));
  v = max(v, uint32_t(MOE_DPP(int(v), 0x141)));
  return max(v, uint32_t(MOE_DPP(int(v), 0x140)));
}

// exp(x) for x <= 0 (0 below 2^-126): the hardware's 2^h of h = x / ln 2, rounded, and the
// first order of x - h ln 2, which the rounding leaves (2^-16 at most): about an ulp of the
// hardware's, where 2^h alone is off by |x| 2^-24 of itself.
__device__ __forceinline__ float exp_below(float x) {
  constexpr double kLn2 = 0.69314718055994530942;
  constexpr float kHigh = float(kLn2), kLow = float(kLn2 - double(kHigh));
  const float h = x * float(1.0 / kLn2), r = __builtin_amdgcn_exp2f(h);
  const float d = fmaf(-h, kLow, fmaf(-h, kHigh, x));
  return fmaf(r, __builtin_amdgcn_fmed3f(d, -0x1p-15f, 0x1p-15f), r);  // d of -inf is NaN, r 0
}
// 1 / a for a from 1 to 2: the hardware's, which is off by an ulp, and a Newton step.
__device__ __forceinline__ float inverse(float a) {
  const float r = __builtin_amdgcn_rcpf(a);
  return fmaf(fmaf(-a, r, 1.f), r, r);
}

// Probabilities of one token: soft the softmax, p the score's, rest 1 - sigmoid
// (sigmoid scores), lse its log-sum-exp.  Places past E hold -inf: 0 in all.
template <int NV> struct Token {
  float soft[NV], p[NV], rest[NV], lse;
  __device__ __forceinline__ void set(const float (&l)[NV], bool sigmoid) {
    float top = l[0];  // of those that are numbers; a NaN reaches the sum
#pragma unroll
    for (int v = 1; v < NV; ++v) top = max_of(top, l[v]);
    top = lanes_max(top);
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      soft[v] = exp_below(l[v] - top);
      sum += soft[v];
    }
    sum = lanes_sum(sum);
    lse = top + logf(sum);
    const float inv = 1.f / sum;
    if (sigmoid) {
      // Where all logits are negative every sigmoid may be tiny: there all of them
      // over exp(top), whose largest is 1 / (1 + exp(top)).
      float all = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const float t = exp_below(-fabsf(l[v])), large = inverse(1.f + t), small = t * large;
        p[v] = l[v] < 0.f ? small : large;
        rest[v] = l[v] < 0.f ? large : small;
        all += p[v];
      }
      if (top <= 0.f) {
        const float down = exp_below(top);
        all = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          p[v] = soft[v] * inverse(1.f + soft[v] * down);
          all += p[v];
        }
      }
      const float a = 1.f / lanes_sum(all);
#pragma unroll
      for (int v = 0; v < NV; ++v) p[v] *= a;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      soft[v] *= inv;
      if (!sigmoid) p[v] = soft[v];
    }
  }
};

// Order of the choice: larger values first, NaN last, 0 and -0 equal; 0 is below all.
__device__ __forceinline__ uint32_t choice_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  const uint32_t key = u & 0x80000000u ? ~u : u | 0x80000000u;
  return v != v ? 1u : max(key, 2u);
}

// The largest key under `below` of a token: the smallest distance to it, which wraps
// around to a large one from `below` upwards.
template <int NV>
__device__ __forceinline__ uint32_t next_below(const uint32_t (&key)[NV], uint32_t below) {
  uint32_t d = ~0u;
#pragma unroll
  for (int v = 0; v < NV; ++v) d = min(d, below - 1u - key[v]);
  return below - 1u - ~lanes_max(~d);
}

// The K-th largest value of a token where no lane has more than four of the largest K
// and none of them equals another one; otherwise some value.
template <int NV>
__device__ __forceinline__ float kth_value(const float (&f)[NV], int K) {
  constexpr int D = 4;
  float m[D];  // the lane's largest ones, descending
#pragma unroll
  for (int i = 0; i < D; ++i) m[i] = -INFINITY;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
#pragma unroll
    for (int i = D - 1; i > 0; --i) m[i] = __builtin_amdgcn_fmed3f(m[i - 1], m[i], f[v]);
    m[0] = max_of(m[0], f[v]);
  }
  float best = INFINITY;
  for (int k = 0; k < K; ++k) {
    best = lanes_max(m[0]);
    const bool took = m[0] == best;
#pragma unroll
    for (int i = 0; i + 1 < D; ++i) m[i] = took ? m[i + 1] : m[i];
    m[D - 1] = took ? -INFINITY : m[D - 1];
  }
  return best;
}

// The K experts of largest value l + b, each counted by the lane that holds it.  Only
// the set matters: a value that exactly K reach tells it.  RARE: equals are rare
// (float32 logits), so such a value is first looked for among the largest few of each
// lane: the loss of 131072 tokens, 8 of 256 sigmoid experts, takes 76 us so and 98
// without; bfloat16 logits, whose equals spoil it for most waves, 115 and 97.
// Otherwise the K-th largest is found by going down from one value to the next;
// everything above it is chosen, and of its equals the first ones by their expert.
template <int NV, bool VEC, bool RARE>
__device__ __forceinline__ void choose(const float (&l)[NV], const float (&b)[NV], int sub, int E, int K,
                                       int (&count)[NV]) {
  float f[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) f[v] = l[v] + b[v];
  if constexpr (RARE) {
    const float last = kth_value(f, K);
    int got = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) got += f[v] >= last;
    if (last > -INFINITY && lanes_sum(got) == K) {  // places past E reach -inf
#pragma unroll
      for (int v = 0; v < NV; ++v) count[v] += f[v] >= last;
      return;
    }
  }
  uint32_t key[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) key[v] = Place<NV, VEC>::expert(sub, v) < E ? choice_key(f[v]) : 0u;
  uint32_t last = ~0u;
  int left = K, equal = 0;  // still to choose; how many equals the last value has
  while (left > 0) {
    last = next_below(key, last);
    equal = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) equal += key[v] == last;
    equal = lanes_sum(equal);
    left -= equal;
  }
  if (left == 0) {
#pragma unroll
    for (int v = 0; v < NV; ++v) count[v] += key[v] >= last;
    return;
  }
  // of the equals of the last value, -left too many: the first take - by their expert
  int take = equal + left;
#pragma unroll
  for (int v = 0; v < NV; ++v) count[v] += key[v] > last;
  for (int k = 0; k < take; ++k) {
    int first = MOE_MAX_EXPERTS;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      first = key[v] == last ? min(first, Place<NV, VEC>::expert(sub, v)) : first;
    first = MOE_MAX_EXPERTS - int(lanes_max(uint32_t(MOE_MAX_EXPERTS - first)));
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (key[v] == last && Place<NV, VEC>::expert(sub, v) == first) {
        key[v] = 0;
        ++count[v];
      }
  }
}

// One chunk's sums: P [E], counts [E], the sum of lse^2, the number of tokens.
__host__ __device__ constexpr int64_t part_words(int64_t E) { return 2 * E + 2; }

// What the backward pass needs: words 0 and 1 the sequences and tokens that count,
// then of every sequence f [E] and its tokens.
constexpr int kStateHead = 4;
__host__ __device__ constexpr int64_t state_words(int64_t B, int64_t E) { return kStateHead + B * (E + 1); }

// Of every sequence, for the sums over them.
struct SeqSum {
  double loss, z;  // f.P, sum of lse^2
  int64_t tokens;
};

// alpha / B' sum f.P + z / n sum lse^2, from the sums over the sequences.
__device__ __forceinline__ float total_loss(double fp, double z, int64_t seqs, int64_t tokens, float alpha,
                                            float z_coef) {
  if (tokens == 0) return 0.f;
  const double balance = double(alpha) * fp / double(seqs);
  return float(z_coef == 0.f ? balance : balance + double(z_coef) * z / double(tokens));  // no 0 * infinity
}
// f_e of a sequence of n tokens.
__device__ __forceinline__ double expert_share(int count, int E, int K, int64_t n) {
  return n == 0 ? 0.0 : double(E) * double(count) / (double(K) * double(n));
}

// Where results go: a chunk's to parts; ONE, of one sequence in one workgroup, itself to
// state, counts and loss.
struct Results {
  float *parts, *state, *loss;
  int32_t* counts;
  float alpha, z_coef;
};

// CHOOSE: counts are of the largest K values, otherwise of topk.  (Kernels of their own: the choice
// takes the registers of half of the waves.)  ROWS tokens at a time.
template <typename T, int NV, bool VEC, bool CHOOSE, bool ONE>
__global__ __launch_bounds__(ONE ? 1024 : 256) void k_balance_parts(
    const T* __restrict__ logits, const int32_t* __restrict__ topk, const float* __restrict__ bias,
    const uint8_t* __restrict__ mask, Results to, int E, int K, int seq_len, int chunk, int chunks, bool sigmoid) {
  constexpr int ROWS = ONE ? kOneRows : kRows, NT = ROWS * kLanes;
  __shared__ float sp[ROWS][NV * kLanes];
  __shared__ float sz[ROWS];
  __shared__ int count[NV * kLanes], tokens;
  const int t = threadIdx.x, sub = t % kLanes, q = t / kLanes;
  for (int i = t; i < NV * kLanes; i += NT) count[i] = 0;
  if (t == 0) tokens = 0;
  __syncthreads();
  const int first = int(blockIdx.x % chunks) * chunk, last = min(first + chunk, seq_len);
  const int64_t row0 = int64_t(blockIdx.x / chunks) * seq_len;
  float p[NV], z = 0.f, l[NV], next[NV];
  int chosen[NV];
  float b[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = Place<NV, VEC>::expert(sub, v);
    b[v] = CHOOSE && bias != nullptr && e < E ? bias[e] : 0.f;
    p[v] = 0.f;
    chosen[v] = 0;
  }
  int mine = 0;
  bool live = false, ahead;
  auto fetch = [&](int r, float (&to)[NV]) {
    const int64_t n = row0 + r;
    const bool is = r < last && (mask == nullptr || mask[n] != 0);
    if (is) load_row<T, NV, VEC>(logits + n * E, sub, E, to);
    return is;
  };
  live = fetch(first + q, l);
  for (int r = first + q; r < last; r += ROWS) {
    ahead = fetch(r + ROWS, next);  // the next token's logits on their way
    if (live) {
      Token<NV> a;
      a.set(l, sigmoid);
#pragma unroll
      for (int v = 0; v < NV; ++v) p[v] += a.p[v];
      z += a.lse * a.lse;
      ++mine;
      if constexpr (CHOOSE) {
        choose<NV, VEC, sizeof(T) == 4>(l, b, sub, E, K, chosen);
      } else if (sub < K) {
        const int e = topk[(row0 + r) * K + sub];
        if (e >= 0 && e < E) atomicAdd(count + e, 1);
      }
    }
    live = ahead;
#pragma unroll
    for (int v = 0; v < NV; ++v) l[v] = next[v];
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    sp[q][Place<NV, VEC>::expert(sub, v)] = p[v];
    if (CHOOSE && chosen[v] > 0) atomicAdd(count + Place<NV, VEC>::expert(sub, v), chosen[v]);
  }
  if (sub == 0) {
    sz[q] = z;
    atomicAdd(&tokens, mine);
  }
  __syncthreads();
  if constexpr (ONE) {
    static_assert(NV * kLanes <= kWave && ROWS == kWave, "a lane for each expert and each row");
    if (t >= kWave) return;
    double p_sum = 0.0, z_sum = double(sz[t]);
    if (t < E) {
      for (int i = 0; i < ROWS; ++i) p_sum += double(sp[i][t]);
      const double f = expert_share(count[t], E, K, tokens);
      to.state[kStateHead + t] = float(f);
      to.counts[t] = count[t];
      p_sum = tokens == 0 ? 0.0 : f * p_sum / double(tokens);
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
      p_sum += __shfl_xor(p_sum, off, kWave);
      z_sum += __shfl_xor(z_sum, off, kWave);
    }
    if (t == 0) {
      int32_t* head = reinterpret_cast<int32_t*>(to.state);
      head[0] = tokens > 0;
      head[1] = head[kStateHead + E] = tokens;
      to.loss[0] = total_loss(p_sum, z_sum, 1, tokens, to.alpha, to.z_coef);
    }
    return;
  }
  float* out = to.parts + int64_t(blockIdx.x) * part_words(E);
  for (int e = t; e < E; e += NT) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) s += sp[i][e];
    out[e] = s;
    reinterpret_cast<int*>(out)[E + e] = count[e];
  }
  if (t == 0) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) s += sz[i];
    out[2 * E] = s;
    reinterpret_cast<int*>(out)[2 * E + 1] = tokens;
  }
}

// A sequence a workgroup of 256 or 1024 threads: its chunks added up by (expert, slice
// of the chunks), eight loads under way; f, its loss, and with one sequence the rest.
__global__ __launch_bounds__(1024) void k_balance_seq(const float* __restrict__ parts, float* __restrict__ state,
                                                      SeqSum* __restrict__ sums, int32_t* __restrict__ seq_counts,
                                                      float* __restrict__ loss, int E, int lanes, int K, int chunks,
                                                      int B, float alpha, float z_coef) {
  __shared__ double sp[1024];
  __shared__ int sc[1024];
  __shared__ double sz[16];
  __shared__ int64_t sn[16];
  const int t = threadIdx.x, nt = blockDim.x, s = blockIdx.x, e = t % lanes, slices = nt / lanes;
  const float* in = parts + int64_t(s) * chunks * part_words(E);
  const int64_t step = part_words(E);
  double p = 0.0;
  int c = 0;
  if (e < E)
    for (int i0 = t / lanes; i0 < chunks; i0 += 8 * slices) {
      float a[8];
      int b[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = i0 + j * slices;
        a[j] = i < chunks ? in[i * step + e] : 0.f;
        b[j] = i < chunks ? reinterpret_cast<const int*>(in)[i * step + E + e] : 0;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p += double(a[j]);
        c += b[j];
      }
    }
  double z = 0.0;
  int64_t n = 0;
  for (int i = t; i < chunks; i += nt) {
    z += double(in[i * step + 2 * E]);
    n += reinterpret_cast<const int*>(in)[i * step + 2 * E + 1];
  }
  auto over_block = [&](double& dv, int64_t& iv) {  // sums over all threads, in a fixed order
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
      dv += __shfl_xor(dv, off, kWave);
      iv += __shfl_xor(iv, off, kWave);
    }
    if (lane_id() == 0) {
      sz[t / kWave] = dv;
      sn[t / kWave] = iv;
    }
    __syncthreads();
    dv = 0.0;
    iv = 0;
    for (int i = 0; i < nt / kWave; ++i) {
      dv += sz[i];
      iv += sn[i];
    }
  };
  sp[t] = p;
  sc[t] = c;
  over_block(z, n);
  for (int off = nt / 2; off >= lanes; off >>= 1) {
    if (t < off) {
      sp[t] += sp[t + off];
      sc[t] += sc[t + off];
    }
    __syncthreads();
  }
  double fp = 0.0;
  if (t < E) {
    c = sc[t];
    const double f = expert_share(c, E, K, n);
    state[kStateHead + int64_t(s) * (E + 1) + t] = float(f);
    seq_counts[int64_t(s) * E + t] = c;  // the counts themselves where there is one sequence
    fp = n == 0 ? 0.0 : f * sp[t] / double(n);
  }
  int64_t none = 0;
  __syncthreads();
  over_block(fp, none);
  if (t == 0) {
    reinterpret_cast<int32_t*>(state)[kStateHead + int64_t(s) * (E + 1) + E] = int32_t(n);
    if (B == 1) {
      reinterpret_cast<int32_t*>(state)[0] = n > 0;
      reinterpret_cast<int32_t*>(state)[1] = int32_t(n);
      loss[0] = total_loss(fp, z, 1, n, alpha, z_coef);
    } else {
      sums[s] = SeqSum{fp, z, n};
    }
  }
}

// Over several sequences: workgroup 0 the loss, the others 16 experts' counts each.
__global__ __launch_bounds__(256) void k_balance_total(const SeqSum* __restrict__ sums,
                                                       const int32_t* __restrict__ seq_counts,
                                                       float* __restrict__ state, int32_t* __restrict__ counts,
                                                       float* __restrict__ loss, int E, int B, float alpha,
                                                       float z_coef) {
  const int t = threadIdx.x;
  if (blockIdx.x == 0) {
    __shared__ double sf[256], sz[256];
    __shared__ int64_t sn[256], ss[256];
    double f = 0.0, z = 0.0;
    int64_t n = 0, seqs = 0;
    for (int i = t; i < B; i += 256) {
      const SeqSum q = sums[i];
      f += q.loss;
      z += q.z;
      n += q.tokens;
      seqs += q.tokens > 0;
    }
    sf[t] = f; sz[t] = z; sn[t] = n; ss[t] = seqs;
    for (int off = 128; off > 0; off >>= 1) {
      __syncthreads();
      if (t < off) {
        sf[t] += sf[t + off]; sz[t] += sz[t + off]; sn[t] += sn[t + off]; ss[t] += ss[t + off];
      }
    }
    if (t == 0) {
      reinterpret_cast<int32_t*>(state)[0] = int32_t(ss[0]);
      reinterpret_cast<int32_t*>(state)[1] = int32_t(sn[0]);
      loss[0] = total_loss(sf[0], sz[0], ss[0], sn[0], alpha, z_coef);
    }
    return;
  }
  __shared__ int sc[256];
  const int e = (int(blockIdx.x) - 1) * 16 + t % 16;
  int c = 0;
  if (e < E)
    for (int s = t / 16; s < B; s += 16) c += seq_counts[int64_t(s) * E + e];
  sc[t] = c;
  __syncthreads();
  if (t < 16 && e < E) {
    c = 0;
    for (int i = 0; i < 16; ++i) c += sc[16 * i + t];
    counts[e] = c;
  }
}

// dlogits may be logits: a lane stores where it alone has loaded.
template <typename T, int NV, bool VEC>
__global__ __launch_bounds__(256) void k_balance_bwd(const T* logits, const uint8_t* __restrict__ mask,
                                                     const float* __restrict__ state, const float* __restrict__ dloss,
                                                     T* dlogits, int64_t N, int E, int seq_len,
                                                     float alpha, float z_coef, bool sigmoid) {
  const int sub = threadIdx.x % kLanes;
  const int64_t n = int64_t(blockIdx.x) * kRows + threadIdx.x / kLanes;
  if (n >= N) return;  // all lanes of a token
  const int32_t* head = reinterpret_cast<const int32_t*>(state);
  float d[NV];
  if (mask == nullptr || mask[n] != 0) {
    float l[NV];
    load_row<T, NV, VEC>(logits + n * E, sub, E, l);
    const float* seq = state + kStateHead + n / seq_len * (E + 1);
    float f[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = Place<NV, VEC>::expert(sub, v);
      f[v] = e < E ? seq[e] : 0.f;
    }
    const float up = dloss == nullptr ? 1.f : dloss[0];
    const float c = up * alpha / (float(head[0]) * float(reinterpret_cast<const int32_t*>(seq)[E]));
    Token<NV> a;
    a.set(l, sigmoid);
    float fp = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) fp += f[v] * a.p[v];
    fp = lanes_sum(fp);
    const float zc = up * 2.f * z_coef / float(head[1]) * a.lse;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float b = c * a.p[v] * (f[v] - fp);
      if (sigmoid) b *= a.rest[v];
      d[v] = z_coef == 0.f ? b : b + zc * a.soft[v];
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) d[v] = 0.f;
  }
  T* p = dlogits + n * E;
  if constexpr (VEC) {
#pragma unroll
    for (int v = 0; v < NV; v += 4) {
      const int e = Place<NV, VEC>::expert(sub, v);
      if (e < E) {
        if constexpr (sizeof(T) == 4)
          *reinterpret_cast<float4*>(p + e) = make_float4(d[v], d[v + 1], d[v + 2], d[v + 3]);
        else
          *reinterpret_cast<uint2*>(p + e) = make_uint2(pack_bf16x2(d[v], d[v + 1]), pack_bf16x2(d[v + 2], d[v + 3]));
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = Place<NV, VEC>::expert(sub, v);
      if (e < E) p[e] = Elt<T>::from_f32(d[v]);
    }
  }
}

// Tokens of a chunk, a whole number of a workgroup's turns: one for each CU, then up to four
// turns, then about kMostChunks chunks (and at least one a sequence).  The next launch reads each
// chunk's sums (16384 tokens of 64 experts as one sequence: chunks of one turn take 6.1 us and the
// next launch 15.7, of four turns 7.8 and 10.1; as four sequences, choice given, 4.4 and 7.7, 5.6
// and 6.4).
int64_t chunk_of(const moe_balance& b) {
  const int64_t per = std::max(std::min<int64_t>(4 * kRows, b.N / 256), (b.N + kMostChunks - 1) / kMostChunks);
  return std::min<int64_t>((per + kRows - 1) / kRows * kRows, (b.seq_len + kRows - 1) / kRows * kRows);
}
int64_t chunks_of(const moe_balance& b) { return (b.seq_len + chunk_of(b) - 1) / chunk_of(b); }

// Few tokens of one sequence, at most 64 experts: all in one workgroup, without the launch that adds
// chunks up.  203 tokens of 8 experts: 6.2 us, 7.0 in two launches, and the call takes the host 2 us less;
// 256: 7.2 and 7.0; 128 tokens of 64 experts: 7.2 and 7.7, 203: 9.8 and 8.4.
bool in_one(const moe_balance& b) {
  return b.N == b.seq_len && b.N <= (b.E <= 16 ? 4 : 2) * kOneRows && b.E <= kWave;
}

size_t pad(size_t n) { return (n + 255) & ~size_t(255); }
size_t parts_bytes(const moe_balance& b) {
  return pad(size_t(b.N / b.seq_len * chunks_of(b)) * part_words(b.E) * 4);
}

// NV and VEC of a launch.
template <typename T, typename F>
hipError_t by_experts(int64_t E, F f) {
  if (E % 4 == 0 && E > 32)
    return E <= 64 ? f(std::integral_constant<int, 4>(), std::true_type())
           : E <= 128 ? f(std::integral_constant<int, 8>(), std::true_type())
                      : f(std::integral_constant<int, 16>(), std::true_type());
  return E <= 16    ? f(std::integral_constant<int, 1>(), std::false_type())
         : E <= 32  ? f(std::integral_constant<int, 2>(), std::false_type())
         : E <= 64  ? f(std::integral_constant<int, 4>(), std::false_type())
         : E <= 128 ? f(std::integral_constant<int, 8>(), std::false_type())
                    : f(std::integral_constant<int, 16>(), std::false_type());
}

template <typename T>
hipError_t loss_t(const moe_balance& b, const T* logits, const int32_t* topk, const float* bias, const uint8_t* mask,
                  float* loss, int32_t* counts, float* state, char* ws, hipStream_t s) {
  const int64_t B = b.N / b.seq_len, chunk = chunk_of(b), chunks = chunks_of(b);
  float* parts = reinterpret_cast<float*>(ws);
  SeqSum* sums = reinterpret_cast<SeqSum*>(ws + parts_bytes(b));
  int32_t* seq_counts = B == 1 ? counts : reinterpret_cast<int32_t*>(ws + parts_bytes(b) + pad(size_t(B) * sizeof(SeqSum)));
  const Results to{parts, state, loss, counts, b.alpha, b.z_coef};
  const bool one = in_one(b);
  const hipError_t st = by_experts<T>(b.E, [&](auto nv, auto vec) {
    const bool sigmoid = b.score == MOE_SCORE_SIGMOID;
    if constexpr (nv.value * kLanes <= kWave)
      if (one) {
        const auto kernel = topk == nullptr ? k_balance_parts<T, nv.value, vec.value, true, true>
                                            : k_balance_parts<T, nv.value, vec.value, false, true>;
        kernel<<<dim3(1), dim3(kOneRows * kLanes), 0, s>>>(logits, topk, bias, mask, to, int(b.E), int(b.K), int(b.N),
                                                           int(b.N), 1, sigmoid);
        return hipGetLastError();
      }
    const auto kernel = topk == nullptr ? k_balance_parts<T, nv.value, vec.value, true, false>
                                        : k_balance_parts<T, nv.value, vec.value, false, false>;
    kernel<<<dim3(unsigned(B * chunks)), dim3(256), 0, s>>>(logits, topk, bias, mask, to, int(b.E), int(b.K),
                                                            int(b.seq_len), int(chunk), int(chunks), sigmoid);
    return hipGetLastError();
  });
  if (st != hipSuccess || one) return st;
  int lanes = 1;
  while (lanes < b.E) lanes *= 2;
  const unsigned threads = lanes * chunks > 2048 ? 1024 : 256;  // lanes is 256 at most
  k_balance_seq<<<dim3(unsigned(B)), dim3(threads), 0, s>>>(parts, state, sums, seq_counts, loss, int(b.E), lanes,
                                                         int(b.K), int(chunks), int(B), b.alpha, b.z_coef);
  if (B > 1)
    k_balance_total<<<dim3(unsigned(1 + (b.E + 15) / 16)), dim3(256), 0, s>>>(sums, seq_counts, state, counts, loss,
                                                                             int(b.E), int(B), b.alpha, b.z_coef);
  return hipGetLastError();
}

template <typename T>
hipError_t bwd_t(const moe_balance& b, const T* logits, const uint8_t* mask, const float* state, const float* dloss,
                 T* dlogits, hipStream_t s) {
  return by_experts<T>(b.E, [&](auto nv, auto vec) {
    k_balance_bwd<T, nv.value, vec.value><<<dim3(unsigned((b.N + kRows - 1) / kRows)), dim3(256), 0, s>>>(
        logits, mask, state, dloss, dlogits, b.N, int(b.E), int(b.seq_len), b.alpha, b.z_coef,
        b.score == MOE_SCORE_SIGMOID);
    return hipGetLastError();
  });
}

}  // namespace

namespace moe_launch {

size_t balance_state(const moe_balance& b) { return size_t(state_words(b.N / b.seq_len, b.E)) * 4; }

size_t balance_ws(const moe_balance& b) {
  const size_t B = size_t(b.N / b.seq_len);
  return parts_bytes(b) + (B == 1 ? 0 : pad(B * sizeof(SeqSum)) + pad(B * b.E * 4));
}

hipError_t balance_loss(const moe_balance& b, const void* logits, const int32_t* topk, const float* bias,
                        const uint8_t* mask, float* loss, int32_t* counts, void* state, void* ws, hipStream_t s) {
  char* w = static_cast<char*>(ws);
  float* st = static_cast<float*>(state);
  return b.dtype == MOE_BF16
             ? loss_t(b, static_cast<const bf16_t*>(logits), topk, bias, mask, loss, counts, st, w, s)
             : loss_t(b, static_cast<const float*>(logits), topk, bias, mask, loss, counts, st, w, s);
}

hipError_t balance_loss_bwd(const moe_balance& b, const void* logits, const uint8_t* mask, const void* state,
                            const float* dloss, void* dlogits, hipStream_t s) {
  const float* st = static_cast<const float*>(state);
  return b.dtype == MOE_BF16
             ? bwd_t(b, static_cast<const bf16_t*>(logits), mask, st, dloss, static_cast<bf16_t*>(dlogits), s)
             : bwd_t(b, static_cast<const float*>(logits), mask, st, dloss, static_cast<float*>(dlogits), s);
}

}  // namespace moe_launch
