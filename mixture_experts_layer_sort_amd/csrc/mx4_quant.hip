// Tensors to microscaled 4-bit floating point and back (moe_mx4 in moe.h):
// blocks of 32 values along the contraction axis with one power of two,
//   s = max(floor(log2 max|v|) - 2, -127),  q = rne(v / 2^s), |q| <= 6.
// floor(log2) is the exponent field of the largest magnitude, so the scale byte
// is max(field - 2, 0) (255 stays: an infinite or NaN value in the block), and the
// hardware's conversions take a scale as a float's exponent field.  They round to
// nearest with ties to even, saturate at 6 and keep subnormal inputs.
// Bound by the bytes read and written.
#include <algorithm>

#include "mx4.h"

namespace {
using namespace moe;

typedef uint32_t words4_t __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t scale_byte(uint32_t field) {
  return field == 255u ? 255u : field > 2u ? field - 2u : 0u;
}
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }
// 255 is NaN.
__device__ __forceinline__ float known_scale(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7fc00000u : byte << 23);
}

// One 16-byte vector of V values of type T, as quantised and dequantised.
template <typename T> struct Vec;
template <> struct Vec<bf16_t> {
  static constexpr int V = 8;
  // exponent fields of the largest magnitudes of the V columns of `n` vectors
  template <int N>
  static __device__ __forceinline__ void fields(const words4_t (&w)[N], uint32_t (&f)[V]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u16x2_t m = {0, 0};
#pragma unroll
      for (int r = 0; r < N; ++r)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, uint32_t(w[r][i] & 0x7fff7fffu)));
      f[2 * i] = m[0] >> 7;
      f[2 * i + 1] = m[1] >> 7;
    }
  }
  // codes of eight rows' values of column j
  static __device__ __forceinline__ uint32_t column(const words4_t* w, int j, float scale) {
    const uint32_t pick = j % 2 ? 0x07060302u : 0x05040100u;
    bf16x2_t p[4];
#pragma unroll
    for (int b = 0; b < 4; ++b)
      p[b] = __builtin_bit_cast(bf16x2_t, __builtin_amdgcn_perm(w[2 * b + 1][j / 2], w[2 * b][j / 2], pick));
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, p[0], scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, p[1], scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, p[2], scale, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, p[3], scale, 3);
  }
  // eight rows of V columns from the columns' codes
  static __device__ __forceinline__ void rows(const uint32_t (&code)[V], const float (&scale)[V], words4_t (&w)[8]) {
    uint32_t d[V][4];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      d[j][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code[j], scale[j], 0));
      d[j][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code[j], scale[j], 1));
      d[j][2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code[j], scale[j], 2));
      d[j][3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code[j], scale[j], 3));
    }
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[r][i] = __builtin_amdgcn_perm(d[2 * i + 1][r / 2], d[2 * i][r / 2], r % 2 ? 0x07060302u : 0x05040100u);
  }
};
template <> struct Vec<float> {
  static constexpr int V = 4;
  template <int N>
  static __device__ __forceinline__ void fields(const words4_t (&w)[N], uint32_t (&f)[V]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int r = 0; r < N; ++r) m = max(m, w[r][i] & 0x7fffffffu);
      f[i] = m >> 23;
    }
  }
  static __device__ __forceinline__ uint32_t column(const words4_t* w, int j, float scale) {
    float v[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) v[r] = __uint_as_float(w[r][j]);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], scale, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], scale, 3);
  }
  static __device__ __forceinline__ void rows(const uint32_t (&code)[V], const float (&scale)[V], words4_t (&w)[8]) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      f32x2_t d[4];
      d[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[j], scale[j], 0);
      d[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[j], scale[j], 1);
      d[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[j], scale[j], 2);
      d[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[j], scale[j], 3);
#pragma unroll
      for (int r = 0; r < 8; ++r) w[r][j] = __float_as_uint(d[r / 2][r % 2]);
    }
  }
};

// Weights [count][K][C].  A wave has 128 rows of V strips of 16 columns; lane (g, o) the
// 32 rows from 32g on of V adjacent columns, one 16-byte load a row (256 contiguous
// bytes for 16 lanes), so that each column's block is in one lane's registers: its
// codes need no exchange, and leave in V * 16 contiguous bytes.  A workgroup is one
// wave, which fills the chip with small tensors too (8 x 512 x 1024 bf16: 5.2 us,
// with four waves 6.7; a scale's bytes meet in the L2).
template <typename T>
__global__ __launch_bounds__(kWave) void k_mx4_weights(const T* __restrict__ v, words4_t* __restrict__ codes,
                                                       uint8_t* __restrict__ scales, int K, int C, int chunks,
                                                       int groups) {
  typedef Vec<T> W;
  constexpr int V = W::V;
  const int g = lane_id() / 16, o = lane_id() % 16;
  const int b = blockIdx.x / (4 * groups), kt = blockIdx.x % (4 * groups), chunk = b % chunks;
  const int64_t m = b / chunks, strip = m * (C / 16) + int64_t(chunk) * V + o * V / 16;
  const int c = o * V % 16;
  uint8_t* mine = scales + ((strip * groups + kt / 4) * kWave + g * 16 + c) * 4 + kt % 4;
  if (kt >= K / kMxTile) {
#pragma unroll
    for (int j = 0; j < V; ++j) mine[4 * j] = 0;
    return;
  }
  const T* p = v + (m * K + kt * kMxTile + 32 * g) * C + int64_t(chunk) * 16 * V + o * V;
  words4_t w[32];
#pragma unroll
  for (int r = 0; r < 32; ++r) w[r] = __builtin_nontemporal_load(reinterpret_cast<const words4_t*>(p + int64_t(r) * C));
  uint32_t f[V];
  W::fields(w, f);
  words4_t* to = codes + (strip * (K / kMxTile) + kt) * kWave + g * 16 + c;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t s = scale_byte(f[j]);
    words4_t out;
#pragma unroll
    for (int d = 0; d < 4; ++d) out[d] = W::column(w + 8 * d, j, scale_of(s));
    to[j] = out;
    mine[4 * j] = uint8_t(s);
  }
}

template <typename T>
__global__ __launch_bounds__(kWave) void k_mx4_weights_back(const words4_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, T* __restrict__ v,
                                                            int K, int C, int chunks) {
  typedef Vec<T> W;
  constexpr int V = W::V;
  const int g = lane_id() / 16, o = lane_id() % 16;
  const int tiles = K / kMxTile, groups = mx_groups(K);
  const int b = blockIdx.x / (4 * groups), kt = blockIdx.x % (4 * groups), chunk = b % chunks;
  if (kt >= tiles) return;
  const int64_t m = b / chunks, strip = m * (C / 16) + int64_t(chunk) * V + o * V / 16;
  const int c = o * V % 16;
  const words4_t* from = codes + (strip * tiles + kt) * kWave + g * 16 + c;
  const uint8_t* s = scales + ((strip * groups + kt / 4) * kWave + g * 16 + c) * 4 + kt % 4;
  words4_t code[V];
  float scale[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    code[j] = from[j];
    scale[j] = known_scale(s[4 * j]);
  }
  T* p = v + (m * K + kt * kMxTile + 32 * g) * C + int64_t(chunk) * 16 * V + o * V;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    uint32_t at[V];
#pragma unroll
    for (int j = 0; j < V; ++j) at[j] = code[j][d];
    words4_t w[8];
    W::rows(at, scale, w);
#pragma unroll
    for (int r = 0; r < 8; ++r) *reinterpret_cast<words4_t*>(p + int64_t(8 * d + r) * C) = w[r];
  }
}

// Eight consecutive values as float.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float* out) {
  Vec16<T>::load(p, out);
  if (Vec16<T>::n == 4) Vec16<T>::load(p + 4, out + 4);
}

// Rows [count][K].  A wave takes 512 values of a row at a time (a group of 16
// scales), a lane eight of them, four lanes a block.
constexpr int kRowItems = 4;  // groups a wave has under way
template <typename T>
__global__ __launch_bounds__(256) void k_mx4_rows(const T* __restrict__ v, uint32_t* __restrict__ codes,
                                                  uint32_t* __restrict__ scales, int64_t items, int K, int groups) {
  const int lane = lane_id();
  const int64_t first = (int64_t(blockIdx.x) * 4 + threadIdx.x / kWave) * kRowItems;
  float x[kRowItems][8];
  int64_t at[kRowItems];
#pragma unroll
  for (int i = 0; i < kRowItems; ++i) {
    const int64_t item = first + i, row = item / groups;
    const int k = int(item - row * groups) * kMxGroup + 8 * lane;
    at[i] = item < items && k < K ? row * K + k : -1;
    if (at[i] >= 0) {
      load8(v + at[i], x[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i][j] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < kRowItems; ++i) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(x[i][j]) & 0x7fffffffu);
    m = max(m, uint32_t(__shfl_xor(int(m), 1, kWave)));
    m = max(m, uint32_t(__shfl_xor(int(m), 2, kWave)));
    const uint32_t s = scale_byte(m >> 23);
    const float scale = scale_of(s);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[i][0], x[i][1], scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[i][2], x[i][3], scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[i][4], x[i][5], scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[i][6], x[i][7], scale, 3);
    if (at[i] >= 0) codes[at[i] / 8] = c;
    // block 4*kt + g of the group is byte kt of word g
    uint32_t word = 0;
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) word |= uint32_t(__shfl(int(s), (4 * kt + lane % 4) * 4, kWave)) << (8 * kt);
    if (lane < 4 && first + i < items) scales[(first + i) * 4 + lane] = word;
  }
}

template <typename T>
__global__ __launch_bounds__(256) void k_mx4_rows_back(const uint32_t* __restrict__ codes,
                                                       const uint8_t* __restrict__ scales, T* __restrict__ v,
                                                       int64_t words, int K, int groups) {
  const int per = K / 8;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < words; i += int64_t(gridDim.x) * 256) {
    const int64_t row = i / per;
    const int b = int(i - row * per) / 4, kt = b / 4, g = b % 4;
    const float s = known_scale(scales[((row * groups + kt / 4) * 4 + g) * 4 + kt % 4]);
    const uint32_t c = codes[i];
    f32x2_t d[4];
    d[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0);
    d[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
    d[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2);
    d[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3);
    float o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = d[j / 2][j % 2];
    Vec16<T>::store(v + i * 8, o);
    if (Vec16<T>::n == 4) Vec16<T>::store(v + i * 8 + 4, o + 4);
  }
}

template <typename T>
hipError_t quantize_t(bool rows, int64_t count, int64_t k, int64_t cols, const T* v, void* codes, void* scales,
                      hipStream_t s) {
  const int groups = mx_groups(k);
  if (rows) {
    const int64_t items = count * groups, per = 4 * kRowItems;
    k_mx4_rows<T><<<dim3(unsigned((items + per - 1) / per)), dim3(256), 0, s>>>(
        v, static_cast<uint32_t*>(codes), static_cast<uint32_t*>(scales), items, int(k), groups);
  } else {
    const int64_t chunks = cols / (16 * Vec<T>::V);
    k_mx4_weights<T><<<dim3(unsigned(count * chunks * groups * 4)), dim3(kWave), 0, s>>>(
        v, static_cast<words4_t*>(codes), static_cast<uint8_t*>(scales), int(k), int(cols), int(chunks), groups);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t dequantize_t(bool rows, int64_t count, int64_t k, int64_t cols, const moe_launch::Mx4& q, T* v,
                        hipStream_t s) {
  const int groups = mx_groups(k);
  if (rows) {
    const int64_t words = count * k / 8;
    k_mx4_rows_back<T><<<dim3(unsigned(std::min<int64_t>((words + 255) / 256, 1 << 20))), dim3(256), 0, s>>>(
        static_cast<const uint32_t*>(q.codes), static_cast<const uint8_t*>(q.scales), v, words, int(k), groups);
  } else {
    const int64_t chunks = cols / (16 * Vec<T>::V);
    k_mx4_weights_back<T><<<dim3(unsigned(count * chunks * groups * 4)), dim3(kWave), 0, s>>>(
        static_cast<const words4_t*>(q.codes), static_cast<const uint8_t*>(q.scales), v, int(k), int(cols),
        int(chunks));
  }
  return hipGetLastError();
}

}  // namespace

namespace moe_launch {

hipError_t mx4_quantize(bool rows, int64_t count, int64_t k, int64_t cols, int dtype, const void* v, void* codes,
                        void* scales, hipStream_t s) {
  return dtype == MOE_BF16 ? quantize_t(rows, count, k, cols, static_cast<const bf16_t*>(v), codes, scales, s)
                           : quantize_t(rows, count, k, cols, static_cast<const float*>(v), codes, scales, s);
}

hipError_t mx4_dequantize(bool rows, int64_t count, int64_t k, int64_t cols, int dtype, const Mx4& q, void* v,
                          hipStream_t s) {
  return dtype == MOE_BF16 ? dequantize_t(rows, count, k, cols, q, static_cast<bf16_t*>(v), s)
                           : dequantize_t(rows, count, k, cols, q, static_cast<float*>(v), s);
}

}  // namespace moe_launch
