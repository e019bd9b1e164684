// Grouped products over many tokens with rows and experts in 4 bits
// (moe_mx4_gate_up, moe_mx4_down in moe.h) on the scaled 16x16x128 matrix
// instruction: products of codes are exact, each block of 32 is scaled by both its
// powers of two, sums are float32.
//
// A workgroup has 16*RG rows of one list tile and 16 strips of 16 columns, each of
// its four waves all the rows and four strips (of gate/up: two strips of both
// matrices, so that the activation is formed in registers).  Per step, 512 values
// of the contraction:
//  - rows: moved by the LDS DMA in the order in which the instruction takes them
//    (a lane's 16 bytes from anywhere, so the gather costs nothing; the LDS reads
//    are contiguous over the lanes), one step ahead, two buffers;
//  - weights: each strip is read by one wave only, so they go straight to
//    registers, a step ahead as well; a load is 1 KiB of contiguous memory;
//  - scales: a word for four tiles of the contraction; the instruction picks the
//    byte.
// Weights are the row operand: a lane ends with four neighbouring columns of a row.
#include <algorithm>

#include "mma_lds.h"
#include "mx4.h"

namespace {
using namespace moe;
using namespace moe_mma;

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

constexpr int kGWaves = 4;
constexpr int kGNT = kGWaves * kWave;
constexpr int kStrips = 4;  // of a wave
constexpr int kStep = 4;    // tiles of a step: a word of scales

template <int RG> struct Stage {
  static constexpr int A = RG * kStep * 1024;  // [row group][tile][lane][16 bytes]
  static constexpr int S = RG * 16 * 16;       // [row][16 bytes]
  static constexpr int BYTES = A + S;
};

__device__ __forceinline__ void dma_bytes(const void* g, char* lds_wave) {
  __builtin_amdgcn_global_load_lds(static_cast<const char*>(g), (LDS_AS void*)lds_wave, 16, 0, 0);
}

// A wave's weights of one step.
struct Weights {
  i32x4_t b[kStep][kStrips];
  int s[kStrips];
};

// acc[row group][strip] += weights . rows over one step of `tiles` tiles.
template <int RG>
__device__ __forceinline__ void step(const char* __restrict__ rows, const Weights& w, int tiles,
                                     f32x4_t (&acc)[RG][kStrips]) {
  const int lane = lane_id(), g = lane / 16, c = lane % 16;
  int s[RG];
#pragma unroll
  for (int r = 0; r < RG; ++r)
    s[r] = *reinterpret_cast<const int*>(rows + Stage<RG>::A + (r * 16 + c) * 16 + g * 4);
  auto tile = [&](auto kt) {
    constexpr int KT = decltype(kt)::value;
#pragma unroll
    for (int r = 0; r < RG; ++r) {
      const i32x4_t a = *reinterpret_cast<const i32x4_t*>(rows + (r * kStep + KT) * 1024 + lane * 16);
      const i32x8_t x = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < kStrips; ++i) {
        const i32x4_t b = w.b[KT][i];
        acc[r][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(i32x8_t{b[0], b[1], b[2], b[3], 0, 0, 0, 0}, x,
                                                                     acc[r][i], 4, 4, KT, w.s[i], KT, s[r]);
      }
    }
  };
  tile(std::integral_constant<int, 0>());
  if (tiles > 1) tile(std::integral_constant<int, 1>());
  if (tiles > 2) tile(std::integral_constant<int, 2>());
  if (tiles > 3) tile(std::integral_constant<int, 3>());
}

// The DMA of one step into `to`, then the step before it from `from`: distinct
// buffers, so that reads of one do not wait for the other.
template <int RG, typename Fetch>
__device__ __forceinline__ void fetch_and_step(char* __restrict__ to, const char* __restrict__ from, bool more,
                                               Fetch fetch, Weights& next, const Weights& w, int tiles,
                                               f32x4_t (&acc)[RG][kStrips]) {
  if (more) fetch(to, next);
  step<RG>(from, w, tiles, acc);
}

struct Rows {
  const char *codes, *scales;
  const int32_t* sorted_flat;  // null: rows as they lie
  int K;                       // row i is row sorted_flat[i] / K
};

// G and U of a workgroup's columns (GATE_UP) or one product.
template <typename T, int RG, bool GATE_UP>
__global__ __launch_bounds__(kGNT, 1) void k_mx4_product(Rows x, const char* __restrict__ codes0,
                                                         const char* __restrict__ scales0,
                                                         const char* __restrict__ codes1,
                                                         const char* __restrict__ scales1,
                                                         const int32_t* __restrict__ tiles,
                                                         const int32_t* __restrict__ num_tiles, T* __restrict__ out,
                                                         int L, int C) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  typedef Stage<RG> St;
  constexpr int SUB = 16 / RG, BN = (GATE_UP ? 2 : 4) * 16 * kGWaves;  // columns
  const int ncols = (C + BN - 1) / BN, nrows = *num_tiles * SUB;
  const int b = xcd_window_block<32>(blockIdx.x, nrows * ncols);
  if (b < 0) return;
  // eight row tiles by turns, then the next columns
  const int group = b / (8 * ncols), in = b % (8 * ncols), high = min(8, nrows - group * 8);
  const int rt = group * 8 + in % high, ct = in / high;
  const int t = rt / SUB, e = tiles[3 * t], row0 = tiles[3 * t + 1] + rt % SUB * 16 * RG;
  const int M = min(16 * RG, tiles[3 * t + 2] - rt % SUB * 16 * RG);
  if (M <= 0) return;
  const int wave = threadIdx.x / kWave, lane = lane_id(), g = lane / 16, c = lane % 16;
  const int kts = L / kMxTile, steps = mx_groups(L);

  // rows past the last repeat it; their results are dropped
  auto source = [&](int r) -> int64_t {
    const int i = row0 + min(r, M - 1);
    return x.sorted_flat != nullptr ? x.sorted_flat[i] / x.K : i;
  };
  const char* px[RG / kGWaves];
#pragma unroll
  for (int j = 0; j < RG / kGWaves; ++j)
    px[j] = x.codes + source((wave * (RG / kGWaves) + j) * 16 + c) * (L / 2) + g * 16;
  // scales of 64 rows an instruction
  const char* ps = x.scales + source((wave * kWave + lane) % (16 * RG)) * steps * 16;

  // the wave's strips; those past the last column repeat it, their results are dropped
  const int64_t strips = C / 16;
  const char *pw[kStrips], *pws[kStrips];
#pragma unroll
  for (int i = 0; i < kStrips; ++i) {
    const int64_t s = GATE_UP ? ct * (BN / 16) + wave * 2 + i % 2
                              : min(int64_t(ct) * (BN / 16) + wave * kStrips + i, strips - 1);
    pw[i] = (GATE_UP && i >= 2 ? codes1 : codes0) + (mx_strip_codes(e * strips + s, L) + lane) * 16;
    pws[i] = (GATE_UP && i >= 2 ? scales1 : scales0) + (mx_strip_scales(e * strips + s, L) + lane) * 4;
  }

  int q = 0;  // the step that fetch() is for
  auto fetch = [&](char* to, Weights& w) {
    const int n = min(kStep, kts - q * kStep);
#pragma unroll
    for (int i = 0; i < kStrips; ++i) w.s[i] = *reinterpret_cast<const int*>(pws[i] + int64_t(q) * kWave * 4);
#pragma unroll
    for (int kt = 0; kt < kStep; ++kt)
      if (kt < n) {
#pragma unroll
        for (int i = 0; i < kStrips; ++i)
          w.b[kt][i] = *reinterpret_cast<const i32x4_t*>(pw[i] + (int64_t(q) * kStep + kt) * 1024);
#pragma unroll
        for (int j = 0; j < RG / kGWaves; ++j)
          dma_bytes(px[j] + (q * kStep + kt) * 64, to + ((wave * (RG / kGWaves) + j) * kStep + kt) * 1024);
      }
    if (wave * kWave < 16 * RG) dma_bytes(ps + q * 16, to + St::A + wave * 1024);
    ++q;
  };

  f32x4_t acc[RG][kStrips];
#pragma unroll
  for (int r = 0; r < RG; ++r)
#pragma unroll
    for (int i = 0; i < kStrips; ++i) acc[r][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  Weights w, next;
  fetch(lds, w);
  for (int i = 0; i < steps; ++i) {
    wait_vm<0>();
    lds_barrier();
    fetch_and_step<RG>(lds + (i + 1) % 2 * St::BYTES, lds + i % 2 * St::BYTES, i + 1 < steps, fetch, next, w,
                       min(kStep, kts - i * kStep), acc);
    w = next;
  }

  constexpr int PAIRS = GATE_UP ? 2 : kStrips;
#pragma unroll
  for (int r = 0; r < RG; ++r) {
    const int row = r * 16 + c;
    if (row >= M) continue;
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
      const int col = (ct * (BN / 16) + wave * PAIRS + i) * 16 + 4 * g;
      if (!GATE_UP && col >= C) continue;
      f32x4_t v = acc[r][i];
      if constexpr (GATE_UP) {
        // the hardware's reciprocal is good to 1 ulp
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = v[k] * __builtin_amdgcn_rcpf(1.0f + expf(-v[k])) * acc[r][i + 2][k];
      }
      T* to = out + int64_t(row0 + row) * C + col;
      if constexpr (sizeof(T) == 4)
        *reinterpret_cast<f32x4_t*>(to) = v;
      else
        *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
  }
}

template <typename T, int RG, bool GATE_UP>
hipError_t product(const moe_launch::Dims& d, const Rows& x, const moe_launch::Mx4& w0, const moe_launch::Mx4& w1,
                   const int32_t* tiles, const int32_t* num_tiles, T* out, int L, int C, hipStream_t s) {
  constexpr int bytes = 2 * Stage<RG>::BYTES, BN = (GATE_UP ? 2 : 4) * 16 * kGWaves;
  const hipError_t e = allow_lds<k_mx4_product<T, RG, GATE_UP>>(bytes);
  if (e != hipSuccess) return e;
  const int64_t blocks = moe_launch::max_tiles(d) * (16 / RG) * ((C + BN - 1) / BN);
  if (blocks > (int64_t(1) << 31) - 256) return hipErrorInvalidValue;
  k_mx4_product<T, RG, GATE_UP><<<dim3(unsigned((blocks + 255) / 256 * 256)), dim3(kGNT), bytes, s>>>(
      x, static_cast<const char*>(w0.codes), static_cast<const char*>(w0.scales),
      static_cast<const char*>(w1.codes), static_cast<const char*>(w1.scales), tiles, num_tiles, out, L, C);
  return hipGetLastError();
}

template <bool GATE_UP>
hipError_t product_any(const moe_launch::Dims& d, const Rows& x, const moe_launch::Mx4& w0, const moe_launch::Mx4& w1,
                       const int32_t* tiles, const int32_t* num_tiles, void* out, int L, int C, hipStream_t s) {
  const double rows = double(d.NK()) / double(d.E);
  auto run = [&](auto rg) {
    constexpr int RG = decltype(rg)::value;
    return d.dtype == MOE_BF16 ? product<bf16_t, RG, GATE_UP>(d, x, w0, w1, tiles, num_tiles,
                                                              static_cast<bf16_t*>(out), L, C, s)
                               : product<float, RG, GATE_UP>(d, x, w0, w1, tiles, num_tiles,
                                                             static_cast<float*>(out), L, C, s);
  };
  return rows <= 64.0    ? run(std::integral_constant<int, 4>())
         : rows <= 160.0 ? run(std::integral_constant<int, 8>())
                         : run(std::integral_constant<int, 16>());
}

Rows rows_of(const moe_launch::Mx4& x, const int32_t* sorted_flat, int64_t K) {
  return Rows{static_cast<const char*>(x.codes), static_cast<const char*>(x.scales), sorted_flat, int(K)};
}

}  // namespace

namespace moe_launch {

hipError_t mx4_gate_up(const Dims& d, const Mx4& x, const int32_t* sorted_flat, const Mx4& wg, const Mx4& wu,
                       const int32_t* tiles, const int32_t* num_tiles, void* act, hipStream_t s) {
  return product_any<true>(d, rows_of(x, sorted_flat, d.K), wg, wu, tiles, num_tiles, act, int(d.H), int(d.F), s);
}

hipError_t mx4_down(const Dims& d, const Mx4& act, const Mx4& wd, const int32_t* tiles, const int32_t* num_tiles,
                    void* ys, hipStream_t s) {
  return product_any<false>(d, rows_of(act, nullptr, 1), wd, wd, tiles, num_tiles, ys, int(d.F), int(d.H), s);
}

}  // namespace moe_launch
