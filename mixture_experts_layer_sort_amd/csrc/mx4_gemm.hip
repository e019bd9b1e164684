// Grouped products over many tokens with rows and experts in 4 bits
// (moe_mx4_gate_up, moe_mx4_down in moe.h) on the scaled 32x32x64 matrix
// instruction: products of codes are exact, each block of 32 is scaled by both its
// powers of two, sums are float32.  (The 16x16x128 form takes as long for half the
// work: 4.9 against 8.3 PFLOP/s in a loop of nothing else.)
//
// A workgroup has 128 rows of one list tile and 16 strips of 16 columns, each of its
// four waves all the rows and four strips (of gate/up: two strips of both matrices, so
// that the activation is formed in registers); two workgroups share a CU, so that one
// of them multiplies while the other waits for its first loads or stores its results.
// Per step, 256 values of the contraction:
//  - rows: moved by the LDS DMA two steps ahead, three buffers; a wave's request takes
//    8 rows of 128 bytes, whole cache lines (the gather costs nothing).  Requests of 64
//    bytes of 16 rows, half a line each, and rows through registers took 2220 us where
//    this takes 1910 to 1980: gate/up of 16384 tokens, H 4096, F 14336, E 8, K 2;
//  - weights: each strip is read by one wave only, so they go straight to
//    registers, of two steps: behind its last product a tile's registers take the same
//    tile of the step after the next (one step ahead and two buffers: 2 to 6 % slower
//    where few rows an expert leave the time to memory);
//  - scales: a word for four tiles of the contraction; the instruction picks the
//    byte.
// Weights are the row operand: a lane ends with groups of four neighbouring columns
// of a row.
// What bounds it there: the instruction runs 56 % of the cycles, at the 1.7 GHz that its
// power leaves on such data; a third of a workgroup's time is first loads, activation and
// stores.
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
constexpr int kPairs = 2;  // pairs of strips of a wave

constexpr int kStep = 2;  // tiles of a step

constexpr int kRows = 128, kGroups = kRows / 32;
// Of a step, in LDS: the rows, [row][(k/32)%8 ^ (row/2)%8][16 bytes], so that a block of 16 rows lies in all
// banks (with row%8 in half of them: 2.3 times the conflicts, 0.5 % more time), and their scales, [row][16 bytes].
constexpr int kRowBytes = kRows * 128, kStageBytes = kRowBytes + kRows * 16;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const char* base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), (short)0, bytes, 0x00020000);
}
// 16 bytes a lane from off to LDS.
__device__ __forceinline__ void dma_bytes(__amdgpu_buffer_rsrc_t r, uint32_t off, char* lds_wave) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LDS_AS void*)lds_wave, 16, int(off), 0, 0, 0);
}
__device__ __forceinline__ i32x4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// A wave's weights of one step: lane (h, c) = (lane / 32, lane % 32) holds of pair p the
// 32 values from 32 (2 * half + h) on of each tile, of column c of the pair.
struct Weights {
  i32x4_t b[kStep][2][kPairs];
};
// Their scales, a word for the four tiles of two steps.
typedef int Scales[2][kPairs];

// acc[row group][pair] += weights . rows over one step, the first (ODD = 0) or second of
// two that share their scales' words; tiles past the last one have zero weights.  Two row
// groups at a time; the next two are read while the products of these run (left to
// itself the compiler reads them right before their use).  behind(n) after batch n of
// products: memory requests that go out there one or two at a time, as a row of them
// holds up the wave, and its products.
constexpr int kBatch = 2, kBatches = 2 * kGroups / kBatch;  // of a tile
template <int ODD, typename Behind>
__device__ __forceinline__ void step(const char* __restrict__ rows, Weights& w, const Scales& ws,
                                     f32x16_t (&acc)[kGroups][kPairs], Behind behind) {
  const int lane = lane_id(), h = lane / 32;
  const char* mine = rows + lane % 32 * 128;
  const int first = (h ^ lane / 2 % 8) * 16;
  int s[2][kGroups];
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int r = 0; r < kGroups; ++r)
      s[f][r] = *reinterpret_cast<const int*>(rows + kRowBytes + (r * 32 + lane % 32) * 16 + (2 * f + h) * 4);
  i32x4_t a[2][kBatch];
  auto read = [&](int n, i32x4_t (&to)[kBatch]) {  // of all tiles' halves' row groups
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int at = n * kBatch + k, r = at % kGroups, f = at / kGroups % 2, kt = at / (2 * kGroups);
      to[k] = *reinterpret_cast<const i32x4_t*>(mine + (first ^ (kt * 64 + f * 32)) + r * 4096);
    }
  };
  read(0, a[0]);
  auto tile = [&](auto kt) {
    constexpr int KT = decltype(kt)::value;
#pragma unroll
    for (int b = 0; b < kBatches; ++b) {
      const int n = KT * kBatches + b;
      if (n + 1 < kStep * kBatches) read(n + 1, a[(n + 1) % 2]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int r = (b * kBatch + k) % kGroups, f = (b * kBatch + k) / kGroups;
        const i32x4_t v = a[n % 2][k];
        const i32x8_t x = {v[0], v[1], v[2], v[3], 0, 0, 0, 0};
#pragma unroll
        for (int p = 0; p < kPairs; ++p) {
          const i32x4_t q = w.b[KT][f][p];
          acc[r][p] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              i32x8_t{q[0], q[1], q[2], q[3], 0, 0, 0, 0}, x, acc[r][p], 4, 4, KT + 2 * ODD, ws[f][p], KT + 2 * ODD, s[f][r]);
          // in this order: without a side effect products sink to the end of the step, and the
          // operands of all of them stay in registers until there
          asm volatile("" : "+v"(acc[r][p]));
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      behind(n);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  tile(std::integral_constant<int, 0>());
  tile(std::integral_constant<int, 1>());
}

// One step from `from`, with the requests for the one after the next, whose rows go to `to`:
// distinct buffers, so that reads of one do not wait for the other.
template <int ODD, typename Request>
__device__ __forceinline__ void step_and_next(char* __restrict__ to, const char* __restrict__ from, Request request,
                                              Weights& w, const Scales& ws, f32x16_t (&acc)[kGroups][kPairs]) {
  step<ODD>(from, w, ws, acc, [&](int n) { request(n, to); });
}

struct Rows {
  const char *codes, *scales;
  const int32_t* sorted_flat;  // gate/up: row i is row sorted_flat[i] / K
  int K;
};

// A lane's 32x32 results, four groups of columns 8q + 4h .. + 3 of row lane % 32, as 16
// neighbouring columns from 16h on: the halves of the wave exchange two groups each.
__device__ __forceinline__ void gather_columns(const f32x16_t& v, float (&out)[16]) {
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[4 * q + k]), __float_as_uint(v[4 * q + 8 + k]),
                                                      false, false);
      out[8 * q + k] = __uint_as_float(x[0]);
      out[8 * q + 4 + k] = __uint_as_float(x[1]);
    }
}

// G and U of a workgroup's columns (GATE_UP) or one product.
template <typename T, bool GATE_UP>
__global__ __launch_bounds__(kGNT, 2) void k_mx4_product(Rows x, const char* __restrict__ codes0,
                                                         const char* __restrict__ scales0,
                                                         const char* __restrict__ codes1,
                                                         const char* __restrict__ scales1,
                                                         const int32_t* __restrict__ tiles,
                                                         const int32_t* __restrict__ num_tiles,
                                                         T* __restrict__ out, int L, int C, bool seconds_last) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  constexpr int SUB = MOE_TILE_M / kRows;
  constexpr int BN = (GATE_UP ? 1 : 2) * 32 * kGWaves;  // columns
  const int ncols = (C + BN - 1) / BN, tile_count = *num_tiles, nrows = tile_count * SUB, all = nrows * ncols;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id();
  const int kts = L / kMxTile, steps = (kts + kStep - 1) / kStep, groups = mx_groups(L);
  const int64_t strips = C / 16;

  // eight row tiles by turns, then the next columns
  const int b = xcd_window_block<32>(blockIdx.x, all);
  if (b < 0) return;
  const int group = b / (8 * ncols), in = b % (8 * ncols), high = min(8, nrows - group * 8);
  const int rt = group * 8 + in % high, ct = in / high;
  const int part = seconds_last ? rt / tile_count : rt % SUB;
  const int32_t* tile = tiles + 3 * (seconds_last ? rt - part * tile_count : rt / SUB);
  auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
  const int e = uniform(tile[0]), row0 = uniform(tile[1]) + part * kRows, M = min(kRows, uniform(tile[2]) - part * kRows);
  if (M <= 0) return;

  // the wave's strips, two a pair; a pair past the last column repeats the last one, its results
  // are dropped (C is a multiple of 32)
  __amdgpu_buffer_rsrc_t pw[kPairs], pws[kPairs];
#pragma unroll
  for (int p = 0; p < kPairs; ++p) {
    const int64_t s = e * strips + min(int64_t(ct) * (BN / 16) + (GATE_UP ? wave * 2 : wave * 4 + 2 * p), strips - 2);
    pw[p] = resource((GATE_UP && p > 0 ? codes1 : codes0) + mx_strip_codes(s, L) * 16, 2 * kts * 1024);
    pws[p] = resource((GATE_UP && p > 0 ? scales1 : scales0) + mx_strip_scales(s, L) * 4, 2 * groups * kWave * 4);
  }
  // a lane's place behind the first strip of a pair
  const uint32_t lane_code = lane % 32 / 16 * uint32_t(kts * 1024) + lane / 32 * 256 + lane % 16 * 16;
  const uint32_t lane_scale = lane % 32 / 16 * uint32_t(groups * 256) + lane / 32 * 64 + lane % 16 * 4;
  auto fetch_scales = [&](int q, Scales& to) {  // of step q and the next one
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int p = 0; p < kPairs; ++p)
        to[f][p] = __builtin_amdgcn_raw_buffer_load_b32(pws[p], lane_scale + q * kStep / 4 * (kWave * 4) + f * 128, 0, 0);
  };
  // Load j (half, pair) of tile k of step q.  Past the last tile it is asked for past the end of the
  // strips, which gives 0 without a branch around the load (its registers would be doubled).
  constexpr int PARTS = 2 * kPairs, LOADS = kStep * PARTS;  // of a tile's, of a step's weights
  auto fetch_tile = [&](int q, int k, int j, Weights& w) {
    const int kt = q * kStep + k;
    const uint32_t at = lane_code + (kt < kts ? uint32_t(kt) * 1024u : 1u << 31);
    w.b[k][j / kPairs][j % kPairs] = load16(pw[j % kPairs], at + j / kPairs * 512);
  };

  // Rows past the last repeat it; their results are dropped.  32-bit offsets: of all tokens for gathered
  // rows, else of the piece's.
  auto source = [&](int r) -> uint32_t {
    const int i = min(r, M - 1);
    return GATE_UP ? uint32_t(x.sorted_flat[row0 + i]) / uint32_t(x.K) : i;
  };
  const char* codes = x.codes + (GATE_UP ? 0 : int64_t(row0) * (L / 2));
  const char* scales = x.scales + (GATE_UP ? 0 : int64_t(row0) * groups * 16);
  // a request takes 8 rows, lane (r, b) the block of row r whose place in LDS is b; the last one scales of 64
  // rows (of waves 0 and 1)
  constexpr int REQUESTS = kRows / 8 / kGWaves, MOVED = REQUESTS + 1;
  auto block = [&](int j) -> uint32_t { return (lane % 8 ^ (lane / 16 + j % 2 * 4)) * 16; };
  uint32_t px[MOVED];
#pragma unroll
  for (int j = 0; j < REQUESTS; ++j) px[j] = source((wave * REQUESTS + j) * 8 + lane / 8) * uint32_t(L / 2) + block(j);
  px[REQUESTS] = source(wave * kWave + lane) * uint32_t(groups * 16);
  // Request n of step q's rows.  An odd last tile is brought twice; past the last step nothing is (zeros).
  auto fetch_rows = [&](int q, int n, char* to) {
    const int live = uniform(q < steps ? -1 : 0);
    if (n < REQUESTS) {
      dma_bytes(resource(codes + q * 128, live), px[n] - (2 * q + 1 < kts ? 0 : block(n) & 64), to + (wave * REQUESTS + n) * 1024);
    } else if (wave * kWave < kRows) {
      dma_bytes(resource(scales + q * kStep / 4 * 16, live), px[REQUESTS], to + kRowBytes + wave * 1024);
    }
  };

  Weights w[2];
  Scales ws, next;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
#pragma unroll
    for (int k = 0; k < MOVED; ++k) fetch_rows(q, k, lds + q * kStageBytes);
    if (q == 0) fetch_scales(0, ws);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < LOADS; ++k) fetch_tile(q, k / PARTS, k % PARTS, w[q]);
    __builtin_amdgcn_sched_barrier(0);
  }
  f32x16_t acc[kGroups][kPairs];
#pragma unroll
  for (int r = 0; r < kGroups; ++r)
#pragma unroll
    for (int p = 0; p < kPairs; ++p)
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[r][p][k] = 0.f;
  // Step i from its buffer, while what step i + 2 needs is asked for: behind the batches of the first tile
  // its rows, behind those of the second the weights of the first.  Past the last step too, where they
  // bring nothing: with as many requests on every path, the compiler's waits need not take the fewest.
  int from = 0;  // buffer of step i
  auto turn = [&](int i, auto odd) {
    constexpr int ODD = decltype(odd)::value;
    // the rows are here; the weights, and what the step before asked for, may still be on their way
    wait_vm<MOVED - 1 + LOADS + (ODD ? 2 * kPairs : 0)>();
    lds_barrier();
    constexpr int EACH = (PARTS + kBatches - 1) / kBatches, TWO = (MOVED + kBatches - 1) / kBatches;
    auto request = [&](int n, char* to) {
      const int b = n % kBatches;
      if (!ODD && n == 0) fetch_scales(i + 2, next);
      if (n < kBatches) {
#pragma unroll
        for (int k = TWO * b; k < TWO * b + TWO; ++k)
          if (k < MOVED) fetch_rows(i + 2, k, to);
      } else {
#pragma unroll
        for (int k = EACH * b; k < EACH * b + EACH; ++k)
          if (k < PARTS) fetch_tile(i + 2, 0, k, w[ODD]);
      }
      if (n + 1 == 2 * kBatches) {
#pragma unroll
        for (int k = 0; k < PARTS; ++k) fetch_tile(i + 2, 1, k, w[ODD]);
      }
    };
    const int to = from == 0 ? 2 : from - 1;
    step_and_next<ODD>(lds + to * kStageBytes, lds + from * kStageBytes, request, w[ODD], ws, acc);
    from = from == 2 ? 0 : from + 1;
  };
#pragma clang loop unroll(disable)
  for (int i = 0; i + 1 < steps; i += 2) {
    turn(i, std::integral_constant<int, 0>());
    turn(i + 1, std::integral_constant<int, 1>());
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int p = 0; p < kPairs; ++p) ws[f][p] = next[f][p];
  }
  if (steps % 2 != 0) turn(steps - 1, std::integral_constant<int, 0>());

  // 32-bit offsets from the piece's first row
  const uint32_t mine = (lane % 32 * uint32_t(C) + lane / 32 * 16) * uint32_t(sizeof(T));
#pragma unroll
  for (int r = 0; r < kGroups; ++r) {
#pragma unroll
    for (int p = 0; p < (GATE_UP ? 1 : kPairs); ++p) {
      const int col = ct * BN + (GATE_UP ? wave * 32 : wave * 64 + 32 * p);
      f32x16_t v = acc[r][p];
      if constexpr (GATE_UP) {
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = silu_f32(v[k]) * acc[r][1][k];
      }
      float o[16];
      gather_columns(v, o);
      char* to = reinterpret_cast<char*>(out + int64_t(row0 + r * 32) * C + col);
      if (r * 32 + lane % 32 < M && col < C) {
#pragma unroll
        for (int k = 0; k < 16; k += Vec16<T>::n)
          Vec16<T>::store(reinterpret_cast<T*>(to + mine + k * sizeof(T)), o + k);
      }
      __builtin_amdgcn_sched_barrier(0);  // one group's registers at a time
    }
  }
  wait_vm<0>();  // the LDS is given back only when nothing more goes there
}

template <typename T, bool GATE_UP>
hipError_t product(const moe_launch::Dims& d, const Rows& x, const moe_launch::Mx4& w0, const moe_launch::Mx4& w1,
                   const int32_t* tiles, const int32_t* num_tiles, T* out, int L, int C, hipStream_t s) {
  constexpr int bytes = 3 * kStageBytes, BN = (GATE_UP ? 1 : 2) * 32 * kGWaves;
  const hipError_t e = allow_lds<k_mx4_product<T, GATE_UP>>(bytes);
  if (e != hipSuccess) return e;
  const int64_t ncols = (C + BN - 1) / BN, pieces = moe_launch::max_tiles(d) * (MOE_TILE_M / kRows) * ncols;
  if (pieces > (int64_t(1) << 31) - 512) return hipErrorInvalidValue;
  // With few rows an expert most list tiles have no second 128 rows: those workgroups, which end at once, hold
  // up the ones behind them, so they come last.  Not where the first halves are half a window of
  // xcd_window_block or less: they would all lie on half of the XCDs.  And not with more rows, where both halves
  // read the expert's weights, side by side.  Times with them last and otherwise:
  //   gate/up of 64 experts, H 2048, F 1408 (704 first halves): 32 rows 42 and 55 us, 96 46 and 66, 128 70 and 70,
  //     144 81 and 67; of 8, H 4096, F 14336 (896): 101 and 125, 106 and 134, 158 and 145, 183 and 146;
  //   down of the same 64 experts (512): 23 and 31, 29 and 40, 41 and 43, 46 and 45; of the 8 (128): 70 and 60, 81
  //     and 70, 85 and 72, 88 and 74;
  //   contraction 8192, 80 rows, gate/up and down with 64 first halves 36 and 30, 42 and 40; 128: 44 and 31, 48 and
  //     43; 192: 45 and 52, 51 and 76; 256: 51 and 74, 60 and 81.
  const bool seconds_last = d.NK() <= 96 * d.E && std::min(d.NK(), d.E) * ncols > 128;
  const unsigned grid = unsigned((pieces + 255) / 256 * 256);
  k_mx4_product<T, GATE_UP><<<dim3(grid), dim3(kGNT), bytes, s>>>(
      x, static_cast<const char*>(w0.codes), static_cast<const char*>(w0.scales),
      static_cast<const char*>(w1.codes), static_cast<const char*>(w1.scales), tiles, num_tiles, out, L, C, seconds_last);
  return hipGetLastError();
}

template <bool GATE_UP>
hipError_t product_any(const moe_launch::Dims& d, const Rows& x, const moe_launch::Mx4& w0, const moe_launch::Mx4& w1,
                       const int32_t* tiles, const int32_t* num_tiles, void* out, int L, int C, hipStream_t s) {
  return d.dtype == MOE_BF16
             ? product<bf16_t, GATE_UP>(d, x, w0, w1, tiles, num_tiles, static_cast<bf16_t*>(out), L, C, s)
             : product<float, GATE_UP>(d, x, w0, w1, tiles, num_tiles, static_cast<float*>(out), L, C, s);
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
