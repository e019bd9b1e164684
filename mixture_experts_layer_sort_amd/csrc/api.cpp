// C ABI of the MoE layer library: argument validation on the host (nothing is
// enqueued when a check fails), then the kernel launches on the caller's
// stream.  No entry point allocates memory, synchronises or reads device
// memory back to the host.
#include <hip/hip_runtime_api.h>

#include <cstdint>

#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

#include "common.h"
#include "moe.h"

namespace {

using moe_launch::Dims;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Shape and limit checks shared by every entry point.
int check_dims(const moe_dims* d, Dims* out) {
  if (d == nullptr) return MOE_EINVAL;
  if (d->gemm_tiles < MOE_TILES_AUTO || d->gemm_tiles > MOE_TILES_128) return MOE_EINVAL;
  if (d->dtype != MOE_F32 && d->dtype != MOE_BF16) return MOE_EUNSUPPORTED;
  if (d->N < 0 || d->H <= 0 || d->F <= 0 || d->E <= 0 || d->K <= 0) return MOE_EINVAL;
  if (d->H % 128 != 0 || d->F % 128 != 0) return MOE_EINVAL;
  if (d->E > MOE_MAX_EXPERTS || d->K > MOE_MAX_TOPK || d->K > d->E) return MOE_EUNSUPPORTED;
  if (d->H > (int64_t(1) << 20) || d->F > (int64_t(1) << 20)) return MOE_EUNSUPPORTED;
  const int64_t lim = int64_t(1) << 31;
  if (d->N >= lim || d->N * d->K >= lim || d->N * d->E >= lim) return MOE_EUNSUPPORTED;
  out->N = d->N;
  out->H = d->H;
  out->F = d->F;
  out->E = d->E;
  out->K = d->K;
  out->dtype = d->dtype;
  out->tiles = d->gemm_tiles;
  return MOE_OK;
}

// Every listed pointer must be non-null and 16-byte aligned.
template <typename... P>
bool ptrs_ok(P... p) {
  const void* arr[] = {static_cast<const void*>(p)...};
  for (const void* q : arr)
    if (q == nullptr || !aligned16(q)) return false;
  return true;
}

int from_hip(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_EHIP; }

// The shared expert's dims: one expert, every token routed to it once.
bool is_shared(const Dims& D) { return D.E == 1 && D.K == 1; }

// Whether [a, a + na) and [b, b + nb) share a byte.
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && p < q + nb && q < p + na;
}

// Bytes of an [N, H] tensor of the element type.
size_t row_bytes(const Dims& D) { return size_t(D.N) * size_t(D.H) * (D.dtype == MOE_BF16 ? 2 : 4); }

// The dims of a decoding call and of its shared expert (may be null).
int check_decode(const moe_dims* d, const moe_dims* ds, Dims* D, int64_t* Fs) {
  int st = check_dims(d, D);
  if (st != MOE_OK) return st;
  *Fs = 0;
  if (ds != nullptr) {
    Dims S;
    st = check_dims(ds, &S);
    if (st != MOE_OK) return st;
    if (!is_shared(S) || S.N != D->N || S.H != D->H || S.dtype != D->dtype) return MOE_EINVAL;
    *Fs = S.F;
  }
  return D->N > MOE_DECODE_MAX_TOKENS ? MOE_EUNSUPPORTED : MOE_OK;
}

// Sizes of a 4-bit tensor; its bytes.
constexpr int64_t kMx4Side = int64_t(1) << 20;
struct Mx4Sizes {
  size_t codes, scales, values;  // values: how many
};
int check_mx4_sizes(int32_t order, int64_t count, int64_t k, int64_t cols, Mx4Sizes* out) {
  if (order != MOE_MX4_WEIGHTS && order != MOE_MX4_ROWS) return MOE_EINVAL;
  if (count < 0 || k <= 0 || cols <= 0 || k % 128 != 0) return MOE_EINVAL;
  if (order == MOE_MX4_ROWS ? cols != 1 : cols % 128 != 0) return MOE_EINVAL;
  if (k > kMx4Side || cols > kMx4Side || count >= int64_t(1) << 27) return MOE_EUNSUPPORTED;
  // a launch has less than 2^32 threads: 2^28 groups of 512 values of a row, and fewer workgroups of weights
  if (count > (int64_t(1) << 36) / k / cols) return MOE_EUNSUPPORTED;
  const size_t n = size_t(count) * size_t(k) * size_t(cols);
  *out = Mx4Sizes{n / 2, size_t(count) * size_t(cols) * size_t((k + 511) / 512) * 16, n};
  return MOE_OK;
}

// moe_mx4_decode's dims: those of moe_decode, sides that a 4-bit tensor can have.
int check_mx4_decode(const moe_dims* d, const moe_dims* ds, Dims* D, int64_t* Fs) {
  const int st = check_decode(d, ds, D, Fs);
  if (st != MOE_OK) return st;
  return D->H > kMx4Side || D->F > kMx4Side || *Fs > kMx4Side ? MOE_EUNSUPPORTED : MOE_OK;
}

bool mx4_ok(const moe_mx4* q) { return q != nullptr && ptrs_ok(q->codes, q->scales); }
moe_launch::Mx4 mx4_of(const moe_mx4* q) {
  return q == nullptr ? moe_launch::Mx4{nullptr, nullptr} : moe_launch::Mx4{q->codes, q->scales};
}

// Codes and scales [count][k][cols] of a tensor, as spans.
struct Span {
  const void* at;
  size_t bytes;
};
void add_mx4(Span* s, int* n, const moe_mx4* q, int64_t count, int64_t k, int64_t cols) {
  s[(*n)++] = Span{q->codes, size_t(count) * size_t(k) * size_t(cols) / 2};
  s[(*n)++] = Span{q->scales, size_t(count) * size_t(cols) * size_t((k + 511) / 512) * 16};
}
// Whether one of the first `written` spans shares a byte with any other one.
bool spans_overlap(const Span* s, int n, int written) {
  for (int i = 0; i < written; ++i)
    for (int j = i + 1; j < n; ++j)
      if (overlap(s[i].at, s[i].bytes, s[j].at, s[j].bytes)) return true;
  return false;
}

// A balance loss's sizes and options.
int check_balance(const moe_balance* b) {
  if (b == nullptr) return MOE_EINVAL;
  if (b->dtype != MOE_F32 && b->dtype != MOE_BF16) return MOE_EUNSUPPORTED;
  if (b->score != MOE_SCORE_SOFTMAX && b->score != MOE_SCORE_SIGMOID) return MOE_EINVAL;
  if (b->N < 0 || b->E <= 0 || b->K <= 0 || b->seq_len <= 0 || b->N % b->seq_len != 0) return MOE_EINVAL;
  if (!std::isfinite(b->alpha) || !std::isfinite(b->z_coef)) return MOE_EINVAL;
  if (b->E > MOE_MAX_EXPERTS || b->K > MOE_MAX_TOPK || b->K > b->E) return MOE_EUNSUPPORTED;
  const int64_t lim = int64_t(1) << 31;
  if (b->N >= lim || b->N * b->K >= lim || b->N * b->E >= lim) return MOE_EUNSUPPORTED;
  // launches of less than 2^32 threads: sixteen for a token, 256 for a sequence
  if (b->N >= int64_t(1) << 28 || b->N / b->seq_len > int64_t(1) << 23) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

// A list of gradients (out: the outputs count too).
int check_grads(const moe_grad* g, int64_t count, bool out) {
  if (count < 0 || (count > 0 && g == nullptr)) return MOE_EINVAL;
  if (count > MOE_GRAD_MAX_TENSORS) return MOE_EUNSUPPORTED;
  // a launch counts chunks in uint32, and steps by its workgroups (2^20 at most) past the last one
  const int64_t chunk = moe_launch::grad_chunk(), most = int64_t(1) << 31;
  int64_t chunks = 0;
  for (int64_t t = 0; t < count; ++t) {
    const moe_grad& q = g[t];
    if (q.n < 0) return MOE_EINVAL;
    if (q.in_dtype != MOE_F32 && q.in_dtype != MOE_BF16) return MOE_EINVAL;
    if (out && q.out_dtype != MOE_F32 && q.out_dtype != MOE_BF16) return MOE_EINVAL;
    if (q.n == 0) continue;
    const uintptr_t ie = q.in_dtype == MOE_BF16 ? 1 : 3, oe = q.out_dtype == MOE_BF16 ? 1 : 3;
    if (q.in == nullptr || (reinterpret_cast<uintptr_t>(q.in) & ie) != 0) return MOE_EINVAL;
    if (out && (q.out == nullptr || (reinterpret_cast<uintptr_t>(q.out) & oe) != 0)) return MOE_EINVAL;
    if (q.n > most * chunk) return MOE_EUNSUPPORTED;
    chunks += (q.n + chunk - 1) / chunk;
    if (chunks > most) return MOE_EUNSUPPORTED;
  }
  return MOE_OK;
}

// Outputs that overlap anything but their own input in place.
int check_grad_overlaps(const moe_grad* g, int64_t count, const void* norm, const void* ws) {
  struct Span {
    uintptr_t lo, hi;
    bool written;
  };
  std::unique_ptr<Span[]> s(new (std::nothrow) Span[size_t(2 * count + 2)]);
  if (s == nullptr) return MOE_EUNSUPPORTED;
  size_t m = 0;
  auto add = [&](const void* p, uintptr_t bytes, bool written) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    s[m++] = Span{lo, lo + bytes, written};
  };
  for (int64_t t = 0; t < count; ++t) {
    const moe_grad& q = g[t];
    if (q.n == 0) continue;
    add(q.out, uintptr_t(q.n) * (q.out_dtype == MOE_BF16 ? 2 : 4), true);
    if (q.in != q.out || q.in_dtype != q.out_dtype) add(q.in, uintptr_t(q.n) * (q.in_dtype == MOE_BF16 ? 2 : 4), false);
  }
  add(norm, sizeof(float), true);
  add(ws, MOE_GRAD_WS_BYTES, true);
  std::sort(s.get(), s.get() + m, [](const Span& a, const Span& b) { return a.lo < b.lo; });
  uintptr_t any = 0, written = 0;  // ends of the spans so far
  for (size_t i = 0; i < m; ++i) {
    if (s[i].lo < (s[i].written ? any : written)) return MOE_EINVAL;
    any = std::max(any, s[i].hi);
    if (s[i].written) written = std::max(written, s[i].hi);
  }
  return MOE_OK;
}

#define MOE_CHECK_DIMS(d, D)            \
  Dims D;                               \
  {                                     \
    int st_ = check_dims((d), &D);      \
    if (st_ != MOE_OK) return st_;      \
  }

}  // namespace

extern "C" {

int moe_abi_version(void) { return MOE_ABI_VERSION; }

const char* moe_status_str(int status) {
  switch (status) {
    case MOE_OK: return "ok";
    case MOE_EINVAL: return "invalid argument (shape, null or misaligned pointer)";
    case MOE_EUNSUPPORTED: return "unsupported configuration (limits or dtype)";
    case MOE_EWORKSPACE: return "workspace missing or too small";
    case MOE_EHIP: return "HIP runtime reported a launch error";
    case MOE_ESCRATCH: return "problem needs more scratch than the no-allocation entry point holds (4 MiB)";
    default: return "unknown status";
  }
}

int64_t moe_max_tiles(const moe_dims* d) {
  Dims D;
  if (check_dims(d, &D) != MOE_OK) return -1;
  return moe_launch::max_tiles(D);
}

size_t moe_workspace_bytes(const moe_dims* d, int32_t entry) {
  Dims D;
  if (check_dims(d, &D) != MOE_OK) return size_t(-1);
  switch (entry) {
    case MOE_ENTRY_PERMUTE_META: return moe_launch::permute_meta_ws(D);
    case MOE_ENTRY_ROUTE_BWD: return moe_launch::route_bwd_ws(D);
    case MOE_ENTRY_PERMUTE_BWD: return moe_launch::permute_bwd_ws(D);
    case MOE_ENTRY_AUX_LOSS: return moe_launch::aux_loss_ws(D);
    case MOE_ENTRY_ROUTE_BWD_AUX: return moe_launch::route_bwd_aux_ws(D);
    case MOE_ENTRY_SHARED_FFN: return is_shared(D) ? moe_launch::shared_ffn_ws(D) : size_t(-1);
    case MOE_ENTRY_SHARED_FFN_BWD: return is_shared(D) ? moe_launch::shared_ffn_bwd_ws(D) : size_t(-1);
    case MOE_ENTRY_ROUTE_META: return moe_launch::route_meta_ws(D);
    case MOE_ENTRY_RMS_NORM_BWD: return D.H <= MOE_NORM_MAX_H ? moe_launch::rms_norm_bwd_ws(D) : size_t(-1);
    default: return size_t(-1);
  }
}

int moe_route(const moe_dims* d, const void* x, const void* w_r, const float* logit_bias, int32_t* topk_idx,
              float* gates, hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!ptrs_ok(x, w_r, topk_idx, gates)) return MOE_EINVAL;
  if (logit_bias != nullptr && !aligned16(logit_bias)) return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  return from_hip(moe_launch::route(D, x, w_r, logit_bias, topk_idx, gates, stream));
}

int moe_route_meta(const moe_dims* d, const void* x, const void* w_r, const float* logit_bias, int32_t capacity,
                   int32_t* topk_idx, float* gates, int32_t* sorted_flat, int32_t* inv, int32_t* counts,
                   int32_t* offsets, int32_t* tiles, int32_t* num_tiles, void* ws, size_t ws_bytes,
                   hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!ptrs_ok(x, w_r, topk_idx, gates, sorted_flat, inv, counts, offsets, tiles, num_tiles)) return MOE_EINVAL;
  if (logit_bias != nullptr && !aligned16(logit_bias)) return MOE_EINVAL;
  if (capacity < 0) return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  const size_t need = moe_launch::route_meta_ws(D);
  if (ws == nullptr || ws_bytes < need || !aligned16(ws)) return MOE_EWORKSPACE;
  return from_hip(moe_launch::route_meta(D, x, w_r, logit_bias, capacity, topk_idx, gates, sorted_flat, inv, counts,
                                         offsets, tiles, num_tiles, ws, stream));
}

int moe_permute_meta_capacity(const moe_dims* d, const int32_t* topk_idx, int32_t capacity, int32_t* sorted_flat,
                              int32_t* inv, int32_t* counts, int32_t* offsets, int32_t* tiles, int32_t* num_tiles,
                              void* ws, size_t ws_bytes, hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!ptrs_ok(topk_idx, sorted_flat, inv, counts, offsets, tiles, num_tiles)) return MOE_EINVAL;
  if (capacity < 0) return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  const size_t need = moe_launch::permute_meta_ws(D);
  if (need > 0 && (ws == nullptr || ws_bytes < need || !aligned16(ws))) return MOE_EWORKSPACE;
  return from_hip(moe_launch::permute_meta(D, topk_idx, capacity, sorted_flat, inv, counts, offsets, tiles, num_tiles,
                                           ws, stream));
}

int moe_permute_meta(const moe_dims* d, const int32_t* topk_idx, int32_t* sorted_flat, int32_t* inv, int32_t* counts,
                     int32_t* offsets, int32_t* tiles, int32_t* num_tiles, void* ws, size_t ws_bytes,
                     hipStream_t stream) {
  return moe_permute_meta_capacity(d, topk_idx, INT32_MAX, sorted_flat, inv, counts, offsets, tiles, num_tiles, ws,
                                   ws_bytes, stream);
}

int moe_permute(const moe_dims* d, const void* x, const int32_t* sorted_flat, void* xs, hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!ptrs_ok(x, sorted_flat, xs)) return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  return from_hip(moe_launch::permute(D, x, sorted_flat, xs, stream));
}

int moe_ffn_gate_up(const moe_dims* d, const void* xs, const void* w_gate, const void* w_up, const int32_t* tiles,
                    const int32_t* num_tiles, void* g_save, void* u_save, void* act, hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!ptrs_ok(xs, w_gate, w_up, tiles, num_tiles, act)) return MOE_EINVAL;
  if ((g_save == nullptr) != (u_save == nullptr)) return MOE_EINVAL;
  if (g_save != nullptr && !ptrs_ok(g_save, u_save)) return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  return from_hip(moe_launch::ffn_gate_up(D, xs, nullptr, w_gate, w_up, tiles, num_tiles, g_save, u_save, act, stream));
}

int moe_ffn_gate_up_gather(const moe_dims* d, const void* x, const int32_t* sorted_flat, const void* w_gate,
                           const void* w_up, const int32_t* tiles, const int32_t* num_tiles, void* g_save,
                           void* u_save, void* act, hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!ptrs_ok(x, sorted_flat, w_gate, w_up, tiles, num_tiles, act)) return MOE_EINVAL;
  if ((g_save == nullptr) != (u_save == nullptr)) return MOE_EINVAL;
  if (g_save != nullptr && !ptrs_ok(g_save, u_save)) return MOE_EINVAL;
  if (D.N * D.H >= (int64_t(1) << 31)) return MOE_EUNSUPPORTED;  // 32-bit row offsets into x
  if (D.N == 0) return MOE_OK;
  return from_hip(
      moe_launch::ffn_gate_up(D, x, sorted_flat, w_gate, w_up, tiles, num_tiles, g_save, u_save, act, stream));
}

int moe_ffn_down(const moe_dims* d, const void* act, const void* w_down, const int32_t* tiles,
                 const int32_t* num_tiles, void* ys, hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!ptrs_ok(act, w_down, tiles, num_tiles, ys)) return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  return from_hip(moe_launch::ffn_down(D, act, w_down, tiles, num_tiles, ys, stream));
}

int moe_expert_ffn(const moe_dims* d, const void* xs, const void* w_gate, const void* w_up, const void* w_down,
                   const int32_t* tiles, const int32_t* num_tiles, void* g_save, void* u_save, void* act, void* ys,
                   hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!ptrs_ok(xs, w_gate, w_up, w_down, tiles, num_tiles, act, ys)) return MOE_EINVAL;
  if ((g_save == nullptr) != (u_save == nullptr)) return MOE_EINVAL;
  if (g_save != nullptr && !ptrs_ok(g_save, u_save)) return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  int st = from_hip(moe_launch::ffn_gate_up(D, xs, nullptr, w_gate, w_up, tiles, num_tiles, g_save, u_save, act, stream));
  if (st != MOE_OK) return st;
  return from_hip(moe_launch::ffn_down(D, act, w_down, tiles, num_tiles, ys, stream));
}

int moe_combine(const moe_dims* d, const void* ys, const float* gates, const int32_t* inv, void* y,
                hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!ptrs_ok(ys, gates, inv, y)) return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  return from_hip(moe_launch::combine(D, ys, gates, inv, nullptr, y, stream));
}

int moe_combine_bwd(const moe_dims* d, const void* dy, const void* ys, const float* gates, const int32_t* inv,
                    void* dys, float* dgates, hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!ptrs_ok(dy, ys, gates, inv, dys, dgates)) return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  return from_hip(moe_launch::combine_bwd(D, dy, ys, gates, inv, dys, dgates, stream));
}

int moe_route_bwd(const moe_dims* d, const void* x, const int32_t* topk_idx, const float* gates,
                  const float* dgates, float* dlogits, float* dw_r, void* ws, size_t ws_bytes, hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!ptrs_ok(x, topk_idx, gates, dgates, dlogits, dw_r)) return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  const size_t need = moe_launch::route_bwd_ws(D);
  if (ws == nullptr || ws_bytes < need || !aligned16(ws)) return MOE_EWORKSPACE;
  return from_hip(moe_launch::route_bwd(D, x, topk_idx, gates, dgates, dlogits, dw_r, ws, stream));
}

int moe_ffn_bwd_dact(const moe_dims* d, const void* dys, const void* w_down, const void* g_save, const void* u_save,
                     const int32_t* tiles, const int32_t* num_tiles, void* dg, void* du, hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!ptrs_ok(dys, w_down, g_save, u_save, tiles, num_tiles, dg, du)) return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  return from_hip(moe_launch::ffn_bwd_dact(D, dys, w_down, g_save, u_save, tiles, num_tiles, dg, du, stream));
}

int moe_ffn_bwd_dx(const moe_dims* d, const void* dg, const void* du, const void* w_gate, const void* w_up,
                   const int32_t* tiles, const int32_t* num_tiles, void* dxs, hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!ptrs_ok(dg, du, w_gate, w_up, tiles, num_tiles, dxs)) return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  return from_hip(moe_launch::ffn_bwd_dx(D, dg, du, w_gate, w_up, tiles, num_tiles, dxs, stream));
}

int moe_ffn_bwd_dw(const moe_dims* d, const void* xs, const void* act, const void* dys, const void* dg,
                   const void* du, const int32_t* offsets, float* dw_gate, float* dw_up, float* dw_down,
                   hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!ptrs_ok(xs, act, dys, dg, du, offsets, dw_gate, dw_up, dw_down)) return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  return from_hip(
      moe_launch::ffn_bwd_dw(D, xs, nullptr, act, dys, dg, du, offsets, dw_gate, dw_up, dw_down, stream));
}

int moe_ffn_bwd_dx_dw(const moe_dims* d, const void* dg, const void* du, const void* w_gate, const void* w_up,
                      const int32_t* tiles, const int32_t* num_tiles, void* dxs, const void* xs, const void* act,
                      const void* dys, const int32_t* offsets, float* dw_gate, float* dw_up, float* dw_down,
                      hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!ptrs_ok(dg, du, w_gate, w_up, tiles, num_tiles, dxs, xs, act, dys, offsets, dw_gate, dw_up, dw_down))
    return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  return from_hip(moe_launch::ffn_bwd_dx_dw(D, dg, du, w_gate, w_up, tiles, num_tiles, dxs, xs, nullptr, act, dys, offsets,
                                            dw_gate, dw_up, dw_down, stream));
}

int moe_ffn_bwd_dx_dw_gather(const moe_dims* d, const void* dg, const void* du, const void* w_gate,
                             const void* w_up, const int32_t* tiles, const int32_t* num_tiles, void* dxs,
                             const void* x, const int32_t* sorted_flat, const void* act, const void* dys,
                             const int32_t* offsets, float* dw_gate, float* dw_up, float* dw_down,
                             hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!ptrs_ok(dg, du, w_gate, w_up, tiles, num_tiles, dxs, x, sorted_flat, act, dys, offsets, dw_gate, dw_up,
               dw_down))
    return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  return from_hip(moe_launch::ffn_bwd_dx_dw(D, dg, du, w_gate, w_up, tiles, num_tiles, dxs, x, sorted_flat, act, dys,
                                            offsets, dw_gate, dw_up, dw_down, stream));
}

int moe_expert_ffn_bwd(const moe_dims* d, const void* dys, const void* xs, const void* w_gate, const void* w_up,
                       const void* w_down, const void* g_save, const void* u_save, const void* act,
                       const int32_t* offsets, const int32_t* tiles, const int32_t* num_tiles, void* dg, void* du,
                       void* dxs, float* dw_gate, float* dw_up, float* dw_down, hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!ptrs_ok(dys, xs, w_gate, w_up, w_down, g_save, u_save, act, offsets, tiles, num_tiles, dg, du, dxs, dw_gate,
               dw_up, dw_down))
    return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  int st = from_hip(moe_launch::ffn_bwd_dact(D, dys, w_down, g_save, u_save, tiles, num_tiles, dg, du, stream));
  if (st != MOE_OK) return st;
  return from_hip(moe_launch::ffn_bwd_dx_dw(D, dg, du, w_gate, w_up, tiles, num_tiles, dxs, xs, nullptr, act, dys, offsets,
                                            dw_gate, dw_up, dw_down, stream));
}

int moe_permute_bwd(const moe_dims* d, const void* dxs, const int32_t* inv, const int32_t* topk_idx,
                    const float* dlogits, const void* w_r, void* dx, void* ws, size_t ws_bytes, hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!ptrs_ok(dxs, inv, topk_idx, dlogits, w_r, dx)) return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  const size_t need = moe_launch::permute_bwd_ws(D);
  if (ws == nullptr || ws_bytes < need || !aligned16(ws)) return MOE_EWORKSPACE;
  return from_hip(moe_launch::permute_bwd(D, dxs, inv, topk_idx, dlogits, w_r, nullptr, dx, ws, stream, false));
}

int moe_permute_bwd_dense(const moe_dims* d, const void* dxs, const int32_t* inv, const int32_t* topk_idx,
                          const float* dlogits, const void* w_r, void* dx, void* ws, size_t ws_bytes,
                          hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!ptrs_ok(dxs, inv, topk_idx, dlogits, w_r, dx)) return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  const size_t need = moe_launch::permute_bwd_ws(D);
  if (ws == nullptr || ws_bytes < need || !aligned16(ws)) return MOE_EWORKSPACE;
  return from_hip(moe_launch::permute_bwd(D, dxs, inv, topk_idx, dlogits, w_r, nullptr, dx, ws, stream, true));
}

int moe_combine_shared(const moe_dims* d, const void* ys, const float* gates, const int32_t* inv,
                       const void* ys_shared, void* y, hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!ptrs_ok(ys, gates, inv, ys_shared, y)) return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  return from_hip(moe_launch::combine(D, ys, gates, inv, ys_shared, y, stream));
}

int moe_permute_bwd_add(const moe_dims* d, const void* dxs, const int32_t* inv, const int32_t* topk_idx,
                        const float* dlogits, const void* w_r, int32_t dense, const void* dx_add, void* dx, void* ws,
                        size_t ws_bytes, hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!ptrs_ok(dxs, inv, topk_idx, dlogits, w_r, dx_add, dx)) return MOE_EINVAL;
  if (dense != 0 && dense != 1) return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  const size_t need = moe_launch::permute_bwd_ws(D);
  if (ws == nullptr || ws_bytes < need || !aligned16(ws)) return MOE_EWORKSPACE;
  return from_hip(moe_launch::permute_bwd(D, dxs, inv, topk_idx, dlogits, w_r, dx_add, dx, ws, stream, dense == 1));
}

int moe_shared_ffn(const moe_dims* ds, const void* x, const void* w_gate, const void* w_up, const void* w_down,
                   void* g_save, void* u_save, void* act, void* ys, void* ws, size_t ws_bytes, hipStream_t stream) {
  MOE_CHECK_DIMS(ds, D);
  if (!is_shared(D)) return MOE_EINVAL;
  if (!ptrs_ok(x, w_gate, w_up, w_down, act, ys)) return MOE_EINVAL;
  if ((g_save == nullptr) != (u_save == nullptr)) return MOE_EINVAL;
  if (g_save != nullptr && !ptrs_ok(g_save, u_save)) return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  const size_t need = moe_launch::shared_ffn_ws(D);
  if (ws == nullptr || ws_bytes < need || !aligned16(ws)) return MOE_EWORKSPACE;
  return from_hip(moe_launch::shared_ffn(D, x, w_gate, w_up, w_down, g_save, u_save, act, ys, ws, stream));
}

int moe_shared_ffn_bwd(const moe_dims* ds, const void* x, const void* dy, const void* w_gate, const void* w_up,
                       const void* w_down, const void* g_save, const void* u_save, const void* act, void* dg, void* du,
                       void* dx_shared, float* dw_gate, float* dw_up, float* dw_down, void* ws, size_t ws_bytes,
                       hipStream_t stream) {
  MOE_CHECK_DIMS(ds, D);
  if (!is_shared(D)) return MOE_EINVAL;
  if (!ptrs_ok(x, dy, w_gate, w_up, w_down, g_save, u_save, act, dg, du, dx_shared, dw_gate, dw_up, dw_down))
    return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  const size_t need = moe_launch::shared_ffn_bwd_ws(D);
  if (ws == nullptr || ws_bytes < need || !aligned16(ws)) return MOE_EWORKSPACE;
  return from_hip(moe_launch::shared_ffn_bwd(D, x, dy, w_gate, w_up, w_down, g_save, u_save, act, dg, du, dx_shared,
                                             dw_gate, dw_up, dw_down, ws, stream));
}

int moe_aux_loss(const moe_dims* d, const void* x, const void* w_r, const float* logit_bias, const int32_t* counts,
                 float alpha, float* probs, float* loss, void* ws, size_t ws_bytes, hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!ptrs_ok(x, w_r, counts, probs, loss)) return MOE_EINVAL;
  if (logit_bias != nullptr && !aligned16(logit_bias)) return MOE_EINVAL;
  if (!std::isfinite(alpha)) return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  const size_t need = moe_launch::aux_loss_ws(D);
  if (ws == nullptr || ws_bytes < need || !aligned16(ws)) return MOE_EWORKSPACE;
  return from_hip(moe_launch::aux_loss(D, x, w_r, logit_bias, counts, alpha, probs, loss, ws, stream));
}

int moe_route_bwd_aux(const moe_dims* d, const void* x, const int32_t* topk_idx, const float* gates,
                      const float* dgates, const float* probs, const int32_t* counts, float aux_scale,
                      float* dlogits, float* dw_r, void* ws, size_t ws_bytes, hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!ptrs_ok(x, topk_idx, gates, dgates, probs, counts, dlogits, dw_r)) return MOE_EINVAL;
  if (!std::isfinite(aux_scale)) return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  const size_t need = moe_launch::route_bwd_aux_ws(D);
  if (ws == nullptr || ws_bytes < need || !aligned16(ws)) return MOE_EWORKSPACE;
  return from_hip(moe_launch::route_bwd_aux(D, x, topk_idx, gates, dgates, probs, counts, aux_scale, dlogits, dw_r,
                                            ws, stream));
}

size_t moe_decode_workspace_bytes(const moe_dims* d, const moe_dims* ds) {
  Dims D;
  int64_t Fs;
  if (check_decode(d, ds, &D, &Fs) != MOE_OK) return size_t(-1);
  return D.N == 0 ? 0 : moe_launch::decode_ws(D, Fs);
}

int moe_decode(const moe_dims* d, const void* x, const void* w_r, const float* logit_bias, const void* w_gate,
               const void* w_up, const void* w_down, const moe_dims* ds, const void* ws_gate, const void* ws_up,
               const void* ws_down, int32_t* topk_idx, float* gates, void* y, void* ws, size_t ws_bytes,
               hipStream_t stream) {
  Dims D;
  int64_t Fs;
  const int st = check_decode(d, ds, &D, &Fs);
  if (st != MOE_OK) return st;
  if (!ptrs_ok(x, w_r, w_gate, w_up, w_down, topk_idx, gates, y)) return MOE_EINVAL;
  if (logit_bias != nullptr && !aligned16(logit_bias)) return MOE_EINVAL;
  if (ds != nullptr ? !ptrs_ok(ws_gate, ws_up, ws_down)
                    : (ws_gate != nullptr || ws_up != nullptr || ws_down != nullptr))
    return MOE_EINVAL;
  const size_t need = D.N == 0 ? 0 : moe_launch::decode_ws(D, Fs), nk = size_t(D.N) * size_t(D.K) * 4;
  // what is written, then what is read: no written one shares a byte with any before or behind it
  const size_t es = D.dtype == MOE_BF16 ? 2 : 4, h = size_t(D.H) * es;
  const size_t wb = D.N == 0 ? 0 : size_t(D.E) * size_t(D.F) * h, sb = D.N == 0 ? 0 : size_t(Fs) * h;
  const size_t rb = D.N == 0 ? 0 : size_t(D.E) * h, bb = logit_bias == nullptr || D.N == 0 ? 0 : size_t(D.E) * 4;
  const void* const at[] = {y, topk_idx, gates, ws, x, w_r, logit_bias, w_gate, w_up, w_down, ws_gate, ws_up, ws_down};
  const size_t bytes[] = {row_bytes(D), nk, nk, need, row_bytes(D), rb, bb, wb, wb, wb, sb, sb, sb};
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 13; ++j)
      if (overlap(at[i], bytes[i], at[j], bytes[j])) return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  if (ws == nullptr || ws_bytes < need || !aligned16(ws)) return MOE_EWORKSPACE;
  return from_hip(moe_launch::decode(D, x, w_r, logit_bias, w_gate, w_up, w_down, Fs, ws_gate, ws_up, ws_down,
                                     topk_idx, gates, y, ws, stream));
}

int moe_rms_norm(const moe_dims* d, const void* x, const void* residual, const void* weight, float eps, void* h,
                 void* y, float* rstd, hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (D.H > MOE_NORM_MAX_H) return MOE_EUNSUPPORTED;
  if (!std::isfinite(eps) || eps <= 0.f) return MOE_EINVAL;
  if (!ptrs_ok(x, weight, y)) return MOE_EINVAL;
  if ((residual == nullptr) != (h == nullptr)) return MOE_EINVAL;
  if (residual != nullptr && !ptrs_ok(residual, h)) return MOE_EINVAL;
  if (rstd != nullptr && !aligned16(rstd)) return MOE_EINVAL;
  const size_t b = row_bytes(D), wb = b / size_t(D.N > 0 ? D.N : 1), rb = size_t(D.N) * 4;
  if (overlap(y, b, x, b) || overlap(y, b, weight, wb)) return MOE_EINVAL;
  if (residual != nullptr) {
    if (overlap(y, b, residual, b) || overlap(y, b, h, b) || overlap(h, b, weight, wb)) return MOE_EINVAL;
    if ((h != x && overlap(h, b, x, b)) || (h != residual && overlap(h, b, residual, b))) return MOE_EINVAL;
  }
  if (rstd != nullptr &&
      (overlap(rstd, rb, x, b) || overlap(rstd, rb, y, b) || overlap(rstd, rb, weight, wb) ||
       (residual != nullptr && (overlap(rstd, rb, residual, b) || overlap(rstd, rb, h, b)))))
    return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  return from_hip(moe_launch::rms_norm(D, x, residual, weight, eps, h, y, rstd, stream));
}

int moe_rms_norm_bwd(const moe_dims* d, const void* dy, const void* h, const void* weight, const float* rstd,
                     const void* dh, void* dx, float* dweight, void* ws, size_t ws_bytes, hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (D.H > MOE_NORM_MAX_H) return MOE_EUNSUPPORTED;
  if (!ptrs_ok(dy, h, weight, rstd, dx, dweight)) return MOE_EINVAL;
  if (dh != nullptr && !aligned16(dh)) return MOE_EINVAL;
  const size_t b = row_bytes(D), wb = b / size_t(D.N > 0 ? D.N : 1), rb = size_t(D.N) * 4;
  if ((dx != dy && overlap(dx, b, dy, b)) || (dh != nullptr && dx != dh && overlap(dx, b, dh, b)) ||
      overlap(dx, b, h, b) || overlap(dx, b, weight, wb) || overlap(dx, b, rstd, rb))
    return MOE_EINVAL;
  const size_t db = size_t(D.H) * 4;
  if (overlap(dweight, db, dx, b) || overlap(dweight, db, dy, b) || overlap(dweight, db, h, b) ||
      overlap(dweight, db, weight, wb) || overlap(dweight, db, rstd, rb) || (dh != nullptr && overlap(dweight, db, dh, b)))
    return MOE_EINVAL;
  const size_t need = D.N == 0 ? 0 : moe_launch::rms_norm_bwd_ws(D);
  if (overlap(ws, need, dweight, db) || overlap(ws, need, dx, b) || overlap(ws, need, dy, b) ||
      overlap(ws, need, h, b) || overlap(ws, need, weight, wb) || overlap(ws, need, rstd, rb) ||
      (dh != nullptr && overlap(ws, need, dh, b)))
    return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  if (ws == nullptr || ws_bytes < need || !aligned16(ws)) return MOE_EWORKSPACE;
  return from_hip(moe_launch::rms_norm_bwd(D, dy, h, weight, rstd, dh, dx, dweight, ws, stream));
}

int moe_grad_norm(const moe_grad* list, int64_t count, float* norm, void* ws, size_t ws_bytes, hipStream_t stream) {
  const int st = check_grads(list, count, false);
  if (st != MOE_OK) return st;
  if (norm == nullptr || (reinterpret_cast<uintptr_t>(norm) & 3u) != 0) return MOE_EINVAL;
  if (ws == nullptr || ws_bytes < MOE_GRAD_WS_BYTES || !aligned16(ws)) return MOE_EWORKSPACE;
  if (overlap(norm, sizeof(float), ws, MOE_GRAD_WS_BYTES)) return MOE_EINVAL;
  for (int64_t t = 0; t < count; ++t) {
    const size_t n = size_t(list[t].n) * (list[t].in_dtype == MOE_BF16 ? 2 : 4);
    if (overlap(list[t].in, n, norm, sizeof(float)) || overlap(list[t].in, n, ws, MOE_GRAD_WS_BYTES)) return MOE_EINVAL;
  }
  return from_hip(moe_launch::grad_norm(list, int(count), norm, ws, stream));
}

int moe_grad_clip(const moe_grad* list, int64_t count, float max_norm, float* norm, void* ws, size_t ws_bytes,
                  hipStream_t stream) {
  int st = check_grads(list, count, true);
  if (st != MOE_OK) return st;
  if (!std::isfinite(max_norm) || max_norm < 0.f) return MOE_EINVAL;
  if (norm == nullptr || (reinterpret_cast<uintptr_t>(norm) & 3u) != 0) return MOE_EINVAL;
  if (ws == nullptr || ws_bytes < MOE_GRAD_WS_BYTES || !aligned16(ws)) return MOE_EWORKSPACE;
  st = check_grad_overlaps(list, count, norm, ws);
  if (st != MOE_OK) return st;
  return from_hip(moe_launch::grad_clip(list, int(count), max_norm, norm, ws, stream));
}

size_t moe_mx4_code_bytes(int32_t order, int64_t count, int64_t k, int64_t cols) {
  Mx4Sizes z;
  return check_mx4_sizes(order, count, k, cols, &z) == MOE_OK ? z.codes : size_t(-1);
}

size_t moe_mx4_scale_bytes(int32_t order, int64_t count, int64_t k, int64_t cols) {
  Mx4Sizes z;
  return check_mx4_sizes(order, count, k, cols, &z) == MOE_OK ? z.scales : size_t(-1);
}

int moe_mx4_quantize(int32_t order, int64_t count, int64_t k, int64_t cols, int32_t dtype, const void* v,
                     const moe_mx4* q, hipStream_t stream) {
  Mx4Sizes z;
  const int st = check_mx4_sizes(order, count, k, cols, &z);
  if (st != MOE_OK) return st;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_EUNSUPPORTED;
  if (!ptrs_ok(v) || !mx4_ok(q)) return MOE_EINVAL;
  const Span s[] = {{q->codes, z.codes}, {q->scales, z.scales}, {v, z.values * (dtype == MOE_BF16 ? 2 : 4)}};
  if (spans_overlap(s, 3, 2)) return MOE_EINVAL;
  if (count == 0) return MOE_OK;
  return from_hip(moe_launch::mx4_quantize(order == MOE_MX4_ROWS, count, k, cols, dtype, v, q->codes, q->scales, stream));
}

int moe_mx4_dequantize(int32_t order, int64_t count, int64_t k, int64_t cols, int32_t dtype, const moe_mx4* q,
                       void* v, hipStream_t stream) {
  Mx4Sizes z;
  const int st = check_mx4_sizes(order, count, k, cols, &z);
  if (st != MOE_OK) return st;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_EUNSUPPORTED;
  if (!ptrs_ok(v) || !mx4_ok(q)) return MOE_EINVAL;
  const Span s[] = {{v, z.values * (dtype == MOE_BF16 ? 2 : 4)}, {q->codes, z.codes}, {q->scales, z.scales}};
  if (spans_overlap(s, 3, 1) || overlap(q->codes, z.codes, q->scales, z.scales)) return MOE_EINVAL;
  if (count == 0) return MOE_OK;
  return from_hip(moe_launch::mx4_dequantize(order == MOE_MX4_ROWS, count, k, cols, dtype, mx4_of(q), v, stream));
}

int moe_mx4_gate_up(const moe_dims* d, const moe_mx4* x, const int32_t* sorted_flat, const moe_mx4* w_gate,
                    const moe_mx4* w_up, const int32_t* tiles, const int32_t* num_tiles, void* act,
                    hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!mx4_ok(x) || !mx4_ok(w_gate) || !mx4_ok(w_up) || !ptrs_ok(sorted_flat, tiles, num_tiles, act)) return MOE_EINVAL;
  if (D.H > kMx4Side || D.F > kMx4Side) return MOE_EUNSUPPORTED;
  // the rows' codes are addressed by 32 bits from the first token's on
  if (D.N * D.H >= int64_t(1) << 33) return MOE_EUNSUPPORTED;
  Span s[10] = {{act, size_t(D.NK()) * size_t(D.F) * (D.dtype == MOE_BF16 ? 2 : 4)},
                {sorted_flat, size_t(D.NK()) * 4},
                {tiles, size_t(moe_launch::max_tiles(D)) * 12},
                {num_tiles, 4}};
  int n = 4;
  add_mx4(s, &n, x, D.N, D.H, 1);
  add_mx4(s, &n, w_gate, D.E, D.H, D.F);
  add_mx4(s, &n, w_up, D.E, D.H, D.F);
  if (D.N == 0) return MOE_OK;
  if (spans_overlap(s, n, 1)) return MOE_EINVAL;
  return from_hip(moe_launch::mx4_gate_up(D, mx4_of(x), sorted_flat, mx4_of(w_gate), mx4_of(w_up), tiles, num_tiles,
                                          act, stream));
}

int moe_mx4_down(const moe_dims* d, const moe_mx4* act, const moe_mx4* w_down, const int32_t* tiles,
                 const int32_t* num_tiles, void* ys, hipStream_t stream) {
  MOE_CHECK_DIMS(d, D);
  if (!mx4_ok(act) || !mx4_ok(w_down) || !ptrs_ok(tiles, num_tiles, ys)) return MOE_EINVAL;
  if (D.H > kMx4Side || D.F > kMx4Side) return MOE_EUNSUPPORTED;
  Span s[7] = {{ys, size_t(D.NK()) * size_t(D.H) * (D.dtype == MOE_BF16 ? 2 : 4)},
               {tiles, size_t(moe_launch::max_tiles(D)) * 12},
               {num_tiles, 4}};
  int n = 3;
  add_mx4(s, &n, act, D.NK(), D.F, 1);
  add_mx4(s, &n, w_down, D.E, D.F, D.H);
  if (D.N == 0) return MOE_OK;
  if (spans_overlap(s, n, 1)) return MOE_EINVAL;
  return from_hip(moe_launch::mx4_down(D, mx4_of(act), mx4_of(w_down), tiles, num_tiles, ys, stream));
}

size_t moe_mx4_decode_workspace_bytes(const moe_dims* d, const moe_dims* ds) {
  Dims D;
  int64_t Fs;
  if (check_mx4_decode(d, ds, &D, &Fs) != MOE_OK) return size_t(-1);
  return D.N == 0 ? 0 : moe_launch::mx4_decode_ws(D, Fs);
}

int moe_mx4_decode(const moe_dims* d, const void* x, const void* w_r, const float* logit_bias, const moe_mx4* w_gate,
                   const moe_mx4* w_up, const moe_mx4* w_down, const moe_dims* ds, const moe_mx4* ws_gate,
                   const moe_mx4* ws_up, const moe_mx4* ws_down, int32_t* topk_idx, float* gates, void* y, void* ws,
                   size_t ws_bytes, hipStream_t stream) {
  Dims D;
  int64_t Fs;
  const int st = check_mx4_decode(d, ds, &D, &Fs);
  if (st != MOE_OK) return st;
  if (!ptrs_ok(x, w_r, topk_idx, gates, y) || !mx4_ok(w_gate) || !mx4_ok(w_up) || !mx4_ok(w_down)) return MOE_EINVAL;
  if (logit_bias != nullptr && !aligned16(logit_bias)) return MOE_EINVAL;
  if (ds != nullptr ? !(mx4_ok(ws_gate) && mx4_ok(ws_up) && mx4_ok(ws_down))
                    : (ws_gate != nullptr || ws_up != nullptr || ws_down != nullptr))
    return MOE_EINVAL;
  if (D.N == 0) return MOE_OK;
  const size_t need = moe_launch::mx4_decode_ws(D, Fs), nk = size_t(D.NK()) * 4;
  Span s[19] = {{y, row_bytes(D)},
                {topk_idx, nk},
                {gates, nk},
                {ws, need},
                {x, row_bytes(D)},
                {w_r, size_t(D.E) * size_t(D.H) * (D.dtype == MOE_BF16 ? 2 : 4)},
                {logit_bias, logit_bias == nullptr ? 0 : size_t(D.E) * 4}};
  int n = 7;
  add_mx4(s, &n, w_gate, D.E, D.H, D.F);
  add_mx4(s, &n, w_up, D.E, D.H, D.F);
  add_mx4(s, &n, w_down, D.E, D.F, D.H);
  if (ds != nullptr) {
    add_mx4(s, &n, ws_gate, 1, D.H, Fs);
    add_mx4(s, &n, ws_up, 1, D.H, Fs);
    add_mx4(s, &n, ws_down, 1, Fs, D.H);
  }
  if (spans_overlap(s, n, 4)) return MOE_EINVAL;
  if (ws == nullptr || ws_bytes < need || !aligned16(ws)) return MOE_EWORKSPACE;
  return from_hip(moe_launch::mx4_decode(D, x, w_r, logit_bias, mx4_of(w_gate), mx4_of(w_up), mx4_of(w_down), Fs,
                                         mx4_of(ws_gate), mx4_of(ws_up), mx4_of(ws_down), topk_idx, gates, y, ws,
                                         stream));
}

size_t moe_balance_state_bytes(const moe_balance* b) {
  if (check_balance(b) != MOE_OK) return size_t(-1);
  return b->N == 0 ? 0 : moe_launch::balance_state(*b);
}

size_t moe_balance_workspace_bytes(const moe_balance* b) {
  if (check_balance(b) != MOE_OK) return size_t(-1);
  return b->N == 0 ? 0 : moe_launch::balance_ws(*b);
}

int moe_balance_loss(const moe_balance* b, const void* logits, const int32_t* topk_idx, const float* logit_bias,
                     const uint8_t* mask, float* loss, int32_t* counts, void* state, size_t state_bytes, void* ws,
                     size_t ws_bytes, hipStream_t stream) {
  const int st = check_balance(b);
  if (st != MOE_OK) return st;
  if (!ptrs_ok(logits, loss, counts)) return MOE_EINVAL;
  if (topk_idx != nullptr && (logit_bias != nullptr || !aligned16(topk_idx))) return MOE_EINVAL;
  if (logit_bias != nullptr && !aligned16(logit_bias)) return MOE_EINVAL;
  if (mask != nullptr && !aligned16(mask)) return MOE_EINVAL;
  if (b->N == 0) return MOE_OK;
  const size_t sb = moe_launch::balance_state(*b), wb = moe_launch::balance_ws(*b);
  const size_t row = size_t(b->E) * (b->dtype == MOE_BF16 ? 2 : 4);
  const Span s[] = {{loss, 4},
                    {counts, size_t(b->E) * 4},
                    {state, sb},
                    {ws, wb},
                    {logits, size_t(b->N) * row},
                    {topk_idx, topk_idx == nullptr ? 0 : size_t(b->N) * size_t(b->K) * 4},
                    {logit_bias, logit_bias == nullptr ? 0 : size_t(b->E) * 4},
                    {mask, mask == nullptr ? 0 : size_t(b->N)}};
  if (spans_overlap(s, 8, 4)) return MOE_EINVAL;
  if (state == nullptr || state_bytes < sb || !aligned16(state)) return MOE_EWORKSPACE;
  if (ws == nullptr || ws_bytes < wb || !aligned16(ws)) return MOE_EWORKSPACE;
  return from_hip(moe_launch::balance_loss(*b, logits, topk_idx, logit_bias, mask, loss, counts, state, ws, stream));
}

int moe_balance_loss_bwd(const moe_balance* b, const void* logits, const uint8_t* mask, const void* state,
                         const float* dloss, void* dlogits, hipStream_t stream) {
  const int st = check_balance(b);
  if (st != MOE_OK) return st;
  if (!ptrs_ok(logits, state, dlogits)) return MOE_EINVAL;
  if (mask != nullptr && !aligned16(mask)) return MOE_EINVAL;
  if (dloss != nullptr && (reinterpret_cast<uintptr_t>(dloss) & 3u) != 0) return MOE_EINVAL;
  if (b->N == 0) return MOE_OK;
  const size_t n = size_t(b->N) * size_t(b->E) * (b->dtype == MOE_BF16 ? 2 : 4);
  const Span s[] = {{dlogits, n},
                    {logits, dlogits == logits ? 0 : n},
                    {mask, mask == nullptr ? 0 : size_t(b->N)},
                    {state, moe_launch::balance_state(*b)},
                    {dloss, dloss == nullptr ? size_t(0) : size_t(4)}};
  if (spans_overlap(s, 5, 1)) return MOE_EINVAL;
  return from_hip(moe_launch::balance_loss_bwd(*b, logits, mask, state, dloss, dlogits, stream));
}

}  // extern "C"
