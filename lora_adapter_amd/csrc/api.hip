// extern "C" entry points of liblora: argument checks on the host (before any
// HIP call), workspace layout, and kernel dispatch on the caller's stream.
#include <string.h>

#include <algorithm>

#include "lora_internal.h"
#include "quantise.h"

using namespace lora;

namespace {

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }

bool dims_ok(int32_t d) { return d > 0 && d % 64 == 0; }

// Checks the descriptor fields every call needs; `need_pages` also asks for
// the factor pages and scales.
int32_t check_pool(const lora_pool_desc *p, bool need_pages) {
  if (!p) return LORA_ERR_INVALID_ARG;
  if (p->dtype != LORA_F32 && p->dtype != LORA_BF16) return LORA_ERR_INVALID_ARG;
  if (p->n_adapters < 1 || p->n_pages < 0 || p->n_page_ids < 0) return LORA_ERR_INVALID_ARG;
  if (!p->rank || !p->page_start || (p->n_page_ids > 0 && !p->page_ids)) return LORA_ERR_INVALID_ARG;
  if (need_pages) {
    if (!p->scale) return LORA_ERR_INVALID_ARG;
    if (p->n_pages > 0 && (!p->a_pages || !p->b_pages)) return LORA_ERR_INVALID_ARG;
    if (!dims_ok(p->d_in) || !dims_ok(p->d_out)) return LORA_ERR_UNSUPPORTED;
  }
  return LORA_OK;
}

int32_t check_batch(int32_t T, int32_t K) {
  if (T < 0 || K < 1 || K > LORA_MAX_K) return LORA_ERR_INVALID_ARG;
  if (int64_t(T) * K > kMaxPairs) return LORA_ERR_UNSUPPORTED;
  return LORA_OK;
}

int32_t dev(hipError_t e) { return e == hipSuccess ? LORA_OK : LORA_ERR_DEVICE; }

// Apply workspace: [split partials][U per slot, slot descriptors (decode
// shapes)][U].  The per-slot U (LORA_MAX_RANK floats per slot) and the slot
// descriptors are written by the per-slot shrink of lora_forward's decode
// launch.
struct ApplyWs {
  GemmConfig cfg;
  size_t partial_bytes;   // aligned
  float *partial;
  float *slot_u;          // decode shapes: [T*K][LORA_MAX_RANK]
  int4 *sdesc;            // decode shapes: [T*K]
  float *U;
  int64_t u_cap;
};

size_t slot_u_only_bytes(int32_t T, int32_t K) {
  return align_up(size_t(T) * size_t(K) * LORA_MAX_RANK * sizeof(float));
}

size_t slot_u_bytes(const GemmConfig &c, int32_t T, int32_t K) {
  return c.kind == 4 ? slot_u_only_bytes(T, K) + align_up(size_t(T) * size_t(K) * sizeof(int4)) : 0;
}

ApplyWs apply_layout(void *ws, size_t ws_bytes, int32_t T, int32_t K, int32_t d_in, int32_t d_out,
                     int32_t dtype) {
  ApplyWs w{};
  w.cfg = choose_gemm(T > 0 ? T : 1, d_in, d_out, dtype);
  w.partial_bytes = align_up(gemm_partial_bytes(w.cfg, T, d_out));
  const size_t head = w.partial_bytes + slot_u_bytes(w.cfg, T, K);
  w.partial = static_cast<float *>(ws);
  if (ws && ws_bytes >= head) {
    w.slot_u = w.cfg.kind == 4
                   ? reinterpret_cast<float *>(static_cast<char *>(ws) + w.partial_bytes) : nullptr;
    w.sdesc = w.cfg.kind == 4
                  ? reinterpret_cast<int4 *>(static_cast<char *>(ws) + w.partial_bytes +
                                             slot_u_only_bytes(T, K)) : nullptr;
    w.U = reinterpret_cast<float *>(static_cast<char *>(ws) + head);
    w.u_cap = int64_t((ws_bytes - head) / sizeof(float));
  } else {
    w.U = nullptr;
    w.u_cap = -1;
  }
  return w;
}

}  // namespace

extern "C" {

int32_t lora_abi_version(void) { return LORA_ABI_VERSION; }

const char *lora_status_string(int32_t status) {
  switch (status) {
    case LORA_OK: return "ok";
    case LORA_ERR_INVALID_ARG: return "invalid argument";
    case LORA_ERR_UNSUPPORTED: return "unsupported shape or dtype";
    case LORA_ERR_CAPACITY: return "buffer too small";
    case LORA_ERR_DEVICE: return "HIP call failed";
    default: return "unknown status";
  }
}

size_t lora_plan_bytes(int32_t T, int32_t K, int32_t n_adapters) {
  if (check_batch(T, K) != LORA_OK || n_adapters < 1) return 0;
  return size_t(plan_layout(int64_t(T) * K, n_adapters).total) * sizeof(int32_t);
}

int32_t lora_plan_layout(int32_t T, int32_t K, int32_t n_adapters, int64_t offsets_out[9]) {
  if (!offsets_out || n_adapters < 1) return LORA_ERR_INVALID_ARG;
  const int32_t st = check_batch(T, K);
  if (st != LORA_OK) return st;
  const PlanLayout L = plan_layout(int64_t(T) * K, n_adapters);
  const int64_t o[9] = {L.hdr, L.pair_tk, L.seg_adapter, L.seg_off, L.seg_row_off,
                        L.bucket_seg_off, L.u_off, L.slot_pos, L.pair_adapter};
  for (int i = 0; i < 9; ++i) offsets_out[i] = o[i] * int64_t(sizeof(int32_t));
  return LORA_OK;
}

int32_t lora_plan(const int32_t *ids, const float *gates, int32_t T, int32_t K,
                  const lora_pool_desc *pool, void *plan, size_t plan_bytes, void *stream) {
  int32_t st = check_batch(T, K);
  if (st != LORA_OK) return st;
  if ((st = check_pool(pool, false)) != LORA_OK) return st;
  if (!plan) return LORA_ERR_INVALID_ARG;
  if (int64_t(T) * K > 0 && (!ids || !gates)) return LORA_ERR_INVALID_ARG;
  if (plan_bytes < lora_plan_bytes(T, K, pool->n_adapters)) return LORA_ERR_CAPACITY;
  return dev(launch_plan(ids, gates, T, K, pool_view(pool), static_cast<int32_t *>(plan),
                         static_cast<hipStream_t>(stream)));
}

int32_t lora_plan_header(const void *plan, int32_t *out, void *stream) {
  if (!plan || !out) return LORA_ERR_INVALID_ARG;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  // the header is the plan buffer's first LORA_PLAN_HEADER_INTS words
  if (hipMemcpyAsync(out, plan, LORA_PLAN_HEADER_INTS * sizeof(int32_t), hipMemcpyDeviceToHost,
                     s) != hipSuccess)
    return LORA_ERR_DEVICE;
  return dev(hipStreamSynchronize(s));
}

size_t lora_apply_workspace_bytes(int32_t T, int32_t K, int32_t d_in, int32_t d_out,
                                  int32_t max_rank, int32_t dtype) {
  if (check_batch(T, K) != LORA_OK || !dims_ok(d_in) || !dims_ok(d_out)) return 0;
  if (max_rank < 0 || max_rank > LORA_MAX_RANK) return 0;
  if (dtype != LORA_F32 && dtype != LORA_BF16) return 0;
  const GemmConfig c = choose_gemm(T > 0 ? T : 1, d_in, d_out, dtype);
  const size_t u = size_t(T) * size_t(K) * size_t(max_rank) * sizeof(float);
  return align_up(gemm_partial_bytes(c, T, d_out)) + slot_u_bytes(c, T, K) + align_up(u > 0 ? u : 1);
}

size_t lora_apply_u_offset(int32_t T, int32_t K, int32_t d_in, int32_t d_out, int32_t dtype) {
  if (check_batch(T, K) != LORA_OK || !dims_ok(d_in) || !dims_ok(d_out)) return 0;
  if (dtype != LORA_F32 && dtype != LORA_BF16) return 0;
  const GemmConfig c = choose_gemm(T > 0 ? T : 1, d_in, d_out, dtype);
  return align_up(gemm_partial_bytes(c, T, d_out)) + slot_u_bytes(c, T, K);
}

namespace {

ShrinkArgs apply_shrink_args(const void *X, const uint8_t *keep_mask, float keep_scale,
                             int32_t T, int32_t K, const float *gates,
                             const lora_pool_desc *pool, const PlanView &pv, const ApplyWs &w) {
  ShrinkArgs a{};
  a.Z = X;
  a.mask = keep_mask;
  a.extra_scale = keep_mask ? keep_scale : 1.0f;
  a.T = T; a.K = K; a.d = pool->d_in;
  a.pages = pool->a_pages;
  a.rank = pool->rank; a.page_start = pool->page_start; a.page_ids = pool->page_ids;
  a.scale = pool->scale;
  a.gates = gates;
  a.plan = pv;
  a.err_word = const_cast<int32_t *>(pv.hdr) + LORA_PH_ERR;
  a.out = w.U;
  a.out_cap = w.u_cap;
  a.big_segments = shrink_tile_enabled(pool->dtype, int64_t(T) * K, pool->d_in, pool->d_out) ? 1 : 0;
  return a;
}

}  // namespace

int32_t lora_shrink(const void *X, const uint8_t *keep_mask, float keep_scale, int32_t T,
                    int32_t K, const float *gates, const lora_pool_desc *pool, const void *plan,
                    void *ws, size_t ws_bytes, void *stream) {
  int32_t st = check_batch(T, K);
  if (st != LORA_OK) return st;
  if ((st = check_pool(pool, true)) != LORA_OK) return st;
  if (!plan) return LORA_ERR_INVALID_ARG;
  if (T == 0) return LORA_OK;
  if (!X || !gates || !ws) return LORA_ERR_INVALID_ARG;
  const ApplyWs w = apply_layout(ws, ws_bytes, T, K, pool->d_in, pool->d_out, pool->dtype);
  if (w.u_cap < 0) return LORA_ERR_CAPACITY;
  const int64_t TK = int64_t(T) * K;
  const PlanView pv = plan_view(plan, TK, pool->n_adapters);
  const ShrinkArgs a = apply_shrink_args(X, keep_mask, keep_scale, T, K, gates, pool, pv, w);
  return dev(launch_shrink(a, pool->dtype, TK, pool->n_adapters, pool->d_in, pool->d_out,
                           static_cast<hipStream_t>(stream)));
}

namespace {

// Shared argument checks and GemmArgs for the two halves of the base stage.
int32_t base_args(const void *X, const void *W_t, void *Y, int32_t T, int32_t K,
                  const lora_pool_desc *pool, const void *plan, void *ws,
                  size_t ws_bytes, GemmConfig &cfg, GemmArgs &g) {
  int32_t st = check_batch(T, K);
  if (st != LORA_OK) return st;
  if ((st = check_pool(pool, true)) != LORA_OK) return st;
  if (!plan) return LORA_ERR_INVALID_ARG;
  if (T == 0) return LORA_OK;
  if (!X || !W_t || !Y || !ws) return LORA_ERR_INVALID_ARG;
  if (Y == X || Y == W_t) return LORA_ERR_INVALID_ARG;
  const ApplyWs w = apply_layout(ws, ws_bytes, T, K, pool->d_in, pool->d_out, pool->dtype);
  if (w.u_cap < 0) return LORA_ERR_CAPACITY;
  const int64_t TK = int64_t(T) * K;
  const PlanView pv = plan_view(plan, TK, pool->n_adapters);
  cfg = w.cfg;
  g = GemmArgs{};
  g.X = X; g.W = W_t; g.M = T; g.N = pool->d_out; g.Kd = pool->d_in;
  g.k_split = w.cfg.k_split;
  g.sk_g = w.cfg.sk;
  g.partial = w.partial;
  g.Y = Y;
  g.ex.K = K;
  g.ex.slot_desc = pv.slot_desc; g.ex.pair_tk = pv.pair_tk; g.ex.page_ids = pool->page_ids;
  g.ex.b_pages = pool->b_pages; g.ex.d_out = pool->d_out;
  g.ex.U = w.U; g.ex.hdr = pv.hdr; g.ex.u_cap = w.u_cap;
  return LORA_OK;
}

}  // namespace

int32_t lora_base_gemm(const void *X, const void *W_t, void *Y, int32_t T, int32_t K,
                       const lora_pool_desc *pool, const void *plan, void *ws,
                       size_t ws_bytes, void *stream) {
  GemmConfig cfg;
  GemmArgs g;
  const int32_t st = base_args(X, W_t, Y, T, K, pool, plan, ws, ws_bytes, cfg, g);
  if (st != LORA_OK || T == 0) return st;
  return dev(launch_base_gemm(cfg, g, static_cast<hipStream_t>(stream)));
}

int32_t lora_expand_epilogue(const void *X, const void *W_t, void *Y, int32_t T, int32_t K,
                             const lora_pool_desc *pool, const void *plan,
                             void *ws, size_t ws_bytes, void *stream) {
  GemmConfig cfg;
  GemmArgs g;
  const int32_t st = base_args(X, W_t, Y, T, K, pool, plan, ws, ws_bytes, cfg, g);
  if (st != LORA_OK || T == 0) return st;
  return dev(launch_epilogue(cfg, g, pool->dtype, static_cast<hipStream_t>(stream)));
}

int32_t lora_base_expand(const void *X, const void *W_t, void *Y, int32_t T, int32_t K,
                         const lora_pool_desc *pool, const void *plan,
                         void *ws, size_t ws_bytes, void *stream) {
  const int32_t st = lora_base_gemm(X, W_t, Y, T, K, pool, plan, ws, ws_bytes, stream);
  if (st != LORA_OK) return st;
  return lora_expand_epilogue(X, W_t, Y, T, K, pool, plan, ws, ws_bytes, stream);
}

int32_t lora_shrink_gemm(const void *X, const void *W_t, void *Y, int32_t T, int32_t K,
                         const float *gates, const uint8_t *keep_mask, float keep_scale,
                         const lora_pool_desc *pool, const void *plan, void *ws,
                         size_t ws_bytes, void *stream) {
  GemmConfig cfg;
  GemmArgs g;
  int32_t st = base_args(X, W_t, Y, T, K, pool, plan, ws, ws_bytes, cfg, g);
  if (st != LORA_OK || T == 0) return st;
  if (!gates) return LORA_ERR_INVALID_ARG;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const ApplyWs w = apply_layout(ws, ws_bytes, T, K, pool->d_in, pool->d_out, pool->dtype);
  const int64_t TK = int64_t(T) * K;
  const PlanView pv = plan_view(plan, TK, pool->n_adapters);
  const ShrinkArgs a = apply_shrink_args(X, keep_mask, keep_scale, T, K, gates, pool, pv, w);
  if (decode_shrink_fusable(cfg, pool->d_in)) {
    hipError_t e = launch_shrink_big(a, pool->dtype, TK, pool->n_adapters, pool->d_in,
                                     pool->d_out, s);
    if (e == hipSuccess) e = launch_decode_gemm_shrink(cfg, g, a, s);
    return dev(e);
  }
  hipError_t e = launch_shrink(a, pool->dtype, TK, pool->n_adapters, pool->d_in, pool->d_out, s);
  if (e == hipSuccess) e = launch_base_gemm(cfg, g, s);
  return dev(e);
}

int32_t lora_apply(const void *X, const void *W_t, void *Y, int32_t T, int32_t K,
                   const float *gates, const uint8_t *keep_mask,
                   float keep_scale, const lora_pool_desc *pool, const void *plan, void *ws,
                   size_t ws_bytes, void *stream) {
  int32_t st = check_batch(T, K);
  if (st != LORA_OK) return st;
  if ((st = check_pool(pool, true)) != LORA_OK) return st;
  if (T > 0 && (!X || !W_t || !Y || !gates || !ws || !plan)) return LORA_ERR_INVALID_ARG;
  st = lora_shrink_gemm(X, W_t, Y, T, K, gates, keep_mask, keep_scale, pool, plan, ws, ws_bytes,
                        stream);
  if (st != LORA_OK) return st;
  return lora_expand_epilogue(X, W_t, Y, T, K, pool, plan, ws, ws_bytes, stream);
}

}  // extern "C"

namespace {

// lora_forward's two halves.  Split GEMM shapes only (gemm_plan_fusable):
//   decode:   first = the plan (built by workgroup 0), GEMM partials and the
//             per-slot shrink (U per slot and slot descriptors), one launch;
//             finish = epilogue from the partials, per-slot U and
//             descriptors, which also stores U in the plan's u_off layout.
//   stream-K: first = GEMM partials with the plan built in the same launch;
//             finish = shrink, then epilogue.
// Other shapes: first = lora_plan, finish = lora_apply.
struct Fwd {
  GemmConfig cfg;
  GemmArgs g;
  bool split;
};

int32_t forward_args(const int32_t *ids, const float *gates, int32_t T, int32_t K, const void *X,
                     const void *W_t, void *Y, const lora_pool_desc *pool, void *plan,
                     size_t plan_bytes, void *ws, size_t ws_bytes, Fwd &f) {
  int32_t st = check_batch(T, K);
  if (st != LORA_OK) return st;
  if ((st = check_pool(pool, true)) != LORA_OK) return st;
  if (!plan) return LORA_ERR_INVALID_ARG;
  if (plan_bytes < lora_plan_bytes(T, K, pool->n_adapters)) return LORA_ERR_CAPACITY;
  f.split = false;
  if (T == 0) return LORA_OK;
  if (!ids || !gates || !X || !W_t || !Y || !ws) return LORA_ERR_INVALID_ARG;
  if ((st = base_args(X, W_t, Y, T, K, pool, plan, ws, ws_bytes, f.cfg, f.g)) != LORA_OK) return st;
  f.split = gemm_plan_fusable(f.cfg);
  return LORA_OK;
}

SlotShrinkArgs slot_shrink_args(const int32_t *ids, const float *gates, int32_t T, int32_t K,
                                const void *X, const uint8_t *keep_mask, float keep_scale,
                                const lora_pool_desc *pool, const ApplyWs &w) {
  SlotShrinkArgs ss{};
  ss.ids = ids; ss.gates = gates; ss.K = K; ss.N = pool->n_adapters;
  ss.Z = X; ss.mask = keep_mask; ss.extra_scale = keep_mask ? keep_scale : 1.0f;
  ss.d = pool->d_in; ss.pages = pool->a_pages;
  ss.rank = pool->rank; ss.page_start = pool->page_start; ss.page_ids = pool->page_ids;
  ss.scale = pool->scale; ss.n_pages = pool->n_pages; ss.n_page_ids = pool->n_page_ids;
  ss.out = w.slot_u; ss.stride = LORA_MAX_RANK; ss.n_slots = T * K; ss.sdesc = w.sdesc;
  return ss;
}

PlanLaunch forward_plan(const int32_t *ids, const float *gates, int32_t T, int32_t K,
                        const lora_pool_desc *pool, void *plan, const Fwd &f, const ApplyWs &w) {
  PlanLaunch pl = plan_setup(ids, gates, T, K, pool_view(pool), static_cast<int32_t *>(plan), 256,
                             plan_lds_cap(f.cfg));
  // decode: the per-slot shrink runs beside the plan, whose U the epilogue
  // later moves to the u_off layout; the decode-shrink wave records are skipped
  if (w.slot_u) pl.a.no_sched = 1;
  return pl;
}

}  // namespace

extern "C" {

int32_t lora_forward_gemm(const int32_t *ids, const float *gates, int32_t T, int32_t K,
                          const void *X, const void *W_t, void *Y, const uint8_t *keep_mask,
                          float keep_scale, const lora_pool_desc *pool, void *plan,
                          size_t plan_bytes, void *ws, size_t ws_bytes, void *stream) {
  Fwd f;
  int32_t st = forward_args(ids, gates, T, K, X, W_t, Y, pool, plan, plan_bytes, ws, ws_bytes, f);
  if (st != LORA_OK) return st;
  if (!f.split) return lora_plan(ids, gates, T, K, pool, plan, plan_bytes, stream);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const ApplyWs w = apply_layout(ws, ws_bytes, T, K, pool->d_in, pool->d_out, pool->dtype);
  if (w.slot_u) {
    const SlotShrinkArgs ss = slot_shrink_args(ids, gates, T, K, X, keep_mask, keep_scale, pool, w);
    return dev(launch_decode_slot_plan(f.cfg, f.g, ss,
                                       forward_plan(ids, gates, T, K, pool, plan, f, w), s));
  }
  return dev(launch_gemm_plan(f.cfg, f.g, forward_plan(ids, gates, T, K, pool, plan, f, w), s));
}

int32_t lora_forward_finish(const int32_t *ids, const float *gates, int32_t T, int32_t K,
                            const void *X, const void *W_t, void *Y, const uint8_t *keep_mask,
                            float keep_scale, const lora_pool_desc *pool, void *plan,
                            size_t plan_bytes, void *ws, size_t ws_bytes, void *stream) {
  Fwd f;
  int32_t st = forward_args(ids, gates, T, K, X, W_t, Y, pool, plan, plan_bytes, ws, ws_bytes, f);
  if (st != LORA_OK || T == 0) return st;
  if (!f.split)
    return lora_apply(X, W_t, Y, T, K, gates, keep_mask, keep_scale, pool, plan, ws, ws_bytes,
                      stream);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const ApplyWs w = apply_layout(ws, ws_bytes, T, K, pool->d_in, pool->d_out, pool->dtype);
  if (w.slot_u)
    return dev(launch_epilogue_ucopy(f.cfg, f.g, pool->dtype, w.slot_u, w.sdesc, w.U, w.u_cap, s));
  st = lora_shrink(X, keep_mask, keep_scale, T, K, gates, pool, plan, ws, ws_bytes, stream);
  if (st != LORA_OK) return st;
  return lora_expand_epilogue(X, W_t, Y, T, K, pool, plan, ws, ws_bytes, stream);
}

int32_t lora_forward(const int32_t *ids, const float *gates, int32_t T, int32_t K,
                     const void *X, const void *W_t, void *Y, const uint8_t *keep_mask,
                     float keep_scale, const lora_pool_desc *pool, void *plan, size_t plan_bytes,
                     void *ws, size_t ws_bytes, void *stream) {
  int32_t st = lora_forward_gemm(ids, gates, T, K, X, W_t, Y, keep_mask, keep_scale, pool, plan,
                                 plan_bytes, ws, ws_bytes, stream);
  if (st != LORA_OK || T == 0) return st;
  return lora_forward_finish(ids, gates, T, K, X, W_t, Y, keep_mask, keep_scale, pool, plan,
                             plan_bytes, ws, ws_bytes, stream);
}

}  // extern "C"

namespace {

MergeArgs merge_args(void *W_t, const lora_pool_desc *pool, const int32_t *merge_ids,
                     const float *coeffs, int32_t m) {
  MergeArgs a{};
  a.W = W_t; a.d_in = pool->d_in; a.d_out = pool->d_out;
  a.a_pages = pool->a_pages; a.b_pages = pool->b_pages;
  a.rank = pool->rank; a.page_start = pool->page_start; a.page_ids = pool->page_ids;
  a.scale = pool->scale;
  a.n_pages = pool->n_pages; a.n_page_ids = pool->n_page_ids; a.n_adapters = pool->n_adapters;
  a.ids = merge_ids; a.coeffs = coeffs; a.m = m;
  return a;
}

}  // namespace

extern "C" {

int32_t lora_merge_delta(void *W_t, const lora_pool_desc *pool, const int32_t *merge_ids,
                         const float *coeffs, int32_t m, void *stream) {
  int32_t st = check_pool(pool, true);
  if (st != LORA_OK) return st;
  if (m < 0 || !W_t) return LORA_ERR_INVALID_ARG;
  if (m == 0) return LORA_OK;
  if (!merge_ids || !coeffs) return LORA_ERR_INVALID_ARG;
  return dev(launch_merge(merge_args(W_t, pool, merge_ids, coeffs, m), pool->dtype,
                          static_cast<hipStream_t>(stream)));
}

int32_t lora_merge_delta_layers(const lora_layer_desc *layers, int32_t n_layers,
                                const int32_t *merge_ids, const float *coeffs, int32_t m,
                                void *stream) {
  if (n_layers < 0 || m < 0 || (n_layers > 0 && !layers)) return LORA_ERR_INVALID_ARG;
  for (int32_t l = 0; l < n_layers; ++l) {
    const int32_t st = check_pool(&layers[l].pool, true);
    if (st != LORA_OK) return st;
    if (!layers[l].W_t || layers[l].pool.dtype != layers[0].pool.dtype) return LORA_ERR_INVALID_ARG;
    for (int32_t q = 0; q < l; ++q)
      if (layers[q].W_t == layers[l].W_t) return LORA_ERR_INVALID_ARG;   // in place, once each
  }
  if (n_layers == 0 || m == 0) return LORA_OK;
  if (!merge_ids || !coeffs) return LORA_ERR_INVALID_ARG;
  constexpr int32_t kChunk = LORA_MERGE_MAX_LAYERS;
  MergeArgs a[kChunk];
  const hipStream_t s = static_cast<hipStream_t>(stream);
  for (int32_t l0 = 0; l0 < n_layers; l0 += kChunk) {
    const int32_t nl = n_layers - l0 < kChunk ? n_layers - l0 : kChunk;
    for (int32_t l = 0; l < nl; ++l)
      a[l] = merge_args(layers[l0 + l].W_t, &layers[l0 + l].pool, merge_ids, coeffs, m);
    const int32_t st = dev(launch_merge_layers(a, nl, layers[0].pool.dtype, s));
    if (st != LORA_OK) return st;
  }
  return LORA_OK;
}

size_t lora_grad_workspace_bytes(int32_t T, int32_t K, int32_t n_adapters, int32_t d_in,
                                 int32_t d_out, int32_t max_rank, int32_t dtype) {
  if (check_batch(T, K) != LORA_OK || !dims_ok(d_in) || !dims_ok(d_out) || n_adapters < 1) return 0;
  if (max_rank < 1 || max_rank > LORA_MAX_RANK) return 0;
  if (dtype != LORA_F32 && dtype != LORA_BF16) return 0;
  const int64_t TK = int64_t(T) * K;
  const size_t g = align_up(size_t(TK) * size_t(max_rank) * sizeof(float) + 4);
  const size_t pieces = size_t(grad_pieces(TK, n_adapters));
  const size_t pa = align_up(pieces * size_t(max_rank) * size_t(d_in) * sizeof(float));
  const size_t pb = align_up(pieces * size_t(max_rank) * size_t(d_out) * sizeof(float));
  // MFMA form: the per-tile dY.B^T partials
  const size_t gp = grad_mfma_form(dtype, TK, d_out)
                        ? align_up(size_t(grad_gpart_tiles(d_out)) * size_t(TK) * size_t(max_rank) *
                                   sizeof(float))
                        : 0;
  return g + pa + pb + gp;
}

int32_t lora_grad(const void *X, const uint8_t *keep_mask, float keep_scale, const void *dY,
                  int32_t T, int32_t K, const float *gates,
                  const lora_pool_desc *pool, const void *plan, const void *apply_ws,
                  size_t apply_ws_bytes, float *dA_pages, float *dB_pages, int32_t max_rank,
                  void *ws, size_t ws_bytes, void *stream) {
  int32_t st = check_batch(T, K);
  if (st != LORA_OK) return st;
  if ((st = check_pool(pool, true)) != LORA_OK) return st;
  if (!plan || max_rank < 1 || max_rank > LORA_MAX_RANK) return LORA_ERR_INVALID_ARG;
  if (T == 0) return LORA_OK;
  if (!X || !dY || !gates || !apply_ws || !dA_pages || !dB_pages || !ws)
    return LORA_ERR_INVALID_ARG;
  const int64_t TK = int64_t(T) * K;
  const size_t need = lora_grad_workspace_bytes(T, K, pool->n_adapters, pool->d_in, pool->d_out,
                                                max_rank, pool->dtype);
  if (ws_bytes < need) return LORA_ERR_CAPACITY;
  const ApplyWs aw = apply_layout(const_cast<void *>(apply_ws), apply_ws_bytes, T, K, pool->d_in,
                              pool->d_out, pool->dtype);
  if (aw.u_cap < 0) return LORA_ERR_CAPACITY;
  const PlanView pv = plan_view(plan, TK, pool->n_adapters);
  int32_t *err_word = const_cast<int32_t *>(pv.hdr) + LORA_PH_ERR;
  const hipStream_t s = static_cast<hipStream_t>(stream);

  char *base = static_cast<char *>(ws);
  const size_t g_bytes = align_up(size_t(TK) * size_t(max_rank) * sizeof(float) + 4);
  const size_t pieces = size_t(grad_pieces(TK, pool->n_adapters));
  const size_t pa = align_up(pieces * size_t(max_rank) * size_t(pool->d_in) * sizeof(float));
  float *G = reinterpret_cast<float *>(base);
  float *partA = reinterpret_cast<float *>(base + g_bytes);
  float *partB = reinterpret_cast<float *>(base + g_bytes + pa);
  const size_t pbytes = align_up(pieces * size_t(max_rank) * size_t(pool->d_out) * sizeof(float));
  const bool fused_g = grad_mfma_form(pool->dtype, TK, pool->d_out);
  float *gpart = fused_g ? reinterpret_cast<float *>(base + g_bytes + pa + pbytes) : nullptr;

  if (fused_g) {
    // prefill-size bf16 batches: dB and the per-tile dY.B^T partials in one
    // pass over dY, then G from the partials, then dA
    SegOuterArgs ob{};
    ob.Z = dY; ob.mask = nullptr; ob.T = T; ob.K = K; ob.d = pool->d_out;
    ob.coef = aw.U; ob.coef_cap = aw.u_cap; ob.plan = pv;
    ob.rank = pool->rank; ob.page_start = pool->page_start; ob.page_ids = pool->page_ids;
    ob.part = partB; ob.max_rank = max_rank; ob.out_pages = dB_pages; ob.err_word = err_word;
    ob.gpart = gpart; ob.b_pages = pool->b_pages;
    GReduceArgs gr{};
    gr.gpart = gpart; gr.n_tiles = grad_gpart_tiles(pool->d_out); gr.TK = TK;
    gr.max_rank = max_rank; gr.plan = pv; gr.rank = pool->rank; gr.scale = pool->scale;
    gr.extra_scale = keep_mask ? keep_scale : 1.0f;
    gr.G = G; gr.g_cap = int64_t(TK) * max_rank;
    // dB with the per-tile partials; its reduction launch also forms G
    hipError_t e = launch_seg_outer(ob, pool->dtype, TK, pool->n_adapters, s, &gr);
    if (e != hipSuccess) return LORA_ERR_DEVICE;
    SegOuterArgs oa = ob;
    oa.Z = X; oa.mask = keep_mask; oa.d = pool->d_in; oa.coef = G; oa.coef_cap = gr.g_cap;
    oa.part = partA; oa.out_pages = dA_pages;
    oa.gpart = nullptr; oa.b_pages = nullptr;
    return dev(launch_seg_outer(oa, pool->dtype, TK, pool->n_adapters, s));
  }

  // G = kappa . g . s . (dY . B_j): the shrink kernel on (dY, B pages)
  ShrinkArgs sa{};
  sa.Z = dY; sa.mask = nullptr; sa.extra_scale = keep_mask ? keep_scale : 1.0f;
  sa.T = T; sa.K = K; sa.d = pool->d_out;
  sa.pages = pool->b_pages;
  sa.rank = pool->rank; sa.page_start = pool->page_start; sa.page_ids = pool->page_ids;
  sa.scale = pool->scale; sa.gates = gates; sa.plan = pv; sa.err_word = err_word;
  sa.out = G; sa.out_cap = int64_t(TK) * max_rank;
  hipError_t e = launch_shrink(sa, pool->dtype, TK, pool->n_adapters, pool->d_in, pool->d_out, s);
  if (e != hipSuccess) return LORA_ERR_DEVICE;

  SegOuterArgs ob{};
  ob.Z = dY; ob.mask = nullptr; ob.T = T; ob.K = K; ob.d = pool->d_out;
  ob.coef = aw.U; ob.coef_cap = aw.u_cap; ob.plan = pv;
  ob.rank = pool->rank; ob.page_start = pool->page_start; ob.page_ids = pool->page_ids;
  ob.part = partB; ob.max_rank = max_rank; ob.out_pages = dB_pages; ob.err_word = err_word;
  SegOuterArgs oa = ob;
  oa.Z = X; oa.mask = keep_mask; oa.d = pool->d_in; oa.coef = G; oa.coef_cap = sa.out_cap;
  oa.part = partA;
  oa.out_pages = dA_pages;
  if (!grad_mfma_form(pool->dtype, TK, pool->d_in))
    return dev(launch_seg_outer_both(ob, oa, pool->dtype, TK, pool->n_adapters, s));
  e = launch_seg_outer(ob, pool->dtype, TK, pool->n_adapters, s);
  if (e != hipSuccess) return LORA_ERR_DEVICE;
  e = launch_seg_outer(oa, pool->dtype, TK, pool->n_adapters, s);
  return dev(e);
}

}  // extern "C"

namespace {

// dX GEMM: dY [T][d_out] times W [d_in][d_out] along d_out, into fp32 partials
// (the epilogue adds the masked LoRA term before the one rounding).
GemmConfig grad_x_config(int32_t T, int32_t d_in, int32_t d_out, int32_t dtype) {
  // the forward's choice: with 256 x 256 tiles the LoRA term and the keep
  // mask go into the GEMM's own epilogue, otherwise split partials and the
  // epilogue launch
  return choose_gemm(T > 0 ? T : 1, d_out, d_in, dtype);
}

}  // namespace

extern "C" {

int32_t lora_transpose(const void *src, void *dst, int32_t rows, int32_t cols, int32_t dtype,
                       void *stream) {
  if (!src || !dst || src == dst || rows < 0 || cols < 0) return LORA_ERR_INVALID_ARG;
  if (dtype != LORA_F32 && dtype != LORA_BF16) return LORA_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return LORA_OK;
  return dev(launch_transpose(src, dst, rows, cols, dtype, static_cast<hipStream_t>(stream)));
}

size_t lora_grad_x_workspace_bytes(int32_t T, int32_t d_in, int32_t d_out, int32_t dtype) {
  if (T < 0 || !dims_ok(d_in) || !dims_ok(d_out)) return 0;
  if (dtype != LORA_F32 && dtype != LORA_BF16) return 0;
  const GemmConfig c = grad_x_config(T, d_in, d_out, dtype);
  const size_t b = gemm_partial_bytes(c, T, d_in);
  return align_up(b > 0 ? b : 1);
}

int32_t lora_grad_x(const void *dY, const void *W, const uint8_t *keep_mask, int32_t T, int32_t K,
                    const lora_pool_desc *pool, const void *plan, const void *grad_ws,
                    size_t grad_ws_bytes, int32_t max_rank, void *dX, void *ws, size_t ws_bytes,
                    void *stream) {
  int32_t st = check_batch(T, K);
  if (st != LORA_OK) return st;
  if ((st = check_pool(pool, true)) != LORA_OK) return st;
  if (!plan || max_rank < 1 || max_rank > LORA_MAX_RANK) return LORA_ERR_INVALID_ARG;
  if (T == 0) return LORA_OK;
  if (!dY || !W || !grad_ws || !dX || !ws) return LORA_ERR_INVALID_ARG;
  if (dX == dY || dX == W) return LORA_ERR_INVALID_ARG;
  if (grad_ws_bytes < lora_grad_workspace_bytes(T, K, pool->n_adapters, pool->d_in, pool->d_out,
                                                max_rank, pool->dtype))
    return LORA_ERR_CAPACITY;
  if (ws_bytes < lora_grad_x_workspace_bytes(T, pool->d_in, pool->d_out, pool->dtype))
    return LORA_ERR_CAPACITY;
  const int64_t TK = int64_t(T) * K;
  const PlanView pv = plan_view(plan, TK, pool->n_adapters);
  const GemmConfig c = grad_x_config(T, pool->d_in, pool->d_out, pool->dtype);
  GemmArgs g{};
  g.X = dY; g.W = W; g.M = T; g.N = pool->d_in; g.Kd = pool->d_out;
  g.k_split = c.k_split;
  g.sk_g = c.sk;
  g.partial = static_cast<float *>(ws);
  g.Y = dX;
  // the expand of the epilogue, on G (lora_grad's workspace starts with it,
  // packed like U) and the A pages, rows of d_in
  g.ex.K = K;
  g.ex.slot_desc = pv.slot_desc; g.ex.pair_tk = pv.pair_tk; g.ex.page_ids = pool->page_ids;
  g.ex.b_pages = pool->a_pages; g.ex.d_out = pool->d_in;
  g.ex.U = static_cast<const float *>(grad_ws); g.ex.hdr = pv.hdr;
  g.ex.u_cap = TK * max_rank;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (c.fused) {
    g.mask = keep_mask;
    return dev(launch_base_gemm(c, g, s));
  }
  hipError_t e = launch_base_gemm(c, g, s);
  if (e == hipSuccess) e = launch_grad_x_epilogue(c, g, pool->dtype, keep_mask, s);
  return dev(e);
}

}  // extern "C"

extern "C" {

size_t lora_tsqr_workspace_bytes(int32_t M, int32_t m, int32_t n) {
  if (!tsqr_shape_ok(M, m, n) || m > (1 << 24)) return 0;
  return align_up(tsqr_workspace_bytes(M, m, n));
}

int32_t lora_tsqr(const void *src, int32_t dtype, const int32_t *cols, int32_t M, int32_t m,
                  int32_t n, float *Qt, float *R, void *ws, size_t ws_bytes, void *stream) {
  if (dtype != LORA_F32 && dtype != LORA_BF16) return LORA_ERR_INVALID_ARG;
  if (M < 0 || m < 1 || n < 1) return LORA_ERR_INVALID_ARG;
  if (M == 0) return LORA_OK;
  if (!tsqr_shape_ok(M, m, n) || m > (1 << 24)) return LORA_ERR_UNSUPPORTED;
  if (!src || !cols || !R || !ws) return LORA_ERR_INVALID_ARG;
  if (ws_bytes < lora_tsqr_workspace_bytes(M, m, n)) return LORA_ERR_CAPACITY;
  return dev(launch_tsqr(src, dtype, cols, M, m, n, Qt, R, ws, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

extern "C" {

size_t lora_compress_workspace_bytes(int32_t M, int32_t d_in, int32_t d_out, int32_t n) {
  if (M < 1 || n < 1 || n > 64 || !dims_ok(d_in) || !dims_ok(d_out) || n > d_in || n > d_out)
    return 0;
  return align_up(compress_workspace_bytes(M, d_in, d_out, n));
}

int32_t lora_compress(const lora_pool_desc *pool, const int32_t *adapters, int32_t M, int32_t n,
                      int32_t policy, float ratio, float energy, int32_t floor_rank, void *out_a,
                      void *out_b, int32_t *out_rank, float *out_sigma, void *ws, size_t ws_bytes,
                      void *stream) {
  int32_t st = check_pool(pool, true);
  if (st != LORA_OK) return st;
  if (M < 0 || n < 1 || (policy != 0 && policy != 1)) return LORA_ERR_INVALID_ARG;
  if (!(ratio > 0.f && ratio <= 1.f) || !(energy > 0.f && energy <= 1.f) || floor_rank < 0)
    return LORA_ERR_INVALID_ARG;
  if (M == 0) return LORA_OK;
  if (n > 64 || n > pool->d_in || n > pool->d_out) return LORA_ERR_UNSUPPORTED;
  if (!adapters || !out_a || !out_b || !out_rank || !out_sigma || !ws || pool->n_pages < 1 ||
      !pool->page_ids)
    return LORA_ERR_INVALID_ARG;
  if (ws_bytes < lora_compress_workspace_bytes(M, pool->d_in, pool->d_out, n)) return LORA_ERR_CAPACITY;
  return dev(launch_compress(pool_view(pool), adapters, M, n, policy, ratio, energy, floor_rank,
                             out_a, out_b, out_rank, out_sigma, ws, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ------------------------------------------------------------ 8-bit base weight

namespace {

int32_t check_weight(const lora_quantised_weight *w, const lora_pool_desc *pool) {
  if (!w) return LORA_ERR_INVALID_ARG;
  if (w->d_in != pool->d_in || w->d_out != pool->d_out) return LORA_ERR_INVALID_ARG;
  if (w->d_in > kQMaxWidth || w->d_out > kQMaxWidth) return LORA_ERR_UNSUPPORTED;
  return LORA_OK;
}

// A quantised GEMM's buffers: fp32 partials and (tile forms) the rows' codes and
// scale bytes.  They lie at the end of a workspace, but that each of the two
// takes room at its start where the first `slab` bytes are free and hold it.
struct QuantTail {
  GemmConfig cfg;
  size_t partial, codes, scales;            // bytes
  bool partial_in, codes_in;                // at the start
  size_t total;                             // bytes at the end
};

int few_adapters(int32_t K, const lora_pool_desc *pool) {
  return K == 1 && pool->n_adapters <= 16 ? pool->n_adapters : 0;
}

QuantTail quant_tail(int32_t T, int few, int32_t d_k, int32_t d_n, int32_t dtype, size_t slab) {
  QuantTail t{};
  t.cfg = choose_quantised_gemm(T > 0 ? T : 1, few, d_k, d_n, dtype);
  t.partial = align_up(gemm_partial_bytes(t.cfg, T, d_n));
  if (t.cfg.kind != 4) {
    t.codes = align_up(size_t(T) * size_t(q_row_bytes(d_k)));
    t.scales = align_up(size_t(q_tile_rows(T)) * size_t(q_row_bytes(d_k) / kQBlock));
  }
  const size_t rows = t.codes + t.scales;
  t.partial_in = t.partial <= slab;
  t.codes_in = (t.partial_in ? t.partial : 0) + rows <= slab;
  t.total = (t.partial_in ? 0 : t.partial) + (t.codes_in ? 0 : rows);
  return t;
}

// The larger tail of the two forms: the size queries do not know the pool.
size_t quant_tail_bytes(int32_t T, int32_t d_k, int32_t d_n, int32_t dtype, size_t slab) {
  const size_t a = quant_tail(T, 1, d_k, d_n, dtype, slab).total;
  const size_t b = quant_tail(T, 0, d_k, d_n, dtype, slab).total;
  return a > b ? a : b;
}

// Fills q for rows [T][d_k] times the weight's codes [d_n][..]; `ws` the
// workspace, `tail` the tail's place in it.  For the tile forms q.g.X is where
// the rows' codes go.
void quantised_args(const QuantTail &t, const void *rows, int32_t T, int32_t d_k, int32_t d_n,
                    const uint8_t *codes, const uint8_t *scale, char *ws, size_t tail, QGemmArgs &q) {
  q.g.X = rows; q.g.W = codes; q.g.M = T; q.g.N = d_n; q.g.Kd = d_k;
  q.g.k_split = t.cfg.k_split; q.g.sk_g = t.cfg.sk;
  q.g.partial = reinterpret_cast<float *>(t.partial_in ? ws : ws + tail);
  q.lda = q.ldb = q_row_bytes(d_k);
  q.lsa = q_tile_rows(T);
  q.lsb = q_scale_bytes(d_k);
  q.sb = scale;
  if (t.cfg.kind != 4) {
    const char *at = ws + (t.codes_in ? (t.partial_in ? t.partial : 0) : tail + (t.partial_in ? 0 : t.partial));
    q.g.X = at;
    q.sa = reinterpret_cast<const uint8_t *>(at) + t.codes;
  }
}

uint8_t *codes_of(const QGemmArgs &q) { return static_cast<uint8_t *>(const_cast<void *>(q.g.X)); }
uint8_t *scales_of(const QGemmArgs &q) { return const_cast<uint8_t *>(q.sa); }

// The product: the rows quantised (tile forms), then the GEMM.
hipError_t run_quantised(const QuantTail &t, const void *rows, int32_t dtype, const QGemmArgs &q,
                         hipStream_t s) {
  if (t.cfg.kind != 4) {
    const hipError_t e = launch_quantise_rows(rows, dtype, q.g.M, q.g.Kd, codes_of(q), scales_of(q), true, s);
    if (e != hipSuccess) return e;
  }
  return launch_quantised_gemm(t.cfg, q, dtype, s);
}

// The checks of the quantised apply, and its workspace: the head is laid out
// as lora_apply's (lora_grad finds U in it; the partials of lora_apply's product
// are the room at its start), the tail ends where the workspace does, so that
// its place needs no max_rank.
struct QuantApply {
  QuantTail t;
  ApplyWs w;
  QGemmArgs q;
  size_t head;            // bytes of the head
};

int32_t quant_apply_args(const void *X, const lora_quantised_weight *W, void *Y, int32_t T,
                         int32_t K, const float *gates, const lora_pool_desc *pool,
                         const void *plan, void *ws, size_t ws_bytes, QuantApply &a) {
  int32_t st = check_batch(T, K);
  if (st != LORA_OK) return st;
  if ((st = check_pool(pool, true)) != LORA_OK) return st;
  if ((st = check_weight(W, pool)) != LORA_OK) return st;
  if (!plan) return LORA_ERR_INVALID_ARG;
  if (T == 0) return LORA_OK;
  if (!X || !Y || !W->q_t || !W->scale || !gates || !ws) return LORA_ERR_INVALID_ARG;
  if (Y == X || Y == W->q_t || Y == W->scale) return LORA_ERR_INVALID_ARG;
  const size_t slab = apply_layout(nullptr, 0, T, K, pool->d_in, pool->d_out, pool->dtype).partial_bytes;
  a.t = quant_tail(T, few_adapters(K, pool), pool->d_in, pool->d_out, pool->dtype, slab);
  if (ws_bytes < a.t.total) return LORA_ERR_CAPACITY;
  const size_t head = a.head = (ws_bytes - a.t.total) / kAlign * kAlign;
  GemmConfig base;
  a.q = QGemmArgs{};
  if ((st = base_args(X, W->q_t, Y, T, K, pool, plan, ws, head, base, a.q.g)) != LORA_OK) return st;
  a.w = apply_layout(ws, head, T, K, pool->d_in, pool->d_out, pool->dtype);
  quantised_args(a.t, X, T, pool->d_in, pool->d_out, W->q_t, W->scale, static_cast<char *>(ws), head, a.q);
  return LORA_OK;
}

// The epilogue counts stream-K units in K tiles of 64: one per 128 codes here.
GemmArgs quant_epilogue_args(const QGemmArgs &q) {
  GemmArgs g = q.g;
  g.Kd = int(q.ldb) / kQBlock * 64;
  return g;
}

}  // namespace

extern "C" {

int64_t lora_quantised_row_bytes(int32_t d) { return d > 0 ? q_row_bytes(d) : 0; }
int64_t lora_quantised_scale_bytes(int32_t d) { return d > 0 ? q_scale_bytes(d) : 0; }

int32_t lora_quantise_rows(const void *X, int32_t dtype, int32_t T, int32_t d, uint8_t *codes,
                           uint8_t *scale, void *stream) {
  if (dtype != LORA_F32 && dtype != LORA_BF16) return LORA_ERR_INVALID_ARG;
  if (T < 0 || T > kMaxPairs) return LORA_ERR_INVALID_ARG;
  if (!dims_ok(d)) return LORA_ERR_UNSUPPORTED;
  if (T == 0) return LORA_OK;
  if (!X || !codes || !scale || X == codes || X == scale || codes == scale) return LORA_ERR_INVALID_ARG;
  return dev(launch_quantise_rows(X, dtype, T, d, codes, scale, false, static_cast<hipStream_t>(stream)));
}

int32_t lora_quantise_weight(const void *W_t, int32_t dtype, const lora_quantised_weight *w,
                             void *stream) {
  if (dtype != LORA_F32 && dtype != LORA_BF16) return LORA_ERR_INVALID_ARG;
  if (!W_t || !w || !w->q_t || !w->scale || (w->q == nullptr) != (w->scale_t == nullptr))
    return LORA_ERR_INVALID_ARG;
  if (!dims_ok(w->d_in) || !dims_ok(w->d_out) || w->d_in > kQMaxWidth || w->d_out > kQMaxWidth)
    return LORA_ERR_UNSUPPORTED;
  const void *b[5] = {W_t, w->q_t, w->scale, w->q, w->scale_t};
  for (int i = 0; i < 5; ++i)
    for (int j = 0; j < i; ++j)
      if (b[i] && b[i] == b[j]) return LORA_ERR_INVALID_ARG;
  return dev(launch_quantise_weight(W_t, dtype, w->d_out, w->d_in, w->q_t, w->q, w->scale, w->scale_t,
                                    static_cast<hipStream_t>(stream)));
}

size_t lora_apply_quantised_workspace_bytes(int32_t T, int32_t K, int32_t d_in, int32_t d_out,
                                            int32_t max_rank, int32_t dtype) {
  const size_t head = lora_apply_workspace_bytes(T, K, d_in, d_out, max_rank, dtype);
  if (!head) return 0;
  const size_t slab = apply_layout(nullptr, 0, T, K, d_in, d_out, dtype).partial_bytes;
  return align_up(head) + quant_tail_bytes(T, d_in, d_out, dtype, slab);
}

int32_t lora_apply_quantised(const void *X, const lora_quantised_weight *W, void *Y, int32_t T,
                             int32_t K, const float *gates, const uint8_t *keep_mask,
                             float keep_scale, const lora_pool_desc *pool, const void *plan, void *ws,
                             size_t ws_bytes, void *stream) {
  QuantApply a;
  const int32_t st = quant_apply_args(X, W, Y, T, K, gates, pool, plan, ws, ws_bytes, a);
  if (st != LORA_OK || T == 0) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t TK = int64_t(T) * K;
  const PlanView pv = plan_view(plan, TK, pool->n_adapters);
  hipError_t e = launch_shrink(apply_shrink_args(X, keep_mask, keep_scale, T, K, gates, pool, pv, a.w),
                               pool->dtype, TK, pool->n_adapters, pool->d_in, pool->d_out, s);
  if (e == hipSuccess) e = run_quantised(a.t, X, pool->dtype, a.q, s);
  if (e == hipSuccess) e = launch_epilogue(a.t.cfg, quant_epilogue_args(a.q), pool->dtype, s);
  return dev(e);
}

int32_t lora_forward_quantised(const int32_t *ids, const float *gates, int32_t T, int32_t K,
                               const void *X, const lora_quantised_weight *W, void *Y,
                               const uint8_t *keep_mask, float keep_scale,
                               const lora_pool_desc *pool, void *plan, size_t plan_bytes, void *ws,
                               size_t ws_bytes, void *stream) {
  QuantApply a;
  int32_t st = quant_apply_args(X, W, Y, T, K, gates, pool, plan, ws, ws_bytes, a);
  if (st != LORA_OK) return st;
  if (plan_bytes < lora_plan_bytes(T, K, pool->n_adapters)) return LORA_ERR_CAPACITY;
  if (T == 0) return lora_plan(ids, gates, T, K, pool, plan, plan_bytes, stream);
  if (!ids) return LORA_ERR_INVALID_ARG;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const PoolView pv = pool_view(pool);
  int32_t *const p = static_cast<int32_t *>(plan);
  hipError_t e;
  if (quantised_gemm_plan_fusable(a.t.cfg)) {
    // the plan beside the GEMM
    PlanLaunch pl = plan_setup(ids, gates, T, K, pv, p, 256, quantised_plan_lds_cap(a.t.cfg));
    if (a.t.cfg.kind == 4 && pool->dtype == LORA_BF16) {
      // decode: the per-slot shrink too, whose U the epilogue moves to the plan's places
      pl.a.no_sched = 1;
      const SlotShrinkArgs ss = slot_shrink_args(ids, gates, T, K, X, keep_mask, keep_scale, pool, a.w);
      e = launch_quantised_gemm_plan(a.t.cfg, a.q, &ss, pl, pool->dtype, s);
      if (e == hipSuccess)
        e = launch_epilogue_ucopy(a.t.cfg, a.q.g, pool->dtype, a.w.slot_u, a.w.sdesc, a.w.U, a.w.u_cap, s);
      return dev(e);
    }
    e = a.t.cfg.kind == 4 ? hipSuccess
                          : launch_quantise_rows(X, pool->dtype, T, pool->d_in, codes_of(a.q), scales_of(a.q),
                                                 true, s);
    if (e == hipSuccess) e = launch_quantised_gemm_plan(a.t.cfg, a.q, nullptr, pl, pool->dtype, s);
    if (e != hipSuccess) return LORA_ERR_DEVICE;
    if ((st = lora_shrink(X, keep_mask, keep_scale, T, K, gates, pool, plan, ws, a.head, stream)) != LORA_OK)
      return st;
  } else {
    // the plan beside the rows' quantisation, then U for the GEMM's epilogue
    const PlanLaunch pl = plan_setup(ids, gates, T, K, pv, p, kPlanThreads, kQPlanRowsLds);
    e = launch_quantise_plan(X, T, pool->d_in, codes_of(a.q), scales_of(a.q), pl, s);
    if (e != hipSuccess) return LORA_ERR_DEVICE;
    if ((st = lora_shrink(X, keep_mask, keep_scale, T, K, gates, pool, plan, ws, a.head, stream)) != LORA_OK)
      return st;
    e = launch_quantised_gemm(a.t.cfg, a.q, pool->dtype, s);
    if (e != hipSuccess) return LORA_ERR_DEVICE;
  }
  return dev(launch_epilogue(a.t.cfg, quant_epilogue_args(a.q), pool->dtype, s));
}

size_t lora_grad_x_quantised_workspace_bytes(int32_t T, int32_t d_in, int32_t d_out, int32_t dtype) {
  if (T < 0 || T > kMaxPairs || !dims_ok(d_in) || !dims_ok(d_out)) return 0;
  if (dtype != LORA_F32 && dtype != LORA_BF16) return 0;
  const size_t n = quant_tail_bytes(T, d_out, d_in, dtype, 0);
  return n > 0 ? n : kAlign;
}

int32_t lora_grad_x_quantised(const void *dY, const lora_quantised_weight *W,
                              const uint8_t *keep_mask, int32_t T, int32_t K,
                              const lora_pool_desc *pool, const void *plan, const void *grad_ws,
                              size_t grad_ws_bytes, int32_t max_rank, void *dX, void *ws,
                              size_t ws_bytes, void *stream) {
  int32_t st = check_batch(T, K);
  if (st != LORA_OK) return st;
  if ((st = check_pool(pool, true)) != LORA_OK) return st;
  if ((st = check_weight(W, pool)) != LORA_OK) return st;
  if (!plan || max_rank < 1 || max_rank > LORA_MAX_RANK) return LORA_ERR_INVALID_ARG;
  if (T == 0) return LORA_OK;
  if (!dY || !W->q || !W->scale_t || !grad_ws || !dX || !ws) return LORA_ERR_INVALID_ARG;
  if (dX == dY || dX == W->q || dX == W->scale_t) return LORA_ERR_INVALID_ARG;
  if (grad_ws_bytes < lora_grad_workspace_bytes(T, K, pool->n_adapters, pool->d_in, pool->d_out,
                                                max_rank, pool->dtype))
    return LORA_ERR_CAPACITY;
  const QuantTail t = quant_tail(T, few_adapters(K, pool), pool->d_out, pool->d_in, pool->dtype, 0);
  if (ws_bytes < t.total) return LORA_ERR_CAPACITY;
  const int64_t TK = int64_t(T) * K;
  const PlanView pv = plan_view(plan, TK, pool->n_adapters);
  QGemmArgs q{};
  q.g.Y = dX;
  // the expand on G and the A pages, as in lora_grad_x
  q.g.ex.K = K;
  q.g.ex.slot_desc = pv.slot_desc; q.g.ex.pair_tk = pv.pair_tk; q.g.ex.page_ids = pool->page_ids;
  q.g.ex.b_pages = pool->a_pages; q.g.ex.d_out = pool->d_in;
  q.g.ex.U = static_cast<const float *>(grad_ws); q.g.ex.hdr = pv.hdr;
  q.g.ex.u_cap = TK * max_rank;
  if (t.cfg.fused) q.g.mask = keep_mask;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  quantised_args(t, dY, T, pool->d_out, pool->d_in, W->q, W->scale_t, static_cast<char *>(ws), 0, q);
  hipError_t e = run_quantised(t, dY, pool->dtype, q, s);
  if (e == hipSuccess && !t.cfg.fused)
    e = launch_grad_x_epilogue(t.cfg, quant_epilogue_args(q), pool->dtype, keep_mask, s);
  return dev(e);
}

}  // extern "C"

// ------------------------------------------------------------ orthogonalised updates

namespace {

constexpr int32_t kMaxOrthAdapters = 16384;

int32_t orth_args(const lora_pool_desc *pool, const int32_t *adapters, int32_t M, int32_t max_rank,
                  int32_t steps, const float *coef, float eps, OrthArgs &a) {
  const int32_t st = check_pool(pool, false);
  if (st != LORA_OK) return st;
  if (M < 0 || max_rank < 1 || max_rank > LORA_MAX_RANK || steps < 1 || steps > LORA_MAX_ORTH_STEPS || !coef)
    return LORA_ERR_INVALID_ARG;
  if (!(eps >= 1e-20f && eps <= 1e20f)) return LORA_ERR_INVALID_ARG;
  if (M > kMaxOrthAdapters) return LORA_ERR_UNSUPPORTED;
  if (M > 0 && !adapters) return LORA_ERR_INVALID_ARG;
  a = OrthArgs{};
  a.pool = pool_view(pool);
  a.adapters = adapters;
  a.M = M; a.max_rank = max_rank; a.steps = steps;
  a.ca = coef[0]; a.cb = coef[1]; a.cc = coef[2]; a.eps = eps;
  return LORA_OK;
}

int32_t orth_factor(const lora_factor_update *u, int32_t d, int32_t dtype, OrthFactor &f) {
  if (!u || !u->pages || !u->momentum || !u->grad) return LORA_ERR_INVALID_ARG;
  // float32 pages may be named as their own master
  float *const master = dtype == LORA_F32 && u->master == u->pages ? nullptr : u->master;
  const void *b[4] = {u->pages, u->momentum, u->grad, master};
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < i; ++j)
      if (b[i] && b[i] == b[j]) return LORA_ERR_INVALID_ARG;
  f.src = u->grad; f.momentum = u->momentum; f.master = master; f.pages = u->pages;
  f.d = d; f.lr = u->lr; f.keep = 1.0f - u->lr * u->decay;
  return LORA_OK;
}

}  // namespace

extern "C" {

size_t lora_orthogonalise_workspace_bytes(int32_t M, int32_t max_rank, int32_t d) {
  if (M < 1 || M > kMaxOrthAdapters || max_rank < 1 || max_rank > LORA_MAX_RANK || !dims_ok(d)) return 0;
  return align_up(orth_workspace_bytes(M, 1, max_rank, d));
}

int32_t lora_orthogonalise(const lora_pool_desc *pool, const int32_t *adapters, int32_t M,
                           int32_t max_rank, const float *src_pages, float *out_pages, int32_t d,
                           int32_t steps, const float *coef, float eps, int32_t *out_rank, void *ws,
                           size_t ws_bytes, void *stream) {
  OrthArgs a;
  const int32_t st = orth_args(pool, adapters, M, max_rank, steps, coef, eps, a);
  if (st != LORA_OK) return st;
  if (!dims_ok(d)) return LORA_ERR_UNSUPPORTED;
  if (M == 0) return LORA_OK;
  if (!src_pages || !out_pages || src_pages == out_pages || !ws) return LORA_ERR_INVALID_ARG;
  if (ws_bytes < lora_orthogonalise_workspace_bytes(M, max_rank, d)) return LORA_ERR_CAPACITY;
  a.f[0].src = src_pages; a.f[0].out = out_pages; a.f[0].d = d;
  a.out_rank = out_rank;
  return dev(launch_orthogonal(a, 1, false, LORA_F32, ws, static_cast<hipStream_t>(stream)));
}

size_t lora_orthogonal_step_workspace_bytes(int32_t M, int32_t max_rank, int32_t d_in, int32_t d_out) {
  if (M < 1 || M > kMaxOrthAdapters || max_rank < 1 || max_rank > LORA_MAX_RANK || !dims_ok(d_in) ||
      !dims_ok(d_out))
    return 0;
  return align_up(orth_workspace_bytes(M, 2, max_rank, d_in > d_out ? d_in : d_out));
}

int32_t lora_orthogonal_step(const lora_pool_desc *pool, const int32_t *adapters, int32_t M,
                             int32_t max_rank, const lora_factor_update *a_update,
                             const lora_factor_update *b_update, float momentum, int32_t nesterov,
                             int32_t steps, const float *coef, float eps, int32_t *out_rank, void *ws,
                             size_t ws_bytes, void *stream) {
  OrthArgs a;
  int32_t st = orth_args(pool, adapters, M, max_rank, steps, coef, eps, a);
  if (st != LORA_OK) return st;
  if (!dims_ok(pool->d_in) || !dims_ok(pool->d_out)) return LORA_ERR_UNSUPPORTED;
  if (M == 0) return LORA_OK;
  if ((st = orth_factor(a_update, pool->d_in, pool->dtype, a.f[0])) != LORA_OK) return st;
  if ((st = orth_factor(b_update, pool->d_out, pool->dtype, a.f[1])) != LORA_OK) return st;
  // what one factor writes is not the other's (their gradients may be the same)
  const void *b[2][4];
  for (int i = 0; i < 2; ++i) {
    b[i][0] = a.f[i].pages; b[i][1] = a.f[i].momentum; b[i][2] = a.f[i].master; b[i][3] = a.f[i].src;
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j)
      if ((i < 3 || j < 3) && b[0][i] && b[0][i] == b[1][j]) return LORA_ERR_INVALID_ARG;
  if (!ws) return LORA_ERR_INVALID_ARG;
  if (ws_bytes < lora_orthogonal_step_workspace_bytes(M, max_rank, pool->d_in, pool->d_out))
    return LORA_ERR_CAPACITY;
  a.mu = momentum; a.nesterov = nesterov ? 1 : 0;
  a.out_rank = out_rank;
  return dev(launch_orthogonal(a, 2, true, pool->dtype, ws, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ------------------------------------------------------------ gated block

namespace {

// The second pool's tables are the first's: one plan serves both.
int32_t check_pair(const lora_pool_desc *a, const lora_pool_desc *b) {
  int32_t st = check_pool(a, true);
  if (st == LORA_OK) st = check_pool(b, true);
  if (st != LORA_OK) return st;
  const bool same = a->dtype == b->dtype && a->d_in == b->d_in && a->d_out == b->d_out &&
                    a->n_adapters == b->n_adapters && a->n_pages == b->n_pages &&
                    a->n_page_ids == b->n_page_ids && a->rank == b->rank &&
                    a->page_start == b->page_start && a->page_ids == b->page_ids;
  return same ? LORA_OK : LORA_ERR_INVALID_ARG;
}

bool activation_ok(int32_t act) {
  return act == LORA_ACT_SILU || act == LORA_ACT_GELU || act == LORA_ACT_GELU_TANH;
}

// out[0 .. n_out) name no buffer twice, and none of in[0 .. n_in).
bool outputs_apart(const void *const *out, int n_out, const void *const *in, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    if (!out[i]) continue;
    for (int j = 0; j < i; ++j)
      if (out[i] == out[j]) return false;
    for (int j = 0; j < n_in; ++j)
      if (out[i] == in[j]) return false;
  }
  return true;
}

// The buffers of a call, to tell whether an output shares memory with another.
struct Ranges {
  struct {
    uintptr_t at, end;
  } r[40];
  int n = 0;
  void add(const void *p, size_t bytes) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    if (p && bytes) r[n++] = {at, at + bytes < at ? UINTPTR_MAX : at + bytes};
  }
  // What kernels read of a pool.
  void add(const lora_pool_desc *p) {
    const size_t e = p->dtype == LORA_BF16 ? 2 : 4, N = size_t(p->n_adapters), pages = size_t(p->n_pages);
    add(p->rank, N * 4);
    add(p->page_start, (N + 1) * 4);
    add(p->page_ids, size_t(p->n_page_ids) * 4);
    add(p->scale, N * 4);
    add(p->a_pages, pages * size_t(p->d_in) * e);
    add(p->b_pages, pages * size_t(p->d_out) * e);
  }
  bool apart(const Ranges &o) const {
    for (int i = 0; i < n; ++i)
      for (int j = 0; j < o.n; ++j)
        if (r[i].at < o.r[j].end && o.r[j].at < r[i].end) return false;
    return true;
  }
  // No two of them overlap.
  bool apart() const {
    for (int i = 0; i < n; ++i)
      for (int j = 0; j < i; ++j)
        if (r[i].at < r[j].end && r[j].at < r[i].end) return false;
    return true;
  }
};

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool aligned16(const void *p) { return aligned(p, 16); }

// Rows of a weight tile, up to 256, are reached by 32-bit byte offsets.
constexpr int32_t kMaxWidth = 1 << 22;

struct GatedCall {
  ApplyWs w[2];
  GemmArgs g[2];
  GemmConfig cfg;
  bool whole;
  GatedArgs a;
  TermsArgs t;
};

TermsArgs terms_args(const PlanView &pv, const lora_pool_desc *pool, int32_t T, int32_t K) {
  TermsArgs t{};
  t.hdr = pv.hdr; t.pair_tk = pv.pair_tk; t.pair_adapter = pv.pair_adapter; t.u_off = pv.u_off;
  t.slot_pos = pv.slot_pos;
  t.rank = pool->rank; t.page_start = pool->page_start; t.page_ids = pool->page_ids;
  t.M = T; t.K = K;
  return t;
}

// What a call may write of an apply workspace.
size_t apply_ws_used(const void *ws, size_t ws_bytes, const ApplyWs &w, int32_t T, int32_t K) {
  const size_t head = size_t(reinterpret_cast<const char *>(w.U) - static_cast<const char *>(ws));
  return std::min(ws_bytes, head + size_t(T) * size_t(K) * LORA_MAX_RANK * sizeof(float));
}

// The checks of the gated forward (T > 0 from the workspaces on), and its
// arguments.
int32_t gated_args(const int32_t *ids, const void *X, const void *W_gate_t, const void *W_up_t, int32_t activation,
                   void *H, void *pre_gate, void *pre_up, int32_t T, int32_t K, const float *gates,
                   const uint8_t *keep_mask, const lora_pool_desc *gate, const lora_pool_desc *up, const void *plan,
                   void *ws_gate, size_t ws_gate_bytes, void *ws_up, size_t ws_up_bytes, GatedCall &c) {
  int32_t st = check_batch(T, K);
  if (st != LORA_OK) return st;
  if ((st = check_pair(gate, up)) != LORA_OK) return st;
  if (!plan || !activation_ok(activation) || !pre_gate != !pre_up) return LORA_ERR_INVALID_ARG;
  if (gate->d_in > kMaxWidth || gate->d_out > kMaxWidth) return LORA_ERR_UNSUPPORTED;
  if (T == 0) return LORA_OK;
  if (!X || !W_gate_t || !W_up_t || !H || !gates || !ws_gate || !ws_up) return LORA_ERR_INVALID_ARG;
  const void *out[] = {H, pre_gate, pre_up, ws_gate, ws_up}, *in[] = {X, W_gate_t, W_up_t, plan};
  if (!outputs_apart(out, 5, in, 4)) return LORA_ERR_INVALID_ARG;
  for (const void *p : {X, W_gate_t, W_up_t, static_cast<const void *>(H), static_cast<const void *>(pre_gate),
                        static_cast<const void *>(pre_up), static_cast<const void *>(ws_gate),
                        static_cast<const void *>(ws_up)})
    if (!aligned16(p)) return LORA_ERR_INVALID_ARG;
  if (!aligned(keep_mask, 8)) return LORA_ERR_INVALID_ARG;
  if ((st = base_args(X, W_gate_t, H, T, K, gate, plan, ws_gate, ws_gate_bytes, c.cfg, c.g[0])) != LORA_OK ||
      (st = base_args(X, W_up_t, H, T, K, up, plan, ws_up, ws_up_bytes, c.cfg, c.g[1])) != LORA_OK)
    return st;
  c.w[0] = apply_layout(ws_gate, ws_gate_bytes, T, K, gate->d_in, gate->d_out, gate->dtype);
  c.w[1] = apply_layout(ws_up, ws_up_bytes, T, K, up->d_in, up->d_out, up->dtype);
  const size_t e = gate->dtype == LORA_BF16 ? 2 : 4, TK = size_t(T) * size_t(K), F = size_t(gate->d_out), d = size_t(gate->d_in);
  Ranges outs, ins;
  for (const void *p : {static_cast<const void *>(H), static_cast<const void *>(pre_gate), static_cast<const void *>(pre_up)})
    outs.add(p, size_t(T) * F * e);
  outs.add(ws_gate, apply_ws_used(ws_gate, ws_gate_bytes, c.w[0], T, K));
  outs.add(ws_up, apply_ws_used(ws_up, ws_up_bytes, c.w[1], T, K));
  outs.add(plan, lora_plan_bytes(T, K, gate->n_adapters));
  ins.add(X, size_t(T) * d * e);
  ins.add(W_gate_t, F * d * e);
  ins.add(W_up_t, F * d * e);
  ins.add(ids, TK * sizeof(int32_t));
  ins.add(gates, TK * sizeof(float));
  ins.add(keep_mask, size_t(T) * d);
  ins.add(gate);
  ins.add(up);
  if (!outs.apart() || !outs.apart(ins)) return LORA_ERR_INVALID_ARG;
  const PlanView pv = plan_view(plan, int64_t(T) * K, gate->n_adapters);
  GatedArgs &a = c.a;
  a = GatedArgs{};
  a.X = X; a.W[0] = W_gate_t; a.W[1] = W_up_t;
  a.M = T; a.N = gate->d_out; a.Kd = gate->d_in;
  a.ex = c.g[0].ex;
  // U of both or of neither
  if (c.w[1].u_cap < a.ex.u_cap) a.ex.u_cap = c.w[1].u_cap;
  a.U_up = c.w[1].U; a.b_up = up->b_pages;
  a.act = activation;
  a.H = H; a.pre_gate = pre_gate; a.pre_up = pre_up;
  a.part[0] = c.g[0].partial; a.part[1] = c.g[1].partial;
  a.splits = c.cfg.splits;
  a.slot_pos = pv.slot_pos;
  c.whole = c.cfg.kind != 4 && gated_whole(T, a.Kd, gate->dtype, c.cfg.fused);
  if (c.cfg.kind == 4 || c.whole) return LORA_OK;
  a.splits = gated_base_splits(T, a.N, a.Kd, gate->dtype, c.cfg.splits);
  TermsArgs &t = c.t;
  t = terms_args(pv, gate, T, K);
  for (int p = 0; p < 2; ++p) {
    t.sums[p] = a.sums[p] = c.g[p].partial;
    // the slots' terms behind, where the partials' room has them
    if (K > 1 && K <= kTermSlots && a.splits + K <= c.cfg.splits)
      t.slots[p] = a.sums[p] + int64_t(a.splits) * T * a.N;
  }
  t.U[0] = a.ex.U; t.U[1] = a.U_up; t.u_cap = a.ex.u_cap;
  t.pages[0] = gate->b_pages; t.pages[1] = up->b_pages;
  t.N = a.N; t.splits = a.splits;
  t.act = activation;
  t.H = H; t.pre_gate = pre_gate; t.pre_up = pre_up;
  return LORA_OK;
}

hipError_t gated_shrinks(const GatedCall &c, const void *X, const uint8_t *keep_mask, float keep_scale,
                         int32_t T, int32_t K, const float *gates, const lora_pool_desc *gate,
                         const lora_pool_desc *up, const PlanView &pv, hipStream_t s) {
  return launch_shrink_pair(apply_shrink_args(X, keep_mask, keep_scale, T, K, gates, gate, pv, c.w[0]),
                            apply_shrink_args(X, keep_mask, keep_scale, T, K, gates, up, pv, c.w[1]), gate->dtype,
                            int64_t(T) * K, gate->n_adapters, gate->d_in, gate->d_out, s);
}

}  // namespace

extern "C" {

int32_t lora_gated_apply(const void *X, const void *W_gate_t, const void *W_up_t, int32_t activation,
                         void *H, void *pre_gate, void *pre_up, int32_t T, int32_t K,
                         const float *gates, const uint8_t *keep_mask, float keep_scale,
                         const lora_pool_desc *gate, const lora_pool_desc *up, const void *plan,
                         void *ws_gate, size_t ws_gate_bytes, void *ws_up, size_t ws_up_bytes,
                         void *stream) {
  GatedCall c;
  const int32_t st = gated_args(nullptr, X, W_gate_t, W_up_t, activation, H, pre_gate, pre_up, T, K, gates, keep_mask,
                                gate, up, plan, ws_gate, ws_gate_bytes, ws_up, ws_up_bytes, c);
  if (st != LORA_OK || T == 0) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const PlanView pv = plan_view(plan, int64_t(T) * K, gate->n_adapters);
  const bool base = c.cfg.kind != 4 && !c.whole;
  hipError_t e = base ? launch_gated_base(c.a, gate->dtype, nullptr, s) : hipSuccess;
  if (e == hipSuccess) e = gated_shrinks(c, X, keep_mask, keep_scale, T, K, gates, gate, up, pv, s);
  if (e != hipSuccess) return LORA_ERR_DEVICE;
  if (base) return dev(launch_terms(c.t, false, gate->dtype, s));
  if (c.whole) return dev(launch_gated(c.a, s));
  e = launch_gated_decode(c.cfg, c.g, s);
  if (e == hipSuccess) e = launch_gated_decode_epilogue(c.a, s);
  return dev(e);
}

int32_t lora_gated_forward(const int32_t *ids, const float *gates, int32_t T, int32_t K,
                           const void *X, const void *W_gate_t, const void *W_up_t,
                           int32_t activation, void *H, void *pre_gate, void *pre_up,
                           const uint8_t *keep_mask, float keep_scale, const lora_pool_desc *gate,
                           const lora_pool_desc *up, void *plan, size_t plan_bytes, void *ws_gate,
                           size_t ws_gate_bytes, void *ws_up, size_t ws_up_bytes, void *stream) {
  GatedCall c;
  int32_t st = gated_args(ids, X, W_gate_t, W_up_t, activation, H, pre_gate, pre_up, T, K, gates, keep_mask, gate, up, plan,
                          ws_gate, ws_gate_bytes, ws_up, ws_up_bytes, c);
  if (st != LORA_OK) return st;
  if (plan_bytes < lora_plan_bytes(T, K, gate->n_adapters)) return LORA_ERR_CAPACITY;
  if (T > 0 && !ids) return LORA_ERR_INVALID_ARG;
  if (T > 0 && c.cfg.kind == 4) {
    // decode: plan, per-slot shrinks and both products' partials in one
    // launch, and an epilogue that also stores U in the plan's layout
    const hipStream_t s = static_cast<hipStream_t>(stream);
    Fwd f{c.cfg, c.g[0], true};
    const SlotShrinkArgs ss[2] = {slot_shrink_args(ids, gates, T, K, X, keep_mask, keep_scale, gate, c.w[0]),
                                  slot_shrink_args(ids, gates, T, K, X, keep_mask, keep_scale, up, c.w[1])};
    const hipError_t e = launch_gated_decode_plan(c.cfg, c.g, ss, forward_plan(ids, gates, T, K, gate, plan, f, c.w[0]), s);
    if (e != hipSuccess) return LORA_ERR_DEVICE;
    c.a.sdesc = c.w[0].sdesc;
    c.a.slot_stride = LORA_MAX_RANK;
    for (int p = 0; p < 2; ++p) c.a.u_out[p] = c.w[p].U;
    c.a.ex.U = c.w[0].slot_u;
    c.a.U_up = c.w[1].slot_u;
    return dev(launch_gated_decode_epilogue(c.a, s));
  }
  if (T > 0 && !c.whole) {
    // the plan beside the base products
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const PlanLaunch pl = gated_base_plan(c.a, gate->dtype, ids, gates, T, K, pool_view(gate), static_cast<int32_t *>(plan));
    if (pl.lds) {
      const PlanView pv = plan_view(plan, int64_t(T) * K, gate->n_adapters);
      hipError_t e = launch_gated_base(c.a, gate->dtype, &pl.a, s);
      if (e == hipSuccess) e = gated_shrinks(c, X, keep_mask, keep_scale, T, K, gates, gate, up, pv, s);
      if (e == hipSuccess) e = launch_terms(c.t, false, gate->dtype, s);
      return dev(e);
    }
  }
  if ((st = lora_plan(ids, gates, T, K, gate, plan, plan_bytes, stream)) != LORA_OK || T == 0) return st;
  return lora_gated_apply(X, W_gate_t, W_up_t, activation, H, pre_gate, pre_up, T, K, gates, keep_mask,
                          keep_scale, gate, up, plan, ws_gate, ws_gate_bytes, ws_up, ws_up_bytes, stream);
}

}  // extern "C"

namespace {

// Workspace of the gated backward: [G of the gate][G of the up projection], and
// where the product is split [the splits' sums][each slot's terms].
struct GatedGradWs {
  int splits;
  size_t g, sums, slots, total;
};

GatedGradWs gated_grad_ws(int32_t T, int32_t K, int32_t d_in, int32_t d_out, int32_t max_rank, int32_t dtype) {
  GatedGradWs w{};
  w.splits = gated_grad_x_splits(T > 0 ? T : 1, d_in, d_out, dtype);
  w.g = align_up(size_t(T) * size_t(K) * size_t(max_rank) * sizeof(float) + 4);
  const size_t one = size_t(T) * size_t(d_in) * sizeof(float);
  w.sums = align_up(size_t(w.splits) * one);
  w.slots = w.splits > 0 && K > 1 && K <= kTermSlots ? align_up(size_t(K) * one) : 0;
  w.total = 2 * w.g + w.sums + w.slots;
  return w;
}

}  // namespace

extern "C" {

size_t lora_gated_grad_workspace_bytes(int32_t T, int32_t K, int32_t d_in, int32_t d_out,
                                       int32_t max_rank, int32_t dtype) {
  if (check_batch(T, K) != LORA_OK || !dims_ok(d_in) || !dims_ok(d_out)) return 0;
  if (max_rank < 1 || max_rank > LORA_MAX_RANK || (dtype != LORA_F32 && dtype != LORA_BF16)) return 0;
  if (d_in > kMaxWidth || d_out > kMaxWidth) return 0;
  return gated_grad_ws(T, K, d_in, d_out, max_rank, dtype).total;
}

int32_t lora_gated_grad(const void *dH, const void *pre_gate, const void *pre_up, int32_t activation,
                        const void *W_gate, const void *W_up, const uint8_t *keep_mask,
                        float keep_scale, int32_t T, int32_t K, const float *gates,
                        const lora_pool_desc *gate, const lora_pool_desc *up, const void *plan,
                        int32_t max_rank, void *d_gate, void *d_up, void *dX, void *ws,
                        size_t ws_bytes, void *stream) {
  int32_t st = check_batch(T, K);
  if (st != LORA_OK) return st;
  if ((st = check_pair(gate, up)) != LORA_OK) return st;
  if (!plan || !activation_ok(activation) || max_rank < 1 || max_rank > LORA_MAX_RANK)
    return LORA_ERR_INVALID_ARG;
  if (gate->d_in > kMaxWidth || gate->d_out > kMaxWidth) return LORA_ERR_UNSUPPORTED;
  if (T == 0) return LORA_OK;
  if (!dH || !pre_gate || !pre_up || !d_gate || !d_up) return LORA_ERR_INVALID_ARG;
  const void *out[] = {d_gate, d_up, dX, ws}, *in[] = {dH, W_gate, W_up, plan, keep_mask};
  if (!outputs_apart(out, 4, in, 5) || d_gate == pre_up || d_up == pre_gate) return LORA_ERR_INVALID_ARG;
  if (dX && (!W_gate || !W_up || !gates || !ws || dX == pre_gate || dX == pre_up)) return LORA_ERR_INVALID_ARG;
  for (const void *p : {dH, pre_gate, pre_up, W_gate, W_up, static_cast<const void *>(d_gate),
                        static_cast<const void *>(d_up), static_cast<const void *>(dX), static_cast<const void *>(ws)})
    if (!aligned16(p)) return LORA_ERR_INVALID_ARG;
  if (!aligned(keep_mask, 8)) return LORA_ERR_INVALID_ARG;
  const int32_t F = gate->d_out, d = gate->d_in, dtype = gate->dtype;
  const GatedGradWs w = gated_grad_ws(T, K, d, F, max_rank, dtype);
  if (dX && ws_bytes < w.total) return LORA_ERR_CAPACITY;
  const size_t e_size = dtype == LORA_BF16 ? 2 : 4, rows = size_t(T) * size_t(F) * e_size;
  Ranges outs, ins;
  outs.add(d_gate, rows);
  outs.add(d_up, rows);
  ins.add(dH, rows);
  if (pre_gate != d_gate) ins.add(pre_gate, rows);      // in place, or apart
  if (pre_up != d_up) ins.add(pre_up, rows);
  if (dX) {
    outs.add(dX, size_t(T) * size_t(d) * e_size);
    outs.add(ws, w.total);
    outs.add(plan, lora_plan_bytes(T, K, gate->n_adapters));
    ins.add(W_gate, size_t(d) * size_t(F) * e_size);
    ins.add(W_up, size_t(d) * size_t(F) * e_size);
    ins.add(gates, size_t(T) * size_t(K) * sizeof(float));
    ins.add(keep_mask, size_t(T) * size_t(d));
    ins.add(gate);
    ins.add(up);
  }
  if (!outs.apart() || !outs.apart(ins)) return LORA_ERR_INVALID_ARG;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = launch_gated_act_grad(dH, pre_gate, pre_up, activation, d_gate, d_up, int64_t(T) * F, dtype, s);
  if (e != hipSuccess || !dX) return dev(e);

  const int64_t TK = int64_t(T) * K;
  const PlanView pv = plan_view(plan, TK, gate->n_adapters);
  char *base = static_cast<char *>(ws);
  const lora_pool_desc *const pool[2] = {gate, up};
  const void *const dY[2] = {d_gate, d_up}, *const W[2] = {W_gate, W_up};
  GatedGradXArgs a{};
  ShrinkArgs shrink[2] = {};
  for (int p = 0; p < 2; ++p) {
    ShrinkArgs &sa = shrink[p];
    sa.Z = dY[p]; sa.extra_scale = keep_mask ? keep_scale : 1.0f;
    sa.T = T; sa.K = K; sa.d = F;
    sa.pages = pool[p]->b_pages;
    sa.rank = gate->rank; sa.page_start = gate->page_start; sa.page_ids = gate->page_ids;
    sa.scale = pool[p]->scale; sa.gates = gates; sa.plan = pv;
    sa.err_word = const_cast<int32_t *>(pv.hdr) + LORA_PH_ERR;
    sa.out = reinterpret_cast<float *>(base + p * w.g); sa.out_cap = TK * max_rank;
    a.dY[p] = dY[p]; a.W[p] = W[p];
  }
  e = launch_shrink_pair(shrink[0], shrink[1], dtype, TK, gate->n_adapters, d, F, s);
  if (e != hipSuccess) return LORA_ERR_DEVICE;
  a.M = T; a.N = d; a.Kd = F;
  a.ex.K = K;
  a.ex.slot_desc = pv.slot_desc; a.ex.pair_tk = pv.pair_tk; a.ex.page_ids = gate->page_ids;
  a.ex.b_pages = gate->a_pages; a.ex.d_out = d;
  a.ex.U = reinterpret_cast<float *>(base); a.ex.hdr = pv.hdr; a.ex.u_cap = TK * max_rank;
  a.U_up = reinterpret_cast<float *>(base + w.g); a.b_up = up->a_pages;
  a.mask = keep_mask; a.dX = dX;
  a.slot_pos = pv.slot_pos;
  a.splits = w.splits;
  TermsArgs t = terms_args(pv, gate, T, K);
  if (w.splits) {
    t.sums[0] = a.sums = reinterpret_cast<float *>(base + 2 * w.g);
    if (w.slots) t.slots[0] = reinterpret_cast<float *>(base + 2 * w.g + w.sums);
    t.U[0] = a.ex.U; t.U[1] = a.U_up; t.u_cap = a.ex.u_cap;
    t.pages[0] = gate->a_pages; t.pages[1] = up->a_pages;
    t.N = d; t.splits = w.splits;
    t.mask = keep_mask; t.dX = dX;
  }
  return dev(launch_gated_grad_x(a, t, dtype, s));
}

}  // extern "C"

// ------------------------------------------------------------ cross entropy

namespace {

int32_t check_entropy(int32_t T, int32_t V, int32_t d, int32_t dtype) {
  if (T < 0 || V < 1 || (dtype != LORA_F32 && dtype != LORA_BF16)) return LORA_ERR_INVALID_ARG;
  if (T > kMaxPairs || V > (1 << 22) || !dims_ok(d) || d > kMaxWidth) return LORA_ERR_UNSUPPORTED;
  return LORA_OK;
}

}  // namespace

extern "C" {

size_t lora_cross_entropy_workspace_bytes(int32_t T, int32_t V, int32_t d, int32_t dtype,
                                          int32_t with_grad) {
  if (check_entropy(T, V, d, dtype) != LORA_OK) return 0;
  return align_up(cross_entropy_workspace_bytes(T > 0 ? T : 1, V, d, dtype, with_grad != 0));
}

int32_t lora_cross_entropy(const void *X, const void *W_t, int32_t dtype, int32_t T, int32_t V,
                           int32_t d, const int32_t *targets, const float *weights,
                           float logit_scale, float *loss, void *dX, void *ws, size_t ws_bytes,
                           void *stream) {
  const int32_t st = check_entropy(T, V, d, dtype);
  if (st != LORA_OK) return st;
  if (!(logit_scale - logit_scale == 0.f) || logit_scale == 0.f) return LORA_ERR_INVALID_ARG;
  if (T == 0) return LORA_OK;
  if (!X || !W_t || !targets || !loss || !ws) return LORA_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(W_t) || !aligned16(dX) || !aligned16(ws)) return LORA_ERR_INVALID_ARG;
  const void *out[] = {loss, dX, ws}, *in[] = {X, W_t, targets, weights};
  if (!outputs_apart(out, 3, in, 4)) return LORA_ERR_INVALID_ARG;
  const size_t need = lora_cross_entropy_workspace_bytes(T, V, d, dtype, dX != nullptr);
  if (ws_bytes < need) return LORA_ERR_CAPACITY;
  const size_t row = size_t(d) * (dtype == LORA_BF16 ? 2 : 4);
  Ranges outs, ins;
  outs.add(loss, size_t(T) * sizeof(float));
  outs.add(dX, size_t(T) * row);
  outs.add(ws, need);
  ins.add(X, size_t(T) * row);
  ins.add(W_t, size_t(V) * row);
  ins.add(targets, size_t(T) * sizeof(int32_t));
  ins.add(weights, size_t(T) * sizeof(float));
  if (!outs.apart() || !outs.apart(ins)) return LORA_ERR_INVALID_ARG;
  CrossEntropyArgs a{};
  a.X = X; a.W = W_t; a.T = T; a.V = V; a.d = d;
  a.targets = targets; a.weights = weights; a.logit_scale = logit_scale;
  a.loss = loss; a.dX = dX;
  return dev(launch_cross_entropy(a, dtype, ws, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ------------------------------------------------------------ gradient clipping

namespace {

constexpr int32_t kMaxClipLayers = 1024;

struct Span {
  uintptr_t at, end;
  int32_t id;          // gradients and what replaces them: 2 x layer + factor
};

Span span(const void *p, size_t bytes, int32_t id) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  return {at, at + bytes, id};
}

// The outputs are apart from each other, and from every input but the gradient
// that they replace in place.
bool spans_apart(Span *out, int n_out, const Span *in, int n_in) {
  std::sort(out, out + n_out, [](const Span &a, const Span &b) { return a.at < b.at; });
  for (int i = 1; i < n_out; ++i)
    if (out[i].at < out[i - 1].end) return false;
  for (int i = 0; i < n_in; ++i) {
    // the first output that ends behind the gradient's start, and those after it
    const Span *o = std::upper_bound(out, out + n_out, in[i].at, [](uintptr_t at, const Span &b) { return at < b.end; });
    for (; o < out + n_out && o->at < in[i].end; ++o)
      if (o->id != in[i].id || o->at != in[i].at) return false;
  }
  return true;
}

}  // namespace

extern "C" {

size_t lora_clip_grad_workspace_bytes(int32_t n_layers, int32_t M, int32_t max_rank) {
  if (n_layers < 0 || n_layers > kMaxClipLayers || M < 0 || M > kMaxOrthAdapters || max_rank < 1 ||
      max_rank > LORA_MAX_RANK)
    return 0;
  return align_up(clip_workspace_bytes(n_layers, M, max_rank) + 8);
}

int32_t lora_clip_grad(const lora_grad_desc *layers, int32_t n_layers, const int32_t *adapters,
                       int32_t M, int32_t max_rank, float max_norm, int32_t together, float *norm,
                       void *ws, size_t ws_bytes, void *stream) {
  if (n_layers < 0 || M < 0 || (n_layers > 0 && !layers) || (M > 0 && !adapters) || !norm || !ws)
    return LORA_ERR_INVALID_ARG;
  if (max_rank < 1 || max_rank > LORA_MAX_RANK || !(max_norm > 0.f)) return LORA_ERR_INVALID_ARG;
  if (n_layers > kMaxClipLayers || M > kMaxOrthAdapters) return LORA_ERR_UNSUPPORTED;
  if (!aligned(norm, sizeof(float)) || !aligned(ws, sizeof(double))) return LORA_ERR_INVALID_ARG;
  ClipLayer l[kMaxClipLayers];
  Span outs[2 * kMaxClipLayers + 2], ins[5 * kMaxClipLayers + 1];
  int n = 0, n_in = 0;
  const size_t need = lora_clip_grad_workspace_bytes(n_layers, M, max_rank);
  outs[n++] = span(norm, (size_t(M) + 1) * sizeof(float), -1);
  outs[n++] = span(ws, need, -2);
  if (M > 0) ins[n_in++] = span(adapters, size_t(M) * sizeof(int32_t), -3);
  for (int32_t i = 0; i < n_layers; ++i) {
    const lora_grad_desc &g = layers[i];
    const int32_t st = check_pool(&g.pool, false);
    if (st != LORA_OK) return st;
    if (!dims_ok(g.pool.d_in) || !dims_ok(g.pool.d_out)) return LORA_ERR_UNSUPPORTED;
    const bool none = g.pool.n_pages == 0;
    const float *in[2] = {g.dA_pages, g.dB_pages};
    float *out[2] = {g.dA_out, g.dB_out};
    l[i] = ClipLayer{{in[0], in[1]}, {out[0], out[1]}, g.pool.rank, g.pool.page_start, g.pool.page_ids,
                     g.pool.n_pages, g.pool.n_page_ids, {g.pool.d_in, g.pool.d_out}, g.pool.n_adapters};
    for (int f = 0; f < 2; ++f) {
      if ((!in[f] || !out[f]) && !none) return LORA_ERR_INVALID_ARG;
      if (!aligned16(in[f]) || !aligned16(out[f])) return LORA_ERR_INVALID_ARG;
      const size_t bytes = size_t(g.pool.n_pages) * size_t(l[i].d[f]) * sizeof(float);
      if (bytes == 0) continue;
      ins[n_in++] = span(in[f], bytes, 2 * i + f);
      outs[n++] = span(out[f], bytes, 2 * i + f);
    }
    ins[n_in++] = span(g.pool.rank, size_t(g.pool.n_adapters) * sizeof(int32_t), -3);
    ins[n_in++] = span(g.pool.page_start, (size_t(g.pool.n_adapters) + 1) * sizeof(int32_t), -3);
    if (g.pool.n_page_ids > 0) ins[n_in++] = span(g.pool.page_ids, size_t(g.pool.n_page_ids) * sizeof(int32_t), -3);
  }
  if (!spans_apart(outs, n, ins, n_in)) return LORA_ERR_INVALID_ARG;
  if (ws_bytes < need) return LORA_ERR_CAPACITY;
  ClipArgs a{};
  a.adapters = adapters; a.M = M; a.max_rank = max_rank; a.together = together ? 1 : 0;
  a.max_norm = max_norm; a.norm = norm;
  return dev(launch_clip(l, n_layers, a, ws, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
