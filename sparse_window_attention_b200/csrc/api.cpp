// C ABI of libbasa: argument checks, then dispatch to the kernel launchers.
// Every check runs on the host before any CUDA call, so an invalid call
// returns its status and launches nothing.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "basa_internal.h"
#include "byte_views.h"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool empty_batch(const basa_params *p) { return p->B == 0 || p->heads == 0; }

// Fewest routing candidates of any window under a radius r >= 1: a corner window
// sees min(r, n - 1) + 1 window positions along an axis of n windows.
int64_t min_candidates(const basa_params *p) {
  const int64_t n[3] = {p->T / p->wt, p->H / p->wh, p->W / p->ww};
  int64_t c = 1;
  for (int a = 0; a < 3; ++a) c *= (n[a] - 1 < p->route_radius ? n[a] - 1 : p->route_radius) + 1;
  return c - 1;
}

// Checks shared by every entry point.
basa_status check_common(const basa_params *p) {
  if (!p) return BASA_ERR_INVALID_ARG;
  if (p->B < 0 || p->heads < 0 || p->n_text < 0 || p->routed_k < 0) return BASA_ERR_INVALID_ARG;
  if (p->dtype != BASA_BF16 && p->dtype != BASA_F32) return BASA_ERR_INVALID_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return BASA_ERR_UNSUPPORTED;
  if (p->T < 1 || p->H < 1 || p->W < 1) return BASA_ERR_SHAPE;
  if (p->wt < 1 || p->wh < 1 || p->ww < 1) return BASA_ERR_SHAPE;
  if (p->T % p->wt || p->H % p->wh || p->W % p->ww) return BASA_ERR_SHAPE;
  if (p->st < 0 || p->st >= p->T || p->sy < 0 || p->sy >= p->H || p->sx < 0 || p->sx >= p->W) return BASA_ERR_SHAPE;
  const bool no_pool = p->pt == 0 && p->ph == 0 && p->pw == 0;
  if (!no_pool) {
    if (p->pt < 1 || p->ph < 1 || p->pw < 1) return BASA_ERR_SHAPE;
    if (p->T % p->pt || p->H % p->ph || p->W % p->pw) return BASA_ERR_SHAPE;
  }
  const int64_t N = int64_t(p->T) * p->H * p->W;
  const int64_t rows = N + p->n_text;
  if (rows >= (int64_t(1) << 31)) return BASA_ERR_UNSUPPORTED;
  const int64_t bh = int64_t(p->B) * p->heads;
  if (bh >= (int64_t(1) << 31)) return BASA_ERR_UNSUPPORTED;
  const int64_t nwin = N / (int64_t(p->wt) * p->wh * p->ww);
  if (p->route_radius < 0) return BASA_ERR_INVALID_ARG;
  if (p->routed_k > 0) {
    if (p->routed_k > basa::kMaxRouted || p->routed_k > nwin - 1) return BASA_ERR_INVALID_ARG;
    if (p->route_radius > 0 && p->routed_k > min_candidates(p)) return BASA_ERR_INVALID_ARG;
  }
  return BASA_OK;
}

bool has_pool(const basa_params *p) { return p->pt > 0; }

// More windows than the bfloat16 backward's lists of them take.
bool too_many_windows(const basa_params *p) {
  const int64_t n = int64_t(p->T / p->wt) * (p->H / p->wh) * (p->W / p->ww);
  return p->dtype == BASA_BF16 && n > (p->routed_k > 0 ? basa::kMaxBwdRouted : basa::kMaxBwdWindows);
}

bool aligned_element(const void *x, const basa_params *p) {
  return (reinterpret_cast<uintptr_t>(x) & (p->dtype == BASA_BF16 ? 1u : 3u)) == 0;
}

// Differential attention: shape (2 heads maps), then the parameters, then the inputs.
basa_status check_diff_shape(const basa_params *p) {
  basa_status st = check_common(p);
  if (st != BASA_OK) return st;
  if (p->dtype == BASA_BF16 && p->head_dim != 128) return BASA_ERR_UNSUPPORTED;
  if (2 * int64_t(p->B) * p->heads >= (int64_t(1) << 31)) return BASA_ERR_UNSUPPORTED;
  return BASA_OK;
}

basa_status check_diff(const basa_diff_params *dp, const basa_params *p) {
  basa_status st = check_diff_shape(p);
  if (st != BASA_OK) return st;
  if (!dp || !aligned_element(dp->lambda, p) || !aligned16(dp->weight)) return BASA_ERR_INVALID_ARG;
  if (dp->weight && (!std::isfinite(dp->gain) || !(dp->eps > 0.f) || !std::isfinite(dp->eps))) return BASA_ERR_INVALID_ARG;
  return BASA_OK;
}

basa_status check_diff_inputs(const void *q, const void *k, const void *v, const void *kp, const void *vp,
                              const int32_t *route_idx, const basa_diff_params *dp, const basa_params *p) {
  for (const void *x : {q, k, v, dp->lambda})
    if (!x) return BASA_ERR_INVALID_ARG;
  for (const void *x : {q, k, v, kp, vp})
    if (!aligned16(x)) return BASA_ERR_INVALID_ARG;
  if (has_pool(p) != (kp != nullptr) || has_pool(p) != (vp != nullptr)) return BASA_ERR_INVALID_ARG;
  if ((p->routed_k > 0) != (route_idx != nullptr) || !aligned4(route_idx)) return BASA_ERR_INVALID_ARG;
  return BASA_OK;
}

basa_status check_rope_params(const basa_rope_params *rp, const basa_params *p) {
  if (!rp) return BASA_ERR_INVALID_ARG;
  for (int m : {rp->dt, rp->dh, rp->dw})
    if (m < 0 || m % 2 || m > p->head_dim) return BASA_ERR_INVALID_ARG;
  if (rp->dt + rp->dh + rp->dw > p->head_dim) return BASA_ERR_INVALID_ARG;
  if (rp->pairs != BASA_ROPE_PAIRS_ADJACENT && rp->pairs != BASA_ROPE_PAIRS_HALVES) return BASA_ERR_INVALID_ARG;
  if (!(rp->theta > 0.0)) return BASA_ERR_INVALID_ARG;
  for (double v : {rp->theta, rp->t0, rp->y0, rp->x0, rp->t_step, rp->y_step, rp->x_step})
    if (!std::isfinite(v)) return BASA_ERR_INVALID_ARG;
  return BASA_OK;
}

bool rope_empty(const basa_rope_tensor &t, const basa_params *p) {
  return p->B == 0 || t.heads == 0 || t.rows == 0;
}

// Strides of a [B, heads, rows, head_dim] view: >= 0 and whole 16-byte steps; a view
// that is written must not meet itself (sorted by stride, each axis steps past the
// extent of the ones before it).
bool rope_strides_ok(const int64_t *stride, const basa_rope_tensor &t, const basa_params *p, bool written) {
  const int64_t vec = p->dtype == BASA_BF16 ? 8 : 4, ext[3] = {p->B, t.heads, t.rows};
  int64_t order[3][2];
  int n = 0;
  for (int a = 0; a < 3; ++a) {
    if (ext[a] == 1) continue;  // never stepped
    if (stride[a] < 0 || stride[a] % vec || stride[a] > (int64_t(1) << 56) / ext[a]) return false;
    int at = n++;
    for (; at > 0 && order[at - 1][0] > stride[a]; --at) std::memcpy(order[at], order[at - 1], sizeof(order[at]));
    order[at][0] = stride[a];
    order[at][1] = ext[a];
  }
  int64_t span = p->head_dim;
  for (int i = 0; i < n && written; ++i) {
    if (order[i][0] < span) return false;
    span += order[i][0] * (order[i][1] - 1);
  }
  return true;
}

bool same_strides(const int64_t *a, const int64_t *b) { return a[0] == b[0] && a[1] == b[1] && a[2] == b[2]; }

using basa::ByteView;
using basa::views_meet;

ByteView rope_view(const void *base, const int64_t *stride, const basa_rope_tensor &t, const basa_params *p) {
  const int64_t size = p->dtype == BASA_BF16 ? 2 : 4, ext[3] = {p->B, t.heads, t.rows};
  ByteView v{reinterpret_cast<uintptr_t>(base), p->head_dim * size, {0, 0, 0}, {1, 1, 1}};
  for (int a = 0; a < 3; ++a) {
    if (ext[a] == 1) continue;
    v.step[a] = stride[a] * size;
    v.ext[a] = ext[a];
  }
  return v;
}

ByteView row_view(const void *base, const basa_params *p) {
  return {reinterpret_cast<uintptr_t>(base), int64_t(p->head_dim) * (p->dtype == BASA_BF16 ? 2 : 4), {0, 0, 0}, {1, 1, 1}};
}

// Nothing that a call writes is anything else that it reads or writes; a tensor may be
// rewritten in place, element by element. Written out over the views that there are, most of
// which are apart as a whole: a call of one token is bound by its checks.
bool rope_disjoint(int n, const basa_rope_tensor *t, bool bwd, const basa_params *p) {
  struct Used {
    ByteView v;
    uintptr_t end;
    int tensor;
    bool written;
    const int64_t *stride;
  } u[5 * BASA_ROPE_MAX_TENSORS];
  int m = 0;
  const auto use = [&](const ByteView &v, int i, bool written, const int64_t *stride) {
    u[m++] = {v, v.end(), i, written, stride};
  };
  for (int i = 0; i < n; ++i) {
    const basa_rope_tensor &r = t[i];
    if (bwd && r.dweight) use(row_view(r.dweight, p), i, true, nullptr);
    if (rope_empty(r, p)) continue;
    use(rope_view(r.y, r.y_stride, r, p), i, true, r.y_stride);
    if (!bwd || r.weight) use(rope_view(r.x, r.x_stride, r, p), i, false, r.x_stride);
    if (bwd) use(rope_view(r.dy, r.dy_stride, r, p), i, false, r.dy_stride);
    if (r.weight) use(row_view(r.weight, p), i, false, nullptr);
  }
  for (int a = 0; a < m; ++a)
    for (int b = 0; b < a; ++b) {
      if (u[a].v.base >= u[b].end || u[b].v.base >= u[a].end || !(u[a].written || u[b].written)) continue;
      const bool in_place = u[a].tensor == u[b].tensor && u[a].v.base == u[b].v.base && u[a].stride && u[b].stride &&
                            same_strides(u[a].stride, u[b].stride);
      if (!in_place && views_meet(u[a].v, u[b].v)) return false;
    }
  return true;
}

basa_status check_rope(int n, const basa_rope_tensor *t, const float *table, float eps, bool bwd,
                       const basa_rope_params *rp, const basa_params *p) {
  basa_status st = check_common(p);
  if (st != BASA_OK) return st;
  if ((st = check_rope_params(rp, p)) != BASA_OK) return st;
  if (n < 1 || n > BASA_ROPE_MAX_TENSORS || !t) return BASA_ERR_INVALID_ARG;
  const int64_t rows = int64_t(p->T) * p->H * p->W + p->n_text;
  const bool turns = rp->dt + rp->dh + rp->dw > 0;
  for (int i = 0; i < n; ++i) {
    const basa_rope_tensor &u = t[i];
    if (u.heads < 0 || u.rows < 0 || u.first_row < 0 || (u.rotate != 0 && u.rotate != 1)) return BASA_ERR_INVALID_ARG;
    if (int64_t(u.first_row) + u.rows > rows) return BASA_ERR_SHAPE;
    if (int64_t(p->B) * u.heads >= (int64_t(1) << 31)) return BASA_ERR_UNSUPPORTED;
    if (u.weight && (!aligned16(u.weight) || !(eps > 0.f) || !std::isfinite(eps))) return BASA_ERR_INVALID_ARG;
    if (bwd && u.dweight && (!u.weight || !aligned16(u.dweight))) return BASA_ERR_INVALID_ARG;
    if (rope_empty(u, p)) continue;
    const bool reads_x = !bwd || u.weight;
    if (!u.y || !aligned16(u.y) || !rope_strides_ok(u.y_stride, u, p, true)) return BASA_ERR_INVALID_ARG;
    if (reads_x && (!u.x || !aligned16(u.x) || !rope_strides_ok(u.x_stride, u, p, false))) return BASA_ERR_INVALID_ARG;
    if (bwd && (!u.dy || !aligned16(u.dy) || !rope_strides_ok(u.dy_stride, u, p, false))) return BASA_ERR_INVALID_ARG;
    if (u.rotate && turns && (!table || !aligned16(table))) return BASA_ERR_INVALID_ARG;
  }
  return rope_disjoint(n, t, bwd, p) ? BASA_OK : BASA_ERR_INVALID_ARG;
}

}  // namespace

extern "C" {

const char *basa_status_string(basa_status s) {
  switch (s) {
    case BASA_OK: return "BASA_OK";
    case BASA_ERR_INVALID_ARG: return "BASA_ERR_INVALID_ARG";
    case BASA_ERR_SHAPE: return "BASA_ERR_SHAPE";
    case BASA_ERR_UNSUPPORTED: return "BASA_ERR_UNSUPPORTED";
    case BASA_ERR_CUDA: return "BASA_ERR_CUDA";
    case BASA_ERR_DEVICE_TIMEOUT: return "BASA_ERR_DEVICE_TIMEOUT";
    case BASA_ERR_BAD_INDEX: return "BASA_ERR_BAD_INDEX";
  }
  return "BASA_ERR_UNKNOWN";
}

basa_status basa_device_error_status(int32_t w) {
  if (w == 0) return BASA_OK;
  return (w & BASA_DEVERR_BAD_ROUTE) ? BASA_ERR_BAD_INDEX : BASA_ERR_DEVICE_TIMEOUT;
}

basa_status basa_pool_kv(const void *k, const void *v, void *kp, void *vp, const basa_params *p,
                         basa_stream_t stream) {
  basa_status st = check_common(p);
  if (st != BASA_OK) return st;
  if (!has_pool(p)) return BASA_ERR_INVALID_ARG;
  if (empty_batch(p)) return BASA_OK;
  if (!k || !v || !kp || !vp) return BASA_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(kp) || !aligned16(vp)) return BASA_ERR_INVALID_ARG;
  return basa::launch_pool_kv(k, v, kp, vp, *p, reinterpret_cast<cudaStream_t>(stream));
}

size_t basa_route_workspace_bytes(const basa_params *p) {
  if (check_common(p) != BASA_OK) return 0;
  const size_t nwin = size_t(p->T / p->wt) * (p->H / p->wh) * (p->W / p->ww);
  return 2 * size_t(p->B) * p->heads * nwin * p->head_dim * sizeof(float);
}

basa_status basa_route_windows(const void *q, const void *k, int32_t *route_idx, float *route_score,
                               void *workspace, const basa_params *p, basa_stream_t stream) {
  basa_status st = check_common(p);
  if (st != BASA_OK) return st;
  if (p->routed_k < 1) return BASA_ERR_INVALID_ARG;
  const int64_t nwin = int64_t(p->T / p->wt) * (p->H / p->wh) * (p->W / p->ww);
  if (nwin > 4096) return BASA_ERR_UNSUPPORTED;
  if (empty_batch(p)) return BASA_OK;
  if (!q || !k || !route_idx || !workspace) return BASA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(workspace) || !aligned4(route_idx)) return BASA_ERR_INVALID_ARG;
  if (route_score && !aligned4(route_score)) return BASA_ERR_INVALID_ARG;
  return basa::launch_route(q, k, route_idx, route_score, workspace, *p, reinterpret_cast<cudaStream_t>(stream));
}

basa_status basa_route_windows_noalloc(const void *q, const void *k, int32_t *route_idx, float *route_score,
                                       const basa_params *p, basa_stream_t stream) {
  basa_status st = check_common(p);
  if (st != BASA_OK) return st;
  if (p->routed_k < 1) return BASA_ERR_INVALID_ARG;
  const int64_t nwin = int64_t(p->T / p->wt) * (p->H / p->wh) * (p->W / p->ww);
  if (nwin > 4096) return BASA_ERR_UNSUPPORTED;
  if (basa_route_workspace_bytes(p) > BASA_NOALLOC_SCRATCH_BYTES) return BASA_ERR_UNSUPPORTED;
  if (empty_batch(p)) return BASA_OK;
  if (!q || !k || !route_idx) return BASA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned4(route_idx)) return BASA_ERR_INVALID_ARG;
  if (route_score && !aligned4(route_score)) return BASA_ERR_INVALID_ARG;
  return basa::launch_route_noalloc(q, k, route_idx, route_score, *p, reinterpret_cast<cudaStream_t>(stream));
}

size_t basa_pool_route_workspace_bytes(const basa_params *p) {
  if (check_common(p) != BASA_OK || !has_pool(p) || p->routed_k < 1) return 0;
  basa::FusedPlan fp;
  if (basa::plan_fused(*p, &fp) != BASA_OK) return 0;
  return fp.means_bytes + fp.part_bytes;
}

basa_status basa_pool_route(const void *q, const void *k, const void *v, void *kp, void *vp, int32_t *route_idx,
                            float *route_score, void *workspace, const basa_params *p, basa_stream_t stream) {
  basa_status st = check_common(p);
  if (st != BASA_OK) return st;
  if (!has_pool(p) || p->routed_k < 1) return BASA_ERR_INVALID_ARG;
  const int64_t nwin = int64_t(p->T / p->wt) * (p->H / p->wh) * (p->W / p->ww);
  if (nwin > 4096) return BASA_ERR_UNSUPPORTED;
  basa::FusedPlan fp;
  st = basa::plan_fused(*p, &fp);
  if (st != BASA_OK) return st;
  if (empty_batch(p)) return BASA_OK;
  if (!q || !k || !v || !kp || !vp || !route_idx || !workspace) return BASA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(kp) || !aligned16(vp) || !aligned16(workspace) ||
      !aligned4(route_idx))
    return BASA_ERR_INVALID_ARG;
  if (route_score && !aligned4(route_score)) return BASA_ERR_INVALID_ARG;
  return basa::launch_pool_route_fused(q, k, v, kp, vp, route_idx, route_score, workspace, *p,
                                       reinterpret_cast<cudaStream_t>(stream));
}

static basa_status attn_common(const void *q, const void *k, const void *v, const void *kp, const void *vp,
                               const int32_t *route_idx, void *out, float *lse, uint32_t keys, const basa_params *p,
                               basa_stream_t stream) {
  basa_status st = check_common(p);
  if (st != BASA_OK) return st;
  if (p->dtype == BASA_BF16 && p->head_dim != 128) return BASA_ERR_UNSUPPORTED;
  if (keys & ~BASA_KEYS_ALL) return BASA_ERR_INVALID_ARG;
  // groups the layer does not have add no keys; the selection must leave some
  const bool any = (keys & BASA_KEYS_WINDOWS) || ((keys & BASA_KEYS_POOLED) && has_pool(p)) ||
                   ((keys & BASA_KEYS_TEXT) && p->n_text > 0);
  if (!any) return BASA_ERR_INVALID_ARG;
  if (empty_batch(p)) return BASA_OK;
  if (!q || !k || !v || !out) return BASA_ERR_INVALID_ARG;
  if (has_pool(p) != (kp != nullptr) || has_pool(p) != (vp != nullptr)) return BASA_ERR_INVALID_ARG;
  if ((p->routed_k > 0) != (route_idx != nullptr)) return BASA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return BASA_ERR_INVALID_ARG;
  if (kp && (!aligned16(kp) || !aligned16(vp))) return BASA_ERR_INVALID_ARG;
  if (route_idx && !aligned4(route_idx)) return BASA_ERR_INVALID_ARG;
  if (lse && !aligned4(lse)) return BASA_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (p->dtype == BASA_F32) return basa::launch_attn_f32(q, k, v, kp, vp, route_idx, out, lse, keys, *p, s);
  return basa::launch_attn_bf16(q, k, v, kp, vp, route_idx, out, lse, keys, *p, s);
}

basa_status basa_window_attn_fwd(const void *q, const void *k, const void *v, const void *kp, const void *vp,
                                 const int32_t *route_idx, void *out, const basa_params *p,
                                 basa_stream_t stream) {
  return attn_common(q, k, v, kp, vp, route_idx, out, nullptr, BASA_KEYS_ALL, p, stream);
}

basa_status basa_window_attn_fwd_lse(const void *q, const void *k, const void *v, const void *kp, const void *vp,
                                     const int32_t *route_idx, void *out, float *lse, uint32_t keys,
                                     const basa_params *p, basa_stream_t stream) {
  return attn_common(q, k, v, kp, vp, route_idx, out, lse, keys, p, stream);
}

size_t basa_text_attn_workspace_bytes(const basa_params *p) {
  if (check_common(p) != BASA_OK || p->n_text < 1 || p->dtype != BASA_BF16) return 0;
  return basa::text_attn_workspace(*p, basa::device_sm_count());
}

basa_status basa_text_attn_fwd(const void *q_text, const void *k, const void *v, void *out_text, void *workspace,
                               const basa_params *p, basa_stream_t stream) {
  basa_status st = check_common(p);
  if (st != BASA_OK) return st;
  if (p->n_text < 1) return BASA_ERR_INVALID_ARG;
  if (p->dtype == BASA_BF16 && p->head_dim != 128) return BASA_ERR_UNSUPPORTED;
  if (empty_batch(p)) return BASA_OK;
  if (!q_text || !k || !v || !out_text) return BASA_ERR_INVALID_ARG;
  if (!aligned16(q_text) || !aligned16(k) || !aligned16(v) || !aligned16(out_text)) return BASA_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (p->dtype == BASA_F32) return basa::launch_attn_text_f32(q_text, k, v, out_text, *p, s);
  const int sms = basa::device_sm_count();
  if (sms <= 0) return BASA_ERR_CUDA;
  if (basa::text_attn_workspace(*p, sms) > 0 && (!workspace || !aligned16(workspace))) return BASA_ERR_INVALID_ARG;
  return basa::launch_attn_text_bf16(q_text, k, v, out_text, workspace, *p, sms, s);
}

size_t basa_window_attn_bwd_workspace_bytes(const basa_params *p) {
  if (check_common(p) != BASA_OK || p->head_dim != 128) return 0;
  return p->dtype == BASA_BF16 ? basa::attn_bwd_bf16_workspace(*p) : basa::attn_bwd_workspace(*p);
}

basa_status basa_window_attn_bwd(const void *q, const void *k, const void *v, const void *kp, const void *vp,
                                 const int32_t *route_idx, const void *out, const float *lse, const void *dout,
                                 void *dq, void *dk, void *dv, void *workspace, const basa_params *p,
                                 basa_stream_t stream) {
  basa_status st = check_common(p);
  if (st != BASA_OK) return st;
  if (p->head_dim != 128) return BASA_ERR_UNSUPPORTED;
  if (too_many_windows(p)) return BASA_ERR_UNSUPPORTED;
  if (empty_batch(p)) return BASA_OK;
  if (!q || !k || !v || !out || !lse || !dout || !dq || !dk || !dv) return BASA_ERR_INVALID_ARG;
  if (has_pool(p) != (kp != nullptr) || has_pool(p) != (vp != nullptr)) return BASA_ERR_INVALID_ARG;
  if ((p->routed_k > 0) != (route_idx != nullptr)) return BASA_ERR_INVALID_ARG;
  for (const void *x : {q, k, v, out, dout, static_cast<const void *>(dq), static_cast<const void *>(dk),
                        static_cast<const void *>(dv)})
    if (!aligned16(x)) return BASA_ERR_INVALID_ARG;
  if (!aligned4(lse) || (route_idx && !aligned4(route_idx))) return BASA_ERR_INVALID_ARG;
  if (kp && (!aligned16(kp) || !aligned16(vp))) return BASA_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (p->dtype == BASA_BF16) {
    const size_t need = basa::attn_bwd_bf16_workspace(*p);
    if (need == 0) return BASA_ERR_UNSUPPORTED;  // the tiling plan does not fit the kernel's limits
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return BASA_ERR_INVALID_ARG;
    return basa::launch_attn_bwd_bf16(q, k, v, kp, vp, route_idx, out, lse, dout, dq, dk, dv, workspace, *p, s);
  }
  if (basa::attn_bwd_workspace(*p) > 0 && (!workspace || !aligned16(workspace))) return BASA_ERR_INVALID_ARG;
  return basa::launch_attn_bwd_f32(q, k, v, kp, vp, route_idx, out, lse, dout, dq, dk, dv, workspace, *p, s);
}

size_t basa_rope_table_bytes(const basa_rope_params *rp, const basa_params *p) {
  if (check_common(p) != BASA_OK || check_rope_params(rp, p) != BASA_OK) return 0;
  return basa::rope_table_bytes(*rp, *p);
}

basa_status basa_rope_table(const float *text_pos, float *table, const basa_rope_params *rp, const basa_params *p,
                            basa_stream_t stream) {
  basa_status st = check_common(p);
  if (st != BASA_OK) return st;
  if ((st = check_rope_params(rp, p)) != BASA_OK) return st;
  if (basa::rope_table_bytes(*rp, *p) == 0) return BASA_OK;
  if (!table || !aligned16(table) || !aligned4(text_pos)) return BASA_ERR_INVALID_ARG;
  return basa::launch_rope_table(text_pos, table, *rp, *p, reinterpret_cast<cudaStream_t>(stream));
}

basa_status basa_rope_fwd(int n, const basa_rope_tensor *t, const float *table, float eps, const basa_rope_params *rp,
                          const basa_params *p, basa_stream_t stream) {
  basa_status st = check_rope(n, t, table, eps, false, rp, p);
  if (st != BASA_OK) return st;
  return basa::launch_rope(n, t, table, eps, nullptr, false, *rp, *p, reinterpret_cast<cudaStream_t>(stream));
}

size_t basa_rope_bwd_workspace_bytes(int n, const basa_rope_tensor *t, const basa_params *p) {
  if (check_common(p) != BASA_OK || n < 1 || n > BASA_ROPE_MAX_TENSORS || !t) return 0;
  return basa::rope_bwd_workspace(n, t, *p);
}

basa_status basa_rope_bwd(int n, const basa_rope_tensor *t, const float *table, float eps, void *workspace,
                          const basa_rope_params *rp, const basa_params *p, basa_stream_t stream) {
  basa_status st = check_rope(n, t, table, eps, true, rp, p);
  if (st != BASA_OK) return st;
  if (basa::rope_bwd_workspace(n, t, *p) > 0 && (!workspace || !aligned16(workspace))) return BASA_ERR_INVALID_ARG;
  return basa::launch_rope(n, t, table, eps, workspace, true, *rp, *p, reinterpret_cast<cudaStream_t>(stream));
}

basa_status basa_diff_pool_kv(const void *k, const void *v, void *kp, void *vp, const basa_params *p,
                              basa_stream_t stream) {
  basa_status st = check_diff_shape(p);
  if (st != BASA_OK) return st;
  if (!has_pool(p)) return BASA_ERR_INVALID_ARG;
  if (empty_batch(p)) return BASA_OK;
  for (const void *x : {k, v, static_cast<const void *>(kp), static_cast<const void *>(vp)})
    if (!x || !aligned16(x)) return BASA_ERR_INVALID_ARG;
  const int units = p->B * p->heads;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if ((st = basa::launch_pool_rows(k, kp, 2 * units, *p, s)) != BASA_OK) return st;
  return basa::launch_pool_rows(v, vp, units, *p, s);
}

basa_status basa_diff_attn_fwd(const void *q, const void *k, const void *v, const void *kp, const void *vp,
                               const int32_t *route_idx, const basa_diff_params *dp, void *out, void *pre, void *second,
                               float *lse, const basa_params *p, basa_stream_t stream) {
  basa_status st = check_diff(dp, p);
  if (st != BASA_OK) return st;
  if (empty_batch(p)) return BASA_OK;
  if ((st = check_diff_inputs(q, k, v, kp, vp, route_idx, dp, p)) != BASA_OK) return st;
  if (!out || !aligned16(out) || !aligned16(pre) || !aligned16(second) || !aligned4(lse)) return BASA_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (p->dtype == BASA_BF16)
    return basa::launch_diff_attn_bf16(q, k, v, kp, vp, route_idx, *dp, out, pre, second, lse, *p, s);
  return basa::launch_diff_attn_f32(q, k, v, kp, vp, route_idx, *dp, out, pre, second, lse, false, *p, s);
}

size_t basa_diff_attn_bwd_workspace_bytes(const basa_diff_params *dp, const basa_params *p) {
  if (check_diff(dp, p) != BASA_OK || empty_batch(p)) return 0;
  return p->dtype == BASA_BF16 ? basa::diff_attn_bwd_bf16_workspace(dp->weight != nullptr, *p)
                               : basa::diff_attn_bwd_f32_workspace(dp->weight != nullptr, *p);
}

basa_status basa_diff_attn_bwd(const void *q, const void *k, const void *v, const void *kp, const void *vp,
                               const int32_t *route_idx, const basa_diff_params *dp, const void *pre, const void *second,
                               const float *lse, const void *dout, void *dq, void *dk, void *dv, void *dlambda,
                               void *dweight, void *workspace, const basa_params *p, basa_stream_t stream) {
  basa_status st = check_diff(dp, p);
  if (st != BASA_OK) return st;
  if (too_many_windows(p)) return BASA_ERR_UNSUPPORTED;
  if (empty_batch(p)) return p->heads > 0 || dp->weight ? BASA_ERR_INVALID_ARG : BASA_OK;
  if ((st = check_diff_inputs(q, k, v, kp, vp, route_idx, dp, p)) != BASA_OK) return st;
  for (const void *x : {pre, second, static_cast<const void *>(lse), dout, static_cast<const void *>(dq),
                        static_cast<const void *>(dk), static_cast<const void *>(dv)})
    if (!x) return BASA_ERR_INVALID_ARG;
  for (const void *x : {pre, second, dout, static_cast<const void *>(dq), static_cast<const void *>(dk),
                        static_cast<const void *>(dv), static_cast<const void *>(dweight)})
    if (!aligned16(x)) return BASA_ERR_INVALID_ARG;
  if (!dlambda || !aligned_element(dlambda, p) || !aligned4(lse)) return BASA_ERR_INVALID_ARG;
  if ((dweight != nullptr) != (dp->weight != nullptr)) return BASA_ERR_INVALID_ARG;
  const size_t need = basa_diff_attn_bwd_workspace_bytes(dp, p);
  if (need == 0) return BASA_ERR_UNSUPPORTED;  // the tiling plan does not fit the kernel's limits
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return BASA_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const auto launch = p->dtype == BASA_BF16 ? basa::launch_diff_attn_bwd_bf16 : basa::launch_diff_attn_bwd_f32;
  return launch(q, k, v, kp, vp, route_idx, *dp, pre, second, lse, dout, dq, dk, dv, dlambda, dweight, workspace, *p, s);
}

size_t basa_diff_text_attn_workspace_bytes(const basa_params *p) {
  if (check_diff_shape(p) != BASA_OK || p->n_text < 1 || empty_batch(p) || p->dtype != BASA_BF16) return 0;
  return basa::diff_text_workspace(*p, basa::device_sm_count());
}

basa_status basa_diff_text_attn_fwd(const void *q_text, const void *k, const void *v, const basa_diff_params *dp,
                                    void *out_text, void *workspace, const basa_params *p, basa_stream_t stream) {
  basa_status st = check_diff(dp, p);
  if (st != BASA_OK) return st;
  if (p->n_text < 1) return BASA_ERR_INVALID_ARG;
  if (empty_batch(p)) return BASA_OK;
  for (const void *x : {q_text, k, v, static_cast<const void *>(out_text)})
    if (!x || !aligned16(x)) return BASA_ERR_INVALID_ARG;
  if (!dp->lambda) return BASA_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (p->dtype == BASA_F32)
    return basa::launch_diff_attn_f32(q_text, k, v, nullptr, nullptr, nullptr, *dp, out_text, nullptr, nullptr, nullptr,
                                      true, *p, s);
  if (!workspace || !aligned16(workspace)) return BASA_ERR_INVALID_ARG;
  const int sms = basa::device_sm_count();
  if (sms <= 0) return BASA_ERR_CUDA;
  return basa::launch_diff_text_bf16(q_text, k, v, *dp, out_text, workspace, *p, sms, s);
}

basa_status basa_merge_branches(int n, const void *const *outs, const float *const *lses, void *out, float *lse,
                                const basa_params *p, basa_stream_t stream) {
  basa_status st = check_common(p);
  if (st != BASA_OK) return st;
  if (n < 1 || n > BASA_MAX_BRANCHES) return BASA_ERR_INVALID_ARG;
  if (empty_batch(p)) return BASA_OK;
  if (!outs || !lses || !out || !aligned16(out)) return BASA_ERR_INVALID_ARG;
  if (lse && !aligned4(lse)) return BASA_ERR_INVALID_ARG;
  for (int b = 0; b < n; ++b)
    if (!outs[b] || !lses[b] || !aligned16(outs[b]) || !aligned4(lses[b])) return BASA_ERR_INVALID_ARG;
  return basa::launch_merge(n, outs, lses, out, lse, *p, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
