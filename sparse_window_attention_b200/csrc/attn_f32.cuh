// Key lists of the float32 attention kernels (CUDA cores): a window's keys by index.
#pragma once

#include "basa_internal.h"

namespace basa {
namespace {

struct F32Args {
  const float *q, *k, *v, *kp, *vp;
  const int32_t *route;
  int32_t *dev_err;  // nullable: BASA_DEVERR_BAD_ROUTE on an out-of-range route id
  float *out;
  float *lse;  // nullable [B*heads][N]
  Geo g;
  int heads, d, n_text, n_pool, routed_k, win_tok, q_chunks;
  int n_vis_keys, n_pool_keys, n_text_keys;  // keys taken from each group (0 = group not selected)
  int dense;  // text-query rows: queries are q_text rows, keys are all N + n_text rows of k, v
  float scale;
};

// A route id outside [0, nWin) is reported (BASA_DEVERR_BAD_ROUTE) and replaced by
// the query's own window, so every access stays inside the tensors.
__device__ __forceinline__ int checked_route(const F32Args &a, int u, int w) {
  if (u >= 0 && u < a.g.nWin) return u;
  if (a.dev_err) atomicOr(a.dev_err, BASA_DEVERR_BAD_ROUTE);
  return w;
}

// Row of key j of window w's key list: [own | routed windows | pooled | text],
// restricted to the selected groups.
__device__ __forceinline__ const float *key_row(const F32Args &a, const float *kv, const float *kvp, long long bh,
                                                const int *wins, int j) {
  const int nvis = a.n_vis_keys;
  const long long rows = (long long)a.g.N + a.n_text;
  if (a.dense) return kv + (bh * rows + j) * a.d;
  if (j < nvis) {
    const int u = wins[j / a.win_tok];
    const int l = j % a.win_tok;
    int ot, oy, ox, type;
    window_origin(a.g, u, &ot, &oy, &ox, &type);
    const int lt = l / (a.g.wh * a.g.ww), ly = (l / a.g.ww) % a.g.wh, lx = l % a.g.ww;
    const int t = (ot + lt) % a.g.T, y = (oy + ly) % a.g.H, x = (ox + lx) % a.g.W;
    return kv + (bh * rows + ((long long)t * a.g.H + y) * a.g.W + x) * a.d;
  }
  j -= nvis;
  if (j < a.n_pool_keys) return kvp + (bh * a.n_pool + j) * a.d;
  j -= a.n_pool_keys;
  return kv + (bh * rows + a.g.N + j) * a.d;
}

}  // namespace
}  // namespace basa
