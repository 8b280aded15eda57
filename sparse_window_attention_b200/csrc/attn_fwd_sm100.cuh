// Pieces shared by the tensor-core forward kernels (window attention and its text rows,
// differential attention): the launch parameters, the key-tile stream of a query window,
// and the softmax of a row.
#pragma once

#include <cuda_bf16.h>

#include "attn_sm100_common.cuh"
#include "basa_internal.h"
#include "sm100_ptx.cuh"

namespace basa {
namespace sm100 {

struct alignas(64) AttnParams {
  CUtensorMap map_q[kMaxShapes];
  CUtensorMap map_k[kMaxShapes];
  CUtensorMap map_v[kMaxShapes];
  CUtensorMap map_o[kMaxShapes];
  CUtensorMap map_kp, map_vp, map_kt, map_vt;
  CUtensorMap map_kp8, map_vp8;  // pooled rows in 8-row boxes (the pooled tail, see below)
  CUtensorMap map_qd, map_od;  // text-query mode: query rows and output rows (d, row, b*head)
  WindowPlan plan;
  const int32_t *route;
  int32_t *dev_err;
  Geo g;
  int routed_k, n_pool, n_text, n_pool_tiles, n_text_tiles;
  // Pooled tail: when the pooled keys past the last full 128-row tile (pool_tail rows,
  // at most 16) fit in free 8-row blocks of the own window's key tile tail_tile[type],
  // they are loaded there (8-row boxes at rows tail_dest[type][b]) instead of taking a
  // key tile of their own; tail_mask[type] marks their rows.
  int pool_tail, tail_blocks;
  int8_t tail_tile[8];
  uint8_t tail_dest[8][2];
  uint32_t tail_mask[8][4];
  float scale_log2;
  int use_windows;  // own and routed windows are keys (else pooled and/or text only)
  // Text-query mode: the queries are the n_text text rows and attend densely to
  // every k/v row, which are streamed as the "text" segment starting at row 0.
  // The key tiles are split into n_splits ranges, one per CTA group.
  int dense, dense_rows, dense_q_tiles, dense_pairs, n_splits, split_tiles, bh_count;
  int text_row0;  // first k/v row of the text segment: N (window mode) or 0
  float *lse;       // nullable: log-sum-exp of each query row's scaled scores [B*heads][N]
  int all_full;  // every key tile of the launch is full: no column masks
  uint32_t flags;
  unsigned long long timeout_ns;
  // differential form: a CTA's unit is a (batch, differential head); map g's q, k, kp are unit 2 * unit + g
  const __nv_bfloat16 *lambda, *norm_weight;  // [heads]; nullable [128]
  __nv_bfloat16 *out, *pre, *second;          // [B*heads][N][128]; pre and second nullable
  int heads, q_tiles, n_items;                // query tiles of a window (at most); work items
  float gain, eps;
  float *part;  // text rows that leave in float32: outputs [split][b*head][n_text][128]
};

// __grid_constant__ kernel parameters are limited to 32764 bytes.
static_assert(sizeof(AttnParams) <= 32764, "window plan too large for the kernel parameter space");

// What a query window's key stream is made of.
struct KeyList {
  int tile0, ntile;  // text-query mode: the range of key tiles
  int wtype[1 + kMaxRouted];
  int org[1 + kMaxRouted][3];
};

// The windows routed to window w (unit `bh` of the routes).
__device__ __forceinline__ void fill_routes(const AttnParams &P, KeyList &c, int bh, int w) {
  for (int r = 0; r < P.routed_k; ++r) {
    int u = P.route[((long long)bh * P.g.nWin + w) * P.routed_k + r];
    if (u < 0 || u >= P.g.nWin) {  // reported, and replaced by the own window: accesses stay in bounds
      if (P.dev_err) atomicOr(P.dev_err, BASA_DEVERR_BAD_ROUTE);
      u = w;
    }
    int a, b, d, t;
    window_origin(P.g, u, &a, &b, &d, &t);
    c.wtype[1 + r] = t;
    c.org[1 + r][0] = a; c.org[1 + r][1] = b; c.org[1 + r][2] = d;
  }
}

// Position in the key-tile stream: segments 0..routed_k are windows (own, then
// routed), then the pooled tokens, then the text tokens.
struct KeyIter {
  int seg, t;
};

__device__ __forceinline__ int seg_tiles(const AttnParams &P, const KeyList &c, int seg) {
  if (seg <= P.routed_k) return P.use_windows ? P.plan.type[c.wtype[seg]].n_tiles : 0;
  if (seg == P.routed_k + 1) return P.n_pool_tiles;
  return P.dense ? c.ntile : P.n_text_tiles;
}
__device__ __forceinline__ void advance(const AttnParams &P, const KeyList &c, KeyIter &it) {
  ++it.t;
  while (it.seg <= P.routed_k + 2 && it.t >= seg_tiles(P, c, it.seg)) {
    ++it.seg;
    it.t = 0;
  }
}

// First key tile of the stream (segments without tiles are skipped).
__device__ __forceinline__ KeyIter first_key(const AttnParams &P, const KeyList &c) {
  KeyIter it{0, 0};
  while (it.seg <= P.routed_k + 2 && seg_tiles(P, c, it.seg) == 0) ++it.seg;
  return it;
}

// The own window's key tile that also carries the pooled tail.
__device__ __forceinline__ bool has_pool_tail(const AttnParams &P, const KeyList &c, const KeyIter &it) {
  return P.pool_tail > 0 && it.seg == 0 && it.t == P.tail_tile[c.wtype[0]];
}

// Bytes the TMA loads of one key (or value) tile deliver.
__device__ __forceinline__ uint32_t key_tile_bytes(const AttnParams &P, const KeyList &c, const KeyIter &it) {
  if (it.seg > P.routed_k) return kTileBytes;  // whole 128-row boxes (rows past the end read as zero)
  uint32_t b = uint32_t(P.plan.tile[P.plan.type[c.wtype[it.seg]].first_tile + it.t].valid_rows) * 256u;
  if (has_pool_tail(P, c, it)) b += uint32_t(P.tail_blocks) * 8u * 256u;
  return b;
}

__device__ __forceinline__ uint32_t load_key_tile(const AttnParams &P, const KeyList &c, const KeyIter &it, bool is_v,
                                                  int bh, uint8_t *dst, uint64_t *bar) {
  if (it.seg <= P.routed_k) {
    const PlanTile &tile = P.plan.tile[P.plan.type[c.wtype[it.seg]].first_tile + it.t];
    uint32_t b = load_window_tile(P.plan, P.g, is_v ? P.map_v : P.map_k, tile, c.org[it.seg], bh, dst, bar);
    if (has_pool_tail(P, c, it)) {
      const CUtensorMap *map = is_v ? &P.map_vp8 : &P.map_kp8;
      for (int i = 0; i < P.tail_blocks; ++i) {
        uint8_t *d = dst + uint32_t(P.tail_dest[c.wtype[0]][i]) * 128u;
        const int row = P.n_pool_tiles * kTileRows + 8 * i;  // rows past n_pool read as zero
        ptx::tma_load_3d(d, map, bar, 0, row, bh);
        ptx::tma_load_3d(d + kHalfBytes, map, bar, 64, row, bh);
        b += 8u * 256u;
      }
    }
    return b;
  }
  const bool pooled = it.seg == P.routed_k + 1;
  const CUtensorMap *map = pooled ? (is_v ? &P.map_vp : &P.map_kp) : (is_v ? &P.map_vt : &P.map_kt);
  const int row = pooled ? it.t * kTileRows : P.text_row0 + (c.tile0 + it.t) * kTileRows;
  ptx::tma_load_3d(dst, map, bar, 0, row, bh);
  ptx::tma_load_3d(dst + kHalfBytes, map, bar, 64, row, bh);
  return kTileBytes;
}

// Column mask of a key tile; returns true when all 128 rows hold keys.
__device__ __forceinline__ bool key_tile_mask(const AttnParams &P, const KeyList &c, const KeyIter &it, uint32_t *m) {
  if (it.seg <= P.routed_k) {
    const PlanTile &tile = P.plan.tile[P.plan.type[c.wtype[it.seg]].first_tile + it.t];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = tile.mask[i];
    if (has_pool_tail(P, c, it)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) m[i] |= P.tail_mask[c.wtype[0]][i];
      return false;
    }
    return tile.valid_rows == kTileRows;
  }
  const bool pooled = it.seg == P.routed_k + 1;
  const int total = pooled ? P.n_pool : (P.dense ? P.dense_rows : P.n_text);
  const int valid = min(kTileRows, total - (pooled ? it.t : c.tile0 + it.t) * kTileRows);
  prefix_mask(valid, m);
  return valid == kTileRows;
}

// The running row max is only raised when a tile's max exceeds it by more than
// 2^8 (log2 units); otherwise the old max is kept and P values up to 256 are
// produced, which float32 sums and bfloat16 P hold exactly as well. This skips
// most rescales of the O accumulator in TMEM.
constexpr float kRescaleLog2 = 8.0f;
// P = 2^x (x = s * scale_log2 - m) for the 128 scores of a row (MUFU ex2), written
// in place as the 64 bfloat16 pairs the P V MMA reads (s[i] = pair (2i, 2i+1), low
// half = even key); each pair is packed as soon as it is computed, so the live
// register set shrinks along the row. Returns the float32 row sum.
__device__ __forceinline__ float exp2_row_packed(uint32_t (&s)[128], float scale_log2, float m) {
  using namespace ptx;
  const uint64_t sc2 = f2_pack(scale_log2, scale_log2), negm2 = f2_pack(-m, -m);
  uint64_t acc0 = f2_pack(0.f, 0.f), acc1 = acc0;
#pragma unroll
  for (int pr = 0; pr < 64; ++pr) {
    const uint64_t x = ffma2(f2_pack(__uint_as_float(s[2 * pr]), __uint_as_float(s[2 * pr + 1])), sc2, negm2);
    float x0, x1;
    f2_unpack(x, x0, x1);
    const float r0 = ex2(x0), r1 = ex2(x1);
    const uint64_t pp = f2_pack(r0, r1);
    if (pr & 1) acc1 = fadd2(acc1, pp);
    else acc0 = fadd2(acc0, pp);
    s[pr] = pack_bf16x2(r0, r1);  // s[pr] was read at pair pr / 2
  }
  float a, b, c, d;
  f2_unpack(acc0, a, b);
  f2_unpack(acc1, c, d);
  return (a + b) + (c + d);
}

// Row max of the N entries of s (raw scores).
template <int N>
__device__ __forceinline__ float row_max(const uint32_t (&s)[N]) {
  float a = __uint_as_float(s[0]), b = __uint_as_float(s[1]), c = __uint_as_float(s[2]), d = __uint_as_float(s[3]);
#pragma unroll
  for (int i = 4; i < N; i += 8) {
    a = ptx::fmax3(a, __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
    b = ptx::fmax3(b, __uint_as_float(s[i + 2]), __uint_as_float(s[i + 3]));
    c = ptx::fmax3(c, __uint_as_float(s[i + 4]), __uint_as_float(s[i + 5]));
    d = ptx::fmax3(d, __uint_as_float(s[i + 6]), __uint_as_float(s[i + 7]));
  }
  return fmaxf(fmaxf(a, b), fmaxf(c, d));
}

// Sets every column whose mask bit is clear to -inf.
template <int N>
__device__ __forceinline__ void apply_mask(uint32_t (&s)[N], const uint32_t *mask) {
#pragma unroll
  for (int wd = 0; wd < N / 32; ++wd) {
    const uint32_t mw = mask[wd];
    if (mw != 0xFFFFFFFFu) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (!((mw >> i) & 1u)) s[32 * wd + i] = __float_as_uint(-INFINITY);
    }
  }
}

}  // namespace sm100

// Parameters of a window-mode launch. `maps` softmax maps share a head's values: q, k, kp
// have maps * heads heads, v, vp and out have heads. `out` may be null: no map of it.
basa_status window_params(sm100::AttnParams &P, const void *q, const void *k, const void *v, const void *kp,
                          const void *vp, const int32_t *route_idx, void *out, float *lse, uint32_t keys,
                          const basa_params &p, int maps);

}  // namespace basa
