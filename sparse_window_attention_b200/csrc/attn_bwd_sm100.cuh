// Pieces shared by the tensor-core backward kernels (window attention, differential
// attention): the launch parameters, the key stream of a query tile, the query stream of a
// key tile, and the moves between TMEM, registers and tiles.
#pragma once

#include <cuda_bf16.h>

#include "attn_sm100_common.cuh"
#include "basa_internal.h"
#include "sm100_ptx.cuh"

namespace basa {
namespace sm100 {

enum Mode { kDq = 0, kDkvWindow = 1, kDkvLong = 2 };

constexpr uint32_t kRecBytes = kTileRows * 16;  // 128 records of 16 bytes
constexpr int kMaxList = 4096;                  // windows whose query tiles one key tile sees

struct alignas(64) BwdParams {
  CUtensorMap map_q[kMaxShapes], map_k[kMaxShapes], map_v[kMaxShapes], map_do[kMaxShapes];
  CUtensorMap map_rec[kMaxShapes];                 // per-token records {-L log2 e, -D, 0, 0}
  CUtensorMap map_dq[kMaxShapes], map_dk[kMaxShapes], map_dv[kMaxShapes];
  CUtensorMap map_kp, map_vp, map_kt, map_vt;      // pooled and text rows, 128-row boxes
  WindowPlan plan;
  const int32_t *route;
  int32_t *dev_err;
  const float4 *rec;  // the records, [bh][N] (dq pass: each thread reads its row's)
  const float *dkvp;  // final pooled-key gradients: dkp [bh][Np][128], then dvp
  float *part;        // long key tiles: [bh][tile][chunk][dK (of each map) | dV][128][128] partial sums
  const __nv_bfloat16 *lambda;  // differential form: [heads]
  __nv_bfloat16 *dq, *dk, *dv;  // differential form: the outputs, stored from registers
  float *dr;                    // differential form: [map][window][query tile][warp] sums of rec.z (sum dS)
  int *next_item;               // differential form: the dq pass's work counter
  int heads, n_items;
  Geo g;
  int bh_count;  // units of v, dout and the routes (differential form: q, k have two for each)
  int routed_k, n_pool, n_text, n_pool_tiles, n_text_tiles, n_long_tiles;
  int pt, ph, pw;
  float inv_patch;
  float scale_log2;  // log2(e) / sqrt(d)
  float scale;       // 1 / sqrt(d)
  uint32_t flags;    // basa_params.flags (test hook: skip the first ring load)
  int all_full;      // every tile of the streams is full: no column masks
  int max_tiles;     // most tiles of a window type
  int n_chunks, chunk_tiles, q_tiles;  // long mode: query tiles of a head, split in chunks
  unsigned long long timeout_ns;
};
static_assert(sizeof(BwdParams) <= 32764, "window plan too large for the kernel parameter space");

// The windows of a query tile's key stream: its own, then the routed ones.
struct RouteList {
  int wtype[1 + kMaxRouted];
  int org[1 + kMaxRouted][3];
};

// ------------------------------------------------------------- dq pass: the key stream
// Segments 0..routed_k are windows (own, then routed), then pooled, then text.
struct KeyIter {
  int seg, t;
};
__device__ __forceinline__ int seg_tiles(const BwdParams &P, const RouteList &c, int seg) {
  if (seg <= P.routed_k) return P.plan.type[c.wtype[seg]].n_tiles;
  return seg == P.routed_k + 1 ? P.n_pool_tiles : P.n_text_tiles;
}
__device__ __forceinline__ void key_first(const BwdParams &P, const RouteList &c, KeyIter &it) {
  it.seg = 0;
  it.t = 0;
  while (it.seg <= P.routed_k + 2 && seg_tiles(P, c, it.seg) == 0) ++it.seg;
}
__device__ __forceinline__ void key_next(const BwdParams &P, const RouteList &c, KeyIter &it) {
  ++it.t;
  while (it.seg <= P.routed_k + 2 && it.t >= seg_tiles(P, c, it.seg)) {
    ++it.seg;
    it.t = 0;
  }
}
__device__ __forceinline__ uint32_t load_key(const BwdParams &P, const RouteList &c, const KeyIter &it, bool is_v, int bh,
                                             uint8_t *dst, uint64_t *bar) {
  if (it.seg <= P.routed_k) {
    const PlanTile &tile = P.plan.tile[P.plan.type[c.wtype[it.seg]].first_tile + it.t];
    load_window_tile(P.plan, P.g, is_v ? P.map_v : P.map_k, tile, c.org[it.seg], bh, dst, bar);
    return uint32_t(tile.valid_rows) * 256u;
  }
  const bool pooled = it.seg == P.routed_k + 1;
  const CUtensorMap *map = pooled ? (is_v ? &P.map_vp : &P.map_kp) : (is_v ? &P.map_vt : &P.map_kt);
  const int row = pooled ? it.t * kTileRows : P.g.N + it.t * kTileRows;
  ptx::tma_load_3d(dst, map, bar, 0, row, bh);
  ptx::tma_load_3d(dst + kHalfBytes, map, bar, 64, row, bh);
  return kTileBytes;
}
__device__ __forceinline__ void key_mask(const BwdParams &P, const RouteList &c, const KeyIter &it, uint32_t *m) {
  if (it.seg <= P.routed_k) {
    const PlanTile &tile = P.plan.tile[P.plan.type[c.wtype[it.seg]].first_tile + it.t];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = tile.mask[i];
    return;
  }
  const bool pooled = it.seg == P.routed_k + 1;
  prefix_mask(min(kTileRows, (pooled ? P.n_pool : P.n_text) - it.t * kTileRows), m);
}

// ------------------------------------------------------------- dK/dV passes: the query stream
// Window list entry li (window mode: the smem list; long mode: window li itself) and
// tile t of it.
struct QIter {
  int li, t, ntiles, type, org[3];
};
__device__ __forceinline__ void q_load(const BwdParams &P, const int16_t *list, int mode, QIter &it) {
  const int w = mode == kDkvLong ? it.li : int(list[it.li]);
  window_origin(P.g, w, &it.org[0], &it.org[1], &it.org[2], &it.type);
  it.ntiles = P.plan.type[it.type].n_tiles;
}
// Positions the iterator at global query tile `skip` of the window sequence.
__device__ __forceinline__ void q_first(const BwdParams &P, const int16_t *list, int mode, int skip, QIter &it) {
  it.li = 0;
  it.t = 0;
  q_load(P, list, mode, it);
  while (skip >= it.ntiles) {
    skip -= it.ntiles;
    ++it.li;
    q_load(P, list, mode, it);
  }
  it.t = skip;
}
__device__ __forceinline__ void q_next(const BwdParams &P, const int16_t *list, int mode, int n_windows, QIter &it) {
  if (++it.t < it.ntiles) return;
  it.t = 0;
  if (++it.li < n_windows) q_load(P, list, mode, it);
}
__device__ __forceinline__ const PlanTile &q_tile(const BwdParams &P, const QIter &it) {
  return P.plan.tile[P.plan.type[it.type].first_tile + it.t];
}

// dq pass ring: key tile j in slot j % 3 (read by S(j) and, much later, dq(j)),
// value tile j in slot 3 + j % 2 (read by dP(j) only), so the next key tiles load
// while earlier ones still wait for their dq product, and value tile j + 1 loads
// while dP(j) is computed and read.
__device__ __forceinline__ int dq_slot(int j, bool is_v) { return is_v ? 3 + (j & 1) : j % 3; }
__device__ __forceinline__ uint32_t dq_phase(int j, bool is_v) { return is_v ? ((j >> 1) & 1) : ((j / 3) & 1); }

// Sets the columns whose mask bit is clear to 0 (m0: columns 0-31, m1: 32-63).
__device__ __forceinline__ void zero_masked(float (&x)[64], uint32_t m0, uint32_t m1) {
#pragma unroll
  for (int i = 0; i < 64; ++i)
    if (!(((i < 32 ? m0 : m1) >> (i & 31)) & 1u)) x[i] = 0.f;
}

// Packs 64 fp32 values (pairs 2i, 2i+1) into 32 bf16x2 words.
__device__ __forceinline__ void pack64(const float (&x)[64], uint32_t (&w)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) w[i] = ptx::pack_bf16x2(x[2 * i], x[2 * i + 1]);
}

// 64 consecutive TMEM columns of this thread's lane, as floats.
__device__ __forceinline__ void tmem_ld64f(uint32_t taddr, float (&x)[64]) {
  uint32_t r[64];
  ptx::tmem_ld64(taddr, r);
  ptx::tmem_ld_wait(r);
#pragma unroll
  for (int i = 0; i < 64; ++i) x[i] = __uint_as_float(r[i]);
}

// Writes 64 bf16 values (columns [64 half, 64 half + 64) of row `row`) into a
// swizzled 128-row staging tile.
__device__ __forceinline__ void stage_row_half(uint8_t *tile, int row, int half, const float (&x)[64]) {
  const uint32_t base = ptx::smem_u32(tile) + uint32_t(half) * kHalfBytes + uint32_t(row) * 128u;
  const uint32_t swz = row & 7;
#pragma unroll
  for (int c = 0; c < 8; ++c)
    ptx::st_shared_v4(base + ((uint32_t(c) ^ swz) << 4), ptx::pack_bf16x2(x[8 * c], x[8 * c + 1]),
                      ptx::pack_bf16x2(x[8 * c + 2], x[8 * c + 3]), ptx::pack_bf16x2(x[8 * c + 4], x[8 * c + 5]),
                      ptx::pack_bf16x2(x[8 * c + 6], x[8 * c + 7]));
}

// Reads 64 bf16 values (columns [64 half, 64 half + 64) of row `row`) from a swizzled
// 128-row tile as 32 bf16x2 words, the layout of an MMA A operand in TMEM.
__device__ __forceinline__ void load_row_half(const uint8_t *tile, int row, int half, uint32_t (&w)[32]) {
  const uint8_t *base = tile + uint32_t(half) * kHalfBytes + uint32_t(row) * 128u;
  const uint32_t swz = row & 7;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint4 v = *reinterpret_cast<const uint4 *>(base + ((uint32_t(c) ^ swz) << 4));
    w[4 * c] = v.x;
    w[4 * c + 1] = v.y;
    w[4 * c + 2] = v.z;
    w[4 * c + 3] = v.w;
  }
}

}  // namespace sm100

// Workspace of a backward over p.heads units of v with `maps` maps for each.
struct BwdLayout {
  size_t rec, part, dkvp, total;
  int n_long, n_chunks, chunk_tiles, q_tiles;
};
BwdLayout bwd_layout(const basa_params &p, const WindowPlan &plan, int maps);

// Parameters of a backward over p.heads units of v with `maps` maps each; the
// workspace starts with a BwdLayout (records, partial sums, pooled gradients).
basa_status bwd_params(sm100::BwdParams &P, BwdLayout &L, const void *q, const void *k, const void *v, const void *kp,
                       const void *vp, const int32_t *route_idx, const void *dout, void *dq, void *dk, void *dv,
                       void *workspace, const basa_params &p, int maps);

// Sums of the pooled and text key tiles' chunks.
basa_status launch_bwd_reduce(const sm100::BwdParams &P, const BwdLayout &L, void *dk, void *dv, const basa_params &p,
                              int maps, cudaStream_t s);

}  // namespace basa
