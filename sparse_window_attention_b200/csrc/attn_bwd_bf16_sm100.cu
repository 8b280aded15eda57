// Backward of the shifted-window attention, bfloat16, head_dim 128, for sm_100a.
//
// Gradients of out = softmax(q K^T / sqrt(d)) V over each query's key list
// [own window | routed windows | pooled | text] (BASA §3.1-§3.3, §A.1), for the
// training step of the dense-teacher adaptation (BASA §3.4). With the forward's
// log-sum-exp L and D_i = dout_i . out_i:
//   P = exp(q K^T / sqrt(d) - L),  dS = P (dout V^T - D),
//   dq = dS K / sqrt(d),  dK = dS^T q / sqrt(d),  dV = P^T dout,
// and the key rows of dK, dV go back to the tokens they came from (pooled keys
// spread evenly over their patch: kp, vp are means).
//
// Every sum has a fixed order and nothing is accumulated with atomics, so the
// results are identical run to run. Launches, in order:
//   records      per query token {-L log2(e), -D} (16-byte records, TMA-loadable with
//                the same boxes as the query tiles; negated for the packed FMA/add)
//   dq pass      one CTA per (b*head, window, query tile): the key stream of the
//                forward; q and dout copied once into TMEM, so S = q K^T and
//                dP = dout V^T read their A operand from TMEM; dS by the compute
//                warps (written over dP), dq += dS K accumulated in TMEM.
//   dK/dV long   (pooled and text key tiles, which every query of the head sees)
//                one CTA per (b*head, key tile, chunk of the head's query tiles):
//                S^T = K q^T, dP^T = V dout^T, dV += P^T dout, dK += dS^T q in TMEM;
//                fp32 partial sums per chunk.
//   reduce       chunks summed in order: pooled-key gradients (float32, for the
//                spread) and the text rows of dk, dv.
//   dK/dV window one CTA per (b*head, window u, key tile of u): the query tiles of
//                u and of every window that routed to u (ascending window id; as often
//                as its key list holds u), same MMAs; the epilogue adds the pooled-key
//                gradient of each token's patch / |patch| and stores dk, dv at the
//                tokens' positions.
//
// Differential form (template argument DIFF; out = O1 - lambda O2 of two maps that share
// their values, the norm's gradient g taken beforehand and D per map in the records): the
// dq pass runs over the maps, with map 2's sums scaled by -lambda in its epilogue, and adds
// up each row's dS (what its D was off by), which lambda's gradient takes in. The
// dK/dV passes run both maps of a (batch, head) in ONE CTA, map 2 first: its dK leaves,
// the dV accumulator is multiplied by -lambda in TMEM, and map 1 adds to it, so the two
// maps' dV meet without a buffer or an atomic. (Both maps at once, sharing dout V^T, would
// take six 128-column accumulators and TMEM holds four.) The passes overlap at their ends by
// programmatic dependent launch: the long pass runs first, on fewer CTAs than there are SMs
// as often as not, and the dq pass, which needs nothing of it, fills the rest. The chunks of a
// long key tile are summed (in their order) by the last CTA of it to finish, so that the window
// pass starts as the dq pass drains and waits for both before its epilogue, with lambda's and
// the weight's sums under its end; or, where too little runs beside that CTA to hide it, by a
// reduction of its own, under which the window pass starts (last_cta_sums).
//
// Roundings, as in the other form: P and dS to bfloat16 for the products that sum them (2^-8
// of each element at most), so dq, dk and dv are off 0.003 of their size where their own
// rounding is 0.0017. Measured, forward and backward, a replayed graph: 12 heads, 64 x 64, 16 x 16 windows, 832
// keys 336 us (18 products of 2 d FLOP a query and key where 12 would do, as the scores and
// dout V^T are taken again in the dK/dV passes, the latter per map); 2 x 3 heads,
// 6 x 18 x 26, 234-token windows, 2 routed 203 us. What bounds them: in the dq and long passes
// the chain score, P, dS of each tile (tensor cores active 30% of the time), in the window pass
// a CTA's start and end around its few query tiles (15%).
//
// Warp roles (320 threads): warp 0 TMA loads, warp 1 issues tcgen05 MMAs (one
// thread), warps 2-9 compute P and dS: two warpgroups, each owning 64 of the 128
// columns of a row (the backward has no row reductions, so the columns split
// freely), a thread per (row, column half). Every wait is bounded (globaltimer):
// on expiry a bit goes to dev_err and the kernel drains and returns.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "attn_sm100_common.cuh"
#include "basa_internal.h"
#include "sm100_ptx.cuh"

namespace basa {
namespace {

using namespace sm100;

enum Mode { kDq = 0, kDkvWindow = 1, kDkvLong = 2 };

constexpr int kThreads = 320;
constexpr int kMaxSlots = 5;
constexpr uint32_t kSmemRow = 0;                            // the two row tiles
constexpr uint32_t kSmemRing = 2 * kTileBytes;              // then a ring of 32 KB tiles
constexpr uint32_t kRecBytes = kTileRows * 16;              // 128 records of 16 bytes
constexpr uint32_t kCtrlBytes = 1024;
constexpr int kMaxList = kMaxBwdRouted;                     // windows whose query tiles one key tile sees (with routing)
constexpr int kIdBits = 27;                                 // of a list entry
static_assert(kMaxBwdWindows == 1 << kIdBits, "window ids in a list entry");
constexpr uint32_t kTmemCols = 512;

constexpr uint32_t kColRecBytes = 8 * 128 * 4;             // per compute warp: 64 x {-L log2 e}, 64 x {-D}

// Shared memory of each pass. dq: row tiles q, dout; five ring slots (three key
// tiles, two value tiles); each thread reads its own row's record from global
// memory. dK/dV: row tiles k, v; four slots (query and dout tiles in turn); two
// record buffers for the streamed query tiles, and per compute warp its 64
// columns' records as two arrays; the window pass adds the list of windows that
// see its key tile.
template <int MODE>
struct Smem {
  static constexpr int slots = MODE == kDq ? 5 : 4;
  static constexpr uint32_t rec = kSmemRing + slots * kTileBytes;
  static constexpr uint32_t col_rec = rec + (MODE == kDq ? 0u : 2 * kRecBytes);
  static constexpr uint32_t ctrl = col_rec + (MODE == kDq ? 0u : kColRecBytes);
  static constexpr uint32_t list = ctrl + kCtrlBytes;
  static constexpr uint32_t place = list + (MODE == kDkvWindow ? kMaxList * 4 : 0);  // differential form
  static constexpr uint32_t bytes = place + (MODE == kDkvWindow ? 256 * 8 : 0) + 1024;  // + alignment slack
  static_assert(bytes <= 227u * 1024u, "shared memory of a pass above the 227 KB a CTA may hold");
};

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
  __nv_bfloat16 *dk;            // differential form: dk itself, for map 2's rows
  float *dr;                    // differential form: [map][window][query tile] sums of rec.z (sum dS)
  int *long_done;               // differential form, nullable: [unit of v][long tile] chunks that are finished
  __nv_bfloat16 *dv;            // (with long_done) for the text rows
  int heads;
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

struct Ctrl {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  // dq pass: a_ready, s_full[0], s_free, dp_full[0], ds_full[0]; dK/dV passes: s_full[0],
  // s_free, dp_full[0], and per compute group ds_full[g]
  uint64_t row_full, row_free, s_full[2], dp_full[2], s_free, a_ready, ds_full[2], acc_full, drain;
  uint32_t tmem_base;
  int abort;
  int n_cols;   // column tiles streamed by this CTA
  int n_list;   // dK/dV window mode: windows in the list
  int wtype[1 + kMaxRouted];
  int org[1 + kMaxRouted][3];
};
static_assert(sizeof(Ctrl) <= kCtrlBytes, "control block too large");

// ------------------------------------------------------------- dq pass: the key stream
// Segments 0..routed_k are windows (own, then routed), then pooled, then text.
struct KeyIter {
  int seg, t;
};
__device__ __forceinline__ int seg_tiles(const BwdParams &P, const Ctrl &c, int seg) {
  if (seg <= P.routed_k) return P.plan.type[c.wtype[seg]].n_tiles;
  return seg == P.routed_k + 1 ? P.n_pool_tiles : P.n_text_tiles;
}
__device__ __forceinline__ void key_first(const BwdParams &P, const Ctrl &c, KeyIter &it) {
  it.seg = 0;
  it.t = 0;
  while (it.seg <= P.routed_k + 2 && seg_tiles(P, c, it.seg) == 0) ++it.seg;
}
__device__ __forceinline__ void key_next(const BwdParams &P, const Ctrl &c, KeyIter &it) {
  ++it.t;
  while (it.seg <= P.routed_k + 2 && it.t >= seg_tiles(P, c, it.seg)) {
    ++it.seg;
    it.t = 0;
  }
}
__device__ __forceinline__ uint32_t load_key(const BwdParams &P, const Ctrl &c, const KeyIter &it, bool is_v, int bh,
                                             uint8_t *dst, uint64_t *bar) {  // bh: unit of the tensor read
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
__device__ __forceinline__ void key_mask(const BwdParams &P, const Ctrl &c, const KeyIter &it, uint32_t *m) {
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
// tile t of it. An entry is a window's id and, above it, how many times more than once its
// key list holds the key tile's window (a route may be repeated, and name its own window):
// its tiles are streamed as often.
struct QIter {
  int li, t, ntiles, type, org[3], more;
};
static_assert(kMaxRouted < 1 << (32 - kIdBits), "a window may list itself kMaxRouted times more");
__device__ __forceinline__ int entry_window(uint32_t e) { return int(e & ((1u << kIdBits) - 1u)); }
__device__ __forceinline__ int entry_more(uint32_t e) { return int(e >> kIdBits); }
__device__ __forceinline__ void q_load(const BwdParams &P, const uint32_t *list, int mode, QIter &it) {
  int w = it.li;
  if (mode == kDkvWindow) {
    const uint32_t e = list[it.li];
    it.more = entry_more(e);
    w = entry_window(e);
  }
  window_origin(P.g, w, &it.org[0], &it.org[1], &it.org[2], &it.type);
  it.ntiles = P.plan.type[it.type].n_tiles;
}
// Positions the iterator at global query tile `skip` of the window sequence.
__device__ __forceinline__ void q_first(const BwdParams &P, const uint32_t *list, int mode, int skip, QIter &it) {
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
__device__ __forceinline__ void q_next(const BwdParams &P, const uint32_t *list, int mode, int n_windows, QIter &it) {
  if (++it.t < it.ntiles) return;
  it.t = 0;
  if (mode == kDkvWindow && --it.more >= 0) return;
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

// Stores the sum of four columns of a long key row's gradient: dK of map `which` of unit bh, or
// (which == maps) dV. Pooled rows to dkvp (float32), text rows to dk, dv.
__device__ __forceinline__ void store_long_sum(const float4 &s, float *dkvp, __nv_bfloat16 *dk, __nv_bfloat16 *dv, int which,
                                               int maps, int bh, int bh_count, bool pooled, int r, int c4, int n_pool,
                                               int n_text, long long N) {
  const bool is_v = which == maps;
  const long long unit = is_v ? bh : (long long)maps * bh + which;
  if (pooled) {
    const long long at = (is_v ? (long long)maps * bh_count : 0) + unit;
    *reinterpret_cast<float4 *>(dkvp + (at * n_pool + r) * 128 + c4 * 4) = s;
  } else {
    const long long o = (unit * (N + n_text) + N + r) * 128 + c4 * 4;
    reinterpret_cast<uint2 *>((is_v ? dv : dk) + o)[0] = make_uint2(ptx::pack_bf16x2(s.x, s.y), ptx::pack_bf16x2(s.z, s.w));
  }
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

template <int MODE, bool DIFF>
__global__ void __launch_bounds__(kThreads, 1) attn_bwd_bf16_kernel(const __grid_constant__ BwdParams P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  using L = Smem<MODE>;
  constexpr int kSlots = L::slots;
  Ctrl &c = *reinterpret_cast<Ctrl *>(smem + L::ctrl);
  uint32_t *list = reinterpret_cast<uint32_t *>(smem + L::list);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (DIFF && MODE != kDkvWindow) ptx::grid_launch_dependents();
  // What follows the dq pass needs the long pass's sums: one CTA of it ends after them.
  const bool last_to_end = DIFF && MODE == kDq && blockIdx.x == gridDim.x - 1 && threadIdx.x == 0;

  // ----------------------------------------------------------- unit of this CTA
  int bh, w = 0, tile_idx = 0, kt = 0, chunk = 0, ot = 0, oy = 0, ox = 0, wtype = 0;
  if (MODE == kDkvLong) {
    chunk = blockIdx.x % P.n_chunks;
    kt = (blockIdx.x / P.n_chunks) % P.n_long_tiles;
    bh = blockIdx.x / (P.n_chunks * P.n_long_tiles);
  } else {
    tile_idx = blockIdx.x % P.max_tiles;
    w = (blockIdx.x / P.max_tiles) % P.g.nWin;
    bh = blockIdx.x / (P.max_tiles * P.g.nWin);
    window_origin(P.g, w, &ot, &oy, &ox, &wtype);
    if (tile_idx >= P.plan.type[wtype].n_tiles) {  // whole CTA: this window type has fewer tiles
      if (DIFF && MODE == kDq && threadIdx.x == 0) P.dr[blockIdx.x] = 0.f;
      if (last_to_end) ptx::grid_wait();
      return;
    }
  }
  // Units: bh counts maps in the dq pass and values (two maps each) in the dK/dV passes.
  const int bh_v = DIFF && MODE == kDq ? bh >> 1 : bh;       // unit of v, dout and the routes
  constexpr int kMaps = DIFF && MODE != kDq ? 2 : 1;         // maps this CTA goes through
  auto map_unit = [&](int m) { return kMaps == 2 ? 2 * bh + 1 - m : bh; };  // unit of q, k of its m-th map
  const float neg_lambda = DIFF ? -__bfloat162float(P.lambda[bh_v % P.heads]) : 1.f;
  const int row_org[3] = {ot, oy, ox};
  const PlanTile &row_tile = P.plan.tile[P.plan.type[wtype].first_tile + tile_idx];  // window modes

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      ptx::mbar_init(&c.full[i], 1);
      ptx::mbar_init(&c.empty[i], 1);
    }
    ptx::mbar_init(&c.row_full, 1);
    ptx::mbar_init(&c.row_free, 1);
    const uint32_t per_group = MODE == kDq ? 256 : 128;  // compute threads that arrive
    for (int g = 0; g < 2; ++g) {
      ptx::mbar_init(&c.s_full[g], 1);
      ptx::mbar_init(&c.dp_full[g], 1);
      ptx::mbar_init(&c.ds_full[g], per_group);
    }
    ptx::mbar_init(&c.s_free, 256);
    ptx::mbar_init(&c.a_ready, 256);
    ptx::mbar_init(&c.acc_full, 1);
    ptx::mbar_init(&c.drain, 1);
    c.abort = 0;
    if (MODE == kDq) {
      c.wtype[0] = wtype;
      c.org[0][0] = ot; c.org[0][1] = oy; c.org[0][2] = ox;
      for (int r = 0; r < P.routed_k; ++r) {
        int u = P.route[((long long)bh_v * P.g.nWin + w) * P.routed_k + r];
        if (u < 0 || u >= P.g.nWin) {  // reported, and replaced by the own window: accesses stay in bounds
          if (P.dev_err) atomicOr(P.dev_err, BASA_DEVERR_BAD_ROUTE);
          u = w;
        }
        int a, b, d, t;
        window_origin(P.g, u, &a, &b, &d, &t);
        c.wtype[1 + r] = t;
        c.org[1 + r][0] = a; c.org[1 + r][1] = b; c.org[1 + r][2] = d;
      }
      int n = 0;
      for (int s = 0; s <= P.routed_k + 2; ++s) n += seg_tiles(P, c, s);
      c.n_cols = n;
    } else if (MODE == kDkvLong) {
      c.n_cols = max(0, min(P.chunk_tiles, P.q_tiles - chunk * P.chunk_tiles));
    }
    ptx::fence_mbar_init();
  }
  if (MODE == kDkvWindow && warp == 0) {
    // The query windows that see key tile (w, tile_idx): w itself, then every window
    // that routed to w, in ascending id (ordered ballot compaction: a fixed order). A
    // route out of range stands for its window itself, as in the forward.
    int n = 1;
    if (lane == 0 && P.routed_k == 0) list[0] = uint32_t(w);
    for (int w0 = 0; P.routed_k > 0 && w0 < P.g.nWin; w0 += 32) {
      const int x = w0 + lane;
      int hits = 0;
      if (x < P.g.nWin) {
        const int32_t *r = P.route + ((long long)bh * P.g.nWin + x) * P.routed_k;
        for (int i = 0; i < P.routed_k; ++i) hits += r[i] == w || (x == w && uint32_t(r[i]) >= uint32_t(P.g.nWin));
        if (x == w) {
          list[0] = uint32_t(w) | uint32_t(hits) << kIdBits;
          hits = 0;
        }
      }
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, hits > 0);
      if (hits > 0) list[n + __popc(m & ((1u << lane) - 1u))] = uint32_t(x) | uint32_t(hits - 1) << kIdBits;
      n += __popc(m);
    }
    __syncwarp();
    int cols = 0;
    for (int i = lane; i < n; i += 32) {
      int a, b, d, t;
      window_origin(P.g, entry_window(list[i]), &a, &b, &d, &t);
      cols += P.plan.type[t].n_tiles * (1 + entry_more(list[i]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) cols += __shfl_xor_sync(0xFFFFFFFFu, cols, o);
    if (lane == 0) {
      c.n_list = n;
      c.n_cols = cols;
    }
  }
  {
    // Rows of a tile that no TMA box writes must hold finite values (their P and dS
    // are 0, and the MMAs multiply them by 0): tiles when the plan has such rows,
    // and always the record buffers.
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const uint32_t first = P.plan.zero_fill ? kSmemRow : L::rec;
    uint4 *z = reinterpret_cast<uint4 *>(smem + first);
    for (uint32_t i = threadIdx.x; i < (L::ctrl - first) / 16; i += kThreads) z[i] = zero;
    ptx::fence_proxy_async_smem();
  }
  if (warp == 1) {
    ptx::tmem_alloc(&c.tmem_base, kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = c.tmem_base;
  const int n_cols = c.n_cols;
  const int n_windows = MODE == kDkvLong ? P.g.nWin : c.n_list;
  uint8_t *row0 = smem + kSmemRow, *row1 = smem + kSmemRow + kTileBytes;

  if (warp == 0) {
    // ------------------------------------------------------------- TMA loader
    if (lane == 0) {
      Waiter wt{&c.abort, P.dev_err, P.timeout_ns, BASA_DEVERR_TIMEOUT_PRODUCER, true};
      Waiter drain{&c.abort, P.dev_err, P.timeout_ns, BASA_DEVERR_TIMEOUT_PRODUCER, false};
      // row tiles: dq pass q, dout; dK/dV passes k, v
      if (MODE == kDq) {
        ptx::mbar_arrive_expect_tx(&c.row_full, uint32_t(row_tile.valid_rows) * 512u);
        load_window_tile(P.plan, P.g, P.map_q, row_tile, row_org, bh, row0, &c.row_full);
        load_window_tile(P.plan, P.g, P.map_do, row_tile, row_org, bh_v, row1, &c.row_full);
      } else if (MODE == kDkvWindow) {
        ptx::mbar_arrive_expect_tx(&c.row_full, uint32_t(row_tile.valid_rows) * 512u);
        load_window_tile(P.plan, P.g, P.map_k, row_tile, row_org, map_unit(0), row0, &c.row_full);
        load_window_tile(P.plan, P.g, P.map_v, row_tile, row_org, bh, row1, &c.row_full);
      } else {
        const bool pooled = kt < P.n_pool_tiles;
        const CUtensorMap *mk = pooled ? &P.map_kp : &P.map_kt, *mv = pooled ? &P.map_vp : &P.map_vt;
        const int row = pooled ? kt * kTileRows : P.g.N + (kt - P.n_pool_tiles) * kTileRows;
        ptx::mbar_arrive_expect_tx(&c.row_full, 2 * kTileBytes);
        ptx::tma_load_3d(row0, mk, &c.row_full, 0, row, map_unit(0));
        ptx::tma_load_3d(row0 + kHalfBytes, mk, &c.row_full, 64, row, map_unit(0));
        ptx::tma_load_3d(row1, mv, &c.row_full, 0, row, bh);
        ptx::tma_load_3d(row1 + kHalfBytes, mv, &c.row_full, 64, row, bh);
      }
      int last = -1, last_k = -1, last_v = -1, row_loads = 1;
      bool skipped0 = false;  // test hook: the first ring item was never loaded
      if (MODE == kDq) {
        KeyIter it;
        key_first(P, c, it);
        for (int j = 0; j < n_cols; ++j) {
          bool ok = true;
          for (int kv = 0; kv < 2; ++kv) {
            const int slot = dq_slot(j, kv == 1);
            if (!wt.wait(&c.empty[slot], dq_phase(j, kv == 1) ^ 1)) { ok = false; break; }
            if (j == 0 && kv == 0 && (P.flags & BASA_FLAG_TEST_SKIP_FIRST_KEY_LOAD)) {
              skipped0 = true;
              last_k = 0;
              continue;
            }
            const uint32_t bytes = it.seg <= P.routed_k
                                       ? uint32_t(P.plan.tile[P.plan.type[c.wtype[it.seg]].first_tile + it.t].valid_rows) * 256u
                                       : kTileBytes;
            ptx::mbar_arrive_expect_tx(&c.full[slot], bytes);
            load_key(P, c, it, kv == 1, kv == 1 ? bh_v : bh, smem + kSmemRing + slot * kTileBytes, &c.full[slot]);
            (kv ? last_v : last_k) = j;
          }
          if (!ok) break;
          key_next(P, c, it);
        }
      } else if (n_cols > 0) {
        bool ok = true;
        for (int m = 0; ok && m < kMaps; ++m) {
          const int unit = map_unit(m);
          if (m == 1) {  // the key tile of map 1, once the last product with map 2's has read it
            if (!wt.wait(&c.row_free, 0)) break;
            const bool pooled = MODE == kDkvLong && kt < P.n_pool_tiles;
            if (MODE == kDkvWindow) {
              ptx::mbar_arrive_expect_tx(&c.row_full, uint32_t(row_tile.valid_rows) * 256u);
              load_window_tile(P.plan, P.g, P.map_k, row_tile, row_org, unit, row0, &c.row_full);
            } else {
              const CUtensorMap *mk = pooled ? &P.map_kp : &P.map_kt;
              const int row = pooled ? kt * kTileRows : P.g.N + (kt - P.n_pool_tiles) * kTileRows;
              ptx::mbar_arrive_expect_tx(&c.row_full, kTileBytes);
              ptx::tma_load_3d(row0, mk, &c.row_full, 0, row, unit);
              ptx::tma_load_3d(row0 + kHalfBytes, mk, &c.row_full, 64, row, unit);
            }
            row_loads = 2;
          }
          QIter it;
          q_first(P, list, MODE, MODE == kDkvLong ? chunk * P.chunk_tiles : 0, it);
          for (int j = m * n_cols; j < (m + 1) * n_cols; ++j) {
            const PlanTile &tile = q_tile(P, it);
            for (int kv = 0; kv < 2; ++kv) {
              const int item = 2 * j + kv, slot = item % kSlots;
              if (!wt.wait(&c.empty[slot], ((item / kSlots) & 1) ^ 1)) { ok = false; break; }
              if (item == 0 && (P.flags & BASA_FLAG_TEST_SKIP_FIRST_KEY_LOAD)) {
                skipped0 = true;
                last = 0;
                continue;
              }
              uint8_t *dst = smem + kSmemRing + slot * kTileBytes;
              if (kv == 0) {  // q tile and its records (record buffer j & 1, freed with the q slot)
                ptx::mbar_arrive_expect_tx(&c.full[slot], uint32_t(tile.valid_rows) * (256u + 16u));
                load_window_tile(P.plan, P.g, P.map_q, tile, it.org, unit, dst, &c.full[slot]);
                load_window_records(P.plan, P.g, P.map_rec, tile, it.org, unit, smem + L::rec + (j & 1) * kRecBytes,
                                    &c.full[slot]);
              } else {
                ptx::mbar_arrive_expect_tx(&c.full[slot], uint32_t(tile.valid_rows) * 256u);
                load_window_tile(P.plan, P.g, P.map_do, tile, it.org, bh, dst, &c.full[slot]);
              }
              last = item;
            }
            if (!ok) break;
            q_next(P, list, MODE, n_windows, it);
          }
        }
      }
      // Drain: wait for the copies still in flight (immediate when all were consumed).
      // A slot's earlier copies completed before the slot was granted again.
      drain.wait(&c.row_full, (row_loads - 1) & 1);
      if (MODE == kDq) {
        for (int j = max(0, last_k - 2); j <= last_k; ++j)
          if (j > 0 || !skipped0) drain.wait(&c.full[dq_slot(j, false)], dq_phase(j, false));
        for (int j = max(0, last_v - 1); j <= last_v; ++j) drain.wait(&c.full[dq_slot(j, true)], dq_phase(j, true));
      }
      for (int item = max(0, last - (kSlots - 1)); item <= last; ++item)
        if (item > 0 || !skipped0) drain.wait(&c.full[item % kSlots], (item / kSlots) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      Waiter wt{&c.abort, P.dev_err, P.timeout_ns, BASA_DEVERR_TIMEOUT_MMA, true};
      Waiter drain{&c.abort, P.dev_err, P.timeout_ns, BASA_DEVERR_TIMEOUT_MMA, false};
      const uint32_t r0 = kDescLoK | (ptx::smem_u32(row0) >> 4), r1 = kDescLoK | (ptx::smem_u32(row1) >> 4);
      const uint32_t ringK = kDescLoK | (ptx::smem_u32(smem + kSmemRing) >> 4);
      const uint32_t ringMn = kDescLoMn | (ptx::smem_u32(smem + kSmemRing) >> 4);
      auto slot_of = [](int item) { return uint32_t(item % kSlots) * kTileDesc; };
      bool ok = n_cols == 0 || wt.wait(&c.row_full, 0);
      if (MODE == kDq && ok && n_cols > 0) {
        // TMEM: S at 0; dP at 128, with dS written over its first halves; dq at 256; the
        // q and dout row tiles at 384 and 448 (bf16), copied there once by the compute
        // warps, so S and dP read their A operand from TMEM and only the key or value
        // tile from shared memory. Order per key tile j: S(j+1) once every thread holds
        // S(j) in registers (it runs while P(j) is computed), then dq(j) += dS(j) K_j,
        // then dP(j+1) over dS(j).
        const uint32_t tS = tmem, tDP = tmem + 128, tDQ = tmem + 256, tQ = tmem + 384, tDO = tmem + 448;
        auto kdesc = [&](int j) { return ringK + uint32_t(dq_slot(j, false)) * kTileDesc; };
        auto wait_k = [&](int j) { return wt.wait(&c.full[dq_slot(j, false)], dq_phase(j, false)); };
        auto wait_v = [&](int j) { return wt.wait(&c.full[dq_slot(j, true)], dq_phase(j, true)); };
        auto vdesc = [&](int j) { return ringK + uint32_t(dq_slot(j, true)) * kTileDesc; };
        ok = wt.wait(&c.a_ready, 0) && wait_k(0);
        if (ok) {
          ptx::tc_fence_after();
          issue_ts_kmajor(tS, tQ, kdesc(0));  // S(0) = q K0^T
          ptx::mma_commit(&c.s_full[0]);
          ok = wait_v(0);
        }
        if (ok) {
          ptx::tc_fence_after();
          issue_ts_kmajor(tDP, tDO, vdesc(0));  // dP(0) = dout V0^T
          ptx::mma_commit(&c.dp_full[0]);
          ptx::mma_commit(&c.empty[dq_slot(0, true)]);
        }
        for (int j = 0; ok && j < n_cols; ++j) {
          const bool more = j + 1 < n_cols;
          if (more) {
            if (!wt.wait(&c.s_free, j & 1) || !wait_k(j + 1)) break;
            ptx::tc_fence_after();
            issue_ts_kmajor(tS, tQ, kdesc(j + 1));  // S(j+1)
            ptx::mma_commit(&c.s_full[0]);
          }
          if (!wt.wait(&c.ds_full[0], j & 1)) break;
          ptx::tc_fence_after();
          issue_ts_split(tDQ, tDP, ringMn + uint32_t(dq_slot(j, false)) * kTileDesc, j > 0);  // dq += dS(j) K_j
          ptx::mma_commit(&c.empty[dq_slot(j, false)]);
          if (more) {
            if (!wait_v(j + 1)) break;
            ptx::tc_fence_after();
            issue_ts_kmajor(tDP, tDO, vdesc(j + 1));  // dP(j+1), after dq(j) has read dS(j)
            ptx::mma_commit(&c.dp_full[0]);
            ptx::mma_commit(&c.empty[dq_slot(j + 1, true)]);
          }
        }
      } else if (MODE != kDq && ok && n_cols > 0) {
        // TMEM: S^T at 0, dP^T at 128, dV at 256, dK at 384. Compute group g owns query
        // columns [64 g, 64 g + 64) of S^T and dP^T, and writes dS^T and P^T (bf16, 32
        // columns each) over its dP^T: S^T is free once it is in registers, so S^T(j+1) is
        // there before the next tile's P is begun (with P^T over S^T it had to wait for dV
        // to read that: 24 heads of 16896 keys 1.38 against 1.36 ms). The dK products are issued per group (the K-steps over its
        // queries) as soon as that group's dS^T is in TMEM, and before those of dV, since
        // the next tile but one's queries, wanted first, take their slot. S^T and dP^T stay
        // whole N = 128 products (an N = 64 half reads the same A operand from shared
        // memory for half the work).
        const uint32_t tS = tmem, tDP = tmem + 128, tDV = tmem + 256, tDK = tmem + 384;
        // Differential form: tiles [0, n_cols) are map 2's, [n_cols, 2 n_cols) map 1's.
        const int total = kMaps * n_cols;
        ok = wt.wait(&c.full[0], 0);
        if (ok) {
          ptx::tc_fence_after();
          issue_ss(tS, r0, ringK + slot_of(0));  // S^T(0) = K q0^T
          ptx::mma_commit(&c.s_full[0]);
          if (kMaps == 2 && n_cols == 1) ptx::mma_commit(&c.row_free);
          ok = wt.wait(&c.full[1], 0);
        }
        if (ok) {
          ptx::tc_fence_after();
          issue_ss(tDP, r1, ringK + slot_of(1));  // dP^T(0) = V dout0^T
          ptx::mma_commit(&c.dp_full[0]);
        }
        for (int j = 0; ok && j < total; ++j) {
          const int qi = 2 * j, di = 2 * j + 1, qn = qi + 2, dn = di + 2;
          const bool more = j + 1 < total;
          const bool map_start = j == 0 || (kMaps == 2 && j == n_cols);
          // Map 2's last tile: its sums first, which do not wait for map 1's key tile.
          const bool boundary = kMaps == 2 && j + 1 == n_cols;
          auto next_scores = [&] {
            if (!wt.wait(&c.s_free, j & 1) || !wt.wait(&c.full[qn % kSlots], (qn / kSlots) & 1)) return false;
            if (boundary && !wt.wait(&c.row_full, 1)) return false;
            ptx::tc_fence_after();
            issue_ss(tS, r0, ringK + slot_of(qn));  // S^T(j+1), while P(j) is computed
            ptx::mma_commit(&c.s_full[0]);
            if (kMaps == 2 && j + 2 == n_cols) ptx::mma_commit(&c.row_free);
            return true;
          };
          if (more && !boundary && !next_scores()) break;
          if (kMaps == 2 && j == n_cols) {
            // both groups have read map 2's dK and rescaled dV before their first P^T
            ok = wt.wait(&c.ds_full[0], j & 1) && wt.wait(&c.ds_full[1], j & 1);
            if (!ok) break;
          }
          for (int g = 0; ok && g < 2; ++g) {
            ok = wt.wait(&c.ds_full[g], j & 1);
            if (!ok) break;
            ptx::tc_fence_after();
            issue_ts_group(tDK, tDP, ringMn + slot_of(qi), g, !map_start || g > 0);  // dK += dS^T(j) q_j
          }
          if (!ok) break;
          ptx::mma_commit(&c.empty[qi % kSlots]);
          for (int g = 0; g < 2; ++g)
            issue_ts_group(tDV, tDP + 32, ringMn + slot_of(di), g, j > 0 || g > 0);  // dV += P^T(j) dout_j
          ptx::mma_commit(&c.empty[di % kSlots]);
          if (boundary) {
            ptx::mma_commit(&c.acc_full);  // map 2 is complete
            if (!next_scores()) break;
          }
          if (more) {
            if (!wt.wait(&c.full[dn % kSlots], (dn / kSlots) & 1)) break;
            ptx::tc_fence_after();
            issue_ss(tDP, r1, ringK + slot_of(dn));  // dP^T(j+1), after the sums have read P^T(j) and dS^T(j)
            ptx::mma_commit(&c.dp_full[0]);
          }
        }
      }
      ptx::mma_commit(&c.acc_full);
      // Every MMA this thread issued must finish before TMEM is freed.
      ptx::mma_commit(&c.drain);
      drain.wait(&c.drain, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- P and dS
    const int g = (warp - 2) / 4;  // column half
    const int sub = warp % 4;      // TMEM lane quarter this warp may access
    const int row = sub * 32 + lane;
    const uint32_t lane_off = uint32_t(sub * 32) << 16;
    const uint32_t col = uint32_t(64 * g);
    Waiter wt{&c.abort, P.dev_err, P.timeout_ns, BASA_DEVERR_TIMEOUT_SOFTMAX, true};
    const float sl2 = P.scale_log2;
    bool ok = true;
    if (MODE == kDq) {
      const uint32_t tS = tmem + lane_off + col, tDP = tmem + lane_off + 128 + col;
      float dr_weight = 0.f;
      uint64_t dr2 = 0;            // sums of this row's dS (even and odd columns)
      uint64_t nl2 = 0, nd2 = 0;  // this row's -L log2 e and -D, paired for packed arithmetic
      int t, y, x;                // (a padding row keeps 0, 0: its dS is 0 as its dout row is 0)
      if (n_cols > 0 && tile_row_token(P.plan, P.g, row_tile, row_org, row, &t, &y, &x)) {
        const float4 rec = P.rec[(long long)bh * P.g.N + ((long long)t * P.g.H + y) * P.g.W + x];
        nl2 = ptx::f2_pack(rec.x, rec.x);
        nd2 = ptx::f2_pack(rec.y, rec.y);
        dr_weight = rec.z;
      }
      if (n_cols > 0) {
        // This row's q and dout (this group's 64 of the head dims) into TMEM, where the
        // MMAs read them as the A operand of S and dP.
        ok = __all_sync(0xFFFFFFFFu, wt.wait(&c.row_full, 0));
        if (ok) {
          uint32_t w[32];
          load_row_half(row0, row, g, w);
          ptx::tmem_st32(tmem + lane_off + 384 + 32 * g, w);
          load_row_half(row1, row, g, w);
          ptx::tmem_st32(tmem + lane_off + 448 + 32 * g, w);
          ptx::tmem_st_wait();
          ptx::tc_fence_before();
          ptx::mbar_arrive(&c.a_ready);
        }
      }
      const uint64_t sl2x2 = ptx::f2_pack(sl2, sl2);
      KeyIter it;
      key_first(P, c, it);
      for (int j = 0; ok && j < n_cols; ++j) {
        ok = __all_sync(0xFFFFFFFFu, wt.wait(&c.s_full[0], j & 1));
        if (!ok) break;
        ptx::tc_fence_after();
        float s[64], dp[64];
        tmem_ld64f(tS, s);
        ptx::tc_fence_before();
        ptx::mbar_arrive(&c.s_free);  // S(j) is in registers: the MMA may overwrite it
        uint32_t m[4] = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
        if (!P.all_full) key_mask(P, c, it, m);
        const uint32_t m0 = m[2 * g], m1 = m[2 * g + 1];
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          float x0, x1;
          ptx::f2_unpack(ptx::ffma2(ptx::f2_pack(s[i], s[i + 1]), sl2x2, nl2), x0, x1);
          s[i] = ptx::ex2(x0);
          s[i + 1] = ptx::ex2(x1);
        }
        ok = __all_sync(0xFFFFFFFFu, wt.wait(&c.dp_full[0], j & 1));
        if (!ok) break;
        ptx::tc_fence_after();
        tmem_ld64f(tDP, dp);
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          float d0, d1;
          ptx::f2_unpack(ptx::fmul2(ptx::f2_pack(s[i], s[i + 1]), ptx::fadd2(ptx::f2_pack(dp[i], dp[i + 1]), nd2)), d0,
                         d1);
          s[i] = d0;
          s[i + 1] = d1;
        }
        if ((m0 & m1) != 0xFFFFFFFFu) zero_masked(s, m0, m1);  // warp-uniform: a partial key tile
        if (DIFF) {
#pragma unroll
          for (int i = 0; i < 64; i += 2) dr2 = ptx::fadd2(dr2, ptx::f2_pack(s[i], s[i + 1]));
        }
        uint32_t pk[32];
        pack64(s, pk);
        ptx::tmem_st32(tDP, pk);  // dS (bf16) over the first half of this thread's dP columns
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(&c.ds_full[0]);
        key_next(P, c, it);
      }
      if (ok) ok = __all_sync(0xFFFFFFFFu, wt.wait(&c.acc_full, 0));
      if (ok) {
        ptx::tc_fence_after();
        float x[64];
        tmem_ld64f(tmem + lane_off + 256 + col, x);
#pragma unroll
        for (int i = 0; i < 64; ++i) x[i] *= DIFF && (bh & 1) ? P.scale * neg_lambda : P.scale;
        stage_row_half(row0, row, g, x);  // the q tile is no longer read
        ptx::fence_proxy_async_smem();
        if (DIFF) {  // the 256 half rows' weighted sums, in a fixed order (the dout tile is no longer read)
          float even, odd;
          ptx::f2_unpack(dr2, even, odd);
          float d = (even + odd) * dr_weight;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, o);
          if (lane == 0) reinterpret_cast<float *>(row1)[warp - 2] = d;
        }
      }
      ptx::named_barrier(1, 256);
      if (DIFF && threadIdx.x == 64) {
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) d += reinterpret_cast<const float *>(row1)[i];
        P.dr[blockIdx.x] = d;  // [map][window][query tile]
      }
      if (threadIdx.x == 64 && ok && !*reinterpret_cast<volatile int *>(&c.abort)) {
        store_window_tile(P.plan, P.g, P.map_dq, row_tile, row_org, bh, row0);
        ptx::tma_store_commit();
        ptx::tma_store_wait_read_all();
      }
    } else {
      const uint32_t tS = tmem + lane_off + col, tDP = tmem + lane_off + 128 + col;
      float *wrec = reinterpret_cast<float *>(smem + L::col_rec) + (warp - 2) * 128;  // [-L log2 e x 64 | -D x 64]
      const float4 *nl4 = reinterpret_cast<const float4 *>(wrec), *nd4 = reinterpret_cast<const float4 *>(wrec + 64);
      // Differential form: this row's token (-1: none) and its patch, kept for the two
      // epilogues in shared memory (registers are full) while the first scores are on their way.
      int2 *place = reinterpret_cast<int2 *>(smem + L::place) + (threadIdx.x - 64);
      auto row_place = [&] {
        int t, y, x;
        if (!tile_row_token(P.plan, P.g, row_tile, row_org, row, &t, &y, &x)) return make_int2(-1, 0);
        return make_int2((t * P.g.H + y) * P.g.W + x,
                         ((t / P.pt) * (P.g.H / P.ph) + y / P.ph) * (P.g.W / P.pw) + x / P.pw);
      };
      if (DIFF && MODE == kDkvWindow) *place = row_place();
      // unrolled: the two maps' epilogues differ (a rolled loop spills over 800 bytes a thread)
#pragma unroll
      for (int m = 0; m < kMaps; ++m) {
        QIter it;
        if (n_cols > 0) q_first(P, list, MODE, MODE == kDkvLong ? chunk * P.chunk_tiles : 0, it);
        for (int j = m * n_cols; ok && j < (m + 1) * n_cols; ++j) {
          ok = __all_sync(0xFFFFFFFFu, wt.wait(&c.s_full[0], j & 1));
          if (!ok) break;
          ptx::tc_fence_after();
          float p[64];
          tmem_ld64f(tS, p);
          ptx::tc_fence_before();
          ptx::mbar_arrive(&c.s_free);  // S^T(j) is in registers: the MMA may overwrite it
          {
            // This warp's 64 query records {-L log2 e, -D, 0, 0}, one load per lane
            // for two columns, rewritten as two arrays that the loops below read four
            // values at a time.
            const float4 *r = reinterpret_cast<const float4 *>(smem + L::rec + (j & 1) * kRecBytes) + col;
            const float4 a = r[lane], b = r[32 + lane];
            __syncwarp();  // every lane has read the previous tile's arrays
            wrec[lane] = a.x;
            wrec[32 + lane] = b.x;
            wrec[64 + lane] = a.y;
            wrec[96 + lane] = b.y;
            __syncwarp();
          }
          uint32_t m0 = 0xFFFFFFFFu, m1 = 0xFFFFFFFFu;
          if (!P.all_full) {
            const PlanTile &qt = q_tile(P, it);
            m0 = qt.mask[2 * g];
            m1 = qt.mask[2 * g + 1];
          }
          const uint64_t sl2x2 = ptx::f2_pack(sl2, sl2);
#pragma unroll
          for (int i = 0; i < 64; i += 4) {
            const float4 nl = nl4[i / 4];
            float x0, x1, x2, x3;
            ptx::f2_unpack(ptx::ffma2(ptx::f2_pack(p[i], p[i + 1]), sl2x2, ptx::f2_pack(nl.x, nl.y)), x0, x1);
            ptx::f2_unpack(ptx::ffma2(ptx::f2_pack(p[i + 2], p[i + 3]), sl2x2, ptx::f2_pack(nl.z, nl.w)), x2, x3);
            p[i] = ptx::ex2(x0);
            p[i + 1] = ptx::ex2(x1);
            p[i + 2] = ptx::ex2(x2);
            p[i + 3] = ptx::ex2(x3);
          }
          const bool partial = (m0 & m1) != 0xFFFFFFFFu;  // warp-uniform: a partial query tile
          if (partial) zero_masked(p, m0, m1);
          ok = __all_sync(0xFFFFFFFFu, wt.wait(&c.dp_full[0], j & 1));
          if (!ok) break;
          ptx::tc_fence_after();
          float dp[64];
          tmem_ld64f(tDP, dp);
#pragma unroll
          for (int i = 0; i < 64; i += 4) {
            const float4 nd = nd4[i / 4];
            float d0, d1, d2, d3;
            ptx::f2_unpack(ptx::fmul2(ptx::f2_pack(p[i], p[i + 1]),
                                      ptx::fadd2(ptx::f2_pack(dp[i], dp[i + 1]), ptx::f2_pack(nd.x, nd.y))),
                           d0, d1);
            ptx::f2_unpack(ptx::fmul2(ptx::f2_pack(p[i + 2], p[i + 3]),
                                      ptx::fadd2(ptx::f2_pack(dp[i + 2], dp[i + 3]), ptx::f2_pack(nd.z, nd.w))),
                           d2, d3);
            dp[i] = d0;
            dp[i + 1] = d1;
            dp[i + 2] = d2;
            dp[i + 3] = d3;
          }
          if (partial) zero_masked(dp, m0, m1);  // dS = 0 there whatever dP holds
          uint32_t pk[32];
          pack64(dp, pk);
          ptx::tmem_st32(tDP, pk);  // dS^T (bf16) over the first half of this thread's dP^T columns,
          pack64(p, pk);
          ptx::tmem_st32(tDP + 32, pk);  // P^T over the second
          ptx::tmem_st_wait();
          ptx::tc_fence_before();
          ptx::mbar_arrive(&c.ds_full[g]);
          q_next(P, list, MODE, n_windows, it);
        }
        if (ok) ok = __all_sync(0xFFFFFFFFu, wt.wait(&c.acc_full, n_cols > 0 ? m : 0));
        if (DIFF && MODE == kDkvWindow) {
          ptx::grid_wait();  // the pooled keys' gradients; after an expired wait too: this launch ends after the others
          ptx::grid_launch_dependents();
        }
        if (!ok) continue;
        ptx::tc_fence_after();
        const bool last_map = m + 1 == kMaps;
        const int unit = map_unit(m);  // of k and dk
        if (!last_map) {  // map 2's part of dV, before map 1 adds to it
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t r[32];
            ptx::tmem_ld32(tmem + lane_off + 256 + col + 32 * h, r);
            ptx::tmem_ld_wait(r);
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * neg_lambda);
            ptx::tmem_st32(tmem + lane_off + 256 + col + 32 * h, r);
          }
        }
        float dv[64], dk[64];
        if (n_cols > 0) {
          tmem_ld64f(tmem + lane_off + 384 + col, dk);
          if (last_map) tmem_ld64f(tmem + lane_off + 256 + col, dv);
        } else {
#pragma unroll
          for (int i = 0; i < 64; ++i) dv[i] = dk[i] = 0.f;
        }
        const float dk_scale = last_map ? P.scale : P.scale * neg_lambda;
#pragma unroll
        for (int i = 0; i < 64; ++i) dk[i] *= dk_scale;
        if (!last_map) {
          ptx::tmem_st_wait();
          ptx::tc_fence_before();
        }
        if (MODE == kDkvLong) {
          // partial sums of this chunk, float32 [dK of each map | dV][row][128]
          float *dst = P.part + ((((long long)bh * P.n_long_tiles + kt) * P.n_chunks + chunk) * (kMaps + 1)) * (kTileRows * 128) +
                       row * 128 + col;
          float4 *pk4 = reinterpret_cast<float4 *>(dst + (kMaps - 1 - m) * (kTileRows * 128));
          float4 *pv4 = reinterpret_cast<float4 *>(dst + kMaps * (kTileRows * 128));
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            pk4[i] = make_float4(dk[4 * i], dk[4 * i + 1], dk[4 * i + 2], dk[4 * i + 3]);
            if (last_map) pv4[i] = make_float4(dv[4 * i], dv[4 * i + 1], dv[4 * i + 2], dv[4 * i + 3]);
          }
        } else {
          int2 at = make_int2(-1, 0);
          if (DIFF) at = *place;
          else if (P.n_pool > 0) at = row_place();
          if (P.n_pool > 0 && at.x >= 0) {
            // the pooled keys' gradient of this token's patch, spread evenly
            const float4 *gk = reinterpret_cast<const float4 *>(P.dkvp + ((long long)unit * P.n_pool + at.y) * 128 + col);
            const float4 *gv = reinterpret_cast<const float4 *>(
                P.dkvp + (((long long)kMaps * P.bh_count + bh) * P.n_pool + at.y) * 128 + col);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float4 a = gk[i];
              dk[4 * i] += a.x * P.inv_patch; dk[4 * i + 1] += a.y * P.inv_patch;
              dk[4 * i + 2] += a.z * P.inv_patch; dk[4 * i + 3] += a.w * P.inv_patch;
              if (last_map) {
                const float4 b = gv[i];
                dv[4 * i] += b.x * P.inv_patch; dv[4 * i + 1] += b.y * P.inv_patch;
                dv[4 * i + 2] += b.z * P.inv_patch; dv[4 * i + 3] += b.w * P.inv_patch;
              }
            }
          }
          if (last_map) {
            stage_row_half(row0, row, g, dk);  // the k and v tiles are no longer read
            stage_row_half(row1, row, g, dv);
            ptx::fence_proxy_async_smem();
          } else {
            // the key tile's place in shared memory is map 1's already
            store_rows64(P.dk + (long long)unit * (P.g.N + P.n_text) * 128 + col,
                         *reinterpret_cast<volatile int *>(&c.abort) ? -1 : at.x, dk, lane);
          }
        }
      }
      if (DIFF && MODE == kDkvLong) __threadfence();  // this chunk's sums, before it counts as finished
      ptx::named_barrier(1, 256);
      if (DIFF && MODE == kDkvLong && P.long_done != nullptr) {
        if (threadIdx.x == 64)
          c.n_list = *reinterpret_cast<volatile int *>(&c.abort) ? -1 : atomicAdd(P.long_done + bh * P.n_long_tiles + kt, 1);
        ptx::named_barrier(1, 256);
        if (c.n_list == P.n_chunks - 1) {  // the last chunk of this key tile: their sums, in order
          __threadfence();
          const bool pooled = kt < P.n_pool_tiles;
          const int tile = pooled ? kt : kt - P.n_pool_tiles, rows = pooled ? P.n_pool : P.n_text;
          const float *base = P.part + (((long long)bh * P.n_long_tiles + kt) * P.n_chunks) * 3 * (kTileRows * 128);
          for (int i = 0; i < 6; ++i) {  // 3 arrays of 128 x 32 groups of four columns, eight a thread at a time
            float4 sum[8];
            const int first = (i & 1) * 2048 + (threadIdx.x - 64);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int ch = 0; ch < P.n_chunks; ++ch) {
              const float4 *p = reinterpret_cast<const float4 *>(base + ((long long)ch * 3 + (i >> 1)) * (kTileRows * 128)) + first;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 x = __ldcg(p + 256 * e);
                sum[e].x += x.x; sum[e].y += x.y; sum[e].z += x.z; sum[e].w += x.w;
              }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int at = first + 256 * e, r = tile * kTileRows + at / 32;
              if (r < rows)
                store_long_sum(sum[e], const_cast<float *>(P.dkvp), P.dk, P.dv, i >> 1, 2, bh, P.bh_count, pooled, r, at % 32,
                               P.n_pool, P.n_text, P.g.N);
            }
          }
        }
      }
      if (MODE == kDkvWindow && threadIdx.x == 64 && ok && !*reinterpret_cast<volatile int *>(&c.abort)) {
        store_window_tile(P.plan, P.g, P.map_dk, row_tile, row_org, map_unit(kMaps - 1), row0);
        store_window_tile(P.plan, P.g, P.map_dv, row_tile, row_org, bh, row1);
        ptx::tma_store_commit();
        ptx::tma_store_wait_read_all();
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
  if (last_to_end) ptx::grid_wait();
}

// Per query token: {-L log2(e), -(dout . out), 0, 0}, two tokens per warp (16 lanes x
// 8 bf16 each), float32 sums in a fixed order.
__global__ void __launch_bounds__(256) bwd_records_kernel(const __nv_bfloat16 *out, const __nv_bfloat16 *dout,
                                                          const float *lse, float4 *rec, long long rows) {
  const long long r = (long long)blockIdx.x * 16 + threadIdx.x / 16;
  const int part = threadIdx.x % 16;
  float acc = 0.f;
  if (r < rows) {
    const uint4 a = reinterpret_cast<const uint4 *>(out + r * 128)[part];
    const uint4 b = reinterpret_cast<const uint4 *>(dout + r * 128)[part];
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc = fmaf(__uint_as_float(aw[i] << 16), __uint_as_float(bw[i] << 16), acc);
      acc = fmaf(__uint_as_float(aw[i] & 0xFFFF0000u), __uint_as_float(bw[i] & 0xFFFF0000u), acc);
    }
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, o);
  if (r < rows && part == 0) rec[r] = make_float4(-lse[r] * 1.4426950408889634f, -acc, 0.f, 0.f);
}

// Sums the chunks of the long key tiles in order: pooled rows -> dkvp (float32),
// text rows -> dk, dv (bf16, rows N.. of each b*head). MAPS dK arrays and one dV for each
// unit of v, all by one thread.
template <int MAPS>
__global__ void __launch_bounds__(256) bwd_reduce_kernel(const float *part, float *dkvp, __nv_bfloat16 *dk,
                                                         __nv_bfloat16 *dv, int bh_count, int n_long, int n_chunks,
                                                         int n_pool, int n_pool_tiles, int n_text, long long N) {
  if (MAPS == 2) ptx::grid_launch_dependents();
  const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;  // (bh, tile, row, 4-column group)
  const long long total = (long long)bh_count * n_long * kTileRows * 32;
  if (idx >= total) return;
  const int c4 = int(idx % 32);
  const int row = int((idx / 32) % kTileRows);
  const int tile = int((idx / (32 * kTileRows)) % n_long);
  const int bh = int(idx / (32LL * kTileRows * n_long));
  const bool pooled = tile < n_pool_tiles;
  const int r = (pooled ? tile : tile - n_pool_tiles) * kTileRows + row;
  if (r >= (pooled ? n_pool : n_text)) return;
  float4 s[MAPS + 1];  // dK of each map, dV
#pragma unroll
  for (int a = 0; a <= MAPS; ++a) s[a] = make_float4(0.f, 0.f, 0.f, 0.f);
  const float *base = part + (((long long)bh * n_long + tile) * n_chunks) * (MAPS + 1) * (kTileRows * 128);
  for (int ch = 0; ch < n_chunks; ++ch) {
    const float *p = base + (long long)ch * (MAPS + 1) * (kTileRows * 128) + row * 128 + c4 * 4;
#pragma unroll
    for (int a = 0; a <= MAPS; ++a) {
      const float4 x = *reinterpret_cast<const float4 *>(p + a * kTileRows * 128);
      s[a].x += x.x; s[a].y += x.y; s[a].z += x.z; s[a].w += x.w;
    }
  }
#pragma unroll
  for (int a = 0; a <= MAPS; ++a)
    store_long_sum(s[a], dkvp, dk, dv, a, MAPS, bh, bh_count, pooled, r, c4, n_pool, n_text, N);
}

// ----------------------------------------------------------------- host side
struct BwdLayout {
  size_t rec, part, dkvp, total;  // of `maps` maps for each unit of v
  int n_long, n_chunks, chunk_tiles, q_tiles;
};

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Query tiles per head: the sum over windows of their type's tile count.
int head_query_tiles(const basa_params &p, const WindowPlan &plan) {
  const Geo g = make_geo(p);
  int n = 0;
  for (int w = 0; w < g.nWin; ++w) {
    int a, b, d, t;
    window_origin(g, w, &a, &b, &d, &t);
    n += plan.type[t].n_tiles;
  }
  return n;
}

// Chunking of the pooled / text key tiles' query range: the chunk count n (at
// least 4 query tiles per chunk) that minimises the estimated time of the launch,
// waves x (tiles per chunk + a CTA's fixed start and end cost in tiles), for a
// 148-SM part. It depends on the shape only, so the workspace size and the order of
// the chunk sums (hence the bits of the results) are the same on every device.
constexpr long long kLongSms = 148;
constexpr double kLongCtaCostTiles = 3.5;
BwdLayout bwd_layout(const basa_params &p, const WindowPlan &plan, int maps) {
  BwdLayout L{};
  const long long bh = (long long)p.B * p.heads;
  const long long N = (long long)p.T * p.H * p.W;
  const int n_pool = p.pt > 0 ? (p.T / p.pt) * (p.H / p.ph) * (p.W / p.pw) : 0;
  L.n_long = (n_pool + kTileRows - 1) / kTileRows + (p.n_text + kTileRows - 1) / kTileRows;
  L.q_tiles = head_query_tiles(p, plan);
  L.n_chunks = 1;
  L.chunk_tiles = L.q_tiles;
  if (L.n_long > 0 && L.q_tiles > 0) {
    const long long units = bh * L.n_long;
    double best = -1.0;
    for (int n = 1; n <= std::max(1, L.q_tiles / 4); ++n) {
      const int tiles = (L.q_tiles + n - 1) / n;
      const int chunks = (L.q_tiles + tiles - 1) / tiles;
      const double cost = double((units * chunks + kLongSms - 1) / kLongSms) * (tiles + kLongCtaCostTiles);
      if (best < 0.0 || cost < best) {
        best = cost;
        L.chunk_tiles = tiles;
        L.n_chunks = chunks;
      }
    }
  }
  L.rec = align256(size_t(maps) * bh * N * 16);
  L.part = align256(size_t(bh) * L.n_long * L.n_chunks * (maps + 1) * kTileRows * 128 * sizeof(float));
  L.dkvp = align256(size_t(bh) * n_pool * 128 * sizeof(float) * (maps + 1));
  L.total = L.rec + L.part + L.dkvp;
  return L;
}

template <int MODE, bool DIFF>
basa_status run_bwd(const BwdParams &P, long long blocks, cudaStream_t s, bool early = false) {
  if (blocks <= 0) return BASA_OK;
  if (blocks >= (1ll << 31)) return BASA_ERR_UNSUPPORTED;
  if (cudaFuncSetAttribute(attn_bwd_bf16_kernel<MODE, DIFF>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Smem<MODE>::bytes) != cudaSuccess)
    return BASA_ERR_CUDA;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Smem<MODE>::bytes;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, attn_bwd_bf16_kernel<MODE, DIFF>, P) == cudaSuccess ? BASA_OK : BASA_ERR_CUDA;
}

// Parameters of a backward over p.heads units of v with `maps` maps each; the
// workspace starts with a BwdLayout (records, partial sums, pooled gradients).
basa_status bwd_params(BwdParams &P, BwdLayout &L, const void *q, const void *k, const void *v, const void *kp,
                       const void *vp, const int32_t *route_idx, const void *dout, void *dq, void *dk, void *dv,
                       void *workspace, const basa_params &p, int maps) {
  if (!tensor_map_encoder()) return BASA_ERR_CUDA;
  std::memset(&P, 0, sizeof(P));
  basa_status st = build_window_plan(p, &P.plan);
  if (st != BASA_OK) return st;
  L = bwd_layout(p, P.plan, maps);
  P.g = make_geo(p);
  if (P.g.nWin > (p.routed_k > 0 ? kMaxBwdRouted : kMaxBwdWindows)) return BASA_ERR_UNSUPPORTED;
  const long long N = P.g.N, kv_rows = N + p.n_text, bh = (long long)p.B * p.heads;
  basa_params pm = p;
  pm.heads = p.heads * maps;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  P.rec = reinterpret_cast<const float4 *>(ws);
  P.part = reinterpret_cast<float *>(ws + L.rec);
  P.dkvp = reinterpret_cast<const float *>(ws + L.rec + L.part);
  for (int i = 0; i < P.plan.n_shapes; ++i) {
    const PlanShape &sh = P.plan.shape[i];
    if (!encode_grid_map(&P.map_q[i], q, pm, N, sh) || !encode_grid_map(&P.map_k[i], k, pm, kv_rows, sh) ||
        !encode_grid_map(&P.map_v[i], v, p, kv_rows, sh) || !encode_grid_map(&P.map_do[i], dout, p, N, sh) ||
        !encode_record_map(&P.map_rec[i], ws, pm, sh) || !encode_grid_map(&P.map_dq[i], dq, pm, N, sh) ||
        !encode_grid_map(&P.map_dk[i], dk, pm, kv_rows, sh) || !encode_grid_map(&P.map_dv[i], dv, p, kv_rows, sh))
      return BASA_ERR_CUDA;
  }
  P.n_pool = p.pt > 0 ? (p.T / p.pt) * (p.H / p.ph) * (p.W / p.pw) : 0;
  P.n_text = p.n_text;
  if (P.n_pool > 0 && (!encode_rows_map(&P.map_kp, kp, pm, P.n_pool) || !encode_rows_map(&P.map_vp, vp, p, P.n_pool)))
    return BASA_ERR_CUDA;
  if (p.n_text > 0 && (!encode_rows_map(&P.map_kt, k, pm, kv_rows) || !encode_rows_map(&P.map_vt, v, p, kv_rows)))
    return BASA_ERR_CUDA;
  P.n_pool_tiles = (P.n_pool + kTileRows - 1) / kTileRows;
  P.n_text_tiles = (p.n_text + kTileRows - 1) / kTileRows;
  P.n_long_tiles = L.n_long;
  P.route = route_idx;
  P.bh_count = int(bh);
  P.dev_err = p.dev_err;
  P.routed_k = p.routed_k;
  P.pt = std::max(p.pt, 1);
  P.ph = std::max(p.ph, 1);
  P.pw = std::max(p.pw, 1);
  P.inv_patch = p.pt > 0 ? 1.0f / float(p.pt * p.ph * p.pw) : 0.f;
  P.scale_log2 = float(1.4426950408889634 / std::sqrt(double(p.head_dim)));
  P.scale = float(1.0 / std::sqrt(double(p.head_dim)));
  P.all_full = (P.n_pool % kTileRows == 0) && (p.n_text % kTileRows == 0);
  P.max_tiles = 0;
  for (int i = 0; i < P.plan.n_tiles; ++i) P.all_full &= P.plan.tile[i].valid_rows == kTileRows;
  for (int t = 0; t < 8; ++t) P.max_tiles = std::max<int>(P.max_tiles, P.plan.type[t].n_tiles);
  P.n_chunks = L.n_chunks;
  P.chunk_tiles = L.chunk_tiles;
  P.q_tiles = L.q_tiles;
  P.timeout_ns = (p.wait_timeout_us ? (unsigned long long)p.wait_timeout_us : 2000000ull) * 1000ull;
  P.flags = p.flags;
  return BASA_OK;
}

basa_status run_reduce(int maps, const BwdParams &P, const BwdLayout &L, void *dk, void *dv, const basa_params &p,
                       cudaStream_t s) {
  const long long threads = (long long)P.bh_count * L.n_long * kTileRows * 32;
  const auto kernel = maps == 2 ? bwd_reduce_kernel<2> : bwd_reduce_kernel<1>;
  kernel<<<unsigned((threads + 255) / 256), 256, 0, s>>>(
      P.part, const_cast<float *>(P.dkvp), static_cast<__nv_bfloat16 *>(dk), static_cast<__nv_bfloat16 *>(dv), P.bh_count,
      L.n_long, L.n_chunks, P.n_pool, P.n_pool_tiles, p.n_text, P.g.N);
  return cudaGetLastError() == cudaSuccess ? BASA_OK : BASA_ERR_CUDA;
}

}  // namespace

size_t attn_bwd_bf16_workspace(const basa_params &p) {
  static thread_local WindowPlan plan;  // large: kept off the stack
  if (build_window_plan(p, &plan) != BASA_OK) return 0;
  return bwd_layout(p, plan, 1).total;
}

basa_status launch_attn_bwd_bf16(const void *q, const void *k, const void *v, const void *kp, const void *vp,
                                 const int32_t *route_idx, const void *out, const float *lse, const void *dout,
                                 void *dq, void *dk, void *dv, void *workspace, const basa_params &p, cudaStream_t s) {
  static thread_local BwdParams P;  // large: kept off the stack
  BwdLayout L;
  basa_status st = bwd_params(P, L, q, k, v, kp, vp, route_idx, dout, dq, dk, dv, workspace, p, 1);
  if (st != BASA_OK) return st;
  const long long rows = (long long)P.bh_count * P.g.N;
  bwd_records_kernel<<<unsigned((rows + 15) / 16), 256, 0, s>>>(
      static_cast<const __nv_bfloat16 *>(out), static_cast<const __nv_bfloat16 *>(dout), lse,
      static_cast<float4 *>(workspace), rows);
  if (cudaGetLastError() != cudaSuccess) return BASA_ERR_CUDA;
  const long long bh = P.bh_count, window_blocks = bh * P.g.nWin * P.max_tiles;
  if ((st = run_bwd<kDq, false>(P, window_blocks, s)) != BASA_OK) return st;
  if (L.n_long > 0) {
    if ((st = run_bwd<kDkvLong, false>(P, bh * L.n_long * L.n_chunks, s)) != BASA_OK) return st;
    if ((st = run_reduce(1, P, L, dk, dv, p, s)) != BASA_OK) return st;
  }
  return run_bwd<kDkvWindow, false>(P, window_blocks, s);
}

namespace {
// Differential form: whether a long key tile's chunks are summed by its last CTA. The sums
// then take that CTA about a key step's time a chunk and more for its start, behind which the
// dq pass's steps run and those of the window pass before its epilogue; where they are too few
// a reduction of its own, by the whole GPU, is sooner done. Steps behind the sums, chunks, and
// the backward's time with a reduction and with the last CTA, us (windows of 16 x 16 but for
// the 6 x 18 x 26 grid's, each in units of v, grid, routes):
//   12, 2:  68 / 70   (12, 32 x 32, 0)      8, 6:  70 / 82   (2, 48 x 64, 0)
//   16, 2: 128 / 121  (24, 32 x 32, 0)     12, 6:  86 / 92   (6, 48 x 64, 0)
//   46, 2: 267 / 254  (12, 64 x 64, 0)     20, 6: 122 / 109  (3, 6 x 18 x 26, 2)
//   14, 3:  98 / 87   (4, 32 x 48, 1)      28, 6: 138 / 141  (6, 6 x 18 x 26, 2)
//   25, 4: 169 / 156  (6, 64 x 64, 0)      18, 8:  94 / 96   (3, 64 x 64, 0)
//   19, 15: 154 / 174 (3, 96 x 96, 0)      34, 8: 241 / 236  (6, 96 x 96, 0)
bool last_cta_sums(const BwdLayout &L, const BwdParams &P, long long dq_ctas) {
  const int seen = 1 + P.routed_k;  // windows of a key list
  const long long dq = (dq_ctas + kLongSms - 1) / kLongSms * (P.max_tiles * seen + L.n_long);
  return L.n_long > 0 && dq + 2 * P.max_tiles * seen >= 11 + L.n_chunks;
}

// Workspace: the layout of two maps, g (with a norm), the partial sums of dlambda and
// dweight, the dq pass's, the counts of finished chunks.
struct DiffLayout {
  size_t g, sums, dr, done, total;
};
DiffLayout diff_layout(bool norm, const basa_params &p, const WindowPlan &plan) {
  int tiles = 0;
  for (int t = 0; t < 8; ++t) tiles = std::max<int>(tiles, plan.type[t].n_tiles);
  const size_t units = size_t(p.B) * p.heads;
  const BwdLayout L = bwd_layout(p, plan, 2);
  DiffLayout D{};
  D.g = L.total;
  D.sums = D.g + (norm ? align256(units * p.T * p.H * p.W * p.head_dim * 2) : 0);
  D.dr = D.sums + align256(diff_prep_workspace(p));
  D.done = D.dr + align256(2 * units * make_geo(p).nWin * tiles * sizeof(float));
  D.total = D.done + align256(units * L.n_long * sizeof(int));
  return D;
}
}  // namespace

size_t diff_attn_bwd_bf16_workspace(bool norm, const basa_params &p) {
  static thread_local WindowPlan plan;
  if (build_window_plan(p, &plan) != BASA_OK) return 0;
  return diff_layout(norm, p, plan).total;
}

basa_status launch_diff_attn_bwd_bf16(const void *q, const void *k, const void *v, const void *kp, const void *vp,
                                      const int32_t *route_idx, const basa_diff_params &dp, const void *pre,
                                      const void *second, const float *lse, const void *dout, void *dq, void *dk,
                                      void *dv, void *dlambda, void *dweight, void *workspace, const basa_params &p,
                                      cudaStream_t s) {
  static thread_local BwdParams P;
  static thread_local WindowPlan plan;
  basa_status st = build_window_plan(p, &plan);
  if (st != BASA_OK) return st;
  const DiffLayout D = diff_layout(dp.weight != nullptr, p, plan);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  BwdLayout L;
  st = bwd_params(P, L, q, k, v, kp, vp, route_idx, dp.weight ? ws + D.g : dout, dq, dk, dv, ws, p, 2);
  if (st != BASA_OK) return st;
  const long long bh = P.bh_count, window_blocks = bh * P.g.nWin * P.max_tiles;
  const bool any_long = L.n_long > 0, last_sums = last_cta_sums(L, P, 2 * window_blocks);
  P.lambda = static_cast<const __nv_bfloat16 *>(dp.lambda);
  P.heads = p.heads;
  P.dk = static_cast<__nv_bfloat16 *>(dk);
  P.dv = static_cast<__nv_bfloat16 *>(dv);
  P.dr = reinterpret_cast<float *>(ws + D.dr);
  P.long_done = last_sums ? reinterpret_cast<int *>(ws + D.done) : nullptr;
  float *sums = reinterpret_cast<float *>(ws + D.sums);
  st = launch_diff_prep(pre, second, lse, dout, dp, ws + D.g, reinterpret_cast<float4 *>(ws), nullptr, sums, P.long_done,
                        L.n_long, p, s);
  if (st != BASA_OK) return st;
  const auto run_sums = [&] {
    return launch_diff_sums(sums, P.dr, 2 * P.g.nWin * P.max_tiles, dp, dlambda, dweight, true, p, s);
  };
  if (any_long && (st = run_bwd<kDkvLong, true>(P, bh * L.n_long * L.n_chunks, s)) != BASA_OK) return st;
  if ((st = run_bwd<kDq, true>(P, 2 * window_blocks, s, any_long)) != BASA_OK) return st;
  if (any_long && !last_sums) {
    if ((st = run_reduce(2, P, L, dk, dv, p, s)) != BASA_OK || (st = run_sums()) != BASA_OK) return st;
    return run_bwd<kDkvWindow, true>(P, window_blocks, s, true);
  }
  if ((st = run_bwd<kDkvWindow, true>(P, window_blocks, s, true)) != BASA_OK) return st;
  return run_sums();
}

}  // namespace basa
