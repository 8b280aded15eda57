// Backward of the differential attention, bfloat16, head_dim 128, for sm_100a.
//
// out = O1 - lambda O2, two softmax maps over one key list that share their values. With g
// the gradient behind the norm and {-L log2 e, -D, weight, token} a record of each map's rows
// (both taken beforehand):
//   P_m = exp(q_m K_m^T / sqrt(d) - L_m),  dS_m = P_m (g V^T - D_m),  f_1 = 1, f_2 = -lambda,
//   dq_m = f_m dS_m K_m / sqrt(d),  dK_m = f_m dS_m^T q_m / sqrt(d),  dV = sum_m f_m P_m^T g.
// The passes are those of the window attention's backward (tile layouts, TMEM use and the
// order of the MMAs within a key or query tile are the same):
//   long     dK/dV of the pooled and text key tiles over chunks of the query tiles
//   dq       the key stream of every query tile
//   reduce   the chunks' sums
//   window   dK/dV of the window key tiles over the query tiles that see them
//
// The dq pass runs over the maps, map 2's sums scaled by -lambda at the end; it also adds up
// each row's dS (what its D was off by), which lambda's gradient takes in. The dK/dV passes
// run both maps of a (batch, head) one after the other, map 2 first: its dK leaves, the dV
// accumulator is multiplied by -lambda in TMEM, and map 1 adds to it, so the two maps' dV meet
// without a buffer or an atomic. (Both maps at once, sharing g V^T, would take six 128-column
// accumulators and TMEM holds four.)
//
// Each pass is one CTA per SM that goes through its work items, so that an item's loads, the
// list of its windows and its rows' places are ready when the one before it ends, and its
// first products run under that one's epilogue: a CTA per item spent 12k cycles on its start
// and 6k on its end beside 4k a tile (the window pass at 16 x 16 windows: 4 tiles). The
// passes overlap at their ends by programmatic dependent launch: the long pass has fewer
// items than there are SMs as often as not, and the dq pass, which needs nothing of it and
// takes its items from a counter, fills the rest; the window pass starts under the reduction
// and waits for it before its first epilogue.
//
// Rows of a tile that no load writes are set to zero beside the load (where a product sums
// over them): what an earlier item left there may be anything, infinities and NaN included.
// Nothing is added atomically: the same bits every run.
#include <algorithm>

#include "attn_bwd_sm100.cuh"

namespace basa {
namespace {

using namespace sm100;

// Warp 0 loads, warp 1 issues MMAs, warps 2-9 compute P and dS (two groups of four, each
// with 64 of the 128 columns of a row), warps 10 and 11 prepare items.
constexpr int kThreads = 384;
constexpr uint32_t kCompute = 256;
constexpr uint32_t kSmemRow = 0;                // the two row tiles
constexpr uint32_t kSmemRing = 2 * kTileBytes;  // then a ring of 32 KB tiles
constexpr uint32_t kCtrlBytes = 1024;
constexpr uint32_t kTmemCols = 512;

// id -> (tile, window, unit) and the window's origin, by unsigned 32-bit division: these stand
// at the head of everything a CTA does.
struct WorkItem {
  int tile, w, bh, wtype, org[3];
};
__device__ __forceinline__ void origin_of(const Geo &g, int w, int *org, int *wtype) {
  const uint32_t row = uint32_t(w) / uint32_t(g.nWx), jt = row / uint32_t(g.nWy);
  const int jx = w - int(row) * g.nWx, jy = int(row - jt * uint32_t(g.nWy));
  org[0] = wrap(int(jt) * g.wt + g.st, g.T);
  org[1] = wrap(jy * g.wh + g.sy, g.H);
  org[2] = wrap(jx * g.ww + g.sx, g.W);
  *wtype = (org[0] + g.wt > g.T ? 1 : 0) | (org[1] + g.wh > g.H ? 2 : 0) | (org[2] + g.ww > g.W ? 4 : 0);
}
__device__ __forceinline__ WorkItem work_item(const BwdParams &P, int id) {
  WorkItem x;
  const uint32_t rest = uint32_t(id) / uint32_t(P.max_tiles);
  x.tile = id - int(rest) * P.max_tiles;
  x.bh = int(rest / uint32_t(P.g.nWin));
  x.w = int(rest) - x.bh * P.g.nWin;
  origin_of(P.g, x.w, x.org, &x.wtype);
  return x;
}

struct Item {
  int n_cols;  // tiles that are streamed (of one map); < 0: there are no more items
  int bh;      // dq: unit of q; dK/dV: unit of v
  int id, tile, chunk, n_list;
  RouteList keys;  // dq: the key stream's windows; window pass: org[0] of the key tile's window
};

// ---------------------------------------------------------------------------- dq pass
constexpr int kDqSlots = 5;
constexpr uint32_t kDqCtrl = kSmemRing + kDqSlots * kTileBytes;
constexpr uint32_t kDqRec = kDqCtrl + kCtrlBytes;  // the rows' {-L log2 e, -D, weight, token}
constexpr uint32_t kDqSmem = kDqRec + kTileRows * 16;
static_assert(kDqSmem <= 227u * 1024u, "shared memory above the 227 KB a CTA may hold");

struct DqCtrl {
  uint64_t full[kDqSlots], empty[kDqSlots];
  uint64_t row_full, a_ready, s_full, s_free, dp_full, ds_full, acc_full, drain;
  uint64_t item_full[2], item_empty[2];
  uint32_t tmem_base;
  int abort;
  Item item[2];
};
static_assert(sizeof(DqCtrl) <= kCtrlBytes, "control block too large");

__global__ void __launch_bounds__(kThreads, 1) diff_dq_kernel(const __grid_constant__ BwdParams P) {
  extern __shared__ __align__(1024) uint8_t smem[];  // whole swizzle atoms: no room for a manual alignment
  DqCtrl &c = *reinterpret_cast<DqCtrl *>(smem + kDqCtrl);
  float4 *recs = reinterpret_cast<float4 *>(smem + kDqRec);  // as loaded; padding rows {0, 0, 0, -1}
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const bool pads = P.plan.zero_fill;  // some window tile has rows that no load writes
  if (threadIdx.x == 0) {
    for (int i = 0; i < kDqSlots; ++i) {
      ptx::mbar_init(&c.full[i], pads && i < 3 ? 2 : 1);
      ptx::mbar_init(&c.empty[i], 1);
    }
    for (uint64_t *b : {&c.s_full, &c.dp_full, &c.acc_full, &c.drain}) ptx::mbar_init(b, 1);
    ptx::mbar_init(&c.row_full, pads ? 2 : 1);
    for (uint64_t *b : {&c.a_ready, &c.s_free, &c.ds_full}) ptx::mbar_init(b, kCompute);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&c.item_full[i], 1);
      ptx::mbar_init(&c.item_empty[i], kCompute + (pads ? 3 : 2));  // compute threads, loader, MMA, warp 11
    }
    c.abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp >= 2 && warp < 10) touch_plan(P.plan, warp - 2, 8);
  if (warp == 1) {
    ptx::tmem_alloc(&c.tmem_base, kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = c.tmem_base;
  uint8_t *row0 = smem + kSmemRow, *row1 = row0 + kTileBytes;
  const auto waiter = [&](int bit, bool honor) { return Waiter{&c.abort, P.dev_err, P.timeout_ns, bit, honor}; };

  if (warp == 0) {
    // ------------------------------------------------------------- TMA loader
    if (lane == 0) {
      const Waiter wt = waiter(BASA_DEVERR_TIMEOUT_PRODUCER, true), drain = waiter(BASA_DEVERR_TIMEOUT_PRODUCER, false);
      const bool skipped0 = P.flags & BASA_FLAG_TEST_SKIP_FIRST_KEY_LOAD;
      int row_loads = 0, col = 0, k_loads = 0, v_loads = 0;
      bool ok = true;
      for (int n = 0; ok; ++n) {
        if (!wt.wait(&c.item_full[n & 1], (n >> 1) & 1)) break;
        const Item &it = c.item[n & 1];
        const int n_cols = it.n_cols, bh = it.bh;
        if (n_cols < 0) break;
        // the row tiles are read once the item before has them in TMEM
        if (n > 0 && !wt.wait(&c.a_ready, (n - 1) & 1)) break;
        const PlanTile &qt = P.plan.tile[it.tile];
        ptx::mbar_arrive_expect_tx(&c.row_full, uint32_t(qt.valid_rows) * (512u + 16u));
        load_window_records(P.plan, P.g, P.map_rec, qt, it.keys.org[0], bh, smem + kDqRec, &c.row_full);
        load_window_tile(P.plan, P.g, P.map_q, qt, it.keys.org[0], bh, row0, &c.row_full);
        load_window_tile(P.plan, P.g, P.map_do, qt, it.keys.org[0], bh >> 1, row1, &c.row_full);
        ++row_loads;
        KeyIter key;
        key_first(P, it.keys, key);
        for (int j = 0; ok && j < n_cols; ++j, ++col) {
          for (int kv = 0; kv < 2; ++kv) {
            const int slot = dq_slot(col, kv == 1);
            ok = wt.wait(&c.empty[slot], dq_phase(col, kv == 1) ^ 1);
            if (!ok) break;
            (kv ? v_loads : k_loads) = col + 1;
            if (col == 0 && kv == 0 && skipped0) continue;
            const uint32_t bytes = key.seg <= P.routed_k
                                       ? uint32_t(P.plan.tile[P.plan.type[it.keys.wtype[key.seg]].first_tile + key.t].valid_rows) * 256u
                                       : kTileBytes;
            ptx::mbar_arrive_expect_tx(&c.full[slot], bytes);
            load_key(P, it.keys, key, kv == 1, kv == 1 ? bh >> 1 : bh, smem + kSmemRing + slot * kTileBytes, &c.full[slot]);
          }
          if (ok) key_next(P, it.keys, key);
        }
        ptx::mbar_arrive(&c.item_empty[n & 1]);
      }
      // Drain: wait for the copies still in flight (immediate when all were consumed). A slot's
      // earlier copies completed before the slot was granted again.
      if (row_loads > 0) drain.wait(&c.row_full, (row_loads - 1) & 1);
      for (int j = max(0, k_loads - 3); j < k_loads; ++j)
        if (j > 0 || !skipped0) drain.wait(&c.full[dq_slot(j, false)], dq_phase(j, false));
      for (int j = max(0, v_loads - 2); j < v_loads; ++j) drain.wait(&c.full[dq_slot(j, true)], dq_phase(j, true));
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      const Waiter wt = waiter(BASA_DEVERR_TIMEOUT_MMA, true), drain = waiter(BASA_DEVERR_TIMEOUT_MMA, false);
      const uint32_t ringK = kDescLoK | (ptx::smem_u32(smem + kSmemRing) >> 4);
      const uint32_t ringMn = kDescLoMn | (ptx::smem_u32(smem + kSmemRing) >> 4);
      // TMEM: S at 0; dP at 128, with dS written over its first halves; dq at 256; the q and
      // g row tiles (bf16) at 384 and 448.
      const uint32_t tS = tmem, tDP = tmem + 128, tDQ = tmem + 256, tQ = tmem + 384, tDO = tmem + 448;
      auto scores = [&](int j) {  // S(j) = q K_j^T
        if (!wt.wait(&c.full[dq_slot(j, false)], dq_phase(j, false))) return false;
        ptx::tc_fence_after();
        issue_ts_kmajor(tS, tQ, ringK + uint32_t(dq_slot(j, false)) * kTileDesc);
        ptx::mma_commit(&c.s_full);
        return true;
      };
      auto dprob = [&](int j) {  // dP(j) = g V_j^T
        if (!wt.wait(&c.full[dq_slot(j, true)], dq_phase(j, true))) return false;
        ptx::tc_fence_after();
        issue_ts_kmajor(tDP, tDO, ringK + uint32_t(dq_slot(j, true)) * kTileDesc);
        ptx::mma_commit(&c.dp_full);
        ptx::mma_commit(&c.empty[dq_slot(j, true)]);
        return true;
      };
      int col = 0;
      for (int n = 0;; ++n) {
        if (!wt.wait(&c.item_full[n & 1], (n >> 1) & 1)) break;
        const int n_cols = c.item[n & 1].n_cols;
        ptx::mbar_arrive(&c.item_empty[n & 1]);
        if (n_cols < 0) break;
        // q and g in TMEM, which also says that the item before has read its S tiles
        bool ok = wt.wait(&c.a_ready, n & 1) && scores(col) && dprob(col);
        for (int j = 0; ok && j < n_cols; ++j, ++col) {
          const bool more = j + 1 < n_cols;
          // S(j+1) once every thread holds S(j); dq += dS(j) K_j; dP(j+1) over dS(j)
          if (more) ok = wt.wait(&c.s_free, col & 1) && scores(col + 1);
          if (ok) ok = wt.wait(&c.ds_full, col & 1);
          if (!ok) break;
          ptx::tc_fence_after();
          issue_ts_split(tDQ, tDP, ringMn + uint32_t(dq_slot(col, false)) * kTileDesc, j > 0);
          ptx::mma_commit(&c.empty[dq_slot(col, false)]);
          if (more) ok = dprob(col + 1);
        }
        if (!ok) break;
        ptx::mma_commit(&c.acc_full);
      }
      // Every MMA this thread issued must finish before TMEM is freed.
      ptx::mma_commit(&c.drain);
      drain.wait(&c.drain, 0);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ------------------------------------------------------------- items
    if (lane == 0) {
      const Waiter wt = waiter(BASA_DEVERR_TIMEOUT_PRODUCER, true);
      for (int n = 0, taken = 0;; ++n) {
        int id;
        WorkItem x;
        for (;; ++taken) {  // the first by the CTA's number, the others from the counter
          id = taken == 0 ? int(blockIdx.x) : int(gridDim.x) + atomicAdd(P.next_item, 1);
          if (id >= P.n_items) break;
          x = work_item(P, id);
          if (x.tile < P.plan.type[x.wtype].n_tiles) {
            ++taken;
            break;
          }
          for (int i = 0; i < 8; ++i) P.dr[8ll * id + i] = 0.f;  // this window type has fewer query tiles
        }
        if (!wt.wait(&c.item_empty[n & 1], ((n >> 1) & 1) ^ 1)) break;
        Item &it = c.item[n & 1];
        it.n_cols = -1;
        if (id < P.n_items) {
          it.bh = x.bh;
          it.id = id;
          it.tile = P.plan.type[x.wtype].first_tile + x.tile;
          it.keys.wtype[0] = x.wtype;
          for (int a = 0; a < 3; ++a) it.keys.org[0][a] = x.org[a];
          for (int r = 0; r < P.routed_k; ++r) {
            int u = P.route[((long long)(x.bh >> 1) * P.g.nWin + x.w) * P.routed_k + r];
            if (u < 0 || u >= P.g.nWin) {  // reported, and replaced by the own window: accesses stay in bounds
              if (P.dev_err) atomicOr(P.dev_err, BASA_DEVERR_BAD_ROUTE);
              u = x.w;
            }
            origin_of(P.g, u, it.keys.org[1 + r], &it.keys.wtype[1 + r]);
          }
          int cols = 0;
          for (int s = 0; s <= P.routed_k + 2; ++s) cols += seg_tiles(P, it.keys, s);
          it.n_cols = cols;
        }
        const bool last = it.n_cols < 0;
        ptx::mbar_arrive(&c.item_full[n & 1]);
        if (last) break;
      }
    }
    __syncwarp();
  } else if (warp == 11) {
    // ------------------------------- what no load writes: records of padding rows, rows of key tiles
    const Waiter wt = waiter(BASA_DEVERR_TIMEOUT_PRODUCER, true);
    int col = 0;
    for (int n = 0; pads; ++n) {
      bool ok = wt.wait(&c.item_full[n & 1], (n >> 1) & 1);
      if (ok && n > 0) ok = wt.wait(&c.a_ready, (n - 1) & 1);  // the records before are read
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      const Item &it = c.item[n & 1];
      if (it.n_cols < 0) break;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!((P.plan.tile[it.tile].mask[i] >> lane) & 1u))
          recs[32 * i + lane] = make_float4(0.f, 0.f, 0.f, __int_as_float(-1));
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&c.row_full);
      const int n_cols = it.n_cols;
      KeyIter key;
      key_first(P, it.keys, key);
      for (int j = 0; ok && j < n_cols; ++j, ++col) {
        const int slot = dq_slot(col, false);
        ok = __all_sync(0xFFFFFFFFu, wt.wait(&c.empty[slot], dq_phase(col, false) ^ 1));
        if (!ok) break;
        uint32_t mk[4];
        key_mask(P, it.keys, key, mk);
        // pooled and text tiles are written whole; rows past their end read as zero
        zero_unwritten_rows(smem + kSmemRing + slot * kTileBytes, mk, lane);
        if (lane == 0) ptx::mbar_arrive(&c.full[slot]);
        key_next(P, it.keys, key);
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&c.item_empty[n & 1]);
    }
  } else {
    // ------------------------------------------------------------- P and dS
    const int g = (warp - 2) / 4;  // column half
    const int sub = warp % 4;      // TMEM lane quarter this warp may access
    const int row = sub * 32 + lane;
    const uint32_t lane_off = uint32_t(sub * 32) << 16;
    const uint32_t col64 = uint32_t(64 * g);
    const uint32_t tS = tmem + lane_off + col64, tDP = tmem + lane_off + 128 + col64;
    const Waiter wt = waiter(BASA_DEVERR_TIMEOUT_SOFTMAX, true);
    const uint64_t sl2x2 = ptx::f2_pack(P.scale_log2, P.scale_log2);
    float4 rec = make_float4(0.f, 0.f, 0.f, 0.f);
    int n_cols = -1;
    // Item n's record, and its q and g row (this group's 64 of the head dims) into TMEM, where
    // the MMAs read them as the A operand of S and dP. The MMAs of the item before are done.
    auto begin = [&](int n) {
      if (!__all_sync(0xFFFFFFFFu, wt.wait(&c.item_full[n & 1], (n >> 1) & 1))) return false;
      n_cols = c.item[n & 1].n_cols;
      if (n_cols < 0) return true;
      if (!__all_sync(0xFFFFFFFFu, wt.wait(&c.row_full, n & 1))) return false;
      rec = recs[row];
      uint32_t w[32];
      load_row_half(row0, row, g, w);
      ptx::tmem_st32(tmem + lane_off + 384 + 32 * g, w);
      load_row_half(row1, row, g, w);
      ptx::tmem_st32(tmem + lane_off + 448 + 32 * g, w);
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      ptx::mbar_arrive(&c.a_ready);
      return true;
    };
    int col = 0;
    bool ok = begin(0);
    for (int n = 0; ok && n_cols >= 0; ++n) {
      const Item &it = c.item[n & 1];
      const uint64_t nl2 = ptx::f2_pack(rec.x, rec.x), nd2 = ptx::f2_pack(rec.y, rec.y);
      const float dr_weight = rec.z;
      const int tok = __float_as_int(rec.w), bh = it.bh, id = it.id;
      uint64_t dr2 = 0;  // sums of this row's dS (even and odd columns)
      KeyIter key;
      key_first(P, it.keys, key);
      const int cols = n_cols;
      for (int j = 0; ok && j < cols; ++j, ++col) {
        ok = __all_sync(0xFFFFFFFFu, wt.wait(&c.s_full, col & 1));
        if (!ok) break;
        ptx::tc_fence_after();
        float s[64], dp[64];
        tmem_ld64f(tS, s);
        ptx::tc_fence_before();
        ptx::mbar_arrive(&c.s_free);  // S(j) is in registers: the MMA may overwrite it
        uint32_t m[4] = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
        if (!P.all_full) key_mask(P, it.keys, key, m);
        const uint32_t m0 = m[2 * g], m1 = m[2 * g + 1];
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          float x0, x1;
          ptx::f2_unpack(ptx::ffma2(ptx::f2_pack(s[i], s[i + 1]), sl2x2, nl2), x0, x1);
          s[i] = ptx::ex2(x0);
          s[i + 1] = ptx::ex2(x1);
        }
        ok = __all_sync(0xFFFFFFFFu, wt.wait(&c.dp_full, col & 1));
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
#pragma unroll
        for (int i = 0; i < 64; i += 2) dr2 = ptx::fadd2(dr2, ptx::f2_pack(s[i], s[i + 1]));
        uint32_t pk[32];
        pack64(s, pk);
        ptx::tmem_st32(tDP, pk);  // dS (bf16) over the first half of this thread's dP columns
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(&c.ds_full);
        key_next(P, it.keys, key);
      }
      if (ok) ok = __all_sync(0xFFFFFFFFu, wt.wait(&c.acc_full, n & 1));
      if (!ok) break;
      ptx::mbar_arrive(&c.item_empty[n & 1]);
      ptx::tc_fence_after();
      ok = begin(n + 1);  // its first products run under what is left of this item
      float x[64];
      tmem_ld64f(tmem + lane_off + 256 + col64, x);
      ptx::tc_fence_before();
      const float f = bh & 1 ? -P.scale * __bfloat162float(P.lambda[(bh >> 1) % P.heads]) : P.scale;
#pragma unroll
      for (int i = 0; i < 64; ++i) x[i] *= f;
      const int row_to = *reinterpret_cast<volatile int *>(&c.abort) ? -1 : tok;
      store_rows64(P.dq + (long long)bh * P.g.N * 128 + col64, row_to, x, lane);
      float even, odd;
      ptx::f2_unpack(dr2, even, odd);
      float d = tok >= 0 ? (even + odd) * dr_weight : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, o);
      if (lane == 0) P.dr[8ll * id + (warp - 2)] = d;
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
  // What follows this launch needs the long pass's sums: one CTA ends after them.
  if (blockIdx.x == 0 && threadIdx.x == 0) ptx::grid_wait();
}

// ---------------------------------------------------------------------------- dK/dV passes
constexpr int kSlots = 4;
constexpr uint32_t kRec = kSmemRing + kSlots * kTileBytes;  // two record buffers of the streamed query tiles
constexpr uint32_t kColRec = kRec + 2 * kRecBytes;          // per compute warp: 64 x {-L log2 e}, 64 x {-D}
constexpr uint32_t kCtrl = kColRec + 8 * 128 * 4;
constexpr uint32_t kPlace = kCtrl + kCtrlBytes;         // two items' rows: token (-1: none) and patch
constexpr uint32_t kList = kPlace + 2 * kTileRows * 8;  // two items' windows that see the key tile
constexpr uint32_t kDkvSmem = kList + 2 * kMaxList * 2 + 1024;  // + alignment slack
static_assert(kDkvSmem <= 227u * 1024u, "shared memory above the 227 KB a CTA may hold");

struct DkvCtrl {
  uint64_t full[kSlots], empty[kSlots];
  uint64_t k_full, k_free, v_full, v_free, s_full, dp_full, p_full[2], ds_full[2], acc_full, drain;
  uint64_t rows_known[2], item_full[2], item_empty[2], place_full[2];
  uint32_t tmem_base;
  int abort;
  Item item[2];
};
static_assert(sizeof(DkvCtrl) <= kCtrlBytes, "control block too large");

template <bool LONG>
__global__ void __launch_bounds__(kThreads, 1) diff_dkv_kernel(const __grid_constant__ BwdParams P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  DkvCtrl &c = *reinterpret_cast<DkvCtrl *>(smem + kCtrl);
  int2 *places = reinterpret_cast<int2 *>(smem + kPlace);
  int16_t *lists = reinterpret_cast<int16_t *>(smem + kList);
  constexpr int kMode = LONG ? kDkvLong : kDkvWindow;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const bool pads = P.plan.zero_fill;  // some window tile has rows that no load writes
  if (LONG) ptx::grid_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      ptx::mbar_init(&c.full[i], pads ? 2 : 1);
      ptx::mbar_init(&c.empty[i], 1);
    }
    for (uint64_t *b : {&c.k_full, &c.k_free, &c.v_full, &c.v_free, &c.s_full, &c.dp_full, &c.acc_full, &c.drain,
                        &c.place_full[0], &c.place_full[1], &c.rows_known[0], &c.rows_known[1]})
      ptx::mbar_init(b, 1);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&c.p_full[i], 128);
      ptx::mbar_init(&c.ds_full[i], 128);
      ptx::mbar_init(&c.item_full[i], 1);
      ptx::mbar_init(&c.item_empty[i], kCompute + (pads ? 3 : 2));  // compute threads, loader, MMA, warp 11
    }
    c.abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp >= 2 && warp < 10) touch_plan(P.plan, warp - 2, 8);
  if (warp == 1) {
    ptx::tmem_alloc(&c.tmem_base, kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = c.tmem_base;
  uint8_t *row0 = smem + kSmemRow, *row1 = row0 + kTileBytes;
  const auto waiter = [&](int bit, bool honor) { return Waiter{&c.abort, P.dev_err, P.timeout_ns, bit, honor}; };
  const auto windows_of = [&](const Item &it) { return LONG ? P.g.nWin : it.n_list; };

  if (warp == 0) {
    // ------------------------------------------------------------- TMA loader
    if (lane == 0) {
      const Waiter wt = waiter(BASA_DEVERR_TIMEOUT_PRODUCER, true), drain = waiter(BASA_DEVERR_TIMEOUT_PRODUCER, false);
      const bool skipped0 = P.flags & BASA_FLAG_TEST_SKIP_FIRST_KEY_LOAD;
      int ring = 0, k_loads = 0, v_loads = 0, tile_no = 0;
      bool ok = true;
      for (int n = 0; ok; ++n) {
        if (!wt.wait(&c.rows_known[n & 1], (n >> 1) & 1)) break;
        const Item &it = c.item[n & 1];
        const int bh = it.bh;
        const int16_t *list = lists + (n & 1) * kMaxList;
        if (*reinterpret_cast<const volatile int *>(&it.n_cols) < 0) break;
        int n_cols = 0, n_windows = 0;
        const bool pooled = LONG && it.tile < P.n_pool_tiles;
        // This item's key tile of map (unit) or its value tile.
        auto load_rows = [&](bool is_v, int unit, uint8_t *dst, uint64_t *bar) {
          if (LONG) {
            const CUtensorMap *map = pooled ? (is_v ? &P.map_vp : &P.map_kp) : (is_v ? &P.map_vt : &P.map_kt);
            const int r = pooled ? it.tile * kTileRows : P.g.N + (it.tile - P.n_pool_tiles) * kTileRows;
            ptx::mbar_arrive_expect_tx(bar, kTileBytes);
            ptx::tma_load_3d(dst, map, bar, 0, r, unit);
            ptx::tma_load_3d(dst + kHalfBytes, map, bar, 64, r, unit);
          } else {
            const PlanTile &tile = P.plan.tile[it.tile];
            ptx::mbar_arrive_expect_tx(bar, uint32_t(tile.valid_rows) * 256u);
            load_window_tile(P.plan, P.g, is_v ? P.map_v : P.map_k, tile, it.keys.org[0], unit, dst, bar);
          }
        };
        for (int m = 0; ok && m < 2; ++m) {
          const int unit = 2 * bh + 1 - m;  // of q, k: map 2 first
          if (k_loads > 0) ok = wt.wait(&c.k_free, (k_loads - 1) & 1);
          if (!ok) break;
          load_rows(false, unit, row0, &c.k_full);
          ++k_loads;
          if (m == 0) {
            if (v_loads > 0) ok = wt.wait(&c.v_free, (v_loads - 1) & 1);
            if (!ok) break;
            load_rows(true, bh, row1, &c.v_full);
            ++v_loads;
            if (!(ok = wt.wait(&c.item_full[n & 1], (n >> 1) & 1))) break;
            n_cols = *reinterpret_cast<const volatile int *>(&it.n_cols);
            n_windows = windows_of(it);
          }
          QIter q;
          q_first(P, list, kMode, LONG ? it.chunk * P.chunk_tiles : 0, q);
          for (int j = 0; ok && j < n_cols; ++j, ++tile_no) {
            const PlanTile &tile = q_tile(P, q);
            for (int kv = 0; kv < 2; ++kv) {
              const int slot = ring % kSlots;
              ok = wt.wait(&c.empty[slot], ((ring / kSlots) & 1) ^ 1);
              if (!ok) break;
              ++ring;
              if (ring == 1 && skipped0) continue;
              uint8_t *dst = smem + kSmemRing + slot * kTileBytes;
              if (kv == 0) {  // q tile and its records (record buffer tile_no & 1, freed with the q slot)
                ptx::mbar_arrive_expect_tx(&c.full[slot], uint32_t(tile.valid_rows) * (256u + 16u));
                load_window_tile(P.plan, P.g, P.map_q, tile, q.org, unit, dst, &c.full[slot]);
                load_window_records(P.plan, P.g, P.map_rec, tile, q.org, unit, smem + kRec + (tile_no & 1) * kRecBytes,
                                    &c.full[slot]);
              } else {
                ptx::mbar_arrive_expect_tx(&c.full[slot], uint32_t(tile.valid_rows) * 256u);
                load_window_tile(P.plan, P.g, P.map_do, tile, q.org, bh, dst, &c.full[slot]);
              }
            }
            if (ok) q_next(P, list, kMode, n_windows, q);
          }
        }
        ptx::mbar_arrive(&c.item_empty[n & 1]);
      }
      // drain, as in the dq pass
      if (k_loads > 0) drain.wait(&c.k_full, (k_loads - 1) & 1);
      if (v_loads > 0) drain.wait(&c.v_full, (v_loads - 1) & 1);
      for (int i = max(0, ring - kSlots); i < ring; ++i)
        if (i > 0 || !skipped0) drain.wait(&c.full[i % kSlots], (i / kSlots) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      const Waiter wt = waiter(BASA_DEVERR_TIMEOUT_MMA, true), drain = waiter(BASA_DEVERR_TIMEOUT_MMA, false);
      const uint32_t r0 = kDescLoK | (ptx::smem_u32(row0) >> 4), r1 = kDescLoK | (ptx::smem_u32(row1) >> 4);
      const uint32_t ringK = kDescLoK | (ptx::smem_u32(smem + kSmemRing) >> 4);
      const uint32_t ringMn = kDescLoMn | (ptx::smem_u32(smem + kSmemRing) >> 4);
      auto slot_of = [](int item) { return uint32_t(item % kSlots) * kTileDesc; };
      // TMEM: S^T at 0, dP^T at 128, dV at 256, dK at 384. Compute group g owns query columns
      // [64 g, 64 g + 64) of S^T and dP^T; the dV and dK products are issued per group as soon
      // as that group's P^T or dS^T is in TMEM.
      const uint32_t tS = tmem, tDP = tmem + 128, tDV = tmem + 256, tDK = tmem + 384;
      int t0 = 0, maps = 0;  // query tiles and maps before this item
      for (int n = 0;; ++n) {
        if (!wt.wait(&c.item_full[n & 1], (n >> 1) & 1)) break;
        const int n_cols = c.item[n & 1].n_cols;
        ptx::mbar_arrive(&c.item_empty[n & 1]);
        if (n_cols < 0) break;
        const int total = 2 * n_cols;  // tiles [0, n_cols) are map 2's, [n_cols, 2 n_cols) map 1's
        auto scores = [&](int j) {     // S^T(j) = K q_j^T
          const int item = 2 * (t0 + j);
          if (!wt.wait(&c.full[item % kSlots], (item / kSlots) & 1)) return false;
          if ((j == 0 || j == n_cols) && !wt.wait(&c.k_full, (maps + (j > 0 ? 1 : 0)) & 1)) return false;
          ptx::tc_fence_after();
          issue_ss(tS, r0, ringK + slot_of(item));
          ptx::mma_commit(&c.s_full);
          if (j + 1 == n_cols || j + 1 == total) ptx::mma_commit(&c.k_free);
          return true;
        };
        auto dprob = [&](int j) {  // dP^T(j) = V g_j^T
          const int item = 2 * (t0 + j) + 1;
          if (!wt.wait(&c.full[item % kSlots], (item / kSlots) & 1)) return false;
          if (j == 0 && !wt.wait(&c.v_full, n & 1)) return false;
          ptx::tc_fence_after();
          issue_ss(tDP, r1, ringK + slot_of(item));
          ptx::mma_commit(&c.dp_full);
          if (j + 1 == total) ptx::mma_commit(&c.v_free);
          return true;
        };
        bool ok = scores(0) && dprob(0);
        for (int j = 0; ok && j < total; ++j) {
          const int t = t0 + j, qi = 2 * t, di = qi + 1;
          const bool map_start = j == 0 || j == n_cols, map_end = j + 1 == n_cols || j + 1 == total;
          // both groups have read the sums before (and rescaled dV) before a map's first P^T
          if (map_start) ok = wt.wait(&c.p_full[0], t & 1) && wt.wait(&c.p_full[1], t & 1);
          for (int g = 0; ok && g < 2; ++g) {
            ok = wt.wait(&c.p_full[g], t & 1);
            if (!ok) break;
            ptx::tc_fence_after();
            issue_ts_group(tDV, tS, ringMn + slot_of(di), g, j > 0 || g > 0);  // dV += P^T(j) g_j
          }
          if (!ok) break;
          ptx::mma_commit(&c.empty[di % kSlots]);
          if (!map_end && !(ok = scores(j + 1))) break;  // P^T(j) has been read by dV
          for (int g = 0; ok && g < 2; ++g) {
            ok = wt.wait(&c.ds_full[g], t & 1);
            if (!ok) break;
            ptx::tc_fence_after();
            issue_ts_group(tDK, tDP, ringMn + slot_of(qi), g, !map_start || g > 0);  // dK += dS^T(j) q_j
          }
          if (!ok) break;
          ptx::mma_commit(&c.empty[qi % kSlots]);
          if (map_end) ptx::mma_commit(&c.acc_full);
          if (j + 1 == n_cols) ok = scores(j + 1);  // map 1's key tile may still be on its way
          if (ok && j + 1 < total) ok = dprob(j + 1);
        }
        if (!ok) break;
        t0 += total;
        maps += 2;
      }
      // Every MMA this thread issued must finish before TMEM is freed.
      ptx::mma_commit(&c.drain);
      drain.wait(&c.drain, 0);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ------------------------------------------------------------- items
    const Waiter wt = waiter(BASA_DEVERR_TIMEOUT_PRODUCER, true);
    int n = 0;
    for (int id = blockIdx.x;; id += gridDim.x) {
      WorkItem x{};
      int chunk = 0, cols = -1;
      if (id < P.n_items) {
        if (LONG) {
          const uint32_t rest = uint32_t(id) / uint32_t(P.n_chunks);
          chunk = id - int(rest) * P.n_chunks;
          x.bh = int(rest / uint32_t(P.n_long_tiles));
          x.tile = int(rest) - x.bh * P.n_long_tiles;
          cols = min(P.chunk_tiles, P.q_tiles - chunk * P.chunk_tiles);
        } else {
          x = work_item(P, id);
          if (x.tile >= P.plan.type[x.wtype].n_tiles) continue;  // this window type has fewer tiles
          x.tile += P.plan.type[x.wtype].first_tile;
          cols = 1;
        }
      }
      if (!__all_sync(0xFFFFFFFFu, wt.wait(&c.item_empty[n & 1], ((n >> 1) & 1) ^ 1))) break;
      if (lane == 0) {  // the key and value tiles can load; how many query tiles there are follows
        Item &it = c.item[n & 1];
        it.n_cols = cols;
        it.bh = x.bh;
        it.tile = x.tile;
        it.chunk = chunk;
        for (int a = 0; a < 3; ++a) it.keys.org[0][a] = x.org[a];
        ptx::mbar_arrive(&c.rows_known[n & 1]);
      }
      if (!LONG && cols > 0) {
        // The query windows that see the key tile: w itself, then every window that routed
        // to w, in ascending id (ordered ballot compaction: a fixed order).
        int16_t *list = lists + (n & 1) * kMaxList;
        int count = 1;
        if (lane == 0) list[0] = int16_t(x.w);
        for (int w0 = 0; P.routed_k > 0 && w0 < P.g.nWin; w0 += 32) {
          const int u = w0 + lane;
          bool hit = false;
          if (u < P.g.nWin && u != x.w) {
            const int32_t *r = P.route + ((long long)x.bh * P.g.nWin + u) * P.routed_k;
            for (int i = 0; i < P.routed_k; ++i) hit |= r[i] == x.w;
          }
          const uint32_t hits = __ballot_sync(0xFFFFFFFFu, hit);
          if (hit) list[count + __popc(hits & ((1u << lane) - 1u))] = int16_t(u);
          count += __popc(hits);
        }
        __syncwarp();
        int total = 0;
        for (int i = lane; i < count; i += 32) {
          int org[3], t;
          origin_of(P.g, list[i], org, &t);
          total += P.plan.type[t].n_tiles;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
        if (lane == 0) {
          c.item[n & 1].n_cols = total;
          c.item[n & 1].n_list = count;
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&c.item_full[n & 1]);
      if (cols < 0) break;
      if (!LONG) {
        for (int r = lane; r < kTileRows; r += 32) {
          int t, y, l;
          int2 at = make_int2(-1, 0);
          if (tile_row_token(P.plan, P.g, P.plan.tile[x.tile], x.org, r, &t, &y, &l))
            at = make_int2((t * P.g.H + y) * P.g.W + l,
                           ((t / P.pt) * (P.g.H / P.ph) + y / P.ph) * (P.g.W / P.pw) + l / P.pw);
          places[(n & 1) * kTileRows + r] = at;
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&c.place_full[n & 1]);
      }
      ++n;
    }
    __syncwarp();
  } else if (warp == 11) {
    // ------------------------------------------------------------- the query tiles' unwritten rows
    const Waiter wt = waiter(BASA_DEVERR_TIMEOUT_PRODUCER, true);
    int ring = 0;
    bool ok = pads;
    for (int n = 0; ok; ++n) {
      ok = __all_sync(0xFFFFFFFFu, wt.wait(&c.item_full[n & 1], (n >> 1) & 1));
      if (!ok) break;
      const Item &it = c.item[n & 1];
      const int n_cols = it.n_cols;
      if (n_cols < 0) break;
      const int16_t *list = lists + (n & 1) * kMaxList;
      for (int m = 0; ok && m < 2; ++m) {
        QIter q;
        q_first(P, list, kMode, LONG ? it.chunk * P.chunk_tiles : 0, q);
        for (int j = 0; ok && j < n_cols; ++j) {
          const PlanTile &tile = q_tile(P, q);
          for (int kv = 0; ok && kv < 2; ++kv, ++ring) {
            const int slot = ring % kSlots;
            ok = __all_sync(0xFFFFFFFFu, wt.wait(&c.empty[slot], ((ring / kSlots) & 1) ^ 1));
            if (!ok) break;
            zero_unwritten_rows(smem + kSmemRing + slot * kTileBytes, tile.mask, lane);
            if (lane == 0) ptx::mbar_arrive(&c.full[slot]);
          }
          q_next(P, list, kMode, windows_of(it), q);
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&c.item_empty[n & 1]);
    }
  } else {
    // ------------------------------------------------------------- P and dS
    const int g = (warp - 2) / 4;  // column half
    const int sub = warp % 4;      // TMEM lane quarter this warp may access
    const int row = sub * 32 + lane;
    const uint32_t lane_off = uint32_t(sub * 32) << 16;
    const uint32_t col = uint32_t(64 * g);
    const uint32_t tS = tmem + lane_off + col, tDP = tmem + lane_off + 128 + col;
    const Waiter wt = waiter(BASA_DEVERR_TIMEOUT_SOFTMAX, true);
    const uint64_t sl2x2 = ptx::f2_pack(P.scale_log2, P.scale_log2);
    float *wrec = reinterpret_cast<float *>(smem + kColRec) + (warp - 2) * 128;  // [-L log2 e x 64 | -D x 64]
    const float4 *nl4 = reinterpret_cast<const float4 *>(wrec), *nd4 = reinterpret_cast<const float4 *>(wrec + 64);
    int t0 = 0;  // query tiles before this map
    bool ok = true;
    for (int n = 0; ok; ++n) {
      ok = __all_sync(0xFFFFFFFFu, wt.wait(&c.item_full[n & 1], (n >> 1) & 1));
      if (!ok) break;
      const Item &it = c.item[n & 1];
      const int n_cols = it.n_cols;
      if (n_cols < 0) break;
      // unrolled: the two maps' epilogues differ
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        QIter q;
        q_first(P, lists + (n & 1) * kMaxList, kMode, LONG ? it.chunk * P.chunk_tiles : 0, q);
        for (int j = 0; ok && j < n_cols; ++j) {
          const int t = t0 + j;
          ok = __all_sync(0xFFFFFFFFu, wt.wait(&c.s_full, t & 1));
          if (!ok) break;
          ptx::tc_fence_after();
          float p[64];
          tmem_ld64f(tS, p);
          {
            // This warp's 64 query records {-L log2 e, -D, ..}, one load per lane for two
            // columns, rewritten as two arrays that the loops below read four at a time.
            const float4 *r = reinterpret_cast<const float4 *>(smem + kRec + (t & 1) * kRecBytes) + col;
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
            const PlanTile &qt = q_tile(P, q);
            m0 = qt.mask[2 * g];
            m1 = qt.mask[2 * g + 1];
          }
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
          uint32_t pk[32];
          pack64(p, pk);
          ptx::tmem_st32(tS, pk);  // P^T (bf16) over the first half of this thread's S^T columns
          ptx::tmem_st_wait();
          ptx::tc_fence_before();
          ptx::mbar_arrive(&c.p_full[g]);
          ok = __all_sync(0xFFFFFFFFu, wt.wait(&c.dp_full, t & 1));
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
          pack64(dp, pk);
          ptx::tmem_st32(tDP, pk);  // dS^T (bf16) over the first half of this thread's dP^T columns
          ptx::tmem_st_wait();
          ptx::tc_fence_before();
          ptx::mbar_arrive(&c.ds_full[g]);
          q_next(P, lists + (n & 1) * kMaxList, kMode, windows_of(it), q);
        }
        t0 += n_cols;
        if (ok) ok = __all_sync(0xFFFFFFFFu, wt.wait(&c.acc_full, m));  // two maps an item
        if (ok && !LONG && m == 0) ok = __all_sync(0xFFFFFFFFu, wt.wait(&c.place_full[n & 1], (n >> 1) & 1));
        if (!ok) continue;
        if (!LONG && n == 0) ptx::grid_wait();  // the pooled keys' gradients
        ptx::tc_fence_after();
        const int bh = it.bh, unit = 2 * bh + 1 - m;  // of v; of k and dk
        const float neg_lambda = -__bfloat162float(P.lambda[bh % P.heads]);
        if (m == 0) {  // map 2's part of dV, before map 1 adds to it
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
        float x[64];
        const bool write = !*reinterpret_cast<volatile int *>(&c.abort);
        // dK of this map, then (with map 1) dV: to the tokens' rows, or to this chunk's sums
#pragma unroll
        for (int which = 0; which <= m; ++which) {
          tmem_ld64f(tmem + lane_off + (which ? 256 : 384) + col, x);
          if (which == m) {
            if (m == 0) ptx::tmem_st_wait();
            ptx::tc_fence_before();
          }
          if (which == 0) {
            const float f = m == 0 ? P.scale * neg_lambda : P.scale;
#pragma unroll
            for (int i = 0; i < 64; ++i) x[i] *= f;
          }
          if (LONG) {
            // float32 [dK of map 1 | dK of map 2 | dV][row][128]
            float *dst = P.part + ((((long long)bh * P.n_long_tiles + it.tile) * P.n_chunks + it.chunk) * 3 +
                                   (which ? 2 : 1 - m)) * (kTileRows * 128) + row * 128 + col;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (write)
                reinterpret_cast<float4 *>(dst)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
          } else {
            const int2 at = places[(n & 1) * kTileRows + row];
            if (P.n_pool > 0 && at.x >= 0) {
              // the pooled keys' gradient of this token's patch, spread evenly
              const long long pu = which ? 2ll * P.bh_count + bh : unit;
              const float4 *gp = reinterpret_cast<const float4 *>(P.dkvp + (pu * P.n_pool + at.y) * 128 + col);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float4 a = gp[i];
                x[4 * i] = fmaf(a.x, P.inv_patch, x[4 * i]);
                x[4 * i + 1] = fmaf(a.y, P.inv_patch, x[4 * i + 1]);
                x[4 * i + 2] = fmaf(a.z, P.inv_patch, x[4 * i + 2]);
                x[4 * i + 3] = fmaf(a.w, P.inv_patch, x[4 * i + 3]);
              }
            }
            const long long rows = P.g.N + P.n_text;
            store_rows64((which ? P.dv + bh * rows * 128 : P.dk + unit * rows * 128) + col, write ? at.x : -1, x, lane);
          }
        }
      }
      ptx::mbar_arrive(&c.item_empty[n & 1]);
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

// ----------------------------------------------------------------- host side
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

int most_tiles(const WindowPlan &plan) {
  int tiles = 0;
  for (int t = 0; t < 8; ++t) tiles = std::max<int>(tiles, plan.type[t].n_tiles);
  return tiles;
}

// Query (and key) tiles of p.heads units of v, those included that a window type lacks.
long long window_items(const basa_params &p, const WindowPlan &plan) {
  return (long long)p.B * p.heads * make_geo(p).nWin * most_tiles(plan);
}

// One CTA per SM at most. An `early` launch may start under the one before it.
basa_status run(void (*kernel)(BwdParams), uint32_t smem, BwdParams &P, long long items, bool early, cudaStream_t s) {
  const int sms = device_sm_count();
  if (sms <= 0) return BASA_ERR_CUDA;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return BASA_ERR_CUDA;
  P.n_items = int(items);
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(std::min<long long>(items, sms)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, P) == cudaSuccess ? BASA_OK : BASA_ERR_CUDA;
}

// Workspace: the layout of two maps, g (with a norm), the partial sums of dlambda and
// dweight, those of the dq pass (eight warps an item), its work counter.
struct DiffLayout {
  size_t g, part, dr, counter, total;
};
DiffLayout diff_layout(bool norm, const basa_params &p, const WindowPlan &plan) {
  DiffLayout L{};
  L.g = bwd_layout(p, plan, 2).total;
  L.part = L.g + (norm ? align256(size_t(p.B) * p.heads * p.T * p.H * p.W * p.head_dim * 2) : 0);
  L.dr = L.part + align256(diff_prep_workspace(p));
  L.counter = L.dr + align256(size_t(2 * window_items(p, plan)) * 8 * sizeof(float));
  L.total = L.counter + 256;
  return L;
}

}  // namespace

size_t diff_attn_bwd_bf16_workspace(bool norm, const basa_params &p) {
  static thread_local WindowPlan plan;  // large: kept off the stack
  if (build_window_plan(p, &plan) != BASA_OK) return 0;
  return diff_layout(norm, p, plan).total;
}

basa_status launch_diff_attn_bwd_bf16(const void *q, const void *k, const void *v, const void *kp, const void *vp,
                                      const int32_t *route_idx, const basa_diff_params &dp, const void *pre,
                                      const void *second, const float *lse, const void *dout, void *dq, void *dk,
                                      void *dv, void *dlambda, void *dweight, void *workspace, const basa_params &p,
                                      cudaStream_t s) {
  static thread_local BwdParams P;  // large: kept off the stack
  static thread_local WindowPlan plan;
  basa_status st = build_window_plan(p, &plan);
  if (st != BASA_OK) return st;
  const DiffLayout D = diff_layout(dp.weight != nullptr, p, plan);
  const long long items = window_items(p, plan);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  BwdLayout L;
  st = bwd_params(P, L, q, k, v, kp, vp, route_idx, dp.weight ? ws + D.g : dout, dq, dk, dv, ws, p, 2);
  if (st != BASA_OK) return st;
  const long long long_items = (long long)P.bh_count * L.n_long * L.n_chunks;
  if (2 * items >= (1ll << 30) || long_items >= (1ll << 30)) return BASA_ERR_UNSUPPORTED;
  P.lambda = static_cast<const __nv_bfloat16 *>(dp.lambda);
  P.heads = p.heads;
  P.dq = static_cast<__nv_bfloat16 *>(dq);
  P.dk = static_cast<__nv_bfloat16 *>(dk);
  P.dv = static_cast<__nv_bfloat16 *>(dv);
  P.dr = reinterpret_cast<float *>(ws + D.dr);
  P.next_item = reinterpret_cast<int *>(ws + D.counter);
  float *sums = reinterpret_cast<float *>(ws + D.part);
  st = launch_diff_prep(pre, second, lse, dout, dp, ws + D.g, reinterpret_cast<float4 *>(ws), nullptr, sums, P.next_item, p,
                        s);
  if (st != BASA_OK) return st;
  const bool any_long = long_items > 0;
  if (any_long && (st = run(diff_dkv_kernel<true>, kDkvSmem, P, long_items, false, s)) != BASA_OK) return st;
  if ((st = run(diff_dq_kernel, kDqSmem, P, 2 * items, any_long, s)) != BASA_OK) return st;
  if (any_long && (st = launch_bwd_reduce(P, L, dk, dv, p, 2, s)) != BASA_OK) return st;
  if ((st = run(diff_dkv_kernel<false>, kDkvSmem, P, items, any_long, s)) != BASA_OK) return st;
  return launch_diff_sums(sums, P.dr, 2 * P.g.nWin * P.max_tiles * 8, dp, dlambda, dweight, p, s);
}

}  // namespace basa
