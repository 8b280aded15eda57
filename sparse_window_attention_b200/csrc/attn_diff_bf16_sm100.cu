// Differential attention forward, bfloat16, head_dim 128, for sm_100a:
//   a = softmax(q1 K1^T / sqrt(d)) V - lambda softmax(q2 K2^T / sqrt(d)) V
//   out = gain * weight * a * rsqrt(mean(a^2) + eps)       (no weight: out = a)
// over the key list of the shifted-window attention, [own window | routed | pooled | text].
//
// A work item is (batch * head, window, 128-row query tile); its two maps run as the two
// softmax groups of the window kernel run two query tiles: key tiles come in pairs K1, K2
// and one V tile serves both maps, so a key step is three tile loads and four 128 x 128 x
// 128 products. Each map is normalised by its own sum only at the end, so both products
// with V are needed (P1 / l1 - lambda P2 / l2 is not known while the sums run); the
// difference and the norm are taken from TMEM in float32 and rounded once. For a backward
// a and O2 are stored too (rounded relative to their own sizes: O1 follows as their sum,
// where a difference of two rounded maps would lose what cancels in it).
//
// The grid is one CTA per SM, each going through its items with everything but the
// softmax running ahead: while the softmax warps finish an item (difference, norm, stores)
// the loader has the next item's queries and first keys under way and the MMA thread its
// first scores. One CTA per item spent 9.3 us of an item on its start and end beside 1.9 us
// a key step (14 steps at 32 x 32 windows, 7 at 16 x 16).
//
// What bounds it: the softmax's chain (scores read, maximum, exponentials, P stored), about
// 3.5k cycles a key step where the four products take 2.1k. Measured at 12 heads (24 maps),
// a graph of ten calls replayed (calls one by one from Python in brackets): a 128 x 128 grid,
// 32 x 32 windows, 1280 + 512 keys 357 us, 0.62 of the tensor cores' measured rate (385, 0.58,
// as a long run meets the power cap); 64 x 64, 16 x 16 windows, 832 keys 66 us (68), 0.39, as 384
// items are three rounds of 148 for the work of 2.6; 21 x 30 x 52, 6 heads, 234-token windows, 4
// routed 369 us (373), 0.44: 117-row tiles.
//
// Roundings: P to bfloat16 for the products with V, at most 2^-8 of each, while the sums it is
// divided by take it in float32: outputs are off 0.002 of their size, of which their own
// rounding is 0.0017.
//
// Warp roles, TMEM (S1, S2, O1, O2) and bounded waits are those of the window kernel:
//   warp 0      loads: publishes the item (windows, routes), then its Q1, Q2 and the
//               K1, K2, V stream through a 5-slot ring that runs on across items
//   warp 1      issues the MMAs
//   warps 2, 3  the next item's column masks, and its rows' tokens (1.4-2.5k and 1.4k cycles
//               of plan lookups that the softmax warps, which bound a step, are spared);
//               warp 2 also zeroes the rows of the V tiles that no load writes: P is 0 there,
//               but what an earlier item left may be infinite or NaN. (The loader doing it
//               cost 20%, doing it for every tile 4%.)
//   warps 4-11  softmax group g for map g, a thread per query row; then group g finishes
//               columns [64 g, 64 g + 64) of the output rows
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>

#include "attn_fwd_sm100.cuh"

namespace basa {
namespace {

using namespace sm100;

constexpr int kThreads = 384;
constexpr int kStages = 5;
constexpr uint32_t kSmemQ = 0;                  // Q1, Q2
constexpr uint32_t kSmemRing = 2 * kTileBytes;  // K1, K2, V ring
constexpr uint32_t kSmemCtrl = kSmemRing + kStages * kTileBytes;
constexpr uint32_t kCtrlBytes = 896;
constexpr int kMaskTable = 36;                          // key tiles whose column masks are tabled
constexpr uint32_t kSmemMask = kSmemCtrl + kCtrlBytes;  // two items' tables
constexpr uint32_t kSmemRows = kSmemMask + 2 * kMaskTable * 16;  // 1 KB: the rows' tokens, then their sums
constexpr uint32_t kSmemBytes = kSmemRows + 1024;
static_assert(kSmemBytes <= 227u * 1024u, "shared memory above the 227 KB a CTA may hold");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSoftmax = 256;  // threads of the two softmax groups

struct Item {
  int n_kt;  // key steps; < 0: there are no more items
  int bh, tile;
  KeyList keys;
};

struct Ctrl {
  uint64_t full[kStages], empty[kStages];
  uint64_t q_full, q_empty, s_full[2], p_full[2], o_full, item_full[2], item_empty[2], mask_full[2], tok_full, o_read, drain;
  uint32_t tmem_base;
  int abort;
  Item item[2];
};
static_assert(sizeof(Ctrl) <= kCtrlBytes, "control block too large");

__global__ void __launch_bounds__(kThreads, 1) attn_diff_bf16_kernel(const __grid_constant__ AttnParams P) {
  extern __shared__ __align__(1024) uint8_t smem[];  // whole swizzle atoms: no room for a manual alignment
  Ctrl &c = *reinterpret_cast<Ctrl *>(smem + kSmemCtrl);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  // Some window tile has rows that no load writes.
  const bool pads = P.plan.zero_fill;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&c.full[i], pads ? 2 : 1);
      ptx::mbar_init(&c.empty[i], 1);
    }
    ptx::mbar_init(&c.q_full, 1);
    ptx::mbar_init(&c.q_empty, 1);
    ptx::mbar_init(&c.o_full, 1);
    ptx::mbar_init(&c.tok_full, 1);
    ptx::mbar_init(&c.o_read, kSoftmax);
    for (int g = 0; g < 2; ++g) {
      ptx::mbar_init(&c.s_full[g], 1);
      ptx::mbar_init(&c.p_full[g], 128);
      ptx::mbar_init(&c.item_full[g], 1);
      ptx::mbar_init(&c.item_empty[g], kSoftmax + (P.all_full ? 1 : 2));
      ptx::mbar_init(&c.mask_full[g], 1);
    }
    ptx::mbar_init(&c.drain, 1);
    c.abort = 0;
    ptx::fence_mbar_init();
  }
  if (pads) {
    uint4 *z = reinterpret_cast<uint4 *>(smem + kSmemRing);
    for (uint32_t i = threadIdx.x; i < kStages * kTileBytes / 16; i += kThreads) z[i] = make_uint4(0, 0, 0, 0);
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

  if (warp == 0) {
    // ------------------------------------------------------------- TMA loader
    if (lane == 0) {
      Waiter wt{&c.abort, P.dev_err, P.timeout_ns, BASA_DEVERR_TIMEOUT_PRODUCER, true};
      Waiter drain{&c.abort, P.dev_err, P.timeout_ns, BASA_DEVERR_TIMEOUT_PRODUCER, false};
      int n = 0, ring = 0;  // items and ring slots so far
      bool ok = true, skipped0 = false;
      for (int id = blockIdx.x; ok && id < P.n_items; id += gridDim.x) {
        const int tile = id % P.q_tiles, w = (id / P.q_tiles) % P.g.nWin, bh = id / (P.q_tiles * P.g.nWin);
        int ot, oy, ox, wtype;
        window_origin(P.g, w, &ot, &oy, &ox, &wtype);
        if (tile >= P.plan.type[wtype].n_tiles) continue;  // this window type has fewer query tiles
        if (!(ok = wt.wait(&c.item_empty[n & 1], ((n >> 1) & 1) ^ 1))) break;
        Item &it = c.item[n & 1];
        it.bh = bh;
        it.tile = P.plan.type[wtype].first_tile + tile;
        it.keys.tile0 = it.keys.ntile = 0;
        it.keys.wtype[0] = wtype;
        it.keys.org[0][0] = ot; it.keys.org[0][1] = oy; it.keys.org[0][2] = ox;
        fill_routes(P, it.keys, bh, w);
        int n_kt = 0;
        for (int s = 0; s <= P.routed_k + 2; ++s) n_kt += seg_tiles(P, it.keys, s);
        it.n_kt = n_kt;
        ptx::mbar_arrive(&c.item_full[n & 1]);

        if (!(ok = wt.wait(&c.q_empty, (n & 1) ^ 1))) break;
        // a tile's TMA boxes deliver 256 bytes per valid row (two 128-byte halves)
        const PlanTile &qt = P.plan.tile[it.tile];
        ptx::mbar_arrive_expect_tx(&c.q_full, uint32_t(qt.valid_rows) * 512u);
        for (int g = 0; g < 2; ++g)
          load_window_tile(P.plan, P.g, P.map_q, qt, it.keys.org[0], 2 * bh + g, smem + kSmemQ + g * kTileBytes,
                           &c.q_full);
        ++n;
        const int item_no = n - 1;
        KeyIter key = first_key(P, it.keys);
        for (int j = 0; ok && j < n_kt; ++j) {
          for (int kv = 0; kv < 3; ++kv, ++ring) {
            const int slot = ring % kStages;
            if (!(ok = wt.wait(&c.empty[slot], ((ring / kStages) & 1) ^ 1))) break;
            if (ring == 0 && (P.flags & BASA_FLAG_TEST_SKIP_FIRST_KEY_LOAD)) {
              skipped0 = true;
              continue;
            }
            ptx::mbar_arrive_expect_tx(&c.full[slot], key_tile_bytes(P, it.keys, key));
            // the second arrival: warp 2's where it zeroes rows, see there
            if (pads && !(kv == 2 && item_no > 0 && j < kStages)) ptx::mbar_arrive(&c.full[slot]);
            load_key_tile(P, it.keys, key, kv == 2, kv == 2 ? bh : 2 * bh + kv, smem + kSmemRing + slot * kTileBytes,
                          &c.full[slot]);
          }
          if (ok) advance(P, it.keys, key);
        }
      }
      if (ok && wt.wait(&c.item_empty[n & 1], ((n >> 1) & 1) ^ 1)) {
        c.item[n & 1].n_kt = -1;
        ptx::mbar_arrive(&c.item_full[n & 1]);
      }
      // Drain: wait for the copies still in flight (immediate when all were consumed).
      if (n > 0) drain.wait(&c.q_full, (n - 1) & 1);
      for (int i = max(0, ring - kStages); i < ring; ++i)
        if (i > 0 || !skipped0) drain.wait(&c.full[i % kStages], (i / kStages) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      Waiter wt{&c.abort, P.dev_err, P.timeout_ns, BASA_DEVERR_TIMEOUT_MMA, true};
      Waiter drain{&c.abort, P.dev_err, P.timeout_ns, BASA_DEVERR_TIMEOUT_MMA, false};
      // low descriptor halves of the query tiles and the ring slots
      const uint32_t sQ = kDescLoK | (ptx::smem_u32(smem + kSmemQ) >> 4);
      const uint32_t sRk = kDescLoK | (ptx::smem_u32(smem + kSmemRing) >> 4);
      const uint32_t sRv = kDescLoMn | (ptx::smem_u32(smem + kSmemRing) >> 4);
      int ring = 0, step = 0;  // ring slots and key steps before this item
      // S_g = Q_g K_g^T with the key tile in ring slot `item`
      auto scores = [&](int g, int item) {
        const int slot = item % kStages;
        if (!wt.wait(&c.full[slot], (item / kStages) & 1)) return false;
        ptx::tc_fence_after();
        issue_ss(tmem + 128 * g, sQ + g * kTileDesc, sRk + slot * kTileDesc);
        ptx::mma_commit(&c.s_full[g]);
        ptx::mma_commit(&c.empty[slot]);
        return true;
      };
      for (int n = 0;; ++n) {
        if (!wt.wait(&c.item_full[n & 1], (n >> 1) & 1)) break;
        const int n_kt = c.item[n & 1].n_kt;
        ptx::mbar_arrive(&c.item_empty[n & 1]);
        if (n_kt < 0) break;
        // Scores over the previous item's P: its last products with V were issued before.
        bool ok = wt.wait(&c.q_full, n & 1) && scores(0, ring) && scores(1, ring + 1);
        if (ok && n_kt == 1) ptx::mma_commit(&c.q_empty);
        for (int j = 0; ok && j < n_kt; ++j) {
          const int vi = ring + 3 * j + 2, vslot = vi % kStages, parity = (step + j) & 1;
          const uint32_t vaddr = sRv + vslot * kTileDesc;
          const bool more = j + 1 < n_kt;
          ok = wt.wait(&c.full[vslot], (vi / kStages) & 1) && wt.wait(&c.p_full[0], parity);
          // both groups read both of the previous item's outputs
          if (ok && j == 0 && n > 0) ok = wt.wait(&c.o_read, (n - 1) & 1);
          if (!ok) break;
          ptx::tc_fence_after();
          issue_ts(tmem + 256, tmem, vaddr, j > 0);
          if (more && !(ok = scores(0, vi + 1))) break;
          if (!(ok = wt.wait(&c.p_full[1], parity))) break;
          ptx::tc_fence_after();
          issue_ts(tmem + 384, tmem + 128, vaddr, j > 0);
          ptx::mma_commit(&c.empty[vslot]);
          if (more && !(ok = scores(1, vi + 2))) break;
          if (j + 2 == n_kt) ptx::mma_commit(&c.q_empty);  // the last scores are issued
        }
        if (!ok) break;
        ptx::mma_commit(&c.o_full);
        ring += 3 * n_kt;
        step += n_kt;
      }
      // Every MMA this thread issued must finish before TMEM is freed.
      ptx::mma_commit(&c.drain);
      drain.wait(&c.drain, 0);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------- column masks
    Waiter wt{&c.abort, P.dev_err, P.timeout_ns, BASA_DEVERR_TIMEOUT_SOFTMAX, true};
    int step = 0;  // key steps before this item
    for (int n = 0; !P.all_full; ++n) {
      // an item is published once the softmax is through with the table of two items before
      if (!__all_sync(0xFFFFFFFFu, wt.wait(&c.item_full[n & 1], (n >> 1) & 1))) break;
      const Item &it = c.item[n & 1];
      if (it.n_kt < 0) break;
      for (int j = lane; j < min(it.n_kt, kMaskTable); j += 32) {
        KeyIter t{0, j};
        while (t.seg <= P.routed_k + 2 && t.t >= seg_tiles(P, it.keys, t.seg)) {
          t.t -= seg_tiles(P, it.keys, t.seg);
          ++t.seg;
        }
        uint32_t mk[4];
        key_tile_mask(P, it.keys, t, mk);
        reinterpret_cast<uint4 *>(smem + kSmemMask)[(n & 1) * kMaskTable + j] = make_uint4(mk[0], mk[1], mk[2], mk[3]);
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&c.mask_full[n & 1]);
      const int n_kt = it.n_kt;
      bool ok = true;
      // V_0 .. V_4 take each ring slot once: after them a slot's unwritten rows hold zeros or
      // rows of this item. (The first item finds the ring zeroed.)
      for (int j = 0; ok && pads && n > 0 && j < min(n_kt, kStages); ++j) {
        const int ring = 3 * (step + j) + 2, slot = ring % kStages;
        ok = __all_sync(0xFFFFFFFFu, wt.wait(&c.empty[slot], ((ring / kStages) & 1) ^ 1));
        if (!ok) break;
        const uint4 t = reinterpret_cast<const uint4 *>(smem + kSmemMask)[(n & 1) * kMaskTable + j];
        const uint32_t mk[4] = {t.x, t.y, t.z, t.w};
        // pooled and text tiles are written whole; rows past their end read as zero
        zero_unwritten_rows(smem + kSmemRing + slot * kTileBytes, mk, lane);
        if (lane == 0) ptx::mbar_arrive(&c.full[slot]);
      }
      if (!ok) break;
      step += n_kt;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&c.item_empty[n & 1]);
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------- the rows' tokens (-1: none)
    Waiter wt{&c.abort, P.dev_err, P.timeout_ns, BASA_DEVERR_TIMEOUT_SOFTMAX, true};
    for (int n = 0;; ++n) {
      bool ok = wt.wait(&c.item_full[n & 1], (n >> 1) & 1);
      // their place holds the previous item's sums until that is finished
      if (ok && n > 0) ok = wt.wait(&c.item_empty[(n - 1) & 1], ((n - 1) >> 1) & 1);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      const Item &it = c.item[n & 1];
      if (it.n_kt < 0) break;
      for (int r = lane; r < kTileRows; r += 32) {
        int t, y, x;
        const bool token = tile_row_token(P.plan, P.g, P.plan.tile[it.tile], it.keys.org[0], r, &t, &y, &x);
        reinterpret_cast<int *>(smem + kSmemRows)[r] = token ? (t * P.g.H + y) * P.g.W + x : -1;
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&c.tok_full);
    }
  } else {
    // ------------------------------------------------------------- softmax
    const int g = (warp - 4) / 4;
    const int sub = warp % 4;  // TMEM lane quarter this warp may access
    const int row = sub * 32 + lane;
    const uint32_t lane_off = uint32_t(sub * 32) << 16;
    const uint32_t tS = tmem + lane_off + g * 128, tO = tmem + lane_off + 256 + g * 128;
    Waiter wt{&c.abort, P.dev_err, P.timeout_ns, BASA_DEVERR_TIMEOUT_SOFTMAX, true};
    const float sl2 = P.scale_log2;
    float *sums = reinterpret_cast<float *>(smem + kSmemRows);  // [2][128]
    int step = 0;
    for (int n = 0;; ++n) {
      bool ok = __all_sync(0xFFFFFFFFu, wt.wait(&c.item_full[n & 1], (n >> 1) & 1));
      const Item &it = c.item[n & 1];
      const int n_kt = ok ? it.n_kt : -1;
      ok = n_kt >= 0;
      const uint4 *masks = reinterpret_cast<const uint4 *>(smem + kSmemMask) + (n & 1) * kMaskTable;
      if (ok && !P.all_full) ok = __all_sync(0xFFFFFFFFu, wt.wait(&c.mask_full[n & 1], (n >> 1) & 1));
      const int bh = ok ? it.bh : 0;
      const float lam = __bfloat162float(P.lambda[bh % P.heads]);
      float m = -INFINITY, l = 0.f;
      KeyIter key{0, 0};  // past the table only
      for (int j = 0; ok && j < n_kt; ++j) {
        ok = __all_sync(0xFFFFFFFFu, wt.wait(&c.s_full[g], (step + j) & 1));
        if (!ok) break;
        ptx::tc_fence_after();
        uint32_t s[128];
        ptx::tmem_ld128(tS, s);
        ptx::tmem_ld_wait(s);
        if (P.all_full) {
        } else if (j < kMaskTable) {
          const uint4 mt = masks[j];
          if ((mt.x & mt.y & mt.z & mt.w) != 0xFFFFFFFFu) {
            const uint32_t mask[4] = {mt.x, mt.y, mt.z, mt.w};
            apply_mask(s, mask);
          }
        } else {
          uint32_t mask[4];
          if (!key_tile_mask(P, it.keys, key, mask)) apply_mask(s, mask);
        }
        const float m_tile = row_max(s) * sl2;
        const bool need = m_tile > m + kRescaleLog2;  // always true on the first tile (m = -inf)
        const float m_new = need ? m_tile : m;
        const float alpha = need ? ptx::ex2(m - m_new) : 1.0f;
        const float sum = exp2_row_packed(s, sl2, m_new);
        l = l * alpha + sum;
        m = m_new;
        // P row -> TMEM over the first 64 columns of S; the MMA that overwrites S
        // next is issued after the P V that reads it.
        ptx::tmem_st64(tS, s);
        if (j > 0 && __any_sync(0xFFFFFFFFu, need)) {
          const uint64_t a2 = ptx::f2_pack(alpha, alpha);
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            uint32_t r[32];
            ptx::tmem_ld32(tO + cc * 32, r);
            ptx::tmem_ld_wait(r);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float lo, hi;
              ptx::f2_unpack(ptx::fmul2(ptx::f2_pack(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), a2), lo, hi);
              r[i] = __float_as_uint(lo);
              r[i + 1] = __float_as_uint(hi);
            }
            ptx::tmem_st32(tO + cc * 32, r);
          }
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(&c.p_full[g]);
        if (j + 1 >= kMaskTable) {
          if (j + 1 == kMaskTable) {  // past the table: walk the stream from its start once
            key = first_key(P, it.keys);
            for (int t = 0; t < kMaskTable; ++t) advance(P, it.keys, key);
          } else {
            advance(P, it.keys, key);
          }
        }
      }
      step += n_kt;
      if (ok) ok = __all_sync(0xFFFFFFFFu, wt.wait(&c.o_full, n & 1) && wt.wait(&c.tok_full, n & 1));
      const int tok = ok ? reinterpret_cast<const int *>(smem + kSmemRows)[row] : -1;
      // Leaving is a common decision (no items left, or a wait has expired): the barriers
      // from here on are met by all 256 threads or by none.
      if (ptx::named_barrier_any(1, kSoftmax, !ok)) break;

      // Group g: columns [64 g, 64 g + 64) of O1 / l1 - lambda O2 / l2 (a TMEM lane holds
      // the same query row of both). The sums cross over in shared memory, twice.
      sums[g * kTileRows + row] = 1.0f / l;
      ptx::named_barrier(1, kSoftmax);
      const float i0 = sums[row], i1 = sums[kTileRows + row];
      // an item cut short has set abort before: nothing of it is stored
      const int row_to = *reinterpret_cast<volatile int *>(&c.abort) ? -1 : tok;
      const long long at = (long long)bh * P.g.N * 128 + 64 * g;
      ptx::tc_fence_after();
      float a[64], o2[64];
      float ss = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int cc = 2 * g + h;
        uint32_t r0[32], r1[32];
        ptx::tmem_ld32(tmem + lane_off + 256 + cc * 32, r0);
        ptx::tmem_ld32(tmem + lane_off + 384 + cc * 32, r1);
        ptx::tmem_ld_wait(r0);
        ptx::tmem_ld_wait(r1);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          o2[32 * h + i] = __uint_as_float(r1[i]) * i1;
          a[32 * h + i] = fmaf(-lam, o2[32 * h + i], __uint_as_float(r0[i]) * i0);
          ss = fmaf(a[32 * h + i], a[32 * h + i], ss);
        }
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(&c.o_read);  // the next item's products with V may start
      if (P.second != nullptr) store_rows64(P.second + at, row_to, o2, lane);
      if (P.pre != nullptr) store_rows64(P.pre + at, row_to, a, lane);
      // log-sum-exp of this row's map: m and l are in base 2 of the scaled scores
      if (row_to >= 0 && P.lse != nullptr)
        P.lse[(long long)(2 * bh + g) * P.g.N + tok] = (m + log2f(l)) * 0.6931471805599453f;
      if (P.norm_weight != nullptr) {
        ptx::named_barrier(1, kSoftmax);
        sums[g * kTileRows + row] = ss;
        ptx::named_barrier(1, kSoftmax);
        const float f = rsqrtf((sums[row] + sums[kTileRows + row]) * (1.0f / 128.0f) + P.eps) * P.gain;
        const uint4 *w4 = reinterpret_cast<const uint4 *>(P.norm_weight + 64 * g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 u = __ldg(w4 + i);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[8 * i + 2 * e] *= f * __uint_as_float(w[e] << 16);
            a[8 * i + 2 * e + 1] *= f * __uint_as_float(w[e] & 0xFFFF0000u);
          }
        }
      }
      ptx::mbar_arrive(&c.item_empty[n & 1]);  // the item and the sums are read
      store_rows64(P.out + at, row_to, a, lane);
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

basa_status launch_diff_attn_bf16(const void *q, const void *k, const void *v, const void *kp, const void *vp,
                                  const int32_t *route_idx, const basa_diff_params &dp, void *out, void *pre,
                                  void *second, float *lse, const basa_params &p, cudaStream_t s) {
  static thread_local AttnParams P;  // large: kept off the stack
  basa_status st = window_params(P, q, k, v, kp, vp, route_idx, nullptr, lse, BASA_KEYS_ALL, p, 2);
  if (st != BASA_OK) return st;
  P.lambda = static_cast<const __nv_bfloat16 *>(dp.lambda);
  P.norm_weight = static_cast<const __nv_bfloat16 *>(dp.weight);
  P.gain = dp.gain;
  P.eps = dp.eps;
  P.heads = p.heads;
  P.out = static_cast<__nv_bfloat16 *>(out);
  P.pre = static_cast<__nv_bfloat16 *>(pre);
  P.second = static_cast<__nv_bfloat16 *>(second);
  for (int t = 0; t < 8; ++t) P.q_tiles = std::max<int>(P.q_tiles, P.plan.type[t].n_tiles);
  const long long items = (long long)p.B * p.heads * P.g.nWin * P.q_tiles;
  if (items >= (1ll << 30)) return BASA_ERR_UNSUPPORTED;
  P.n_items = int(items);
  const int sms = device_sm_count();
  if (sms <= 0) return BASA_ERR_CUDA;
  if (cudaFuncSetAttribute(attn_diff_bf16_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) !=
      cudaSuccess)
    return BASA_ERR_CUDA;
  attn_diff_bf16_kernel<<<unsigned(std::min<long long>(items, sms)), kThreads, kSmemBytes, s>>>(P);
  return cudaGetLastError() == cudaSuccess ? BASA_OK : BASA_ERR_CUDA;
}

}  // namespace basa
