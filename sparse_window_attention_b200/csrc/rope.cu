// Rotary positions along the t, y and x axes of the token grid (HBM-bound), with the
// per-head RMS norm of queries and keys before the rotation, and the gradients of both.
//
//   xn = x * rsqrt(mean(x^2) + eps) * weight        (a tensor without weight: xn = x)
//   (y_a, y_b) = (xn_a cos - xn_b sin, xn_a sin + xn_b cos)  for each channel pair (a, b),
// the angle of pair i of an axis that owns m channels being position * theta^(-2 i / m).
//
// What bounds it: one read and one write of the tensors. A row's cos and sin depend on
// the token only, so a thread keeps those of its channels in registers and walks the
// (batch, head) units of its row: the angle tables are read once per row and not once
// per head. A thread owns two 16-byte chunks of a row, half a head apart, so both
// pairings (adjacent channels, or channel i with i + d/2) find their partners in the
// thread's own registers, and the norm's sum of squares is a few shuffles. The arithmetic
// is in packed float32 pairs, two channel pairs an instruction, with the norm's weight
// multiplied into the cos and sin beforehand: element by element, and with the unit's
// index divided out for every load, the kernel was bound by its instructions (half of
// all issue slots, 4.6 TB/s). Measured: q, k, v of 24 heads and 16384 + 512 rows (623 MB in
// and out) 107 us, 5.8 of the 6.55 TB/s that a copy reaches; forward and backward of 12
// heads and 32760 rows (1.41 GB) 247 us, 5.7 TB/s; one row 3.4 us, a launch's latency.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "basa_internal.h"
#include "sm100_ptx.cuh"

namespace basa {
namespace {

constexpr int kRopeThreads = 256;
// Units a thread loads before it works on the first: 2 * 16 bytes each (backward: twice that).
constexpr int kUnrollFwd = 4, kUnrollBwd = 3, kUnrollCopy = 8;

struct RopeTensorArgs {
  const void *x, *dy, *weight;
  void *y;
  float *part;  // backward: per-block partial weight gradients [blocks][d]
  long long xs[3], ys[3], ds[3];  // element strides (batch, head, row)
  int heads, rows, first_row, rotate;
  int first_block, row_blocks, groups, group_units;  // blocks = row_blocks x groups of (batch, head) units
};

struct RopeArgs {
  RopeTensorArgs t[BASA_ROPE_MAX_TENSORS];
  int n;
  const float2 *table;
  int N, H, W, B;
  int nt, nh, nw;                     // pairs of each axis
  long long tab_y, tab_x, tab_text;   // offsets of the tables (the t axis starts at 0)
  float eps;
};

template <typename T>
struct Vec {
  static constexpr int n = 16 / sizeof(T);
};

// A thread's channels: VEC pairs (a, b), held as VEC / 2 packed float32 pairs of a's and
// of b's. With HALVES the first chunk holds the a's and the second the b's; with adjacent
// pairs each 32-bit word of bfloat16 (or each two floats) is a pair.
template <bool HALVES>
__device__ __forceinline__ void unpack(const uint4 &u, const uint4 &v, uint64_t *a, uint64_t *b, const __nv_bfloat16 *) {
  const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
  const auto lo = [](uint32_t x) { return __uint_as_float(x << 16); };
  const auto hi = [](uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = HALVES ? ptx::f2_pack(lo(w[i]), hi(w[i])) : ptx::f2_pack(lo(w[2 * i]), lo(w[2 * i + 1]));
    b[i] = HALVES ? ptx::f2_pack(lo(w[4 + i]), hi(w[4 + i])) : ptx::f2_pack(hi(w[2 * i]), hi(w[2 * i + 1]));
  }
}
template <bool HALVES>
__device__ __forceinline__ void unpack(const uint4 &u, const uint4 &v, uint64_t *a, uint64_t *b, const float *) {
  const auto f = [](uint32_t x) { return __uint_as_float(x); };
  a[0] = HALVES ? ptx::f2_pack(f(u.x), f(u.y)) : ptx::f2_pack(f(u.x), f(u.z));
  a[1] = HALVES ? ptx::f2_pack(f(u.z), f(u.w)) : ptx::f2_pack(f(v.x), f(v.z));
  b[0] = HALVES ? ptx::f2_pack(f(v.x), f(v.y)) : ptx::f2_pack(f(u.y), f(u.w));
  b[1] = HALVES ? ptx::f2_pack(f(v.z), f(v.w)) : ptx::f2_pack(f(v.y), f(v.w));
}
// The only rounding: float32 results to the element type, to nearest even.
template <bool HALVES>
__device__ __forceinline__ void pack(const uint64_t *a, const uint64_t *b, uint4 &u, uint4 &v, const __nv_bfloat16 *) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a0, a1, b0, b1;
    ptx::f2_unpack(a[i], a0, a1);
    ptx::f2_unpack(b[i], b0, b1);
    w[HALVES ? i : 2 * i] = HALVES ? ptx::pack_bf16x2(a0, a1) : ptx::pack_bf16x2(a0, b0);
    w[HALVES ? 4 + i : 2 * i + 1] = HALVES ? ptx::pack_bf16x2(b0, b1) : ptx::pack_bf16x2(a1, b1);
  }
  u = make_uint4(w[0], w[1], w[2], w[3]);
  v = make_uint4(w[4], w[5], w[6], w[7]);
}
template <bool HALVES>
__device__ __forceinline__ void pack(const uint64_t *a, const uint64_t *b, uint4 &u, uint4 &v, const float *) {
  float x[8];  // a0 a1 a2 a3 b0 b1 b2 b3
  ptx::f2_unpack(a[0], x[0], x[1]);
  ptx::f2_unpack(a[1], x[2], x[3]);
  ptx::f2_unpack(b[0], x[4], x[5]);
  ptx::f2_unpack(b[1], x[6], x[7]);
  const auto w = [&](int i) { return __float_as_uint(x[i]); };
  u = HALVES ? make_uint4(w(0), w(1), w(2), w(3)) : make_uint4(w(0), w(4), w(1), w(5));
  v = HALVES ? make_uint4(w(4), w(5), w(6), w(7)) : make_uint4(w(2), w(6), w(3), w(7));
}

// Pair index of a thread's i-th pair (chunk column c).
template <int D, int VEC, bool HALVES>
__device__ __forceinline__ int pair_index(int c, int i) {
  if (HALVES) return VEC * c + i;
  return i < VEC / 2 ? VEC / 2 * c + i : D / 4 + VEC / 2 * c + (i - VEC / 2);
}

__device__ __forceinline__ uint64_t f2_both(float x) { return ptx::f2_pack(x, x); }
__device__ __forceinline__ uint64_t f2_neg(uint64_t x) { return x ^ 0x8000000080000000ull; }
__device__ __forceinline__ float f2_sum(uint64_t x) {
  float a, b;
  ptx::f2_unpack(x, a, b);
  return a + b;
}

// Sum over the LPR lanes that share a row (aligned groups of lanes).
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

// cos and sin of a thread's pairs in row `row` of the key sequence. Pairs behind the axes'
// channels are left as they are.
template <int D, int VEC, bool HALVES>
__device__ __forceinline__ void load_angles(const RopeArgs &a, int row, int c, uint64_t *cs, uint64_t *sn) {
  const int P = a.nt + a.nh + a.nw;
  const int t = row / (a.H * a.W), y = (row / a.W) % a.H, x = row % a.W;
  float co[VEC], si[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int p = pair_index<D, VEC, HALVES>(c, i);
    long long at;
    if (row >= a.N) at = a.tab_text + (long long)(row - a.N) * P + p;
    else if (p < a.nt) at = (long long)t * a.nt + p;
    else if (p < a.nt + a.nh) at = a.tab_y + (long long)y * a.nh + (p - a.nt);
    else at = a.tab_x + (long long)x * a.nw + (p - a.nt - a.nh);
    float2 e = make_float2(1.f, 0.f);
    if (p < P) e = __ldg(a.table + at);
    co[i] = e.x;
    si[i] = e.y;
  }
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) {
    cs[i] = ptx::f2_pack(co[2 * i], co[2 * i + 1]);
    sn[i] = ptx::f2_pack(si[2 * i], si[2 * i + 1]);
  }
}

// The walk over a group's (batch, head) units: element offsets without a division a step.
struct UnitWalk {
  long long at, step, wrap;
  int h, heads;
  __device__ UnitWalk(const long long *stride, int unit, int n_heads) {
    heads = n_heads;
    h = unit % n_heads;
    at = (unit / n_heads) * stride[0] + h * stride[1];
    step = stride[1];
    wrap = stride[0] - (n_heads - 1) * stride[1];
  }
  __device__ __forceinline__ long long next() {
    const long long here = at;
    at += ++h == heads ? wrap : step;
    if (h == heads) h = 0;
    return here;
  }
};

// One CTA = (tensor, block of 256 / LPR rows, group of (batch, head) units); a thread
// owns chunk column c of one row and walks the group's units.
//
// The backward turns dy back (g = R^T dy) and, behind a norm with xh = x * r,
// r = rsqrt(mean(x^2) + eps):  dweight = sum g * xh,
// dx = r * (g w - xh * mean(g w * xh)). Each block sums its rows' weight gradients in a
// fixed order; rope_dweight_kernel adds the blocks, so nothing depends on timing.
template <typename T, int D, bool HALVES, bool BWD>
__global__ void __launch_bounds__(kRopeThreads, BWD ? 2 : 3) rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int VEC = Vec<T>::n, LPR = D / 2 / VEC, ROWS = kRopeThreads / LPR, H2 = VEC / 2;
  int ti = 0;
  while (ti + 1 < a.n && int(blockIdx.x) >= a.t[ti + 1].first_block) ++ti;
  const RopeTensorArgs &t = a.t[ti];
  const int blk = int(blockIdx.x) - t.first_block;
  const int group = blk / t.row_blocks;
  const int c = threadIdx.x % LPR;
  const int r = (blk % t.row_blocks) * ROWS + threadIdx.x / LPR;
  const bool valid = r < t.rows;
  const bool norm = t.weight != nullptr;
  const int u0 = group * t.group_units, n_units = min(t.group_units, a.B * t.heads - u0);
  const T *kind = nullptr;
  // A row past the end works on zeros (shuffles want every lane) and writes nothing.
  const long long row = valid ? r : 0;
  const T *x0 = static_cast<const T *>(t.x) + row * t.xs[2] + c * VEC;
  T *y0 = static_cast<T *>(t.y) + row * t.ys[2] + c * VEC;
  const T *d0 = static_cast<const T *>(t.dy) + row * t.ds[2] + c * VEC;
  UnitWalk yw(t.ys, u0, t.heads);
  const auto load = [valid](const T *p, uint4 &u, uint4 &v) {
    u = v = make_uint4(0, 0, 0, 0);
    if (!valid) return;
    u = __ldcs(reinterpret_cast<const uint4 *>(p));
    v = __ldcs(reinterpret_cast<const uint4 *>(p + D / 2));
  };
  const auto store = [&](const uint4 &u, const uint4 &v) {
    T *p = y0 + yw.next();
    if (valid) {
      *reinterpret_cast<uint4 *>(p) = u;
      *reinterpret_cast<uint4 *>(p + D / 2) = v;
    }
  };

  if (!norm && !t.rotate) {  // a tensor that is only laid out: its bits
    const T *s0 = BWD ? d0 : x0;
    UnitWalk sw(BWD ? t.ds : t.xs, u0, t.heads);
    for (int u = 0; u < n_units; u += kUnrollCopy) {
      uint4 p[kUnrollCopy], q[kUnrollCopy];
#pragma unroll
      for (int k = 0; k < kUnrollCopy; ++k)
        if (u + k < n_units) load(s0 + sw.next(), p[k], q[k]);
#pragma unroll
      for (int k = 0; k < kUnrollCopy; ++k)
        if (u + k < n_units) store(p[k], q[k]);
    }
    return;
  }

  uint64_t cs[H2], sn[H2], wa[H2], wb[H2];
#pragma unroll
  for (int i = 0; i < H2; ++i) {
    cs[i] = wa[i] = wb[i] = f2_both(1.f);
    sn[i] = f2_both(0.f);
  }
  if (t.rotate) load_angles<D, VEC, HALVES>(a, t.first_row + int(row), c, cs, sn);
  if (norm) {
    const uint4 *wp = reinterpret_cast<const uint4 *>(t.weight);
    unpack<HALVES>(__ldg(wp + c), __ldg(wp + LPR + c), wa, wb, kind);
  }
  UnitWalk xw(t.xs, u0, t.heads);

  if constexpr (!BWD) {
    // y_a = x_a (w_a cos) - x_b (w_b sin), y_b = x_a (w_a sin) + x_b (w_b cos), times r
    uint64_t ac[H2], as[H2], bc[H2], bs[H2];
#pragma unroll
    for (int i = 0; i < H2; ++i) {
      ac[i] = ptx::fmul2(wa[i], cs[i]);
      as[i] = ptx::fmul2(wa[i], sn[i]);
      bc[i] = ptx::fmul2(wb[i], cs[i]);
      bs[i] = f2_neg(ptx::fmul2(wb[i], sn[i]));
    }
    for (int u = 0; u < n_units; u += kUnrollFwd) {
      uint4 p[kUnrollFwd], q[kUnrollFwd];
#pragma unroll
      for (int k = 0; k < kUnrollFwd; ++k)
        if (u + k < n_units) load(x0 + xw.next(), p[k], q[k]);
#pragma unroll
      for (int k = 0; k < kUnrollFwd; ++k) {
        if (u + k >= n_units) break;
        uint64_t xa[H2], xb[H2];
        unpack<HALVES>(p[k], q[k], xa, xb, kind);
        if (norm) {
          uint64_t ss = f2_both(0.f);
#pragma unroll
          for (int i = 0; i < H2; ++i) ss = ptx::ffma2(xb[i], xb[i], ptx::ffma2(xa[i], xa[i], ss));
          const uint64_t rms = f2_both(rsqrtf(row_sum<LPR>(f2_sum(ss)) * (1.f / D) + a.eps));
#pragma unroll
          for (int i = 0; i < H2; ++i) {
            xa[i] = ptx::fmul2(xa[i], rms);
            xb[i] = ptx::fmul2(xb[i], rms);
          }
        }
#pragma unroll
        for (int i = 0; i < H2; ++i) {
          const uint64_t ya = ptx::ffma2(xa[i], ac[i], ptx::fmul2(xb[i], bs[i]));
          xb[i] = ptx::ffma2(xa[i], as[i], ptx::fmul2(xb[i], bc[i]));
          xa[i] = ya;
        }
        pack<HALVES>(xa, xb, p[k], q[k], kind);
        store(p[k], q[k]);
      }
    }
  } else {
    uint64_t dwa[H2], dwb[H2];
#pragma unroll
    for (int i = 0; i < H2; ++i) dwa[i] = dwb[i] = f2_both(0.f);
    UnitWalk dw(t.ds, u0, t.heads);
    for (int u = 0; u < n_units; u += kUnrollBwd) {
      uint4 p[kUnrollBwd], q[kUnrollBwd], gp[kUnrollBwd], gq[kUnrollBwd];
#pragma unroll
      for (int k = 0; k < kUnrollBwd; ++k) {
        if (u + k >= n_units) break;
        if (norm) load(x0 + xw.next(), p[k], q[k]);
        load(d0 + dw.next(), gp[k], gq[k]);
      }
#pragma unroll
      for (int k = 0; k < kUnrollBwd; ++k) {
        if (u + k >= n_units) break;
        uint64_t ga[H2], gb[H2];
        unpack<HALVES>(gp[k], gq[k], ga, gb, kind);
#pragma unroll
        for (int i = 0; i < H2; ++i) {  // the turn by -angle
          const uint64_t g = ptx::ffma2(ga[i], cs[i], ptx::fmul2(gb[i], sn[i]));
          gb[i] = ptx::ffma2(gb[i], cs[i], ptx::fmul2(ga[i], f2_neg(sn[i])));
          ga[i] = g;
        }
        if (norm) {
          uint64_t xa[H2], xb[H2], ss = f2_both(0.f), dot = f2_both(0.f);
          unpack<HALVES>(p[k], q[k], xa, xb, kind);
#pragma unroll
          for (int i = 0; i < H2; ++i) ss = ptx::ffma2(xb[i], xb[i], ptx::ffma2(xa[i], xa[i], ss));
          const float rms = rsqrtf(row_sum<LPR>(f2_sum(ss)) * (1.f / D) + a.eps);
          const uint64_t rms2 = f2_both(rms);
#pragma unroll
          for (int i = 0; i < H2; ++i) {
            const uint64_t pa = ptx::fmul2(ga[i], xa[i]), pb = ptx::fmul2(gb[i], xb[i]);
            dwa[i] = ptx::ffma2(pa, rms2, dwa[i]);
            dwb[i] = ptx::ffma2(pb, rms2, dwb[i]);
            dot = ptx::ffma2(pb, wb[i], ptx::ffma2(pa, wa[i], dot));
          }
          // dx = r g w - x r^3 mean(g w x)
          const float mean = row_sum<LPR>(f2_sum(dot)) * (1.f / D);
          const uint64_t kx = f2_both(-(rms * rms) * (rms * mean));
#pragma unroll
          for (int i = 0; i < H2; ++i) {
            ga[i] = ptx::ffma2(xa[i], kx, ptx::fmul2(ptx::fmul2(ga[i], wa[i]), rms2));
            gb[i] = ptx::ffma2(xb[i], kx, ptx::fmul2(ptx::fmul2(gb[i], wb[i]), rms2));
          }
        }
        pack<HALVES>(ga, gb, gp[k], gq[k], kind);
        store(gp[k], gq[k]);
      }
    }
    if (t.part == nullptr) return;  // the same in the whole block
    __shared__ float red[kRopeThreads / 32][D];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
    for (int i = 0; i < H2; ++i) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float v[2];
        ptx::f2_unpack(half ? dwb[i] : dwa[i], v[0], v[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int o = LPR; o < 32; o <<= 1) v[e] += __shfl_xor_sync(0xFFFFFFFFu, v[e], o);
          const int pair = pair_index<D, VEC, HALVES>(c, 2 * i + e);
          if (lane < LPR) red[warp][HALVES ? pair + half * (D / 2) : 2 * pair + half] = v[e];
        }
      }
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < kRopeThreads / 32; ++k) s += red[k][threadIdx.x];
      t.part[(long long)blk * D + threadIdx.x] = s;
    }
  }
}

// dweight[col] = sum over the blocks of their partial sums: one CTA per (tensor, 32
// columns), 32 slices of the blocks, added in a fixed order.
struct DweightArgs {
  const float *part[BASA_ROPE_MAX_TENSORS];
  void *dst[BASA_ROPE_MAX_TENSORS];
  int blocks[BASA_ROPE_MAX_TENSORS];
  int d;
};

template <typename T>
__global__ void __launch_bounds__(1024) rope_dweight_kernel(const __grid_constant__ DweightArgs a) {
  __shared__ float red[32][33];
  const int ti = blockIdx.y, col = blockIdx.x * 32 + threadIdx.x % 32, slice = threadIdx.x / 32;
  const float *p = a.part[ti] + col;
  float s = 0.f;
#pragma unroll 8
  for (int b = slice; b < a.blocks[ti]; b += 32) s += p[(long long)b * a.d];
  red[slice][threadIdx.x % 32] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) sum += red[k][threadIdx.x];
    static_cast<T *>(a.dst[ti])[col] = T(sum);
  }
}

// cos and sin tables: [T][nt], [H][nh], [W][nw], [n_text][nt + nh + nw]. The angle is a
// float64 product reduced in float64, so far positions keep their fraction of a turn;
// a few thousand entries, computed once for a grid.
struct TableArgs {
  float2 *table;
  const float *text_pos;  // nullable: text rows are not turned
  double log_theta, origin[3], step[3];
  int ext[3], pairs[3], n_text;
};

__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ TableArgs a) {
  long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x, left = i;
  double pos = 0.0;
  int axis = 0, p = 0;
  bool found = false;
  for (int k = 0; k < 3 && !found; ++k) {
    const long long n = (long long)a.ext[k] * a.pairs[k];
    if (left < n) {
      axis = k;
      p = int(left % a.pairs[k]);
      pos = a.origin[k] + a.step[k] * double(left / a.pairs[k]);
      found = true;
    } else {
      left -= n;
    }
  }
  if (!found) {
    const int P = a.pairs[0] + a.pairs[1] + a.pairs[2];
    if (left >= (long long)a.n_text * P) return;
    const long long row = left / P;
    p = int(left % P);
    while (p >= a.pairs[axis]) p -= a.pairs[axis++];
    if (a.text_pos) pos = double(a.text_pos[3 * row + axis]);
  }
  double s, c;
  sincos(pos * exp(-a.log_theta * double(p) / double(a.pairs[axis])), &s, &c);
  a.table[i] = make_float2(float(c), float(s));
}

template <typename T, int D, bool HALVES>
void run_rope(const RopeArgs &a, bool bwd, unsigned blocks, cudaStream_t s) {
  if (bwd) rope_kernel<T, D, HALVES, true><<<blocks, kRopeThreads, 0, s>>>(a);
  else rope_kernel<T, D, HALVES, false><<<blocks, kRopeThreads, 0, s>>>(a);
}

template <typename T, int D>
void run_rope(const RopeArgs &a, bool bwd, bool halves, unsigned blocks, cudaStream_t s) {
  if (halves) run_rope<T, D, true>(a, bwd, blocks, s);
  else run_rope<T, D, false>(a, bwd, blocks, s);
}

// Blocks of a tensor list: rows in blocks of 256 threads, and the (batch, head) units
// in as many groups as it takes to give the GPU about kTargetBlocks blocks: 8 for each of
// 148 SMs, where 3 (backward: 2) run at a time, so that the last ones leave an SM idle for a
// small part of the whole, and a block still walks enough units for its cos and sin. Twice as
// many took 107 us at 24 heads of 16384 + 512 rows and 34 at 4096 + 512, four times as many
// 104 and 37; this many 107 and 32. Depends on the shapes only, so the order of the weight
// gradients' sums does too. Returns the block count (< 0: too many).
constexpr long long kTargetBlocks = 8 * 148;
bool has_rows(const basa_rope_tensor &t, const basa_params &p) { return p.B > 0 && t.heads > 0 && t.rows > 0; }
long long plan_blocks(int n, const basa_rope_tensor *t, const basa_params &p, RopeArgs *a) {
  const int rows_per_block = kRopeThreads / (p.head_dim / 2 / (p.dtype == BASA_BF16 ? 8 : 4));
  long long row_blocks = 0;
  for (int i = 0; i < n; ++i)
    if (has_rows(t[i], p)) row_blocks += (t[i].rows + rows_per_block - 1) / rows_per_block;
  long long blocks = 0;
  a->n = 0;
  for (int i = 0; i < n; ++i) {
    if (!has_rows(t[i], p)) continue;
    RopeTensorArgs &r = a->t[a->n++];
    const long long units = (long long)p.B * t[i].heads;
    const long long want = std::min(units, std::max(1ll, kTargetBlocks / row_blocks));
    r.row_blocks = (t[i].rows + rows_per_block - 1) / rows_per_block;
    r.group_units = int((units + want - 1) / want);
    r.groups = int((units + r.group_units - 1) / r.group_units);
    r.first_block = int(std::min(blocks, (1ll << 31) - 1));
    blocks += (long long)r.row_blocks * r.groups;
  }
  return blocks < (1ll << 31) ? blocks : -1;
}

}  // namespace

size_t rope_table_bytes(const basa_rope_params &rp, const basa_params &p) {
  const size_t entries = size_t(p.T) * (rp.dt / 2) + size_t(p.H) * (rp.dh / 2) + size_t(p.W) * (rp.dw / 2) +
                         size_t(p.n_text) * ((rp.dt + rp.dh + rp.dw) / 2);
  return entries * sizeof(float2);
}

basa_status launch_rope_table(const float *text_pos, float *table, const basa_rope_params &rp, const basa_params &p,
                              cudaStream_t s) {
  TableArgs a{};
  a.table = reinterpret_cast<float2 *>(table);
  a.text_pos = text_pos;
  a.log_theta = log(rp.theta);
  const double origin[3] = {rp.t0, rp.y0, rp.x0}, step[3] = {rp.t_step, rp.y_step, rp.x_step};
  const int ext[3] = {p.T, p.H, p.W}, pairs[3] = {rp.dt / 2, rp.dh / 2, rp.dw / 2};
  for (int k = 0; k < 3; ++k) {
    a.origin[k] = origin[k];
    a.step[k] = step[k];
    a.ext[k] = ext[k];
    a.pairs[k] = pairs[k];
  }
  a.n_text = p.n_text;
  const size_t entries = rope_table_bytes(rp, p) / sizeof(float2);
  if (entries == 0) return BASA_OK;
  const size_t blocks = (entries + 255) / 256;
  if (blocks >= (size_t(1) << 31)) return BASA_ERR_UNSUPPORTED;
  rope_table_kernel<<<unsigned(blocks), 256, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? BASA_OK : BASA_ERR_CUDA;
}

size_t rope_bwd_workspace(int n, const basa_rope_tensor *t, const basa_params &p) {
  RopeArgs a{};
  if (plan_blocks(n, t, p, &a) < 0) return 0;
  size_t rows = 0;
  for (int i = 0, j = 0; i < n; ++i) {
    if (!has_rows(t[i], p)) continue;
    if (t[i].dweight) rows += size_t(a.t[j].row_blocks) * a.t[j].groups;
    ++j;
  }
  return rows * p.head_dim * sizeof(float);
}

basa_status launch_rope(int n, const basa_rope_tensor *t, const float *table, float eps, void *workspace, bool bwd,
                        const basa_rope_params &rp, const basa_params &p, cudaStream_t s) {
  RopeArgs a{};
  const long long blocks = plan_blocks(n, t, p, &a);
  if (blocks < 0) return BASA_ERR_UNSUPPORTED;
  a.table = reinterpret_cast<const float2 *>(table);
  a.N = p.T * p.H * p.W;
  a.H = p.H;
  a.W = p.W;
  a.B = p.B;
  a.nt = rp.dt / 2;
  a.nh = rp.dh / 2;
  a.nw = rp.dw / 2;
  a.tab_y = (long long)p.T * a.nt;
  a.tab_x = a.tab_y + (long long)p.H * a.nh;
  a.tab_text = a.tab_x + (long long)p.W * a.nw;
  a.eps = eps;
  DweightArgs d{};
  d.d = p.head_dim;
  int n_dw = 0;
  float *part = static_cast<float *>(workspace);
  for (int i = 0, j = 0; i < n; ++i) {
    const basa_rope_tensor &u = t[i];
    int part_blocks = 0;
    if (has_rows(u, p)) {
      RopeTensorArgs &r = a.t[j++];
      r.x = u.x;
      r.y = u.y;
      r.dy = u.dy;
      r.weight = u.weight;
      const int ext[3] = {p.B, u.heads, u.rows};
      for (int k = 0; k < 3; ++k) {  // an axis with one entry is never stepped
        r.xs[k] = ext[k] > 1 ? u.x_stride[k] : 0;
        r.ys[k] = ext[k] > 1 ? u.y_stride[k] : 0;
        r.ds[k] = ext[k] > 1 ? u.dy_stride[k] : 0;
      }
      r.heads = u.heads;
      r.rows = u.rows;
      r.first_row = u.first_row;
      r.rotate = u.rotate && a.nt + a.nh + a.nw > 0;
      if (bwd && u.dweight) {
        part_blocks = r.row_blocks * r.groups;
        r.part = part;
      }
    }
    if (bwd && u.dweight) {  // a part without rows gets a gradient of zero
      d.part[n_dw] = part;
      d.dst[n_dw] = u.dweight;
      d.blocks[n_dw++] = part_blocks;
      part += size_t(part_blocks) * p.head_dim;
    }
  }
  if (blocks > 0) {
    const bool halves = rp.pairs == BASA_ROPE_PAIRS_HALVES;
    const unsigned b = unsigned(blocks);
    if (p.dtype == BASA_BF16) {
      if (p.head_dim == 128) run_rope<__nv_bfloat16, 128>(a, bwd, halves, b, s);
      else run_rope<__nv_bfloat16, 64>(a, bwd, halves, b, s);
    } else {
      if (p.head_dim == 128) run_rope<float, 128>(a, bwd, halves, b, s);
      else run_rope<float, 64>(a, bwd, halves, b, s);
    }
    if (cudaGetLastError() != cudaSuccess) return BASA_ERR_CUDA;
  }
  if (n_dw > 0) {
    const dim3 grid(unsigned(p.head_dim / 32), unsigned(n_dw));
    if (p.dtype == BASA_BF16) rope_dweight_kernel<__nv_bfloat16><<<grid, 1024, 0, s>>>(d);
    else rope_dweight_kernel<float><<<grid, 1024, 0, s>>>(d);
    if (cudaGetLastError() != cudaSuccess) return BASA_ERR_CUDA;
  }
  return BASA_OK;
}

}  // namespace basa
