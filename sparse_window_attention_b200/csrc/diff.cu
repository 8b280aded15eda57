// Differential attention around the attention kernels (HBM-bound passes):
//
//   a = O1 - lambda O2,   out = gain * weight * a * rsqrt(mean(a^2) + eps)   (no weight: out = a)
//
// combine   takes the maps' float32 outputs (or their partial results over key ranges,
//           joined by log-sum-exp) to out: the text-query rows.
// prepare   the start of the backward: with xh = a r and G = gain * dout
//             dweight = sum G xh,  g = r (G w - xh mean(G w xh)),
//             D2 = g . O2,  D1 = g . O1 = g . a + lambda D2,  dlambda = -sum g . O2;
//           the maps' outputs are rounded here, so D is a little off the rows' true sum
//           R = sum_j P dP. The dq pass, which has P in float32, finds by how much: sum_j dS
//           = R - D. And where a stands in for the true one, g . a is known (mean(G w xh) d
//           eps r^2), but with the true one, R1 - lambda R2, it is something else, so with
//           c = O2 . a / (a . a + d eps) what is summed is
//             g . O2 - c (g . a) + c mean(G w xh) d eps r^2  +  (1 + c lambda) dR2 - c dR1
//           (dR of the dq pass, weighted by the records). This c takes out what a's error e
//           does to g . O2 through mean(G w e): r^3 / d (a . O2) (G w . e), as r^2 = d / (a . a
//           + d eps). Maps that are nearly alike would otherwise leave dlambda 5% off, and a sum
//           over rows that cancels 2%. (Without d eps, c grows without bound where a is small
//           against sqrt(eps), where g hardly depends on a, and dlambda is up to half off.)
//           g goes on as the output gradient of both maps (map 2's factor -lambda is put
//           on its dq, dK and dV sums), D1 and D2 as their rows' softmax corrections.
// reduce    the blocks' partial sums of dlambda and dweight, in a fixed order.
#include <cuda_bf16.h>

#include <algorithm>

#include "basa_internal.h"
#include "sm100_ptx.cuh"

namespace basa {
namespace {

constexpr int kDiffThreads = 256;

// Eight elements as they lie in memory, and unpacked.
template <typename T>
struct Raw {
  uint4 u[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T *p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < int(sizeof(T) / 2); ++i) r.u[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
  return r;
}
__device__ __forceinline__ void unpack8(const Raw<__nv_bfloat16> &r, float *v) {
  const uint4 u = r.u[0];
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack8(const Raw<float> &r, float *v) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[4 * i] = __uint_as_float(r.u[i].x);
    v[4 * i + 1] = __uint_as_float(r.u[i].y);
    v[4 * i + 2] = __uint_as_float(r.u[i].z);
    v[4 * i + 3] = __uint_as_float(r.u[i].w);
  }
}
template <typename T>
__device__ __forceinline__ void load8(const T *p, float *v) {
  unpack8(load_raw(p), v);
}
// Rounds v to the element type (once, to nearest even) and stores it; v then holds the
// values that were stored.
__device__ __forceinline__ void store8(__nv_bfloat16 *p, float *v) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
    v[2 * i] = __uint_as_float(r[i] << 16);
    v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(r[0], r[1], r[2], r[3]);
}
__device__ __forceinline__ void store8(float *p, float *v) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }

// Sum over the LPR lanes of a row (aligned groups of lanes).
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

struct CombineArgs {
  const float *part;  // [n_splits][B][2 heads][rows][d]
  const float *lse;   // [n_splits][B][2 heads][rows] (n_splits > 1)
  const void *lambda, *weight;
  void *out;          // [B][heads][rows][d]
  int n_splits, heads;
  long long rows, units;  // rows of a unit; B * heads
  float gain, eps;
};

// A map's row from its key-range splits: sum_i exp(L_i - max L) O_i / sum_i exp(L_i - max L).
template <int D>
__device__ __forceinline__ void joined_row(const CombineArgs &a, long long map_row, int c, float *v) {
  const long long stride = 2 * a.units * a.rows;
  if (a.n_splits == 1) {
    load8(a.part + map_row * D + 8 * c, v);
    return;
  }
  float m = -INFINITY, tot = 0.f;
  for (int i = 0; i < a.n_splits; ++i) m = fmaxf(m, __ldg(a.lse + i * stride + map_row));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  for (int i = 0; i < a.n_splits; ++i) {
    const float w = expf(__ldg(a.lse + i * stride + map_row) - m);
    float x[8];
    load8(a.part + (i * stride + map_row) * D + 8 * c, x);
    tot += w;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = fmaf(w, x[k], v[k]);
  }
  const float inv = 1.0f / tot;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= inv;
}

// D / 8 lanes per row, 8 channels a lane.
template <typename T, int D>
__global__ void __launch_bounds__(kDiffThreads) diff_combine_kernel(const __grid_constant__ CombineArgs a) {
  constexpr int LPR = D / 8, ROWS = kDiffThreads / LPR;
  const long long r = (long long)blockIdx.x * ROWS + threadIdx.x / LPR;
  const int c = threadIdx.x % LPR;
  const bool valid = r < a.units * a.rows;
  const long long unit = valid ? r / a.rows : 0, row = valid ? r % a.rows : 0;
  float x[8], o2[8];
  joined_row<D>(a, (2 * unit) * a.rows + row, c, x);
  joined_row<D>(a, (2 * unit + 1) * a.rows + row, c, o2);
  const float lam = to_float(static_cast<const T *>(a.lambda)[unit % a.heads]);
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = fmaf(-lam, o2[i], x[i]);
    ss = fmaf(x[i], x[i], ss);
  }
  if (a.weight) {
    const float f = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + a.eps) * a.gain;
    float w[8];
    load8(static_cast<const T *>(a.weight) + 8 * c, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= f * w[i];
  }
  if (!valid) return;
  store8(static_cast<T *>(a.out) + (unit * a.rows + row) * D + 8 * c, x);
}

// Rows of one (batch, head) that a block of the backward's start goes through: a few
// passes, so that the partial sums are a small part of the traffic and the blocks still
// fill the GPU (12 heads of 4096 rows: 768 blocks).
constexpr int kPrepRows = 64;

struct PrepArgs {
  const void *pre, *second, *dout, *lambda, *weight;
  const float *lse;  // [units][2][rows]
  void *g;           // [units][rows][d]; unused without weight (g = dout)
  float4 *rec;       // nullable: records {-L log2 e, -D, weight of dR in -dlambda, 0} [units][2][rows]
  float *drow;       // nullable: D alone, [units][2][rows]
  int *zeros;        // nullable: [units][n_zeros], set to 0
  float *part;       // [blocks][1 + d]: sum g . O2, then the weight's gradient
  int heads, blocks_per_unit, n_zeros;
  long long rows;
  float gain, eps;
};

template <typename T, int D>
__global__ void __launch_bounds__(kDiffThreads) diff_prep_kernel(const __grid_constant__ PrepArgs a) {
  constexpr int LPR = D / 8, ROWS = kDiffThreads / LPR;
  __shared__ float red[kDiffThreads / 32][D + 1];
  const long long unit = blockIdx.x / a.blocks_per_unit;
  const long long r0 = (long long)(blockIdx.x % a.blocks_per_unit) * kPrepRows;
  const long long r1 = min(a.rows, r0 + kPrepRows);
  if (a.zeros != nullptr && r0 == 0)
    for (int i = threadIdx.x; i < a.n_zeros; i += kDiffThreads) a.zeros[unit * a.n_zeros + i] = 0;
  const int c = threadIdx.x % LPR;
  const float lam = to_float(static_cast<const T *>(a.lambda)[unit % a.heads]);
  float w[8], dw[8], dl = 0.f;
  if (a.weight) load8(static_cast<const T *>(a.weight) + 8 * c, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = 0.f;
  // A pass's rows are loaded while the one before is worked on: a row's sums are five chains
  // of shuffles, which the loads waited for otherwise (19 us against 17 at 12 heads of 4096
  // rows of bfloat16, caches cold; 50 MB are 7.7 us, the rest is instructions: 58% of issue).
  Raw<T> rx{}, ro{}, rg{};
  auto load_rows = [&](long long r) {
    rx = ro = rg = Raw<T>{};
    if (r >= r1) return;
    const long long at = (unit * a.rows + r) * D + 8 * c;
    rx = load_raw(static_cast<const T *>(a.pre) + at);
    ro = load_raw(static_cast<const T *>(a.second) + at);
    rg = load_raw(static_cast<const T *>(a.dout) + at);
  };
  load_rows(r0 + threadIdx.x / LPR);
  for (long long base = r0; base < r1; base += ROWS) {  // the same trip count in every lane (shuffles)
    const long long r = base + threadIdx.x / LPR;
    const bool valid = r < r1;
    const long long at = (unit * a.rows + r) * D + 8 * c;
    float x[8], o2[8], g[8];
    unpack8(rx, x);
    unpack8(ro, o2);
    unpack8(rg, g);
    load_rows(r + ROWS);
    float ga = 0.f, c2 = 0.f;  // this lane's part of g . a; c
    if (a.weight) {
      float ss = 0.f, so = 0.f, dot = 0.f, xh[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(x[i], x[i], ss);
        so = fmaf(x[i], o2[i], so);
      }
      ss = row_sum<LPR>(ss);
      so = row_sum<LPR>(so);
      c2 = so / fmaf(float(D), a.eps, ss);
      const float rms = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xh[i] = x[i] * rms;
        g[i] *= a.gain;
        dw[i] = fmaf(g[i], xh[i], dw[i]);
        g[i] *= w[i];
        dot = fmaf(g[i], xh[i], dot);
      }
      dot = row_sum<LPR>(dot) * (1.f / D);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = rms * (g[i] - xh[i] * dot);
      if (c == 0) ga = dot * (float(D) * a.eps * rms * rms);
      dl = fmaf(c2, ga, dl);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) ga = fmaf(g[i], x[i], ga);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) dl = fmaf(g[i], fmaf(-c2, x[i], o2[i]), dl);
    // D1 and D2 are those of the rounded g, which the products with V see
    float d2 = 0.f, da = ga, g0[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) g0[i] = g[i];
    if (a.weight && valid) store8(static_cast<T *>(a.g) + at, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      d2 = fmaf(g[i], o2[i], d2);
      da = fmaf(g[i] - g0[i], x[i], da);
    }
    d2 = row_sum<LPR>(d2);
    da = row_sum<LPR>(da);
    if (valid && c < 2) {
      const long long m = (2 * unit + c) * a.rows + r;
      const float d = c == 0 ? fmaf(lam, d2, da) : d2;
      if (a.rec) a.rec[m] = make_float4(-a.lse[m] * 1.4426950408889634f, -d, c == 0 ? -c2 : fmaf(c2, lam, 1.f), 0.f);
      if (a.drow) a.drow[m] = d;
    }
  }
  // lanes with the same channels, then the warps, in order
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) dl += __shfl_xor_sync(0xFFFFFFFFu, dl, o);
  if (lane == 0) red[warp][D] = dl;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) dw[i] += __shfl_xor_sync(0xFFFFFFFFu, dw[i], o);
    if (lane < LPR) red[warp][8 * c + i] = dw[i];
  }
  __syncthreads();
  if (threadIdx.x <= D) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kDiffThreads / 32; ++k) s += red[k][threadIdx.x];
    a.part[(long long)blockIdx.x * (D + 1) + (threadIdx.x == D ? 0 : 1 + threadIdx.x)] = s;
  }
}

// One CTA per head: dlambda[h] = -(its blocks' sums, and the dq pass's); then one per 32
// channels of dweight.
struct SumArgs {
  const float *part, *dr;  // dr nullable: [B][heads][dr_per_unit] sums of weighted dR
  void *dlambda, *dweight;
  int B, heads, blocks_per_unit, dr_per_unit, d;
};

template <typename T>
__global__ void __launch_bounds__(1024) diff_sum_kernel(const __grid_constant__ SumArgs a) {
  __shared__ float red[32][33];
  ptx::grid_launch_dependents();
  const int lane = threadIdx.x % 32, slice = threadIdx.x / 32;
  const long long stride = a.d + 1;
  float s = 0.f;
  if (int(blockIdx.x) < a.heads) {
    const int n = a.B * a.blocks_per_unit;
    for (int i = threadIdx.x; i < n; i += 1024) {
      const long long unit = (long long)(i / a.blocks_per_unit) * a.heads + blockIdx.x;
      s += __ldcg(a.part + (unit * a.blocks_per_unit + i % a.blocks_per_unit) * stride);
    }
    for (int b = 0; a.dr != nullptr && b < a.B; ++b) {
      const float *p = a.dr + ((long long)b * a.heads + blockIdx.x) * a.dr_per_unit;
      for (int i = threadIdx.x; i < a.dr_per_unit; i += 1024) s += __ldcg(p + i);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (lane == 0) red[slice][0] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
      float t = 0.f;
#pragma unroll
      for (int k = 0; k < 32; ++k) t += red[k][0];
      static_cast<T *>(a.dlambda)[blockIdx.x] = T(-t);
    }
  } else {
    const int col = (blockIdx.x - a.heads) * 32 + lane;
    const long long n = (long long)a.B * a.heads * a.blocks_per_unit;
#pragma unroll 4
    for (long long i = slice; i < n; i += 32) s += __ldcg(a.part + i * stride + 1 + col);
    red[slice][lane] = s;
    __syncthreads();
    if (slice == 0) {
      float t = 0.f;
#pragma unroll
      for (int k = 0; k < 32; ++k) t += red[k][lane];
      static_cast<T *>(a.dweight)[col] = T(t);
    }
  }
  // what follows may need what came before this launch
  if (blockIdx.x == 0 && threadIdx.x == 0) ptx::grid_wait();
}

long long prep_blocks_per_unit(const basa_params &p) {
  return ((long long)p.T * p.H * p.W + kPrepRows - 1) / kPrepRows;
}

}  // namespace

basa_status launch_diff_combine(int n_splits, const float *part, const float *part_lse, long long rows,
                                const basa_diff_params &dp, void *out, const basa_params &p, cudaStream_t s) {
  CombineArgs a{};
  a.part = part;
  a.lse = part_lse;
  a.lambda = dp.lambda;
  a.weight = dp.weight;
  a.out = out;
  a.n_splits = n_splits;
  a.heads = p.heads;
  a.rows = rows;
  a.units = (long long)p.B * p.heads;
  a.gain = dp.gain;
  a.eps = dp.eps;
  constexpr int D = 128, ROWS = kDiffThreads / (D / 8);
  const long long blocks = (a.units * a.rows + ROWS - 1) / ROWS;
  if (blocks >= (1ll << 31)) return BASA_ERR_UNSUPPORTED;
  diff_combine_kernel<__nv_bfloat16, D><<<unsigned(blocks), kDiffThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? BASA_OK : BASA_ERR_CUDA;
}

size_t diff_prep_workspace(const basa_params &p) {
  return size_t(p.B) * p.heads * prep_blocks_per_unit(p) * (p.head_dim + 1) * sizeof(float);
}

basa_status launch_diff_prep(const void *pre, const void *second, const float *lse, const void *dout,
                             const basa_diff_params &dp, void *g, float4 *rec, float *drow, float *part,
                             int *zeros, int n_zeros, const basa_params &p, cudaStream_t s) {
  PrepArgs a{};
  a.pre = pre;
  a.second = second;
  a.dout = dout;
  a.lambda = dp.lambda;
  a.weight = dp.weight;
  a.lse = lse;
  a.g = g;
  a.rec = rec;
  a.drow = drow;
  a.part = part;
  a.zeros = zeros;
  a.n_zeros = n_zeros;
  a.heads = p.heads;
  a.rows = (long long)p.T * p.H * p.W;
  a.gain = dp.gain;
  a.eps = dp.eps;
  const long long per_unit = prep_blocks_per_unit(p), blocks = per_unit * p.B * p.heads;
  if (blocks >= (1ll << 31)) return BASA_ERR_UNSUPPORTED;
  a.blocks_per_unit = int(per_unit);
  if (p.dtype == BASA_BF16) diff_prep_kernel<__nv_bfloat16, 128><<<unsigned(blocks), kDiffThreads, 0, s>>>(a);
  else if (p.head_dim == 128) diff_prep_kernel<float, 128><<<unsigned(blocks), kDiffThreads, 0, s>>>(a);
  else diff_prep_kernel<float, 64><<<unsigned(blocks), kDiffThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? BASA_OK : BASA_ERR_CUDA;
}

basa_status launch_diff_sums(const float *part, const float *dr, int dr_per_unit, const basa_diff_params &dp,
                             void *dlambda, void *dweight, bool early, const basa_params &p, cudaStream_t s) {
  SumArgs r{part, dr, dlambda, dweight, p.B, p.heads, int(prep_blocks_per_unit(p)), dr_per_unit, p.head_dim};
  const unsigned ctas = unsigned(p.heads + (dp.weight ? p.head_dim / 32 : 0));
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = early ? 1 : 0;
  const cudaError_t e = p.dtype == BASA_BF16 ? cudaLaunchKernelEx(&cfg, diff_sum_kernel<__nv_bfloat16>, r)
                                             : cudaLaunchKernelEx(&cfg, diff_sum_kernel<float>, r);
  return e == cudaSuccess ? BASA_OK : BASA_ERR_CUDA;
}

}  // namespace basa
