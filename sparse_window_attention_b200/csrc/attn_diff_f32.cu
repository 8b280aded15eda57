// Differential attention forward in float32 on the CUDA cores (no TF32, as in the window
// attention): the windows' rows, and the text queries' rows dense over every key.
//
//   a = softmax(q1 K1^T / sqrt(d)) V - lambda softmax(q2 K2^T / sqrt(d)) V,
//   out = gain * weight * a * rsqrt(mean(a^2) + eps)       (no weight: out = a)
//
// One CTA = (batch * head, window, 16 queries), both maps: warps 0-3 run map 1, warps 4-7
// map 2, four queries a warp, over key tiles of 32 rows K1, K2, V that cp.async brings in
// two deep. A lane is a key for the scores (its key row against four broadcast queries:
// no shuffles but the row maximum's) and a group of channels for the product with V (the
// probabilities read back as broadcasts). Few queries a CTA because the layers that run in
// float32 are small and bound by latency: with a thread a query and a launch a map, 2 heads
// of 16 windows of 64 tokens (128 keys each) took 57 us, so 19 us (1, 2 and 8 queries a warp 26,
// 20 and 29).
#include "attn_f32.cuh"

namespace basa {
namespace {

constexpr int kThreads = 256;
constexpr int kKeyTile = 32;
constexpr int kWarpQ = 4;            // queries of a warp
constexpr int kQueries = 4 * kWarpQ;  // of a CTA

struct DiffF32Args {
  F32Args f;  // q, k, kp of 2 heads maps; v, vp, route, out of heads
  const float *lambda, *weight;
  float *pre, *second;  // nullable
  float gain, eps;
};

template <int D>
struct DiffSmem {
  static constexpr int stride = D + 4;  // a row's 16-byte steps fall on different banks for 8 rows in turn
  float q[2][kQueries][D];
  float k[2][2][kKeyTile][stride];  // [stage][map]
  float v[2][kKeyTile][D];
  float p[8][kWarpQ][kKeyTile];
  float o2[kQueries][D];
  int wins[1 + kMaxRouted];
};

__device__ __forceinline__ void copy16(float *dst, const float *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(uint32_t(__cvta_generic_to_shared(dst))), "l"(src)
               : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads) attn_diff_f32_kernel(const __grid_constant__ DiffF32Args A) {
  constexpr int C = D / 32;  // channels of a lane in the product with V
  extern __shared__ __align__(16) uint8_t smem_raw[];
  DiffSmem<D> &sm = *reinterpret_cast<DiffSmem<D> *>(smem_raw);
  const F32Args &a = A.f;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, map = warp / 4;
  const int n_win = a.dense ? 1 : a.g.nWin;
  const int chunk = blockIdx.x % a.q_chunks, w = (blockIdx.x / a.q_chunks) % n_win;
  const long long bh = blockIdx.x / (a.q_chunks * n_win);
  const int n_queries = a.dense ? a.n_text : a.win_tok;
  const long long q_rows = a.dense ? a.n_text : a.g.N;
  if (threadIdx.x == 0) sm.wins[0] = w;
  if (!a.dense && threadIdx.x > 0 && threadIdx.x <= a.routed_k)
    sm.wins[threadIdx.x] = checked_route(a, a.route[(bh * a.g.nWin + w) * a.routed_k + threadIdx.x - 1], w);

  // Row of the CTA's query i inside its unit: a token of the grid, or a text row.
  auto query_row = [&](int i) -> long long {
    const int lq = chunk * kQueries + i;
    if (a.dense) return lq;
    int ot, oy, ox, type;
    window_origin(a.g, w, &ot, &oy, &ox, &type);
    const int lt = lq / (a.g.wh * a.g.ww), ly = (lq / a.g.ww) % a.g.wh, lx = lq % a.g.ww;
    return ((long long)((ot + lt) % a.g.T) * a.g.H + (oy + ly) % a.g.H) * a.g.W + (ox + lx) % a.g.W;
  };
  for (int i = threadIdx.x; i < 2 * kQueries * (D / 4); i += kThreads) {
    const int c4 = i % (D / 4), qi = (i / (D / 4)) % kQueries, m = i / (D / 4 * kQueries);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (chunk * kQueries + qi < n_queries)
      x = reinterpret_cast<const float4 *>(a.q + ((2 * bh + m) * q_rows + query_row(qi)) * D)[c4];
    reinterpret_cast<float4 *>(sm.q[m][qi])[c4] = make_float4(x.x * a.scale, x.y * a.scale, x.z * a.scale, x.w * a.scale);
  }
  __syncthreads();

  const int nk = a.dense ? a.g.N + a.n_text : a.n_vis_keys + a.n_pool_keys + a.n_text_keys;
  const int n_tiles = (nk + kKeyTile - 1) / kKeyTile;
  // Eight threads a key row. Rows past the end repeat the last key; their probability is 0.
  auto load = [&](int tile) {
    if (tile < n_tiles) {
      const int r = threadIdx.x / 8, j = min(tile * kKeyTile + r, nk - 1), st = tile & 1;
      const float *k0 = key_row(a, a.k, a.kp, 2 * bh, sm.wins, j), *k1 = key_row(a, a.k, a.kp, 2 * bh + 1, sm.wins, j);
      const float *v0 = key_row(a, a.v, a.vp, bh, sm.wins, j);
#pragma unroll
      for (int c = threadIdx.x % 8; c < D / 4; c += 8) {
        copy16(&sm.k[st][0][r][4 * c], k0 + 4 * c);
        copy16(&sm.k[st][1][r][4 * c], k1 + 4 * c);
        copy16(&sm.v[st][r][4 * c], v0 + 4 * c);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  float m[kWarpQ], l[kWarpQ], o[kWarpQ][C];
#pragma unroll
  for (int i = 0; i < kWarpQ; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;  // of this lane's keys
#pragma unroll
    for (int c = 0; c < C; ++c) o[i][c] = 0.f;
  }
  load(0);
  for (int tile = 0; tile < n_tiles; ++tile) {
    load(tile + 1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    const int st = tile & 1;
    float s[kWarpQ];
#pragma unroll
    for (int i = 0; i < kWarpQ; ++i) s[i] = 0.f;
    const float4 *kr = reinterpret_cast<const float4 *>(sm.k[st][map][lane]);
#pragma unroll
    for (int c = 0; c < D / 4; ++c) {
      const float4 k4 = kr[c];
#pragma unroll
      for (int i = 0; i < kWarpQ; ++i) {
        const float4 q4 = reinterpret_cast<const float4 *>(sm.q[map][(warp % 4) * kWarpQ + i])[c];
        s[i] = fmaf(q4.x, k4.x, fmaf(q4.y, k4.y, fmaf(q4.z, k4.z, fmaf(q4.w, k4.w, s[i]))));
      }
    }
    const bool key = tile * kKeyTile + lane < nk;
#pragma unroll
    for (int i = 0; i < kWarpQ; ++i) {
      float mt = key ? s[i] : -INFINITY;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xFFFFFFFFu, mt, x));
      const float mn = fmaxf(m[i], mt);  // finite: the tile has a key
      const float alpha = expf(m[i] - mn), p = key ? expf(s[i] - mn) : 0.f;
      m[i] = mn;
      l[i] = fmaf(l[i], alpha, p);
#pragma unroll
      for (int c = 0; c < C; ++c) o[i][c] *= alpha;
      sm.p[warp][i][lane] = p;
    }
    __syncwarp();
#pragma unroll 2
    for (int j = 0; j < kKeyTile; j += 4) {
      float pv[kWarpQ][4];
#pragma unroll
      for (int i = 0; i < kWarpQ; ++i)
        *reinterpret_cast<float4 *>(pv[i]) = *reinterpret_cast<const float4 *>(&sm.p[warp][i][j]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x[C];
        if (C == 4) *reinterpret_cast<float4 *>(x) = *reinterpret_cast<const float4 *>(&sm.v[st][j + e][C * lane]);
        else *reinterpret_cast<float2 *>(x) = *reinterpret_cast<const float2 *>(&sm.v[st][j + e][C * lane]);
#pragma unroll
        for (int i = 0; i < kWarpQ; ++i)
#pragma unroll
          for (int c = 0; c < C; ++c) o[i][c] = fmaf(pv[i][e], x[c], o[i][c]);
      }
    }
    __syncthreads();  // the stage is read: load(tile + 2) may overwrite it
  }

  const float lam = A.lambda[bh % a.heads];
#pragma unroll
  for (int i = 0; i < kWarpQ; ++i) {
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], x);
    const float inv = 1.0f / l[i];
    const int qi = (warp % 4) * kWarpQ + i;
    const bool active = chunk * kQueries + qi < n_queries;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      o[i][c] *= inv;
      if (map == 1) sm.o2[qi][C * lane + c] = o[i][c];
    }
    if (active && a.lse && lane == 0) a.lse[(2 * bh + map) * q_rows + query_row(qi)] = m[i] + logf(l[i]);
  }
  __syncthreads();
  if (map == 1) return;
#pragma unroll
  for (int i = 0; i < kWarpQ; ++i) {
    const int qi = warp * kWarpQ + i;
    if (chunk * kQueries + qi >= n_queries) break;  // the same in the whole warp
    const long long at = (bh * q_rows + query_row(qi)) * D + C * lane;
    float ss = 0.f, o2[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      o2[c] = sm.o2[qi][C * lane + c];
      o[i][c] = fmaf(-lam, o2[c], o[i][c]);
      ss = fmaf(o[i][c], o[i][c], ss);
      if (A.second) A.second[at + c] = o2[c];
      if (A.pre) A.pre[at + c] = o[i][c];
    }
    if (A.weight) {
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, x);
      const float f = rsqrtf(ss * (1.f / D) + A.eps) * A.gain;
#pragma unroll
      for (int c = 0; c < C; ++c) o[i][c] *= f * A.weight[C * lane + c];
    }
#pragma unroll
    for (int c = 0; c < C; ++c) a.out[at + c] = o[i][c];
  }
}

template <int D>
basa_status run(const DiffF32Args &a, long long blocks, cudaStream_t s) {
  if (cudaFuncSetAttribute(attn_diff_f32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(DiffSmem<D>)) !=
      cudaSuccess)
    return BASA_ERR_CUDA;
  attn_diff_f32_kernel<D><<<unsigned(blocks), kThreads, sizeof(DiffSmem<D>), s>>>(a);
  return cudaGetLastError() == cudaSuccess ? BASA_OK : BASA_ERR_CUDA;
}

}  // namespace

basa_status launch_diff_attn_f32(const void *q, const void *k, const void *v, const void *kp, const void *vp,
                                 const int32_t *route_idx, const basa_diff_params &dp, void *out, void *pre,
                                 void *second, float *lse, bool dense, const basa_params &p, cudaStream_t s) {
  DiffF32Args A{};
  F32Args &a = A.f;
  a.q = static_cast<const float *>(q);
  a.k = static_cast<const float *>(k);
  a.v = static_cast<const float *>(v);
  a.kp = static_cast<const float *>(kp);
  a.vp = static_cast<const float *>(vp);
  a.route = route_idx;
  a.dev_err = p.dev_err;
  a.out = static_cast<float *>(out);
  a.lse = lse;
  a.g = make_geo(p);
  a.heads = p.heads;
  a.d = p.head_dim;
  a.n_text = p.n_text;
  a.n_pool = p.pt > 0 ? (p.T / p.pt) * (p.H / p.ph) * (p.W / p.pw) : 0;
  a.routed_k = dense ? 0 : p.routed_k;
  a.win_tok = p.wt * p.wh * p.ww;
  a.n_vis_keys = a.win_tok * (1 + a.routed_k);
  a.n_pool_keys = a.n_pool;
  a.n_text_keys = p.n_text;
  a.dense = dense;
  a.scale = 1.0f / sqrtf(float(p.head_dim));
  a.q_chunks = ((dense ? p.n_text : a.win_tok) + kQueries - 1) / kQueries;
  A.lambda = static_cast<const float *>(dp.lambda);
  A.weight = static_cast<const float *>(dp.weight);
  A.pre = static_cast<float *>(pre);
  A.second = static_cast<float *>(second);
  A.gain = dp.gain;
  A.eps = dp.eps;
  const long long blocks = (long long)p.B * p.heads * (dense ? 1 : a.g.nWin) * a.q_chunks;
  if (blocks >= (1ll << 31)) return BASA_ERR_UNSUPPORTED;
  return p.head_dim == 64 ? run<64>(A, blocks, s) : run<128>(A, blocks, s);
}

}  // namespace basa
