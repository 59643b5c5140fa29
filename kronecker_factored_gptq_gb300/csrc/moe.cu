// bakron_moe: a mixture-of-experts layer over packed experts, for few tokens.
//
//   l_te = sum_j x_tj router_ej, the top_k experts of each token with weights q,
//   h = silu(gate_e x) * (up_e x),   y_t = sum over its experts of q (w_out_e h).
//
// The layer is bound by the bytes of the experts that any token chose: every
// expert's matrices are read once for all its tokens.  Two launches:
//
// moe_in_kernel.  Which experts to read is known only after routing, so the
// routing must not take a launch of its own: each cluster of 8 blocks computes
// all logits, an eighth of the experts per block, and exchanges them through
// distributed shared memory; every block then selects the experts itself
// (the router is small and comes from L2).  The work that follows is a list of
// (chosen expert, 16 rows of gate and the same 16 of up) dealt to the blocks in
// turn.  A block's warps split the columns; the tokens of the expert are the
// columns of the matrix instructions (qmma.cuh), gathered from x by index.
// h leaves multiplied by q, in two bf16 terms (three for fp32), so that the
// second product sees it to 2^-16 (2^-24).
//
// moe_out_kernel.  A block owns 16 rows of y for all tokens and runs over the
// chosen experts one after the other: a token that did not choose the expert has
// a zero column.  So the sum over experts stays in the accumulators, in expert
// order, and nothing is joined by atomics.  When there are few row tiles the
// list of (expert, chunk) is also split over the blocks of a cluster.
#include <cooperative_groups.h>

#include <algorithm>

#include "linear.cuh"
#include "qmma.cuh"

namespace bakron {

namespace cg = cooperative_groups;

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kCluster = 8;
constexpr int kMaxTokens = BAKRON_MOE_TOKENS;
constexpr int kMaxTopK = 16;
constexpr int kMaxExperts = 1024;

struct MoeArgs {
  const void* x;        // T x d
  const void* router;   // E x d
  const uint8_t* xp;    // activations as 16-bit terms: x itself or planes in the workspace
  int64_t xp_pitch;     // bytes between its rows
  int64_t xp_plane;     // bytes between its terms
  int64_t xp_cols;      // columns that exist in a row (a multiple of 8)
  int T, E, k;
  int renormalize;
  int vec_ok;           // x and router rows are 16-byte aligned
  int64_t d, f, fp;     // fp: f rounded up to 128
  PackedView wi, wo;
  uint8_t* h;           // terms x (T k) x fp 16-bit values
  int64_t h_plane;
  int* active;          // [0] chosen experts na, then their indices
  int16_t* pair;        // [na][T]: t k + slot where token t chose the expert, else -1
  void* y;
};

template <typename TX>
__device__ __forceinline__ void load8(float (&v)[8], const TX* p, bool vec, int64_t left) {
  if (vec && left >= 8) {
    if constexpr (sizeof(TX) == 2) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
      const TX* e = reinterpret_cast<const TX*>(&u);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = to_float(e[i]);
    } else {
      const float4 a = __ldg(reinterpret_cast<const float4*>(p));
      const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? to_float(p[i]) : 0.f;
  }
}

// Logits of this block's experts (rank, rank + 8, ...) for every token, into
// every block of the cluster.  The warps split an expert's columns when there
// are fewer experts than warps; the parts are added in a fixed order.
template <typename TX>
__device__ void router_logits(const MoeArgs& a, cg::cluster_group& cluster, float* logits, float* parts) {
  constexpr int TT = 4;                      // tokens at a time
  const int rank = (int)cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mine = (a.E - rank + kCluster - 1) / kCluster;     // experts of this block
  if (mine > 0) {
    int split = 1;                           // warps per expert
    while (split < kWarps && mine * split * 2 <= kWarps) split *= 2;
    const int at_once = kWarps / split;
    const int part = warp % split;
    const TX* x = static_cast<const TX*>(a.x);
    for (int i0 = 0; i0 < mine; i0 += at_once) {
      const int i = i0 + warp / split;
      if (i < mine) {
        const TX* r = static_cast<const TX*>(a.router) + (int64_t)(rank + i * kCluster) * a.d;
        for (int t0 = 0; t0 < a.T; t0 += TT) {
          float acc[TT];
#pragma unroll
          for (int t = 0; t < TT; ++t) acc[t] = 0.f;
          for (int64_t c = 8 * (lane + 32 * part); c < a.d; c += 8 * 32 * split) {
            float w[8];
            load8(w, r + c, a.vec_ok != 0, a.d - c);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
              if (t0 + t < a.T) {
                float v[8];
                load8(v, x + (int64_t)(t0 + t) * a.d + c, a.vec_ok != 0, a.d - c);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[t] = fmaf(v[e], w[e], acc[t]);
              }
            }
          }
#pragma unroll
          for (int t = 0; t < TT; ++t) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
            if (lane == 0 && t0 + t < a.T) parts[warp * kMaxTokens + t0 + t] = acc[t];
          }
        }
      }
      __syncthreads();
      for (int q = threadIdx.x; q < at_once * a.T; q += kThreads) {
        const int il = q / a.T, t = q - il * a.T;
        if (i0 + il < mine) {
          float v = 0.f;
          for (int p = 0; p < split; ++p) v += parts[(il * split + p) * kMaxTokens + t];
          const int at = t * a.E + rank + (i0 + il) * kCluster;
          for (int b = 0; b < kCluster; ++b) cluster.map_shared_rank(logits, b)[at] = v;
        }
      }
      __syncthreads();
    }
  }
  __syncwarp();
  cluster.sync();
}

// The experts of one token (one warp): choice[i], weight[i] for i < k, the
// largest logits first, a tie to the lowest index.  NaN logits rank last and
// make the weights NaN.
__device__ void select_experts(const float* l, int E, int k, bool renormalize, int* choice, float* weight,
                               int lane) {
  uint32_t taken = 0;                        // bit i: expert lane + 32 i (E <= 1024)
  float top = 0.f, mine = 0.f;
  for (int i = 0; i < k; ++i) {
    float best = 0.f;
    int at = -1;
    for (int j = 0; 32 * j + lane < E; ++j) {
      if (taken >> j & 1) continue;
      float v = l[32 * j + lane];
      if (v != v) v = -INFINITY;
      if (at < 0 || v > best) { best = v; at = 32 * j + lane; }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float ov = __shfl_xor_sync(0xffffffffu, best, o);
      const int oa = __shfl_xor_sync(0xffffffffu, at, o);
      if (oa >= 0 && (at < 0 || ov > best || (ov == best && oa < at))) { best = ov; at = oa; }
    }
    if ((at & 31) == lane) taken |= 1u << (at >> 5);
    if (i == 0) top = best;
    if (lane == 0) choice[i] = at;
    if (lane == i) mine = l[at];
  }
  float sum = 0.f;
  if (renormalize) {
    sum = lane < k ? expf(mine - top) : 0.f;
  } else {
    for (int e = lane; e < E; e += 32) sum += expf(l[e] - top);
  }
  bool bad = false;
  for (int e = lane; e < E; e += 32) bad |= l[e] != l[e];
  bad = __any_sync(0xffffffffu, bad);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane < k) weight[lane] = bad ? NAN : expf(mine - top) / sum;
}

// Shared memory of the routing, after the logits.
struct Routing {
  int choice[kMaxTokens][kMaxTopK];
  float weight[kMaxTokens][kMaxTopK];
  int na;
  int active[kMaxTokens * kMaxTopK];
  float parts[kWarps * kMaxTokens];
};

template <typename TX, typename H, int TERMS, int HT, int NT, int NS>
__global__ void __launch_bounds__(kThreads, 2) moe_in_kernel(const __grid_constant__ MoeArgs a) {
  extern __shared__ __align__(16) uint8_t dsm[];
  __shared__ Routing R;
  __shared__ float red[kWarps][NT * 8][33];
  float* logits = reinterpret_cast<float*>(dsm);          // [T][E]
  int* slot_of = reinterpret_cast<int*>(logits + a.T * a.E);   // [E]: index among the chosen, or -1
  cg::cluster_group cluster = cg::this_cluster();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  router_logits<TX>(a, cluster, logits, R.parts);
  for (int t = warp; t < a.T; t += kWarps)
    select_experts(logits + t * a.E, a.E, a.k, a.renormalize != 0, R.choice[t], R.weight[t], lane);
  for (int e = threadIdx.x; e < a.E; e += kThreads) slot_of[e] = -1;
  __syncthreads();
  // the chosen experts in ascending order
  for (int i = threadIdx.x; i < a.T * a.k; i += kThreads) slot_of[R.choice[i / a.k][i % a.k]] = 0;
  __syncthreads();
  if (warp == 0) {
    int n = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const bool in = e0 + lane < a.E && slot_of[e0 + lane] == 0;
      const uint32_t m = __ballot_sync(0xffffffffu, in);
      if (in) {
        const int at = n + __popc(m & ((1u << lane) - 1));
        R.active[at] = e0 + lane;
      }
      n += __popc(m);
    }
    if (lane == 0) R.na = n;
  }
  __syncthreads();
  const int na = R.na;
  if (blockIdx.x == 0) {
    // for the second launch: the chosen experts, and who chose them
    if (threadIdx.x == 0) a.active[0] = na;
    for (int i = threadIdx.x; i < na; i += kThreads) a.active[1 + i] = R.active[i];
    for (int i = threadIdx.x; i < na * a.T; i += kThreads) {
      const int e = R.active[i / a.T], t = i % a.T;
      int p = -1;
      for (int s = 0; s < a.k; ++s)
        if (R.choice[t][s] == e) p = t * a.k + s;
      a.pair[i] = (int16_t)p;
    }
  }
  // zeros past f, for the padded columns of w_out
  if (a.fp > a.f) {
    const int64_t per = a.fp - a.f;
    for (int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x; i < HT * a.T * a.k * per;
         i += (int64_t)gridDim.x * kThreads) {
      const int64_t row = i / per, c = a.f + i % per;
      const int64_t q = row / (a.T * a.k), p = row % (a.T * a.k);
      *reinterpret_cast<uint16_t*>(a.h + q * a.h_plane + (p * a.fp + c) * 2) = 0;
    }
  }

  const int tiles = (int)((a.f + 15) / 16);
  const int64_t items = (int64_t)na * tiles;
  const int nc = (int)a.wi.nc;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int ai = (int)(it / tiles);
    const int64_t row0 = (it - (int64_t)ai * tiles) * 16;
    const int e = R.active[ai];
    // the expert's tokens, by ballot: thread's column 8 j + lane / 4
    uint32_t who = 0;
    int my_slot = -1;
    if (lane < a.T)
      for (int s = 0; s < a.k; ++s)
        if (R.choice[lane][s] == e) my_slot = s;
    who = __ballot_sync(0xffffffffu, my_slot >= 0);
    const int cnt = __popc(who);
    const int live = (cnt + 7) / 8;
    const uint8_t* xr[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int c = 8 * j + (lane >> 2);
      xr[j] = nullptr;
      if (c < cnt) xr[j] = a.xp + (int64_t)__fns(who, 0, c + 1) * a.xp_pitch + (lane & 3) * 16;
    }
    const qm::TileRef tile[2] = {qm::tile_ref(a.wi, e, row0, lane), qm::tile_ref(a.wi, e, a.f + row0, lane)};
    float tot[2][NT][4];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) tot[r][j][i] = 0.f;
    qm::Chunk16<NS> f[2];
    if (warp < nc) {
      qm::load_chunk<NS>(f[0], a.wi, tile[0], warp);
      qm::load_chunk<NS>(f[1], a.wi, tile[1], warp);
    }
    for (int c = warp; c < nc; c += kWarps) {
      const qm::Chunk16<NS> g[2] = {f[0], f[1]};
      if (c + kWarps < nc) {
        qm::load_chunk<NS>(f[0], a.wi, tile[0], c + kWarps);
        qm::load_chunk<NS>(f[1], a.wi, tile[1], c + kWarps);
      }
      const int64_t k0 = (int64_t)c * 128 + 8 * (lane & 3);
      qm::chunk_product<H, TERMS, 2, NT, NS>(
          tot, g, a.wi.zero != nullptr, a.wi.zu, live, [&](int j, int q, int s) {
            if (xr[j] == nullptr || k0 + 32 * s >= a.xp_cols) return make_uint4(0, 0, 0, 0);
            return __ldg(reinterpret_cast<const uint4*>(xr[j] + q * a.xp_plane + (int64_t)c * 256 + s * 64));
          });
    }
    // gate and up in turn through the same array
    float gate[NT], up[NT];       // of outputs threadIdx.x + 256 j: row i & 15, column i / 16
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int rr = lane >> 2, cc = 8 * j + 2 * (lane & 3);
        red[warp][cc][rr] = tot[r][j][0];
        red[warp][cc + 1][rr] = tot[r][j][1];
        red[warp][cc][rr + 8] = tot[r][j][2];
        red[warp][cc + 1][rr + 8] = tot[r][j][3];
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < (NT + 1) / 2; ++j) {
        const int i = threadIdx.x + kThreads * j;
        if (i < NT * 8 * 16) {
          float v = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) v += red[w][i >> 4][i & 15];
          (r == 0 ? gate : up)[j] = v;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < (NT + 1) / 2; ++j) {
      const int i = threadIdx.x + kThreads * j;
      const int c = i >> 4;
      const int64_t row = row0 + (i & 15);
      if (i < NT * 8 * 16 && c < cnt && row < a.f) {
        const int t = (int)__fns(who, 0, c + 1);
        int s = 0;
        for (int q = 0; q < a.k; ++q)
          if (R.choice[t][q] == e) s = q;
        const float g = gate[j];
        const float v = g / (1.f + expf(-g)) * up[j] * R.weight[t][s];
        float p[3];
        split3(v, p[0], p[1], p[2]);
        uint8_t* o = a.h + ((int64_t)(t * a.k + s) * a.fp + row) * 2;
#pragma unroll
        for (int q = 0; q < HT; ++q) *reinterpret_cast<uint16_t*>(o + q * a.h_plane) = bf16_bits(p[q]);
      }
    }
  }
}

template <typename TX, int HT, int NT, int NS>
__global__ void __launch_bounds__(kThreads, 2) moe_out_kernel(const __grid_constant__ MoeArgs a) {
  __shared__ float red[kWarps][NT * 8][17];
  __shared__ float part[NT * 8 * 16];
  cg::cluster_group cluster = cg::this_cluster();
  const int S = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row0 = (int64_t)(blockIdx.x / S) * 16;
  const int na = a.active[0];
  const int nc = (int)a.wo.nc;
  const int64_t units = (int64_t)na * nc;          // (expert, chunk)
  const int64_t u0 = units * rank / S, u1 = units * (rank + 1) / S;
  float tot[1][NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) tot[0][j][i] = 0.f;
  const int live = (a.T + 7) / 8;

  int cur = -1;
  qm::TileRef tile;
  qm::Chunk16<NS> f[1];
  auto load = [&](int64_t u) {
    const int ai = (int)(u / nc);
    if (ai != cur) {
      cur = ai;
      tile = qm::tile_ref(a.wo, a.active[1 + ai], row0, lane);
    }
    qm::load_chunk<NS>(f[0], a.wo, tile, u - (int64_t)ai * nc);
  };
  int have = -1;
  const uint8_t* hr[NT];
  if (u0 + warp < u1) load(u0 + warp);
  for (int64_t u = u0 + warp; u < u1; u += kWarps) {
    const qm::Chunk16<NS> g[1] = {f[0]};
    if (u + kWarps < u1) load(u + kWarps);
    const int ai = (int)(u / nc), c = (int)(u - (int64_t)ai * nc);
    if (ai != have) {
      have = ai;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int t = 8 * j + (lane >> 2);
        const int p = t < a.T ? a.pair[ai * a.T + t] : -1;
        hr[j] = p < 0 ? nullptr : a.h + (int64_t)p * a.fp * 2 + (lane & 3) * 16;
      }
    }
    qm::chunk_product<__nv_bfloat16, HT, 1, NT, NS>(
        tot, g, a.wo.zero != nullptr, a.wo.zu, live, [&](int j, int q, int s) {
          if (hr[j] == nullptr) return make_uint4(0, 0, 0, 0);
          return *reinterpret_cast<const uint4*>(hr[j] + q * a.h_plane + (int64_t)c * 256 + s * 64);
        });
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int rr = lane >> 2, cc = 8 * j + 2 * (lane & 3);
    red[warp][cc][rr] = tot[0][j][0];
    red[warp][cc + 1][rr] = tot[0][j][1];
    red[warp][cc][rr + 8] = tot[0][j][2];
    red[warp][cc + 1][rr + 8] = tot[0][j][3];
  }
  __syncthreads();
  TX* y = static_cast<TX*>(a.y);
  for (int i = threadIdx.x; i < NT * 8 * 16; i += kThreads) {
    const int t = i >> 4, r = i & 15;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += red[w][t][r];
    if (S > 1) part[i] = v;
    else if (t < a.T && row0 + r < a.d) y[(int64_t)t * a.d + row0 + r] = from_float<TX>(v);
  }
  if (S > 1) {
    __syncwarp();
    cluster.sync();
    if (rank == 0) {
      for (int i = threadIdx.x; i < NT * 8 * 16; i += kThreads) {
        const int t = i >> 4, r = i & 15;
        if (t >= a.T || row0 + r >= a.d) continue;
        float v = 0.f;
        for (int k = 0; k < S; ++k) v += cluster.map_shared_rank(part, k)[i];
        y[(int64_t)t * a.d + row0 + r] = from_float<TX>(v);
      }
    }
    __syncwarp();
    cluster.sync();
  }
}

cudaError_t launch_cluster(const void* k, unsigned grid, unsigned cluster, size_t smem, MoeArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  void* args[] = {&a};
  count_launch();
  return cudaLaunchKernelExC(&cfg, k, args);
}

constexpr size_t kMaxDynamic = (size_t)kMaxTokens * kMaxExperts * 4 + kMaxExperts * 4;

template <typename TX, typename H, int TERMS, int HT, int NT, int NS, int NSO>
cudaError_t run(MoeArgs& a, cudaStream_t s) {
  const void* k1 = (const void*)moe_in_kernel<TX, H, TERMS, HT, NT, NS>;
  const void* k2 = (const void*)moe_out_kernel<TX, HT, NT, NSO>;
  static std::atomic<unsigned long long> done;
  cudaError_t e = ensure_smem_limit(k1, kMaxDynamic, done);
  if (e != cudaSuccess) return e;
  const size_t smem = (size_t)a.T * a.E * 4 + (size_t)a.E * 4;
  const int64_t most = (int64_t)std::min(a.E, a.T * a.k) * ((a.f + 15) / 16);
  // two blocks per SM, not more than there can be items
  int64_t clusters = std::min<int64_t>(2 * sm_count() / kCluster, (most + kCluster - 1) / kCluster);
  e = launch_cluster(k1, (unsigned)(clusters * kCluster), kCluster, smem, a, s);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (a.d + 15) / 16;
  const int64_t units = (int64_t)std::min(a.E, a.T * a.k) * a.wo.nc;
  int S = 1;
  while (S < 8 && tiles * S < 2 * sm_count() && units >= (int64_t)2 * S * kWarps) S *= 2;
  return launch_cluster(k2, (unsigned)(tiles * S), (unsigned)S, 0, a, s);
}

template <typename TX, typename H, int TERMS, int HT, int NT>
cudaError_t by_groups(MoeArgs& a, cudaStream_t s) {
  const bool wi = a.wi.ng == 1 || a.wi.g % 128 == 0, wo = a.wo.ng == 1 || a.wo.g % 128 == 0;
  if (wi && wo) return run<TX, H, TERMS, HT, NT, 1, 1>(a, s);
  if (wi) return run<TX, H, TERMS, HT, NT, 1, 4>(a, s);
  if (wo) return run<TX, H, TERMS, HT, NT, 4, 1>(a, s);
  return run<TX, H, TERMS, HT, NT, 4, 4>(a, s);
}

template <typename TX, typename H, int TERMS, int HT>
cudaError_t by_tokens(MoeArgs& a, cudaStream_t s) {
  if (a.T <= 8) return by_groups<TX, H, TERMS, HT, 1>(a, s);
  if (a.T <= 16) return by_groups<TX, H, TERMS, HT, 2>(a, s);
  return by_groups<TX, H, TERMS, HT, 4>(a, s);
}

struct MoeLayout {
  size_t xp, h, active, pair, total;
  int64_t dp, fp;
};

MoeLayout moe_layout(int64_t T, int64_t d, int64_t f, int64_t E, int k, int dtype) {
  MoeLayout L;
  const int64_t t = std::min<int64_t>(T, kMaxTokens);
  L.dp = (d + 127) / 128 * 128;
  L.fp = (f + 127) / 128 * 128;
  size_t off = 0;
  auto take = [&](size_t b) { const size_t o = off; off += (b + 255) / 256 * 256; return o; };
  L.xp = take((size_t)(dtype == BAKRON_F32 ? 3 : 1) * t * L.dp * 2);
  L.h = take((size_t)(dtype == BAKRON_F32 ? 3 : 2) * t * k * L.fp * 2);
  L.active = take((size_t)(1 + std::min<int64_t>(E, t * k)) * 4);
  L.pair = take((size_t)std::min<int64_t>(E, t * k) * t * 2);
  L.total = off;
  return L;
}

bool moe_views(const bakron_packed* w_in, const bakron_packed* w_out, int64_t T, int top_k, int dtype,
               PackedView* wi, PackedView* wo) {
  if (!dtype_ok(dtype) || T < 0 || T > (int64_t(1) << 28)) return false;
  if (!packed_view(w_in, wi) || !packed_view(w_out, wo)) return false;
  return wi->count == wo->count && wi->count <= kMaxExperts && wi->n == wo->m && wi->m == 2 * wo->n &&
         top_k >= 1 && top_k <= kMaxTopK && top_k <= wi->count;
}

}  // namespace
}  // namespace bakron

using namespace bakron;

extern "C" bakron_status bakron_moe_workspace_size(const bakron_packed* w_in,
                                                   const bakron_packed* w_out, int64_t T, int top_k,
                                                   int dtype, size_t* bytes) {
  PackedView wi, wo;
  if (!bytes || !moe_views(w_in, w_out, T, top_k, dtype, &wi, &wo)) return BAKRON_ERR_INVALID_ARG;
  *bytes = moe_layout(T, wi.n, wo.n, wi.count, top_k, dtype).total;
  return BAKRON_OK;
}

extern "C" bakron_status bakron_moe(const void* X, int64_t T, int dtype, const void* router,
                                    const bakron_packed* w_in, const bakron_packed* w_out, int top_k,
                                    int renormalize, void* Y, void* ws, size_t ws_bytes,
                                    void* stream) {
  MoeArgs a = {};
  if (!moe_views(w_in, w_out, T, top_k, dtype, &a.wi, &a.wo)) return BAKRON_ERR_INVALID_ARG;
  if (T == 0) return BAKRON_OK;
  const size_t es = dtype_size(dtype);
  if (!X || !router || !Y || !ws || !aligned_to(X, es) || !aligned_to(router, es) || !aligned_to(Y, es) ||
      !aligned_to(ws, 256))
    return BAKRON_ERR_INVALID_ARG;
  a.d = a.wi.n;
  a.f = a.wo.n;
  a.E = (int)a.wi.count;
  a.k = top_k;
  a.renormalize = renormalize;
  a.router = router;
  const MoeLayout L = moe_layout(T, a.d, a.f, a.E, top_k, dtype);
  if (ws_bytes < L.total) return BAKRON_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  uint8_t* base = static_cast<uint8_t*>(ws);
  a.fp = L.fp;
  a.h = base + L.h;
  a.active = reinterpret_cast<int*>(base + L.active);
  a.pair = reinterpret_cast<int16_t*>(base + L.pair);
  for (int64_t t0 = 0; t0 < T; t0 += kMaxTokens) {
    a.T = (int)std::min<int64_t>(kMaxTokens, T - t0);
    a.x = static_cast<const uint8_t*>(X) + (size_t)(t0 * a.d) * es;
    a.y = static_cast<uint8_t*>(Y) + (size_t)(t0 * a.d) * es;
    a.h_plane = (int64_t)a.T * a.k * a.fp * 2;
    const bool rows16 = (a.d * es) % 16 == 0;
    a.vec_ok = rows16 && aligned_to(a.x, 16) && aligned_to(router, 16);
    cudaError_t e = cudaSuccess;
    if (dtype != BAKRON_F32 && rows16 && aligned_to(a.x, 16)) {
      a.xp = static_cast<const uint8_t*>(a.x);
      a.xp_pitch = a.d * 2;
      a.xp_plane = 0;
      a.xp_cols = a.d;
    } else {
      a.xp = base + L.xp;
      a.xp_pitch = L.dp * 2;
      a.xp_plane = (int64_t)a.T * L.dp * 2;
      a.xp_cols = L.dp;
      e = launch_planes(a.x, dtype, a.T, a.d, L.dp, base + L.xp, s);
    }
    if (e == cudaSuccess) {
      switch (dtype) {
        case BAKRON_F32: e = by_tokens<float, __nv_bfloat16, 3, 3>(a, s); break;
        case BAKRON_BF16: e = by_tokens<__nv_bfloat16, __nv_bfloat16, 1, 2>(a, s); break;
        default: e = by_tokens<__half, __half, 1, 2>(a, s); break;
      }
    }
    if (e != cudaSuccess) return BAKRON_ERR_CUDA;
  }
  return BAKRON_OK;
}
