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
constexpr int kDepthIn = 4;      // chunks in flight per warp
constexpr int kDepthOut = 6;

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

// Index of the c-th set bit (from 0).
__device__ __forceinline__ int nth_bit(uint32_t m, int c) {
  for (int i = 0; i < c; ++i) m &= m - 1;
  return __ffs((int)m) - 1;
}

// Shared memory of the routing.
struct Routing {
  int choice[kMaxTokens][kMaxTopK];
  float weight[kMaxTokens][kMaxTopK];
  int na;
  int active[kMaxTokens * kMaxTopK];
  uint32_t who[kMaxTokens * kMaxTopK];                    // bit t: token t chose the expert
  float parts[kWarps * kMaxTokens];
};

template <typename TX, typename H, int TERMS, int HT, int NT, int NS>
__global__ void __launch_bounds__(kThreads, 2) moe_in_kernel(const __grid_constant__ MoeArgs a) {
  extern __shared__ __align__(16) uint8_t dsm[];
  __shared__ Routing R;
  using P = qm::Pipe<2, NS, kDepthIn>;
  // the routing's arrays end before the chunks' slots and the joins begin
  float* red = reinterpret_cast<float*>(dsm + kWarps * P::kBytes);
  float* logits = reinterpret_cast<float*>(dsm);               // [T][E]
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
        slot_of[e0 + lane] = at;
      }
      n += __popc(m);
    }
    if (lane == 0) R.na = n;
  }
  __syncthreads();
  const int na = R.na;
  for (int i = threadIdx.x; i < na; i += kThreads) R.who[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * a.k; i += kThreads)
    atomicOr(&R.who[slot_of[R.choice[i / a.k][i % a.k]]], 1u << (i / a.k));
  __syncthreads();
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

  // Items: (chosen expert, row tile), a gate tile and its up tile each, for
  // groups of G warps that split the columns: as many groups as the items can
  // feed.  A warp runs through its (item, chunk) pairs as one sequence, so the
  // copies of the next item start while this one ends.
  const int tiles = (int)((a.f + 15) / 16);
  const int64_t items = (int64_t)na * tiles;
  const int nc = (int)a.wi.nc;
  int G = 1;
  while (G < kWarps && items * 2 * G <= (int64_t)gridDim.x * kWarps && nc >= 2 * G) G *= 2;
  const int group = warp / G, part = warp % G;
  const int64_t groups = (int64_t)gridDim.x * (kWarps / G);
  const int64_t first = (int64_t)blockIdx.x + (int64_t)gridDim.x * group;
  const int c_lo = nc * part / G, c_hi = nc * (part + 1) / G;

  P pipe;
  pipe.base = (uint32_t)__cvta_generic_to_shared(dsm) + (uint32_t)warp * P::kBytes;
  auto open_item = [&](qm::TileRef<2>& t, int64_t it) {
    const int ai = (int)(it / tiles);
    const int64_t r0 = (it - (int64_t)ai * tiles) * 16;
    const int64_t rows[2] = {r0, a.f + r0};
    qm::tile_ref<2>(t, a.wi, R.active[ai], rows, lane);
  };
  qm::TileRef<2> t_ahead, t_now;
  int64_t it_ahead = first;
  int c_ahead = c_lo;
  if (it_ahead < items) open_item(t_ahead, it_ahead);
  auto issue = [&]() {
    pipe.issue(a.wi, t_ahead, c_ahead, it_ahead < items, lane);
    if (it_ahead < items && ++c_ahead == c_hi) {
      c_ahead = c_lo;
      it_ahead += groups;
      if (it_ahead < items) open_item(t_ahead, it_ahead);
    }
  };
#pragma unroll
  for (int p = 0; p < kDepthIn - 1; ++p) issue();

  for (int64_t it = first; it < items; it += groups) {
    const int ai = (int)(it / tiles);
    const int64_t row0 = (it - (int64_t)ai * tiles) * 16;
    const int e = R.active[ai];
    if (a.wi.zero) open_item(t_now, it);
    // the expert's tokens: thread's column 8 j + lane / 4
    const uint32_t who = R.who[ai];
    const int cnt = __popc(who);
    const int live = (cnt + 7) / 8;
    const uint8_t* xr[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int c = 8 * j + (lane >> 2);
      xr[j] = c < cnt ? a.xp + (int64_t)nth_bit(who, c) * a.xp_pitch + (lane & 3) * 16 : nullptr;
    }
    float tot[2][NT][4];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) tot[r][j][i] = 0.f;
    uint32_t z[2][2][NS];
    qm::load_zeros<2, NS>(z, a.wi, t_now, c_lo);
    for (int c = c_lo; c < c_hi; ++c) {
      qm::Chunk16<NS> f[2];
      issue();
      pipe.take(f, lane);
      qm::set_zeros<2, NS>(f, z);
      if (c + 1 < c_hi) qm::load_zeros<2, NS>(z, a.wi, t_now, c + 1);
      const int64_t k0 = (int64_t)c * 128 + 8 * (lane & 3);
      qm::chunk_product<H, TERMS, 2, NT, NS>(
          tot, f, a.wi.zero != nullptr, a.wi.zu, live, [&](int j, int q, int s) {
            if (xr[j] == nullptr || k0 + 32 * s >= a.xp_cols) return make_uint4(0, 0, 0, 0);
            return __ldg(reinterpret_cast<const uint4*>(xr[j] + q * a.xp_plane + (int64_t)c * 256 + s * 64));
          });
    }
    // the group's sums of gate and up (thread: rows lane / 4 and + 8, columns
    // 2 (lane & 3) and + 1 of each column tile)
    if (G > 1) {
      float* mine = red + (size_t)warp * (2 * NT * 4 * 32) + lane;
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) mine[((r * NT + j) * 4 + i) * 32] = tot[r][j][i];
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * G) : "memory");
      if (part == 0) {
        for (int w = 1; w < G; ++w) {
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) tot[r][j][i] += mine[(size_t)w * (2 * NT * 4 * 32) + ((r * NT + j) * 4 + i) * 32];
        }
      }
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * G) : "memory");
    }
    if (part == 0) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = 8 * j + 2 * (lane & 3) + (i & 1);
          const int64_t row = row0 + (lane >> 2) + 8 * (i >> 1);
          if (c < cnt && row < a.f) {
            const int t = nth_bit(who, c);
            int s = 0;
            for (int q = 0; q < a.k; ++q)
              if (R.choice[t][q] == e) s = q;
            const float g = tot[0][j][i];
            const float v = g / (1.f + expf(-g)) * tot[1][j][i] * R.weight[t][s];
            float p[3];
            split3(v, p[0], p[1], p[2]);
            uint8_t* o = a.h + ((int64_t)(t * a.k + s) * a.fp + row) * 2;
#pragma unroll
            for (int q = 0; q < HT; ++q) *reinterpret_cast<uint16_t*>(o + q * a.h_plane) = bf16_bits(p[q]);
          }
        }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <typename TX, int HT, int NT, int NS>
__global__ void __launch_bounds__(kThreads, 2) moe_out_kernel(const __grid_constant__ MoeArgs a) {
  using P = qm::Pipe<1, NS, kDepthOut>;
  extern __shared__ __align__(16) uint8_t dsm[];
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

  // this warp's run of the list
  const int64_t v0 = u0 + (u1 - u0) * warp / kWarps, v1 = u0 + (u1 - u0) * (warp + 1) / kWarps;
  P pipe;
  pipe.base = (uint32_t)__cvta_generic_to_shared(dsm) + (uint32_t)warp * P::kBytes;
  qm::TileRef<1> t_ahead, t_now;
  int ai_ahead = (int)(v0 / nc), c_ahead = (int)(v0 - (int64_t)ai_ahead * nc);
  int64_t v_ahead = v0;
  const int64_t rows[1] = {row0};
  if (v0 < v1) qm::tile_ref<1>(t_ahead, a.wo, a.active[1 + ai_ahead], rows, lane);
  auto issue = [&]() {
    pipe.issue(a.wo, t_ahead, c_ahead, v_ahead < v1, lane);
    if (v_ahead < v1) {
      ++v_ahead;
      if (++c_ahead == nc && v_ahead < v1) {
        c_ahead = 0;
        ++ai_ahead;
        qm::tile_ref<1>(t_ahead, a.wo, a.active[1 + ai_ahead], rows, lane);
      }
    }
  };
#pragma unroll
  for (int p = 0; p < kDepthOut - 1; ++p) issue();
  int ai = (int)(v0 / nc), c = (int)(v0 - (int64_t)ai * nc);
  int have = -1;
  const uint8_t* hr[NT];
  for (int64_t v = v0; v < v1; ++v) {
    if (ai != have) {
      have = ai;
      if (a.wo.zero) qm::tile_ref<1>(t_now, a.wo, a.active[1 + ai], rows, lane);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int t = 8 * j + (lane >> 2);
        const int p = t < a.T ? a.pair[ai * a.T + t] : -1;
        hr[j] = p < 0 ? nullptr : a.h + (int64_t)p * a.fp * 2 + (lane & 3) * 16;
      }
    }
    uint32_t z[1][2][NS];
    qm::load_zeros<1, NS>(z, a.wo, t_now, c);
    issue();
    qm::Chunk16<NS> f[1];
    pipe.take(f, lane);
    qm::set_zeros<1, NS>(f, z);
    qm::chunk_product<__nv_bfloat16, HT, 1, NT, NS>(
        tot, f, a.wo.zero != nullptr, a.wo.zu, live, [&](int j, int q, int s) {
          if (hr[j] == nullptr) return make_uint4(0, 0, 0, 0);
          return __ldg(reinterpret_cast<const uint4*>(hr[j] + q * a.h_plane + (int64_t)c * 256 + s * 64));
        });
    if (++c == nc) {
      c = 0;
      ++ai;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
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

template <typename TX, typename H, int TERMS, int HT, int NT, int NS, int NSO>
cudaError_t run(MoeArgs& a, cudaStream_t s) {
  const void* k1 = (const void*)moe_in_kernel<TX, H, TERMS, HT, NT, NS>;
  const void* k2 = (const void*)moe_out_kernel<TX, HT, NT, NSO>;
  constexpr size_t in_fixed = kWarps * (size_t)qm::Pipe<2, NS, kDepthIn>::kBytes + kWarps * 2 * NT * 4 * 32 * 4;
  constexpr size_t in_most = std::max(in_fixed, (size_t)(8 * NT + 1) * kMaxExperts * 4);
  constexpr size_t out_bytes = kWarps * (size_t)qm::Pipe<1, NSO, kDepthOut>::kBytes;
  static std::atomic<unsigned long long> done, done2;
  cudaError_t e = ensure_smem_limit(k1, in_most, done);
  if (e == cudaSuccess) e = ensure_smem_limit(k2, out_bytes, done2);
  if (e != cudaSuccess) return e;
  const size_t smem = std::max(in_fixed, (size_t)(a.T + 1) * a.E * 4);
  const int64_t most = (int64_t)std::min(a.E, a.T * a.k) * ((a.f + 15) / 16);
  // two blocks per SM, not more than there can be items
  int64_t clusters = std::min<int64_t>(2 * sm_count() / kCluster, (most + kCluster - 1) / kCluster);
  e = launch_cluster(k1, (unsigned)(clusters * kCluster), kCluster, smem, a, s);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (a.d + 15) / 16;
  const int64_t units = (int64_t)std::min(a.E, a.T * a.k) * a.wo.nc;
  int S = 1;
  while (S < 8 && tiles * S < 2 * sm_count() && units >= (int64_t)2 * S * kWarps) S *= 2;
  return launch_cluster(k2, (unsigned)(tiles * S), (unsigned)S, out_bytes, a, s);
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
    if (e != cudaSuccess) return launch_status(e);
  }
  return BAKRON_OK;
}
