// bakron_moe: a mixture-of-experts layer over packed experts, for few tokens.
//
//   l_te = sum_j x_tj router_ej, the top_k experts of each token with weights q,
//   h = silu(gate_e x) * (up_e x),   y_t = sum over its experts of q (w_out_e h).
//
// The layer is bound by the bytes of the experts that any token chose: every
// expert's matrices are read once for all its tokens.  Three launches, or four:
//
// moe_route_kernel forms the logits, one block per expert and two tokens.  (Formed
// by every block of the next launch instead, the same rows went to all SMs and
// took 58 us at 16 tokens x 8 experts x 4096 and 5.6 us at 1 x 32 x 1024; this
// launch, chained to the next without a gap, takes about 3.)
//
// moe_in_kernel.  Every block selects the experts from the logits.  The work
// that follows is a list of (chosen expert, 16 rows of gate and the same 16 of up), cut into
// equal runs, one per block, so that a block meets one expert or two and holds
// that expert's tokens in shared memory; they are the columns of the matrix
// instructions (qmma.cuh).  A warp takes whole items, or a part of the columns
// of one when there are fewer items than warps.  h leaves multiplied by q, in two
// bf16 terms, rounded, so that the second product sees it to 2^-17 (cut off: 2^-15,
// always towards zero); fp32's three terms hold it whole.
//
// moe_out_kernel.  A block owns 256 rows of y (32 per warp) and a run of the list
// of (chosen expert, chunk of f); the expert's tokens are again the columns, and
// their sums go to the block's part of the workspace when the expert changes (kept
// in shared memory instead, 32 tokens' sums left room for one block per SM).
// The blocks that share rows are joined in rank order: for up to four tokens by
// the last of them to arrive (a counter that the launch before cleared), so
// nothing depends on who was last; for more by moe_join_kernel, as one block
// per row group was slow to read many tokens' sums (32 tokens, 8 experts of 4096 x 4096,
// with the sums moved: 209 -> 128 us).
// (As clusters of 16 with the sums in distributed shared memory not all blocks fitted
// at once: 184 us against 122 at 16 tokens x 8 experts of 4096 x 14336.)
//
// Measured: 16 tokens, 8 experts of 4096 x 14336, two each, bf16: 231 to 262 us by routing
// (an expert with more than eight tokens takes the loop for two column tiles), of which
// the two products about 130 and 100 alone, against 111 for the experts' bytes: latency
// and the instructions per code bound them, as in the few-token product (50 to 54 % of
// the issue slots, 24 % of the warps).  All loops of a kernel share 128 registers and
// spill; 2 to 3 % of the executed instructions are spills' there, 4 in fp32, 7 for one
// token.  One token, 4 of 32 experts of 1024 x 704: 27 us, latencies of the launches and
// of the selection.  Every 32 tokens read their experts again: 2048 tokens, 8 experts of
// 4096 x 4096, take 8.4 ms.
#include <algorithm>
#include <type_traits>

#include "linear.cuh"
#include "qmma.cuh"

namespace bakron {

namespace {

constexpr int kInWarps = 16, kInThreads = 32 * kInWarps;
constexpr int kOutWarps = 8, kOutThreads = 32 * kOutWarps;
constexpr int kOutRows = 32 * kOutWarps;
constexpr int kRouteWarps = 8, kRouteTokens = 2;
constexpr int kLastTokens = 4;                  // up to which moe_out_kernel joins its blocks' sums itself
constexpr int kMaxTokens = BAKRON_MOE_TOKENS;
constexpr int kMaxTopK = 16;
constexpr int kMaxExperts = 1024;
constexpr int kDepthIn = 2, kDepthOut = 2;      // slots of two chunks per warp
template <int NS>
constexpr uint32_t kInX = NS == 1 ? 64 * 1024 : 48 * 1024;     // shared memory for an expert's tokens
template <int NS>
constexpr uint32_t kOutX = NS == 1 ? 40 * 1024 : 28 * 1024;    // and for their h: two blocks per SM
// Tokens of one launch: fp32 ones take three times the room.
constexpr int launch_tokens(int terms) { return terms == 1 ? kMaxTokens : kMaxTokens / 2; }

struct MoeArgs {
  const void* x;        // T x d
  const void* router;   // E x d
  int T, E, k;
  int renormalize;
  int x_vec, vec_ok;    // rows of x (of x and the router) are 16-byte aligned
  int64_t d, f, fp;     // fp: f rounded up to 128
  PackedView wi, wo;
  uint8_t* h;           // terms x (T k) x fp 16-bit values
  int64_t h_plane;
  int* active;          // [0] chosen experts na, then their indices
  uint32_t* who;        // [na]: bit t set where token t chose the expert
  uint8_t* slot;        // [na][T]: which of its choices
  float* logits;        // [T][E]
  int* arrived;         // [row groups of y], for up to kLastTokens tokens
  float* part;          // [row groups][S][T][256]
  int row_groups, S;    // blocks per row group of y
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

// logits[t][e] of one expert and kRouteTokens tokens; the warps split the columns
// and their parts are added in a fixed order.
template <typename TX>
__global__ void __launch_bounds__(32 * kRouteWarps) moe_route_kernel(const __grid_constant__ MoeArgs a) {
  __shared__ float parts[kRouteWarps][kRouteTokens];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e = blockIdx.x, t0 = blockIdx.y * kRouteTokens;
  const TX* r = static_cast<const TX*>(a.router) + (int64_t)e * a.d;
  const TX* x = static_cast<const TX*>(a.x) + (int64_t)t0 * a.d;
  grid_dep_wait();
  grid_dep_launch();
  float acc[kRouteTokens];
#pragma unroll
  for (int t = 0; t < kRouteTokens; ++t) acc[t] = 0.f;
#pragma unroll 2
  for (int64_t c = 8 * threadIdx.x; c < a.d; c += 8 * 32 * kRouteWarps) {
    float w[8];
    load8(w, r + c, a.vec_ok != 0, a.d - c);
#pragma unroll
    for (int t = 0; t < kRouteTokens; ++t) {
      if (t0 + t < a.T) {
        float v[8];
        load8(v, x + (int64_t)t * a.d + c, a.vec_ok != 0, a.d - c);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[t] = fmaf(v[i], w[i], acc[t]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < kRouteTokens; ++t) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
    if (lane == 0) parts[warp][t] = acc[t];
  }
  __syncthreads();
  if (threadIdx.x < kRouteTokens && t0 + (int)threadIdx.x < a.T) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kRouteWarps; ++w) v += parts[w][threadIdx.x];
    a.logits[(t0 + threadIdx.x) * a.E + e] = v;
  }
}

// A key that orders floats as unsigned integers; NaN lowest.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0u;
  const uint32_t u = __float_as_uint(v == 0.f ? 0.f : v);   // -0 ties with 0
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// The experts of one token (one warp): choice[i], weight[i] for i < k, the
// largest logits first, a tie to the lowest index.  NaN logits rank last and
// make the weights NaN.
__device__ void select_experts(const float* l, int E, int k, bool renormalize, int* choice, float* weight,
                               int lane) {
  uint32_t taken = 0;                        // bit j: expert lane + 32 j (E <= 1024)
  float top = 0.f, mine = 0.f;
  bool bad = false;
  for (int e = lane; e < E; e += 32) bad |= l[e] != l[e];
  for (int i = 0; i < k; ++i) {
    uint32_t best = 0;
    int at = 0x7fffffff;                     // this lane's best that is not taken
    for (int j = 0; 32 * j + lane < E; ++j) {
      if (taken >> j & 1) continue;
      const uint32_t v = order_key(l[32 * j + lane]);
      if (at == 0x7fffffff || v > best) { best = v; at = 32 * j + lane; }
    }
    const uint32_t most = __reduce_max_sync(0xffffffffu, best);
    at = (int)__reduce_min_sync(0xffffffffu, best == most ? (unsigned)at : 0x7fffffffu);
    if ((at & 31) == lane) taken |= 1u << (at >> 5);
    const float v = l[at];
    if (i == 0) top = v;
    if (lane == i) {
      mine = v;
      choice[i] = at;
    }
  }
  float sum = 0.f;
  if (renormalize) {
    sum = lane < k ? expf(mine - top) : 0.f;
  } else {
    for (int e = lane; e < E; e += 32) sum += expf(l[e] - top);
  }
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

// Calls f with the number of column tiles as a constant: a kernel holds the loop
// for 1, 2 and 4 tiles of 8 tokens, and an expert with few tokens does not pay
// for registers and instructions of many.
template <typename F>
__device__ __forceinline__ void by_columns(int live, F f) {
  if (live <= 1) f(std::integral_constant<int, 1>());
  else if (live == 2) f(std::integral_constant<int, 2>());
  else f(std::integral_constant<int, 4>());
}

// Shared memory of the routing.
struct Routing {
  int choice[kMaxTokens][kMaxTopK];
  float weight[kMaxTokens][kMaxTopK];
  int na;
  int active[kMaxTokens * kMaxTopK];
  uint32_t who[kMaxTokens * kMaxTopK];                    // bit t: token t chose the expert
};

template <typename TX, typename H, int TERMS, int HT, int NS>
__global__ void __launch_bounds__(kInThreads, 1) moe_in_kernel(const __grid_constant__ MoeArgs a) {
  constexpr int kWarps = kInWarps, kThreads = kInThreads;
  extern __shared__ __align__(16) uint8_t dsm[];
  __shared__ Routing R;
  using P = qm::Pipe<2, NS, kDepthIn>;
  // the routing's arrays end before the chunks' slots and the tokens begin
  uint8_t* xs = dsm + kWarps * P::kBytes;
  float* logits = reinterpret_cast<float*>(dsm);               // [T][E]
  int* slot_of = reinterpret_cast<int*>(logits + a.T * a.E);   // [E]: index among the chosen, or -1
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  grid_dep_launch();
  for (int i = threadIdx.x; i < a.T * a.E; i += kThreads) logits[i] = __ldcg(a.logits + i);
  for (int e = threadIdx.x; e < a.E; e += kThreads) slot_of[e] = -1;
  __syncthreads();
  for (int t = warp; t < a.T; t += kWarps)
    select_experts(logits + t * a.E, a.E, a.k, a.renormalize != 0, R.choice[t], R.weight[t], lane);
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
  if (blockIdx.x == 0) {
    // for the second launch: the chosen experts, and who chose them
    for (int i = threadIdx.x; i < a.T * a.k; i += kThreads)
      a.slot[slot_of[R.choice[i / a.k][i % a.k]] * a.T + i / a.k] = (uint8_t)(i % a.k);
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < a.row_groups; i += kThreads) a.arrived[i] = 0;
    if (threadIdx.x == 0) a.active[0] = na;
    for (int i = threadIdx.x; i < na; i += kThreads) {
      a.active[1 + i] = R.active[i];
      a.who[i] = R.who[i];
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

  // This block's run of items (expert, row tile); G warps per item.
  const int tiles = (int)((a.f + 15) / 16);
  const int64_t items = (int64_t)na * tiles;
  const int i_lo = (int)(items * blockIdx.x / gridDim.x), i_hi = (int)(items * (blockIdx.x + 1) / gridDim.x);
  const int nc = (int)a.wi.nc;
  const int np = (nc + 1) / 2;             // pairs of chunks
  auto segment_end = [&](int it) { return min(i_hi, (it / tiles + 1) * tiles); };
  // warps per item: as many as the run's fullest expert leaves without one
  int most = 1;
  for (int it = i_lo; it < i_hi;) {
    const int end = segment_end(it);
    most = max(most, end - it);
    it = end;
  }
  int G = 1;
  while (2 * G * most <= kWarps && 2 * G <= np) G *= 2;
  const int group = warp / G, part = warp % G, groups = kWarps / G;
  const int c_lo = np * part / G * 2, c_hi = min(nc, np * (part + 1) / G * 2);

  P pipe;
  pipe.base = (uint32_t)__cvta_generic_to_shared(dsm) + (uint32_t)warp * P::kBytes;
  auto open_item = [&](qm::TileRef<2>& t, int it) {
    const int ai = it / tiles;
    const int64_t r0 = (int64_t)(it - ai * tiles) * 16;
    const int64_t rows[2] = {r0, a.f + r0};
    qm::tile_ref<2>(t, a.wi, R.active[ai], rows, lane);
  };
  // a warp's items: group, group + groups, ... of each expert's part of the run
  auto next_item = [&](int it, int seg_end) { return it + groups < seg_end ? it + groups : -1; };
  qm::TileRef<2> t_ahead, t_now;
  int seg_a = i_lo, seg_a_end = i_lo < i_hi ? segment_end(i_lo) : i_lo;   // where the copies are
  int it_ahead = -1, c_ahead = c_lo;
  auto settle = [&]() {      // first item of this warp at or after segment seg_a
    while (it_ahead < 0 && seg_a < i_hi) {
      if (seg_a + group < seg_a_end) {
        it_ahead = seg_a + group;
      } else {
        seg_a = seg_a_end;
        if (seg_a < i_hi) seg_a_end = segment_end(seg_a);
      }
    }
    if (it_ahead >= 0) open_item(t_ahead, it_ahead);
  };
  settle();
  auto issue = [&]() {
    const int n = it_ahead >= 0 ? min(2, c_hi - c_ahead) : 0;
    pipe.issue(a.wi, t_ahead, c_ahead, n, lane);
    c_ahead += n;
    if (it_ahead >= 0 && c_ahead == c_hi) {
      c_ahead = c_lo;
      it_ahead = next_item(it_ahead, seg_a_end);
      if (it_ahead < 0) {
        seg_a = seg_a_end;
        if (seg_a < i_hi) seg_a_end = segment_end(seg_a);
        settle();
      } else {
        open_item(t_ahead, it_ahead);
      }
    }
  };
  __syncthreads();             // the routing's arrays are done with
#pragma unroll
  for (int p = 0; p < kDepthIn - 1; ++p) issue();

  const uint32_t xs_addr = (uint32_t)__cvta_generic_to_shared(xs);
  for (int seg = i_lo; seg < i_hi;) {
    const int end = segment_end(seg);
    const int ai = seg / tiles, e = R.active[ai];
    const uint32_t who = R.who[ai];
    const int cnt = __popc(who), live = (cnt + 7) / 8;
    // the expert's tokens: all columns at once, or slab by slab
    const int room = (int)((kInX<NS> / (uint32_t)(TERMS * cnt) - 64) / 256);
    const int slab = room >= nc ? nc : room & ~1;
    const uint32_t pitch = qm::x_pitch(slab), plane = pitch * (uint32_t)cnt;
    auto stage = [&](int s0) {
      qm::stage_x<TX, TERMS>(xs, plane, pitch, static_cast<const TX*>(a.x), a.d, cnt,
                             [&](int r) { return (int64_t)nth_bit(who, r); }, (int64_t)s0 * 128, min(slab, nc - s0),
                             a.d, a.x_vec != 0);
    };
    __syncthreads();
    if (slab == nc) {
      stage(0);
      __syncthreads();
    }
    const int rounds = (end - seg + groups - 1) / groups;    // the same for every warp
    // NT column tiles of tokens
    auto rounds_of = [&](auto nt_) {
    constexpr int NT = decltype(nt_)::value;
    uint32_t col[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
      col[j] = xs_addr + (uint32_t)min(8 * j + (lane >> 2), cnt - 1) * pitch + (uint32_t)(lane & 3) * 16;
    for (int r = 0; r < rounds; ++r) {
      const int it = seg + r * groups + group;
      const bool on = it < end;
      const int64_t row0 = (int64_t)(it - ai * tiles) * 16;
      if (on && a.wi.zero) open_item(t_now, it);
      float tot[2][NT][4];
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) tot[q][j][i] = 0.f;
      uint32_t z[2][2][NS];
      if (on) qm::load_zeros<2, NS>(z, a.wi, t_now, c_lo);
      for (int s0 = 0; s0 < nc; s0 += slab) {
        if (slab < nc) {
          __syncthreads();
          stage(s0);
          __syncthreads();
        }
        if (on) {
          // slabs are even and so is each warp's first chunk: a slot never straddles two
          const int s1 = min(s0 + slab, c_hi);
          for (int c = max(s0, c_lo); c < s1; c += 2) {
            issue();
            pipe.wait();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (c + h < s1) {
                qm::Chunk16<NS> f[2];
                pipe.take(f, h, lane);
                qm::set_zeros<2, NS>(f, z);
                if (c + h + 1 < c_hi) qm::load_zeros<2, NS>(z, a.wi, t_now, c + h + 1);
                const uint32_t xc = (uint32_t)(c + h - s0) * 256;
                qm::chunk_product<H, TERMS, 2, NT, NS>(
                    tot, f, a.wi.zero != nullptr, a.wi.zu,
                    [&](int j, int q, int s) { return qm::lds128(col[j] + q * plane + xc + s * 64); });
              }
            }
            pipe.release();
          }
        }
      }
      // the group's sums of gate and up (thread: rows lane / 4 and + 8, columns
      // 2 (lane & 3) and + 1 of each column tile); the joins use the tokens' area, which
      // is free: G > 1 where no expert of the run has more items than there are
      // groups, so this is the only round
      if (G > 1) {
        float* mine = reinterpret_cast<float*>(xs) + (size_t)warp * (NT * 4 * 32) + lane;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          __syncthreads();
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) mine[(j * 4 + i) * 32] = tot[q][j][i];
          __syncthreads();
          if (part == 0) {
            for (int w = 1; w < G; ++w) {
#pragma unroll
              for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) tot[q][j][i] += mine[(size_t)w * (NT * 4 * 32) + (j * 4 + i) * 32];
            }
          }
        }
      }
      if (on && part == 0) {
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
              if constexpr (HT == 2) split3_near(v, p[0], p[1], p[2]);
              else split3(v, p[0], p[1], p[2]);
              uint8_t* o = a.h + ((int64_t)(t * a.k + s) * a.fp + row) * 2;
#pragma unroll
              for (int q = 0; q < HT; ++q) *reinterpret_cast<uint16_t*>(o + q * a.h_plane) = bf16_bits(p[q]);
            }
          }
      }
    }
    };
    by_columns(live, rounds_of);
    seg = end;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Rows 4 i .. 4 i + 3 (over the tokens) of a row group of y: its blocks' sums in
// rank order.
template <typename TX>
__device__ __forceinline__ void join_sums(const MoeArgs& a, int rg, int i) {
  const int n4 = a.T * kOutRows / 4;
  const float4* all = reinterpret_cast<const float4*>(a.part) + (int64_t)rg * a.S * n4 + i;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < a.S; k0 += 8) {       // eight blocks' sums on their way at a time
    float4 p[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      p[k] = k0 + k < a.S ? __ldcg(all + (int64_t)(k0 + k) * n4) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v.x += p[k].x;
      v.y += p[k].y;
      v.z += p[k].z;
      v.w += p[k].w;
    }
  }
  const int64_t row = (int64_t)rg * kOutRows + 4 * i % kOutRows;
  TX* o = static_cast<TX*>(a.y) + (int64_t)(4 * i / kOutRows) * a.d + row;
  if (row < a.d) o[0] = from_float<TX>(v.x);
  if (row + 1 < a.d) o[1] = from_float<TX>(v.y);
  if (row + 2 < a.d) o[2] = from_float<TX>(v.z);
  if (row + 3 < a.d) o[3] = from_float<TX>(v.w);
}

template <typename TX, int HT, int NS>
__global__ void __launch_bounds__(kOutThreads, 2) moe_out_kernel(const __grid_constant__ MoeArgs a) {
  constexpr int kWarps = kOutWarps, kThreads = kOutThreads;
  using P = qm::Pipe<2, NS, kDepthOut>;
  extern __shared__ __align__(16) uint8_t dsm[];
  uint8_t* hs = dsm + kWarps * P::kBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = a.S, rank = blockIdx.x % S, rg = blockIdx.x / S;
  __shared__ int last;
  const int64_t row0 = (int64_t)rg * kOutRows;
  grid_dep_wait();
  grid_dep_launch();
  const int na = a.active[0];
  const int nc = (int)a.wo.nc;
  const int units = na * nc;                                // (expert, chunk)
  const int u0 = (int)((int64_t)units * rank / S), u1 = (int)((int64_t)units * (rank + 1) / S);
  // the block's sums [T][256].  A token is another column, and so another lane's, for each
  // expert; what its sums were is seen because the warps meet (__syncthreads) when the
  // next expert's h is staged
  float* mine = a.part + ((int64_t)rg * S + rank) * a.T * kOutRows;
  uint32_t seen = 0;                                        // tokens that have sums

  // chunks of an expert's h that are staged at a time, of `part` chunks in all:
  // an even number, unless it is all of them or there is room for one only
  auto slab_of = [&](int ai, int part) {
    const int room = (int)((kOutX<NS> / (uint32_t)(HT * __popc(a.who[ai])) - 64) / 256);
    return room >= part ? part : max(1, room & ~1);
  };
  const int64_t rows[2] = {row0 + 32 * warp, row0 + 32 * warp + 16};
  P pipe;
  pipe.base = (uint32_t)__cvta_generic_to_shared(dsm) + (uint32_t)warp * P::kBytes;
  qm::TileRef<2> t_ahead, t_now;
  int u_ahead = u0, ai_ahead = u0 / nc, c_ahead = u0 - ai_ahead * nc;
  if (u0 < u1) qm::tile_ref<2>(t_ahead, a.wo, a.active[1 + ai_ahead], rows, lane);
  // two chunks at a time, fewer at the end of an expert's part of the run or of
  // what is staged of its h
  int slab_ahead = u0 < u1 ? slab_of(ai_ahead, min(nc, c_ahead + (u1 - u0)) - c_ahead) : 0;
  int left = slab_ahead;                                    // of the slab
  auto issue = [&]() {
    const int n = u_ahead < u1 ? min(min(2, left), min(u1 - u_ahead, nc - c_ahead)) : 0;
    pipe.issue(a.wo, t_ahead, c_ahead, n, lane);
    u_ahead += n;
    c_ahead += n;
    left -= n;
    if (left == 0) left = slab_ahead;
    if (n > 0 && c_ahead == nc && u_ahead < u1) {
      c_ahead = 0;
      ++ai_ahead;
      left = slab_ahead = slab_of(ai_ahead, min(nc, u1 - u_ahead));
      qm::tile_ref<2>(t_ahead, a.wo, a.active[1 + ai_ahead], rows, lane);
    }
  };
#pragma unroll
  for (int p = 0; p < kDepthOut - 1; ++p) issue();

  const uint32_t hs_addr = (uint32_t)__cvta_generic_to_shared(hs);
  for (int u = u0; u < u1;) {
    const int ai = u / nc, c0 = u - ai * nc;
    const int c1 = min(nc, c0 + (u1 - u));                  // this block's chunks of the expert
    const uint32_t who = a.who[ai];
    const int cnt = __popc(who), live = (cnt + 7) / 8;
    if (a.wo.zero) qm::tile_ref<2>(t_now, a.wo, a.active[1 + ai], rows, lane);
    const int slab = slab_of(ai, c1 - c0);
    const uint32_t pitch = qm::x_pitch(slab), plane = pitch * (uint32_t)cnt;
    auto chunks_of = [&](auto nt_) {
    constexpr int NT = decltype(nt_)::value;
    uint32_t col[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
      col[j] = hs_addr + (uint32_t)min(8 * j + (lane >> 2), cnt - 1) * pitch + (uint32_t)(lane & 3) * 16;
    float tot[2][NT][4];
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) tot[q][j][i] = 0.f;
    uint32_t z[2][2][NS];
    qm::load_zeros<2, NS>(z, a.wo, t_now, c0);
    for (int s0 = c0; s0 < c1; s0 += slab) {
      const int s1 = min(s0 + slab, c1);
      __syncthreads();
      const int per = (s1 - s0) * 16;
      for (int i = threadIdx.x; i < HT * cnt * per; i += kThreads) {
        const int row = i / per, p = i - row * per;
        const int q = row / cnt, t = nth_bit(who, row - q * cnt);
        const uint8_t* src = a.h + q * a.h_plane + (int64_t)(t * a.k + a.slot[ai * a.T + t]) * a.fp * 2;
        *reinterpret_cast<uint4*>(hs + q * plane + (row - q * cnt) * pitch + p * 16) =
            *reinterpret_cast<const uint4*>(src + (int64_t)s0 * 256 + p * 16);
      }
      __syncthreads();
      for (int c = s0; c < s1; c += 2) {
        issue();
        pipe.wait();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (c + h < s1) {
            qm::Chunk16<NS> f[2];
            pipe.take(f, h, lane);
            qm::set_zeros<2, NS>(f, z);
            if (c + h + 1 < c1) qm::load_zeros<2, NS>(z, a.wo, t_now, c + h + 1);
            const uint32_t hc = (uint32_t)(c + h - s0) * 256;
            qm::chunk_product<__nv_bfloat16, HT, 2, NT, NS>(
                tot, f, a.wo.zero != nullptr, a.wo.zu,
                [&](int j, int q, int s) { return qm::lds128(col[j] + q * plane + hc + s * 64); });
          }
        }
        pipe.release();
      }
    }
    // to the tokens' sums
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = 8 * j + 2 * (lane & 3) + i;
        if (c < cnt) {
          const int t = nth_bit(who, c);
          float* to = mine + t * kOutRows + 32 * warp + (lane >> 2);
          const bool more = seen >> t & 1;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float v = tot[q >> 1][j][i + 2 * (q & 1)];
            to[8 * q] = more ? to[8 * q] + v : v;
          }
        }
      }
    };
    by_columns(live, chunks_of);
    seen |= who;
    u += c1 - c0;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  for (int i = threadIdx.x; i < a.T * kOutRows; i += kThreads)
    if (!(seen >> (i / kOutRows) & 1)) mine[i] = 0.f;
  if (a.T > kLastTokens) return;             // moe_join_kernel follows
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(&a.arrived[rg], 1) == S - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  for (int i = threadIdx.x; i < a.T * kOutRows / 4; i += kThreads) join_sums<TX>(a, rg, i);
}

// One block per row group and 256 groups of four rows of a token.
template <typename TX>
__global__ void __launch_bounds__(kOutThreads) moe_join_kernel(const __grid_constant__ MoeArgs a) {
  const int i = blockIdx.y * kOutThreads + threadIdx.x;
  grid_dep_wait();
  grid_dep_launch();
  if (i < a.T * kOutRows / 4) join_sums<TX>(a, blockIdx.x, i);
}

// Blocks that share a row group of y: two blocks per SM in all, each with a
// unit at least.
int out_split(int64_t d, int64_t T, int64_t E, int k, int64_t nc) {
  const int64_t groups = (d + kOutRows - 1) / kOutRows;
  const int64_t units = std::min<int64_t>(E, T * k) * nc;
  return (int)std::max<int64_t>(1, std::min<int64_t>(2 * sm_count() / groups, units));
}

template <typename TX, typename H, int TERMS, int HT, int NS, int NSO>
cudaError_t run(MoeArgs& a, cudaStream_t s) {
  auto k1 = moe_in_kernel<TX, H, TERMS, HT, NS>;
  auto k2 = moe_out_kernel<TX, HT, NSO>;
  static_assert(kInX<NS> / (TERMS * launch_tokens(TERMS)) >= 2 * 256 + 64, "two chunks of every token fit");
  static_assert(kOutX<NSO> / (HT * launch_tokens(TERMS)) >= 256 + 64, "one chunk of every token's h fits");
  constexpr size_t pipes = kInWarps * (size_t)qm::Pipe<2, NS, kDepthIn>::kBytes;
  static_assert(kInWarps * (kMaxTokens / 8) * 4 * 32 * 4 <= kInX<NS>, "the joins fit the tokens' area");
  constexpr size_t in_bytes = std::max(pipes + kInX<NS>, (size_t)(kMaxTokens + 1) * kMaxExperts * 4);
  constexpr size_t out_bytes = kOutWarps * (size_t)qm::Pipe<2, NSO, kDepthOut>::kBytes + kOutX<NSO>;
  static_assert(2 * (out_bytes + 1024 + 64) <= 228 * 1024, "two blocks per SM");
  static std::atomic<unsigned long long> done, done2;
  cudaError_t e = ensure_smem_limit((const void*)k1, in_bytes, done);
  if (e == cudaSuccess)
    e = ensure_smem_limit((const void*)k2, out_bytes, done2);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)a.E, (unsigned)((a.T + kRouteTokens - 1) / kRouteTokens));
  cfg.blockDim = dim3(32 * kRouteWarps);
  count_launch(a.T > kLastTokens ? 4 : 3);
  e = cudaLaunchKernelEx(&cfg, moe_route_kernel<TX>, a);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)sm_count());    // one block per SM
  cfg.blockDim = dim3(kInThreads);
  cfg.dynamicSmemBytes = in_bytes;
  e = cudaLaunchKernelEx(&cfg, k1, a);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)(a.row_groups * a.S));
  cfg.blockDim = dim3(kOutThreads);
  cfg.dynamicSmemBytes = out_bytes;
  e = cudaLaunchKernelEx(&cfg, k2, a);
  if (e != cudaSuccess || a.T <= kLastTokens) return e;
  cfg.gridDim = dim3((unsigned)a.row_groups, (unsigned)((a.T * kOutRows / 4 + kOutThreads - 1) / kOutThreads));
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, moe_join_kernel<TX>, a);
}

template <typename TX, typename H, int TERMS, int HT>
cudaError_t by_groups(MoeArgs& a, cudaStream_t s) {
  const bool wi = a.wi.ng == 1 || a.wi.g % 128 == 0, wo = a.wo.ng == 1 || a.wo.g % 128 == 0;
  if (wi && wo) return run<TX, H, TERMS, HT, 1, 1>(a, s);
  if (wi) return run<TX, H, TERMS, HT, 1, 4>(a, s);
  if (wo) return run<TX, H, TERMS, HT, 4, 1>(a, s);
  return run<TX, H, TERMS, HT, 4, 4>(a, s);
}

struct MoeLayout {
  size_t h, active, who, slot, logits, arrived, part, total;
  int64_t fp;
};

MoeLayout moe_layout(int64_t T, int64_t d, int64_t f, int64_t E, int k, int dtype) {
  MoeLayout L;
  const int64_t t = std::min<int64_t>(T, kMaxTokens);
  const int64_t na = std::min<int64_t>(E, t * k), groups = (d + kOutRows - 1) / kOutRows;
  L.fp = (f + 127) / 128 * 128;
  size_t off = 0;
  auto take = [&](size_t b) { const size_t o = off; off += (b + 255) / 256 * 256; return o; };
  L.h = take((size_t)(dtype == BAKRON_F32 ? 3 : 2) * t * k * L.fp * 2);
  L.active = take((size_t)(1 + na) * 4);
  L.who = take((size_t)na * 4);
  L.slot = take((size_t)(na * t));
  L.logits = take((size_t)(t * E) * 4);
  L.arrived = take((size_t)groups * 4);
  // at most two blocks per SM in all (a smaller last launch may split more finely)
  L.part = take((size_t)std::max<int64_t>(groups, 2 * sm_count()) * t * kOutRows * 4);
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
  a.who = reinterpret_cast<uint32_t*>(base + L.who);
  a.slot = base + L.slot;
  a.logits = reinterpret_cast<float*>(base + L.logits);
  a.arrived = reinterpret_cast<int*>(base + L.arrived);
  a.part = reinterpret_cast<float*>(base + L.part);
  a.row_groups = (int)((a.d + kOutRows - 1) / kOutRows);
  const int64_t most = launch_tokens(dtype == BAKRON_F32 ? 3 : 1);
  for (int64_t t0 = 0; t0 < T; t0 += most) {
    a.T = (int)std::min<int64_t>(most, T - t0);
    a.x = static_cast<const uint8_t*>(X) + (size_t)(t0 * a.d) * es;
    a.y = static_cast<uint8_t*>(Y) + (size_t)(t0 * a.d) * es;
    a.h_plane = (int64_t)a.T * a.k * a.fp * 2;
    a.S = out_split(a.d, a.T, a.E, a.k, a.wo.nc);
    a.x_vec = (a.d * es) % 16 == 0 && aligned_to(a.x, 16);
    a.vec_ok = a.x_vec && aligned_to(router, 16);
    cudaError_t e;
    switch (dtype) {
      case BAKRON_F32: e = by_groups<float, __nv_bfloat16, 3, 3>(a, s); break;
      case BAKRON_BF16: e = by_groups<__nv_bfloat16, __nv_bfloat16, 1, 2>(a, s); break;
      default: e = by_groups<__half, __half, 1, 2>(a, s); break;
    }
    if (e != cudaSuccess) return launch_status(e);
  }
  return BAKRON_OK;
}
