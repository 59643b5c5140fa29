// Building blocks of the linear layer's tcgen05 kernels: 16-bit matrix
// instructions, TMEM access, waits and the position in a ring of stages.
#pragma once

#include <algorithm>

#include "act.cuh"
#include "linear.cuh"
#include "tc_common.cuh"

namespace bakron {
namespace tc {

__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

template <typename H>
struct IdescType;
template <>
struct IdescType<__half> { static constexpr uint32_t v = 0; };
template <>
struct IdescType<__nv_bfloat16> { static constexpr uint32_t v = 1; };
template <typename H>
__device__ __forceinline__ uint32_t idesc_f16(int n) {
  return (1u << 4) | (IdescType<H>::v << 7) | (IdescType<H>::v << 10) | ((uint32_t)(n >> 3) << 17) |
         ((128u >> 4) << 24);
}

// Bounded wait; the clock is read only once the first try has failed.  When it
// runs out the block records BAKRON_ERR_TIMEOUT and its other roles stop.
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, int* abort, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  volatile int* ab = abort;
  if (mbar_wait(bar, parity, ab)) return true;
  atomicCAS(status, 0, (int)BAKRON_ERR_TIMEOUT);
  *ab = 1;
  return false;
}
// Position in a ring of stages, advanced without divisions: stage s and the
// parity of its current use.
struct Ring {
  int s = 0;
  uint32_t parity = 0;
  bool first = true;      // first time round: the stage is free
  __device__ __forceinline__ void advance(int by, int stages) {
    s += by;
    if (s >= stages) {
      s -= stages;
      parity ^= 1;
      first = false;
    }
  }
};
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}


// What a tcgen05 product computes: Y = X V^T, the same with bakron_linear_act's
// epilogue, or the experts' products over rows sorted by expert (and likewise their
// gradients).
enum Product { kPlain, kWithAct, kExperts };

// A tile of the output: 128 rows m of expert e's matrix, tokens t0 to end.
struct Place {
  int m, e;
  int64_t t0, end;
};

constexpr int kTileThreads = 512;            // that fill an experts' table
constexpr int kTileBounds = 4;               // boundaries each
constexpr uint32_t kTableBytes = 2 * (kMaxGroupedExperts + 1) * 4;
static_assert(kTileThreads * kTileBounds > kMaxGroupedExperts);

// The tiles of a product.  Experts: `bounds` are the boundaries of their rows, `first`
// their first token tiles (e = 0 .. E, in shared memory).
template <Product P, typename Args>
struct Tiles {
  const Args& a;        // tiles (not for experts), tiles_m, N, T
  int64_t own;          // tiles of the experts
  const int* bounds;
  const int* first;
  int E;

  __device__ __forceinline__ int64_t count() const { return P == kExperts ? own : a.tiles; }
  __device__ __forceinline__ Place at(int64_t tile) const {
    if constexpr (P != kExperts) {
      return Place{(int)(tile % a.tiles_m), 0, tile / a.tiles_m * a.N, a.T};
    } else {
      const int tt = (int)(tile / a.tiles_m);
      int e = 0, hi = E;                     // the last expert whose first tile is at most tt
      while (hi - e > 1) {
        const int mid = (e + hi) >> 1;
        if (first[mid] <= tt) e = mid;
        else hi = mid;
      }
      return Place{(int)(tile % a.tiles_m), e, bounds[e] + (int64_t)(tt - first[e]) * a.N, bounds[e + 1]};
    }
  }
};

// Token tiles of N: at most, as each expert's rows may end within one, and
// likely, where tokens are spread about evenly.
inline int64_t token_tiles(const LinearArgs& a, int N) {
  return (a.T + N - 1) / N + (a.offsets ? std::min<int64_t>(a.w.count, a.T) : 0);
}
inline int64_t likely_tiles(const LinearArgs& a, int N) {
  if (!a.offsets) return (a.T + N - 1) / N;
  const int64_t live = std::min<int64_t>(a.w.count, a.T);
  return std::max<int64_t>(live, a.T / N + (live + 1) / 2);
}

// Fills an experts' table from their offsets (device, E + 1), a block of at least
// kTileThreads threads together; returns the number of token tiles.  An offset below an earlier
// one or outside 0 .. T counts as the nearest that is not: whatever the offsets, every
// tile lies inside the rows and no two share one.
__device__ inline int expert_tiles(const int* offsets, int E, int T, int N, int* bounds, int* first,
                                   int (*sums)[kTileThreads / 32]) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool in = tid < kTileThreads;
  int v[kTileBounds], most = 0;
#pragma unroll
  for (int i = 0; i < kTileBounds; ++i) {
    const int b = kTileBounds * tid + i;
    v[i] = in && b <= E ? min(max(__ldg(offsets + b), 0), T) : 0;
    most = v[i] = max(v[i], most);
  }
  int up = most;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up = max(up, u);
  }
  if (in && lane == 31) sums[0][warp] = up;
  int before = __shfl_up_sync(0xffffffffu, up, 1);
  if (lane == 0) before = 0;
  __syncthreads();
  if (in) {
    for (int w = 0; w < warp; ++w) before = max(before, sums[0][w]);
#pragma unroll
    for (int i = 0; i < kTileBounds; ++i)
      if (kTileBounds * tid + i <= E) bounds[kTileBounds * tid + i] = max(before, v[i]);
  }
  __syncthreads();
  int sum = 0;
#pragma unroll
  for (int i = 0; i < kTileBounds; ++i) {
    const int e = kTileBounds * tid + i;
    v[i] = sum;
    if (in && e < E) sum += (bounds[e + 1] - bounds[e] + N - 1) / N;
  }
  up = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += u;
  }
  if (in && lane == 31) sums[1][warp] = up;
  before = up - sum;
  __syncthreads();
  if (in) {
    for (int w = 0; w < warp; ++w) before += sums[1][w];
#pragma unroll
    for (int i = 0; i < kTileBounds; ++i)
      if (kTileBounds * tid + i <= E) first[kTileBounds * tid + i] = before + v[i];
  }
  __syncthreads();
  return first[E];
}

}  // namespace tc
}  // namespace bakron
