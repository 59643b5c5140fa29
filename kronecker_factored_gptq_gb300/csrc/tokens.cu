// Tokens sorted by expert and back: bakron_sort_tokens, bakron_dispatch, bakron_combine and
// bakron_combine_grad.
//
// The sort is a counting sort of n = T k choices in one launch: a block, or the blocks of a
// cluster, of up to 32 warps; each warp has a run of consecutive choices and counts them by
// expert in a row of shared memory of its own.  The sums over warps, blocks (through
// distributed shared memory) and experts turn the counts into the first place of every
// (expert, warp); then each warp walks through its run again, 32 choices at a time, and a choice's
// place is its expert's next one plus the number of lower lanes with the same expert.  Only
// whole numbers are added, and every place follows from the order of choice, so it is stable
// and the same in every run.  What bounds it is the instructions of the warps' walks, some 200 a step of
// 32 choices (one ballot a bit of the expert's number instead of the match was no faster): 64 choices 2.9 us,
// 49152 of 64 experts 11 us in a cluster of eight blocks, 16 in one of four, 50 in one block.
//
// The others move rows and are bound by their bytes: a warp takes a part of a token's row and
// every row of the token's choices, so that dispatch reads x once, whatever k.  The gradient of combine takes
// a token's choices two at a time over whole rows (their sums stay in two registers), so dy is read once for
// every two, from L1 or L2 after the first: 4096 tokens of 6 choices, rows of 4096 bf16, 70 us (the bytes, dy once:
// 64), of 8 90 (84); 1024 of 8, rows of 16384, 102 (84).  They go through
// choice order, in which the reads of x and the writes of y are consecutive.  Four blocks an SM, 64 registers a
// thread, keep enough bytes in flight; with 128 and more combine took 93 to 123 us instead of 38.
// Measured, bf16 rows of 4096 (the bytes at 6.80 TB/s): dispatch of 8192 tokens to 6 experts, 5 % padding, 71 us
// (66); combine of 8192 x 2 38 us (30), its gradient 53 us (49).  Rows that do not begin on 16 bytes take pieces of
// 8, 4 or 2 bytes.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "piece.cuh"

namespace bakron {

namespace cg = cooperative_groups;

namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxChoices = 32;              // of a token: a lane each
constexpr int64_t kMaxRows = int64_t(1) << 28;
constexpr int kMaxBlocks = 8;                // of the sort: a cluster
constexpr int kKept = 8;                     // choices of a lane at a time
constexpr int64_t kMaxWidth = int64_t(1) << 20;

// ---------------------------------------------------------------- sort

struct SortArgs {
  const void* choice;
  int n, E;
  int32_t* offsets;
  int32_t* place;
};

template <typename I>
__global__ void __launch_bounds__(1024) sort_kernel(const __grid_constant__ SortArgs a) {
  extern __shared__ int smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5, E = a.E;
  int* total = smem;                         // [E]: choices of this block
  int* first = smem + E;                     // [E]: first place
  int* count = smem + 2 * E;                 // [warps][E]
  int* mine = count + warp * E;
  __shared__ int sums[32];
  for (int i = threadIdx.x; i < warps * E; i += blockDim.x) count[i] = 0;
  __syncthreads();
  const I* choice = static_cast<const I*>(a.choice);
  // runs of whole 32s
  const int steps = (a.n + 31) / 32, w = rank * warps + warp, W = C * warps;
  const int lo = (int)((int64_t)steps * w / W) * 32, hi = min(a.n, (int)((int64_t)steps * (w + 1) / W) * 32);
  // the run's first choices stay in registers for the second walk
  int kept[kKept];
#pragma unroll
  for (int q = 0; q < kKept; ++q) {
    const int i = lo + 32 * q + lane;
    const I e = i < hi ? choice[i] : (I)-1;
    kept[q] = e >= 0 && e < E ? (int)e : -1;
  }
#pragma unroll
  for (int q = 0; q < kKept; ++q)
    if (kept[q] >= 0) atomicAdd(&mine[kept[q]], 1);
#pragma unroll 4
  for (int i = lo + 32 * kKept + lane; i < hi; i += 32) {
    const I e = choice[i];
    if (e >= 0 && e < E) atomicAdd(&mine[(int)e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int sum = 0;
    for (int v0 = 0; v0 < warps; v0 += 8) {
      int c[8];
#pragma unroll
      for (int v = 0; v < 8; ++v) c[v] = v0 + v < warps ? count[(v0 + v) * E + e] : 0;
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        if (v0 + v < warps) count[(v0 + v) * E + e] = sum;
        sum += c[v];
      }
    }
    total[e] = sum;
  }
  cluster.sync();
  // first place of each expert in this block: all choices of lower experts, and its own in
  // lower blocks
  int run = 0;                               // choices of the experts before this turn's
  for (int e0 = 0; e0 < E; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x;
    int all = 0, before = 0;
    if (e < E) {
      int c[kMaxBlocks];
#pragma unroll
      for (int q = 0; q < kMaxBlocks; ++q) c[q] = q < C ? cluster.map_shared_rank(total, q)[e] : 0;
#pragma unroll
      for (int q = 0; q < kMaxBlocks; ++q) {
        if (q < rank) before += c[q];
        all += c[q];
      }
    }
    int up = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += u;
    }
    if (lane == 31) sums[warp] = up;
    __syncthreads();
    int lower = run, whole = 0;
    for (int v = 0; v < warps; ++v) {
      if (v < warp) lower += sums[v];
      whole += sums[v];
    }
    if (e < E) {
      first[e] = lower + up - all + before;
      if (rank == 0) a.offsets[e] = lower + up - all;
    }
    run += whole;
    __syncthreads();
  }
  if (rank == 0 && threadIdx.x == 0) a.offsets[E] = run;
  // (the barrier that ended the last turn is between first[] and its use)
  auto put = [&](int i, int e) {
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    const int lower = __popc(same & ((1u << lane) - 1));
    int at = -1;
    if (e >= 0) at = first[e] + mine[e] + lower;
    __syncwarp();
    if (e >= 0 && lower == 0) mine[e] += __popc(same);
    __syncwarp();
    if (i < hi) a.place[i] = at;
  };
#pragma unroll
  for (int q = 0; q < kKept; ++q)
    if (lo + 32 * q < hi) put(lo + 32 * q + lane, kept[q]);
  for (int i0 = lo + 32 * kKept; i0 < hi; i0 += 32 * kKept) {
#pragma unroll
    for (int q = 0; q < kKept; ++q) {
      const int i = i0 + 32 * q + lane;
      const I e = i < hi ? choice[i] : (I)-1;
      kept[q] = e >= 0 && e < E ? (int)e : -1;
    }
#pragma unroll
    for (int q = 0; q < kKept; ++q)
      if (i0 + 32 * q < hi) put(i0 + 32 * q + lane, kept[q]);
  }
  __syncwarp();
  cluster.sync();                            // no block leaves while its totals are read
}

template <typename I>
cudaError_t run_sort(const SortArgs& a, cudaStream_t s) {
  auto k = sort_kernel<I>;
  // a warp per 64 choices and a thread per expert; beyond 32 warps, more blocks
  const int warps = std::min(32, std::max({4, (a.n + 63) / 64, (a.E + 31) / 32}));
  int C = 1;
  while (C < kMaxBlocks && a.n > C * 32 * 64) C *= 2;
  const size_t smem = (size_t)(warps + 2) * a.E * sizeof(int);
  static std::atomic<unsigned long long> done;
  if (smem > 46 * 1024) {
    const cudaError_t e = ensure_smem_limit((const void*)k, (size_t)34 * kMaxExperts * sizeof(int), done);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)C);
  cfg.blockDim = dim3((unsigned)(32 * warps));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, k, a);
}

// ---------------------------------------------------------------- rows

struct RowArgs {
  const void* in;       // x, rows or dy
  const void* rows;     // gradient: the rows of the forward pass
  void* out;            // rows, y or drows
  const int32_t* place;
  const float* weight;
  float* dweight;
  int64_t T, R, d;
  int k;
  int64_t vecs;         // of a row
  int64_t parts;        // warps' parts of a row
  int narrow;           // T parts is below 2^32
};

template <typename TX, int VB>
__device__ __forceinline__ Piece<TX, VB> load(const void* base, int64_t i) {
  return static_cast<const Piece<TX, VB>*>(base)[i];
}

constexpr int kThreads = 256;
// Pieces of a lane at a time: 64 bytes where they are whole, and 32 where several rows are at hand;
// more of the narrow ones (rows of 4097 bf16: combine of 4096 x 2 55 us, with two 91; rows of 4096 22).
template <int VB>
constexpr int kVecs = VB == 16 ? 4 : 8;
template <int VB>
constexpr int kWideOf = VB == 16 ? 2 : VB == 8 ? 4 : 8;

// Unit u of a.parts a token: the token (division of 32 bits where the units fit).
__device__ __forceinline__ int64_t token_of(const RowArgs& a, int64_t u) {
  return a.narrow ? (int64_t)((uint32_t)u / (uint32_t)a.parts) : u / a.parts;
}

// A token's places and weights: lane j holds choice j (R where there is none).
__device__ __forceinline__ void load_choices(const RowArgs& a, int64_t t, int lane, int& at, float& w) {
  at = -1;
  w = 1.f;
  if (lane < a.k) {
    at = __ldg(a.place + t * a.k + lane);
    if (at >= a.R) at = -1;
    if (a.weight) w = __ldg(a.weight + t * a.k + lane);
  }
}

template <typename TX, int VB, bool kWeight>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const __grid_constant__ RowArgs a) {
  using P = Piece<TX, VB>;
  const int lane = threadIdx.x & 31;
  const int64_t units = a.T * a.parts;
  for (int64_t u = blockIdx.x * (int64_t)(kThreads / 32) + (threadIdx.x >> 5); u < units;
       u += (int64_t)gridDim.x * (kThreads / 32)) {
    const int64_t t = token_of(a, u), v0 = (u - t * a.parts) * (32 * kVecs<VB>) + lane;
    int at;
    float w;
    load_choices(a, t, lane, at, w);
    P x[kVecs<VB>];
#pragma unroll
    for (int i = 0; i < kVecs<VB>; ++i)
      if (v0 + 32 * i < a.vecs) x[i] = load<TX, VB>(a.in, t * a.vecs + v0 + 32 * i);
    for (int j = 0; j < a.k; ++j) {
      const int64_t r = __shfl_sync(0xffffffffu, at, j);
      const float f = kWeight ? __shfl_sync(0xffffffffu, w, j) : 1.f;
      if (r < 0) continue;
#pragma unroll
      for (int i = 0; i < kVecs<VB>; ++i) {
        if (v0 + 32 * i >= a.vecs) continue;
        P o = x[i];
        if constexpr (kWeight) {
          float v[P::V];
#pragma unroll
          for (int e = 0; e < P::V; ++e) v[e] = f * x[i].get(e);
          o.set(v);
        }
        static_cast<P*>(a.out)[r * a.vecs + v0 + 32 * i] = o;
      }
    }
  }
}

template <typename TX, int VB>
__global__ void __launch_bounds__(kThreads, 4) combine_kernel(const __grid_constant__ RowArgs a) {
  using P = Piece<TX, VB>;
  constexpr int kAtOnce = 2, kWide = kWideOf<VB>;
  const int lane = threadIdx.x & 31;
  const int64_t units = a.T * a.parts, step = (int64_t)gridDim.x * (kThreads / 32);
  int64_t u = blockIdx.x * (int64_t)(kThreads / 32) + (threadIdx.x >> 5);
  int at_next = -1;
  float w_next = 1.f;
  if (u < units) load_choices(a, token_of(a, u), lane, at_next, w_next);
  for (; u < units; u += step) {
    const int64_t t = token_of(a, u), v0 = (u - t * a.parts) * (32 * kWide) + lane;
    const int at = at_next;
    const float w = w_next;
    if (u + step < units) load_choices(a, token_of(a, u + step), lane, at_next, w_next);
    float sum[kWide][P::V];
#pragma unroll
    for (int i = 0; i < kWide; ++i)
#pragma unroll
      for (int e = 0; e < P::V; ++e) sum[i][e] = 0.f;
    for (int j0 = 0; j0 < a.k; j0 += kAtOnce) {
      P x[kAtOnce][kWide];
      float f[kAtOnce];
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q) {
        const int r = __shfl_sync(0xffffffffu, at, (j0 + q) & 31);
        const bool there = r >= 0 && j0 + q < a.k;
        f[q] = __shfl_sync(0xffffffffu, w, (j0 + q) & 31);
        const P* row = static_cast<const P*>(a.in) + (int64_t)(there ? r : 0) * a.vecs + v0;
#pragma unroll
        for (int i = 0; i < kWide; ++i) {
          if (there && v0 + 32 * i < a.vecs) x[q][i] = row[32 * i];
        }
        if (!there) f[q] = 0.f;
        if (!there) {
#pragma unroll
          for (int i = 0; i < kWide; ++i) x[q][i] = P{};
        }
      }
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q)
#pragma unroll
        for (int i = 0; i < kWide; ++i)
#pragma unroll
          for (int e = 0; e < P::V; ++e) sum[i][e] = fmaf(f[q], x[q][i].get(e), sum[i][e]);
    }
#pragma unroll
    for (int i = 0; i < kWide; ++i) {
      if (v0 + 32 * i >= a.vecs) continue;
      P o;
      o.set(sum[i]);
      static_cast<P*>(a.out)[t * a.vecs + v0 + 32 * i] = o;
    }
  }
}

// A block per token (or a warp, blockDim 32 x several tokens): dy's row meets every row of the
// token's choices, kAtOnce of them together; the products are joined over the lanes and then
// the warps in a fixed order.
template <typename TX, int VB, bool kBlock>
__global__ void __launch_bounds__(kThreads, 4) combine_grad_kernel(const __grid_constant__ RowArgs a) {
  using P = Piece<TX, VB>;
  constexpr int kAtOnce = 2, kWide = kWideOf<VB>;
  __shared__ float red[2][kAtOnce][kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t step = kBlock ? gridDim.x : (int64_t)gridDim.x * warps;
  const int first = kBlock ? threadIdx.x : lane, width = kBlock ? blockDim.x : 32;
  int slot = 0, at_next = -1;
  float w_next = 1.f;
  int64_t t = kBlock ? blockIdx.x : blockIdx.x * (int64_t)warps + warp;
  if (t < a.T) load_choices(a, t, lane, at_next, w_next);
  for (; t < a.T; t += step) {
    const int at = at_next;
    const float w = w_next;
    if (t + step < a.T) load_choices(a, t + step, lane, at_next, w_next);
    for (int j0 = 0; j0 < a.k; j0 += kAtOnce) {
      int r[kAtOnce];
      float f[kAtOnce], dot[kAtOnce];
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q) {
        r[q] = __shfl_sync(0xffffffffu, at, (j0 + q) & 31);
        f[q] = __shfl_sync(0xffffffffu, w, (j0 + q) & 31);
        if (j0 + q >= a.k) r[q] = -1;
        dot[q] = 0.f;
      }
      for (int64_t v = first; v < a.vecs; v += (int64_t)width * kWide) {
        P d[kWide], x[kAtOnce][kWide];
#pragma unroll
        for (int i = 0; i < kWide; ++i) {
          const int64_t c = v + (int64_t)i * width;
          if (c >= a.vecs) continue;
          d[i] = load<TX, VB>(a.in, t * a.vecs + c);
#pragma unroll
          for (int q = 0; q < kAtOnce; ++q)
            if (r[q] >= 0) x[q][i] = load<TX, VB>(a.rows, (int64_t)r[q] * a.vecs + c);
        }
#pragma unroll
        for (int i = 0; i < kWide; ++i) {
          const int64_t c = v + (int64_t)i * width;
          if (c >= a.vecs) continue;
#pragma unroll
          for (int q = 0; q < kAtOnce; ++q) {
            if (r[q] < 0) continue;
            P o;
            float v[P::V];
#pragma unroll
            for (int e = 0; e < P::V; ++e) {
              const float g = d[i].get(e);
              dot[q] = fmaf(g, x[q][i].get(e), dot[q]);
              v[e] = f[q] * g;
            }
            o.set(v);
            static_cast<P*>(a.out)[(int64_t)r[q] * a.vecs + c] = o;
          }
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) dot[q] += __shfl_xor_sync(0xffffffffu, dot[q], o);
      if constexpr (kBlock) {
        // the slots alternate: one is written again only after the barrier in between
        if (lane == 0) {
#pragma unroll
          for (int q = 0; q < kAtOnce; ++q) red[slot][q][warp] = dot[q];
        }
        __syncthreads();
        if (threadIdx.x < kAtOnce && j0 + (int)threadIdx.x < a.k) {
          float v = 0.f;
          for (int u = 0; u < warps; ++u) v += red[slot][threadIdx.x][u];
          a.dweight[t * a.k + j0 + threadIdx.x] = v;
        }
        slot ^= 1;
      } else {
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q)
          if (lane == q && j0 + q < a.k) a.dweight[t * a.k + j0 + q] = dot[q];
      }
    }
  }
}

enum class Op { kDispatch, kCombine, kCombineGrad };

template <typename TX, int VB>
cudaError_t launch_rows(RowArgs& a, Op op, cudaStream_t s) {
  a.vecs = a.d * (int64_t)sizeof(TX) / VB;
  const int per = 32 * (op == Op::kCombine ? kWideOf<VB> : kVecs<VB>);
  a.parts = (a.vecs + per - 1) / per;
  a.narrow = a.T * a.parts < (int64_t(1) << 32);
  // dispatch_kernel's warps take a unit or few, the others loop, with the next choices on their way
  const int64_t most = (int64_t)sm_count() * (op == Op::kDispatch ? 64 : 4);
  const unsigned blocks = (unsigned)std::min<int64_t>(most, (a.T * a.parts + kThreads / 32 - 1) / (kThreads / 32));
  count_launch();
  if (op == Op::kDispatch) {
    if (a.weight) dispatch_kernel<TX, VB, true><<<blocks, kThreads, 0, s>>>(a);
    else dispatch_kernel<TX, VB, false><<<blocks, kThreads, 0, s>>>(a);
  } else if (op == Op::kCombine) {
    combine_kernel<TX, VB><<<blocks, kThreads, 0, s>>>(a);
  } else if (a.vecs <= 128) {
    combine_grad_kernel<TX, VB, false><<<(unsigned)std::min<int64_t>(most, (a.T + 7) / 8), kThreads, 0, s>>>(a);
  } else {
    combine_grad_kernel<TX, VB, true><<<(unsigned)std::min<int64_t>(most, a.T), kThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

// The widest pieces that rows and addresses allow.
template <typename TX>
cudaError_t by_width(RowArgs& a, Op op, cudaStream_t s) {
  const uintptr_t all = (uintptr_t)(a.d * (int64_t)sizeof(TX)) | reinterpret_cast<uintptr_t>(a.in) |
                        reinterpret_cast<uintptr_t>(a.out) | reinterpret_cast<uintptr_t>(a.rows);
  if (all % 16 == 0) return launch_rows<TX, 16>(a, op, s);
  if (all % 8 == 0) return launch_rows<TX, 8>(a, op, s);
  if constexpr (sizeof(TX) == 4) return launch_rows<TX, 4>(a, op, s);
  else return all % 4 == 0 ? launch_rows<TX, 4>(a, op, s) : launch_rows<TX, 2>(a, op, s);
}

bakron_status run_rows(RowArgs& a, int dtype, Op op, void* stream) {
  cudaStream_t s = (cudaStream_t)stream;
  switch (dtype) {
    case BAKRON_F32: return launch_status(by_width<float>(a, op, s));
    case BAKRON_BF16: return launch_status(by_width<__nv_bfloat16>(a, op, s));
    default: return launch_status(by_width<__half>(a, op, s));
  }
}

// What the calls on rows share; `one` is the array of T x d, `many` that of R x d.
bool row_args(const void* one, const void* many, int64_t T, int64_t R, int64_t d, int dtype, const int32_t* place,
              int k, const float* weight, RowArgs* a) {
  if (!dtype_ok(dtype) || T < 0 || T > kMaxRows || R < 0 || R > kMaxRows || d < 1 || d > kMaxWidth || k < 1 ||
      k > kMaxChoices || T * k > kMaxRows)
    return false;
  const size_t es = dtype_size(dtype);
  if (T > 0 && (!one || !place || !aligned_to(one, es) || !aligned_to(place, 4) || !aligned_to(weight, 4))) return false;
  if (T > 0 && R > 0 && (!many || !aligned_to(many, es))) return false;
  *a = {};
  a->T = T;
  a->R = R;
  a->d = d;
  a->k = k;
  a->place = place;
  a->weight = weight;
  return true;
}

}  // namespace
}  // namespace bakron

using namespace bakron;

extern "C" bakron_status bakron_sort_tokens(const void* choice, int choice_bytes, int64_t T, int k, int E,
                                            int32_t* offsets, int32_t* place, void* stream) {
  if ((choice_bytes != 4 && choice_bytes != 8) || T < 0 || T > kMaxRows || k < 1 || k > kMaxChoices ||
      T * k > kMaxRows || E < 1 || E > kMaxExperts || !offsets || !aligned_to(offsets, 4))
    return BAKRON_ERR_INVALID_ARG;
  if (T > 0 && (!choice || !place || !aligned_to(choice, (size_t)choice_bytes) || !aligned_to(place, 4)))
    return BAKRON_ERR_INVALID_ARG;
  SortArgs a = {choice, (int)(T * k), E, offsets, place};
  cudaStream_t s = (cudaStream_t)stream;
  return launch_status(choice_bytes == 4 ? run_sort<int32_t>(a, s) : run_sort<int64_t>(a, s));
}

extern "C" bakron_status bakron_dispatch(const void* X, int64_t T, int64_t d, int dtype, const int32_t* place,
                                         int k, const float* weight, void* rows, int64_t R, void* stream) {
  RowArgs a;
  if (!row_args(X, rows, T, R, d, dtype, place, k, weight, &a)) return BAKRON_ERR_INVALID_ARG;
  if (T == 0 || R == 0) return BAKRON_OK;
  a.in = X;
  a.out = rows;
  return run_rows(a, dtype, Op::kDispatch, stream);
}

extern "C" bakron_status bakron_combine(const void* rows, int64_t R, int64_t d, int dtype, const int32_t* place,
                                        int64_t T, int k, const float* weight, void* Y, void* stream) {
  RowArgs a;
  if (!row_args(Y, rows, T, R, d, dtype, place, k, weight, &a)) return BAKRON_ERR_INVALID_ARG;
  if (T == 0) return BAKRON_OK;
  a.in = rows;
  a.out = Y;
  return run_rows(a, dtype, Op::kCombine, stream);
}

extern "C" bakron_status bakron_combine_grad(const void* dY, const void* rows, int64_t R, int64_t d, int dtype,
                                             const int32_t* place, int64_t T, int k, const float* weight,
                                             void* drows, float* dweight, void* stream) {
  RowArgs a;
  if (!row_args(dY, rows, T, R, d, dtype, place, k, weight, &a)) return BAKRON_ERR_INVALID_ARG;
  if (T == 0) return BAKRON_OK;
  if (!weight || !dweight || !aligned_to(dweight, 4) || (R > 0 && (!drows || !aligned_to(drows, dtype_size(dtype)))))
    return BAKRON_ERR_INVALID_ARG;
  a.in = dY;
  a.rows = rows;
  a.out = drows;
  a.dweight = dweight;
  return run_rows(a, dtype, Op::kCombineGrad, stream);
}
