// Layer norm over rows and its gradients.
//
// Forward: mu = mean(x), var = mean((x - mu)^2), r = 1 / sqrt(var + eps),
// y = (x - mu) r gamma + beta.  Backward, with h = (x - mu) r, a = dy gamma:
//   dx = r (a - mean(a) - h mean(a h)),  dgamma = sum_t dy h,  dbeta = sum_t dy.
// Both are bound by HBM: forward reads and writes each element once, backward
// reads two and writes one.  A row stays in registers between its reductions
// (the variance from the deviations, not from a difference of two large
// sums), so nothing is read twice: one warp per row while a warp's registers
// hold it, else one block per row.  A block's barriers leave the memory idle unless
// the rows after the one at hand are on their way, so the block-per-row kernels
// copy them asynchronously into shared memory, a few rows ahead; a thread
// copies what it reads itself, so the copies need no barrier.  A thread owns the
// same columns of every row that its block takes, so the sums over rows of
// dgamma and dbeta grow in registers and leave the block once, into a row of the
// workspace; a second launch adds the blocks' rows in a fixed order (no atomics,
// so the bits do not depend on the run).  Up to a row per SM, each row has a block, and
// blocks of their own sum the columns beside them (37 x 1111 fp32: 3.4 us, 6.1 with the
// second launch).
//
// Rows that do not begin on 16 bytes (an odd d, or an odd address): a warp copies
// the aligned 16-byte pieces that hold its columns, a thread moves its columns
// into place out of two of them, and the results are exchanged through shared
// memory so that they leave by whole words in order.  (Copies of 4 bytes, which
// need no moving, took 172 us instead of 113 for the gradient of 8192 x 4097 bf16;
// one column per load took 165.)
//
// Measured, forward and gradient: 8192 x 4096 bf16 31 and 43 us (4.3 and 4.7 TB/s; the bytes
// at 6.68 TB/s 20 and 30), 2048 x 14336 fp16 32 and 54 (one block per SM, one row at a
// time), 8192 x 1024 8.7 and 19, 8192 x 4097 65 and 115 (instructions per column),
// 37 x 1111 fp32 3.0 and 3.2 (launch and latency).  Past 14336 columns a
// thread of the gradient holds 32 columns, in a kernel that is compiled for 1024 threads and
// spills at its 64 registers (9 % of the executed instructions): 2048 x 14344 fp16 117,
// 2048 x 16384 bf16 126.
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "packed.cuh"
#include "rows_copy.h"

namespace bakron {
namespace {

struct NormArgs {
  const void* x;
  const void* dy;
  int64_t T, d;
  const float* gamma;
  const float* beta;
  float eps;
  void* y;               // y, or dx
  float* mean;
  float* rstd;
  const float* mean_in;
  const float* rstd_in;
  float* part;           // [blocks][2][d], NULL without weight gradients or with few rows
  float* dgamma;         // of few rows
  float* dbeta;
  int depth;             // slots of rows in shared memory
  bool vectors;          // gamma and beta on 32 bytes
};

constexpr int kMaxWarps = 32;

// Sums of N values over the threads that share a row: the warp, or the block.
// `slot` alternates between calls, so one barrier per call is enough: a
// slot is written again only after the barrier of the call in between.
template <bool kBlock, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[4][kMaxWarps], int& slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if constexpr (kBlock) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) red[slot][k][threadIdx.x >> 5] = v[k];
    }
    __syncthreads();
    // every warp adds the warps' sums in the same way
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = lane < warps ? red[slot][k][lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (o < warps) {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
      }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = __shfl_sync(0xffffffffu, v[k], 0);
    slot ^= 1;
  }
}

// V consecutive elements.
template <typename TX, int V>
struct alignas(sizeof(TX) * V) Vec {
  TX v[V];
};

// The 16 bytes that begin `at` bytes into 32 (at < 16, the same for the whole warp).
template <int ES>
__device__ __forceinline__ uint4 window(const uint4& a, const uint4& b, uint32_t at) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int k = 0; k < 6; ++k) w[k] = at & 8 ? w[k + 2] : w[k];
#pragma unroll
  for (int k = 0; k < 5; ++k) w[k] = at & 4 ? w[k + 1] : w[k];
  if constexpr (ES == 2) {
    const uint32_t bits = (at & 2) * 8;
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], bits);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 ld_piece(uint32_t at) {
  uint4 u;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "r"(at)
               : "memory");
  return u;
}

// Shared memory of a warp's columns of one array's row, and of its results, when
// rows have any alignment.
template <int NV>
constexpr uint32_t kWarpRow = NV * 512 + 16;
constexpr uint32_t kWarpOut = 512;

// The rows of a block (or warp), copied to shared memory `depth` - 1 rows
// ahead.  kShift: rows of any alignment.
template <typename TX, int V, int NV, int ARRAYS, bool kBlock, bool kShift>
struct Rows {
  const TX* src[ARRAYS];
  int64_t d, step, T;
  int64_t next;             // next row to copy
  uint32_t slot, bytes;     // the slots of this block (warp), and their bytes
  uint32_t mine;            // this thread's place in them
  uint32_t fill = 0, read = 0;
  int tid, tpr, depth;

  // The vectors of a thread; a warp has neighbouring ones when it shares pieces.
  __device__ __forceinline__ int vec(int i) const {
    return kShift ? (tid & ~31) * NV + (tid & 31) + i * 32 : tid + i * tpr;
  }
  __device__ __forceinline__ uint32_t array_bytes() const {
    return kShift ? (uint32_t)(tpr >> 5) * kWarpRow<NV> : (uint32_t)(NV * tpr) * 16u;
  }
  __device__ __forceinline__ uint32_t slot_bytes() const { return ARRAYS * array_bytes(); }
  // Bytes by which a row misses a 16-byte boundary.
  __device__ __forceinline__ uint32_t past(const TX* row) const { return (uint32_t)(uintptr_t)row & 15u; }

  // A warp's pieces of one array: those of its columns, with what lies in front of
  // them in the first where that is the array's (piece_bytes), zeros past the
  // row's end.  `front`: the array's bytes in front of the row, 16 for more.
  __device__ __forceinline__ void copy_pieces(const TX* row, int front, uint32_t to) {
    const int lane = tid & 31, c0 = (tid & ~31) * NV * V;
    const uint32_t shift = past(row);
    const int before = c0 > 0 ? 16 : front;
    const char* from = reinterpret_cast<const char*>(row + c0) - shift + lane * 16;
    const int left = ((int)d - c0) * (int)sizeof(TX) + (int)shift;     // bytes from piece 0 on
    to += (tid >> 5) * kWarpRow<NV> + lane * 16;
    if (left >= (int)kWarpRow<NV> && before >= (int)shift) {
#pragma unroll
      for (int i = 0; i <= NV; ++i)
        if (i < NV || lane == 0)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * 512), "l"(from + i * 512)
                       : "memory");
    } else if (left > 0) {
#pragma unroll
      for (int i = 0; i <= NV; ++i) {
        const int at = lane * 16 + i * 512;
        if (i == NV && lane > 0) break;
        const PieceBytes p = piece_bytes(before, (int)shift, left, at);
        if (p.from > 0) {
          // the array begins inside this piece
          for (int b = p.from; b < p.to; b += sizeof(TX)) {
            if constexpr (sizeof(TX) == 2)
              asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + b), "h"(*reinterpret_cast<const uint16_t*>(from + b))
                           : "memory");
            else
              asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + b), "r"(*reinterpret_cast<const uint32_t*>(from + b))
                           : "memory");
          }
          for (int b = max(p.from, p.to); b < 16; b += sizeof(TX)) {
            if constexpr (sizeof(TX) == 2)
              asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + b), "h"((uint16_t)0) : "memory");
            else
              asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + b), "r"(0u) : "memory");
          }
          continue;
        }
        const int n = p.to;
        // (nothing is read from the address that goes with n = 0)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + i * 512),
                     "l"(n ? from + i * 512 : from - lane * 16), "r"(n)
                     : "memory");
      }
    }
  }
  __device__ __forceinline__ void copy() {
    if (next < T) {
      const int front = next >= 16 ? 16 : min(16, (int)next * (int)d * (int)sizeof(TX));
#pragma unroll
      for (int k = 0; k < ARRAYS; ++k) {
        if constexpr (kShift) {
          copy_pieces(src[k] + next * d, front, slot + fill + k * array_bytes());
        } else {
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int c = vec(i) * V;
            if (c < (int)d)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                               mine + fill + (uint32_t)((k * NV + i) * tpr) * 16u),
                           "l"(src[k] + next * d + c)
                           : "memory");
          }
        }
      }
      next += step;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    fill = fill + slot_bytes() == bytes ? 0 : fill + slot_bytes();
  }
  __device__ __forceinline__ void start(int64_t first, void* smem) {
    next = first;
    bytes = slot_bytes() * (uint32_t)depth;
    slot = (uint32_t)__cvta_generic_to_shared(smem) + (kBlock ? 0u : (threadIdx.x >> 5) * bytes);
    mine = slot + (kShift ? (tid >> 5) * kWarpRow<NV> + (tid & 31) * 16u : tid * 16u);
    for (int p = 0; p < depth - 1; ++p) copy();
  }
  // Row `row`, the successor of the one asked for before.
  __device__ __forceinline__ void get(int64_t row, Vec<TX, V> (&v)[ARRAYS][NV]) {
    if constexpr (kShift) __syncwarp();     // the slot to be filled has been read
    copy();
    // `depth` is 1 to 4
    if (depth == 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (depth == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (depth == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
    if constexpr (kShift) __syncwarp();     // the other lanes' pieces
#pragma unroll
    for (int k = 0; k < ARRAYS; ++k) {
      const uint32_t shift = kShift ? past(src[k] + row * d) : 0u;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (vec(i) * V < (int)d) {
          const uint32_t at = kShift ? mine + read + k * array_bytes() + i * 512u
                                     : mine + read + (uint32_t)((k * NV + i) * tpr) * 16u;
          uint4 u = ld_piece(at);
          if constexpr (kShift) u = window<sizeof(TX)>(u, ld_piece(at + 16u), shift);
          v[k][i] = *reinterpret_cast<const Vec<TX, V>*>(&u);
        }
      }
    }
    read = read + slot_bytes() == bytes ? 0 : read + slot_bytes();
  }
};

// A row of results, vector by vector in the order of Rows::vec.  With kShift all
// lanes of a warp come here for every i, whether they have columns or not, and
// `stage` is the warp's kWarpOut bytes of shared memory.
template <typename TX, int V, int NV, bool kShift>
struct RowOut {
  TX* y;                 // the row
  uint32_t stage;
  int d;
  uint32_t before = 0;   // the last word of this lane's vector before

  __device__ __forceinline__ RowOut(TX* row, int64_t d_, uint32_t stage_) : y(row), stage(stage_), d((int)d_) {}
  __device__ __forceinline__ void put(int i, int vec, const Vec<TX, V>& o) {
    const int c = vec * V;
    if constexpr (!kShift) {
      *reinterpret_cast<Vec<TX, V>*>(y + c) = o;
      return;
    }
    const int lane = threadIdx.x & 31;
    if (c - lane * V >= d) return;       // the whole warp
    uint4 u = *reinterpret_cast<const uint4*>(&o);
    uint32_t half = 0;
    if constexpr (sizeof(TX) == 2) {
      half = ((uint32_t)(uintptr_t)y >> 1) & 1u;
      if (half) {      // one column on: the lane's first is the last of the lane before
        const uint32_t p = __shfl_sync(0xffffffffu, lane == 31 ? before : u.w, (lane + 31) & 31);
        before = u.w;
        u.w = __funnelshift_l(u.z, u.w, 16);
        u.z = __funnelshift_l(u.y, u.z, 16);
        u.y = __funnelshift_l(u.x, u.y, 16);
        u.x = __funnelshift_l(p, u.x, 16);
      }
    }
    __syncwarp();      // the vector before has been read
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * 16), "r"(u.x), "r"(u.y),
                 "r"(u.z), "r"(u.w)
                 : "memory");
    __syncwarp();
    constexpr int N = 4 / sizeof(TX);                          // columns of a word
    const int c0 = c - lane * (V - N) - (int)half;             // of this lane's first word
    uint32_t* to = reinterpret_cast<uint32_t*>(y + c0);
    const bool inside = (i > 0 || !half) && c + (32 - lane) * V <= d;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t w;
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(stage + lane * 4 + j * 128) : "memory");
      if (inside || (c0 + j * 32 * N + N <= d && !(half && i == 0 && j == 0 && lane == 0))) {
        to[j * 32] = w;
      } else if constexpr (N == 2) {
        // the first or the last column of a word
        const int a = c0 + j * 64;
        TX* one = y + a;
        if (half && i == 0 && j == 0 && lane == 0) {
          if (a + 1 < d) *reinterpret_cast<uint16_t*>(one + 1) = (uint16_t)(w >> 16);
        } else if (a < d) {
          *reinterpret_cast<uint16_t*>(one) = (uint16_t)w;
        }
      }
    }
    // the last column of the warp begins a word that is not its own
    if constexpr (N == 2)
      if (half && lane == 31 && (i == NV - 1 || c + V == d) && c + V - 1 < d) y[c + V - 1] = o.v[V - 1];
  }
};

// Two fp32 values at a time: one instruction for two additions, products or
// fused ones.  What bounds the block-per-row kernels after HBM is the number of
// instructions per element.
struct F2 {
  float x, y;
};
__device__ __forceinline__ F2 f2(float v) { return F2{v, v}; }
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("{\n .reg .b64 a, b, r;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 r, a, b;\n"
      " mov.b64 {%0, %1}, r;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("{\n .reg .b64 a, b, r;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 r, a, b;\n"
      " mov.b64 {%0, %1}, r;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("{\n .reg .b64 a, b, c, r;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 r, a, b, c;\n mov.b64 {%0, %1}, r;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

// V elements to and from fp32, two at a time for the 16-bit types.
template <typename TX, int V>
__device__ __forceinline__ void widen(float (&f)[V], const Vec<TX, V>& v) {
  if constexpr (sizeof(TX) == 2) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      if constexpr (std::is_same<TX, __half>::value) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&u[e]));
        f[2 * e] = p.x;
        f[2 * e + 1] = p.y;
      } else {
        f[2 * e] = __uint_as_float(u[e] << 16);
        f[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = v.v[e];
  }
}
template <typename TX, int V>
__device__ __forceinline__ void narrow(Vec<TX, V>& v, const float (&f)[V]) {
  if constexpr (sizeof(TX) == 2) {
    uint32_t* u = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      if constexpr (std::is_same<TX, __half>::value) {
        const __half2 h = __floats2half2_rn(f[2 * e], f[2 * e + 1]);
        u[e] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
        u[e] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) v.v[e] = f[e];
  }
}

// V values of gamma or beta (`none` where there is no array, or no column).
template <int V, bool kShift>
__device__ __forceinline__ Vec<float, V> param(const float* g, float none, int c, int d, bool vectors) {
  Vec<float, V> r;
  if (g && (kShift ? vectors && c + V <= d : c < d)) {
    r = *reinterpret_cast<const Vec<float, V>*>(g + c);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) r.v[e] = kShift && g && c + e < d ? g[c + e] : none;
  }
  return r;
}

// Columns past the row's end become `v` (they are 0 as copied, which is right for
// every sum but that of the squared deviations).
template <int V>
__device__ __forceinline__ void fill_tail(float (&f)[V], int c, int d, float v) {
  if (c + V > d) {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (c + e >= d) f[e] = v;
  }
}

template <typename TX, int V, int NV, bool kBlock, bool kShift, int MAXB>
__global__ void __launch_bounds__(MAXB, MAXB <= 256 ? 2 : 1) norm_kernel(const __grid_constant__ NormArgs p) {
  extern __shared__ __align__(16) uint8_t dsm[];
  __shared__ float red[2][4][kMaxWarps];
  int slot = 0;
  const int tid = kBlock ? threadIdx.x : threadIdx.x & 31;
  const int tpr = kBlock ? blockDim.x : 32;
  const int rows_at_once = kBlock ? 1 : blockDim.x >> 5;
  const int64_t row0 = (int64_t)blockIdx.x * rows_at_once + (kBlock ? 0 : threadIdx.x >> 5);
  const int64_t step = (int64_t)gridDim.x * rows_at_once;
  const float inv_d = 1.f / (float)p.d;
  const int d = (int)p.d;
  // R rows at a time: their sums share the barriers and the shuffles' latency
  constexpr int R = kBlock && MAXB <= 512 ? 2 : 1;
  Rows<TX, V, NV, 1, kBlock, kShift> rows;
  rows.src[0] = static_cast<const TX*>(p.x);
  rows.d = p.d;
  rows.step = step;
  rows.T = p.T;
  rows.tid = tid;
  rows.tpr = tpr;
  rows.depth = p.depth;
  rows.start(row0, dsm);
  const uint32_t stage = rows.slot + rows.bytes * (kBlock ? 1 : rows_at_once - (threadIdx.x >> 5)) +
                         (threadIdx.x >> 5) * kWarpOut;     // after all slots
  for (int64_t row = row0; row < p.T; row += R * step) {
    float f[R][NV][V];
    float sum[R], sq[R];
    F2 p2[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      Vec<TX, V> v[1][NV];
      rows.get(row + q * step, v);
      p2[q] = f2(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = rows.vec(i) * V;
        if (c < d) {
          widen(f[q][i], v[0][i]);
#pragma unroll
          for (int e = 0; e < V; e += 2) p2[q] = add2(p2[q], F2{f[q][i][e], f[q][i][e + 1]});
        }
      }
      sum[q] = p2[q].x + p2[q].y;
    }
    row_sums<kBlock, R>(sum, red, slot);
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const float mu = sum[q] * inv_d;
      sum[q] = mu;
      p2[q] = f2(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = rows.vec(i) * V;
        if (c < d) {
          if constexpr (kShift) fill_tail(f[q][i], c, d, mu);
#pragma unroll
          for (int e = 0; e < V; e += 2) {
            const F2 t = add2(F2{f[q][i][e], f[q][i][e + 1]}, f2(-mu));
            p2[q] = fma2(t, t, p2[q]);
            f[q][i][e] = t.x;
            f[q][i][e + 1] = t.y;
          }
        }
      }
      sq[q] = p2[q].x + p2[q].y;
    }
    row_sums<kBlock, R>(sq, red, slot);
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const int64_t at = row + q * step;
      if (at >= p.T) break;
      const float r = rsqrtf(sq[q] * inv_d + p.eps);
      if (tid == 0) {
        if (p.mean) p.mean[at] = sum[q];
        if (p.rstd) p.rstd[at] = r;
      }
      RowOut<TX, V, NV, kShift> out(static_cast<TX*>(p.y) + at * p.d, p.d, stage);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = rows.vec(i) * V;
        if (!kShift && c >= d) continue;
        Vec<TX, V> o;
        if (c < d) {
          const Vec<float, V> g = param<V, kShift>(p.gamma, 1.f, c, d, p.vectors);
          const Vec<float, V> b = param<V, kShift>(p.beta, 0.f, c, d, p.vectors);
#pragma unroll
          for (int e = 0; e < V; e += 2) {
            const F2 t = fma2(mul2(F2{f[q][i][e], f[q][i][e + 1]}, f2(r)), F2{g.v[e], g.v[e + 1]},
                              F2{b.v[e], b.v[e + 1]});
            f[q][i][e] = t.x;
            f[q][i][e + 1] = t.y;
          }
          narrow(o, f[q][i]);
        }
        out.put(i, rows.vec(i), o);
      }
    }
  }
}

// dgamma and dbeta of 32 columns over few rows: a warp takes every W-th row, the
// warps' sums are added in order.  mean and rstd are given, so this needs nothing of
// the rows' own blocks and runs beside them.
template <typename TX>
__device__ __forceinline__ void column_sums(const NormArgs& p, int block, float* sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t c = (int64_t)block * 32 + lane;
  const TX* x = static_cast<const TX*>(p.x) + c;
  const TX* dy = static_cast<const TX*>(p.dy) + c;
  float g = 0.f, b = 0.f;
  if (c < p.d) {
#pragma unroll 8
    for (int64_t t = warp; t < p.T; t += warps) {
      const float w = to_float(dy[t * p.d]), h = (to_float(x[t * p.d]) - p.mean_in[t]) * p.rstd_in[t];
      g = fmaf(w, h, g);
      b += w;
    }
  }
  sum[warp * 64 + lane] = g;
  sum[warp * 64 + 32 + lane] = b;
  __syncthreads();
  if (warp < 2 && c < p.d) {
    float v = 0.f;
    for (int w = 0; w < warps; ++w) v += sum[w * 64 + threadIdx.x];
    (warp == 0 ? p.dgamma : p.dbeta)[c] = v;
  }
}

template <typename TX, int V, int NV, bool kBlock, bool kShift, int MAXB>
__global__ void __launch_bounds__(MAXB, MAXB <= 256 ? 2 : 1) norm_grad_kernel(const __grid_constant__ NormArgs p) {
  extern __shared__ __align__(16) uint8_t dsm[];
  if constexpr (NV == 1) {        // few rows, one per block; the blocks after them sum columns
    if (blockIdx.x >= p.T) {
      column_sums<TX>(p, (int)(blockIdx.x - p.T), reinterpret_cast<float*>(dsm));
      return;
    }
  }
  __shared__ float red[2][4][kMaxWarps];
  int slot = 0;
  const int tid = kBlock ? threadIdx.x : threadIdx.x & 31;
  const int tpr = kBlock ? blockDim.x : 32;
  const int rows_at_once = kBlock ? 1 : blockDim.x >> 5;
  const int64_t lead = (int64_t)blockIdx.x * rows_at_once + (kBlock ? 0 : threadIdx.x >> 5);
  const int64_t step = (int64_t)gridDim.x * rows_at_once;
  const float inv_d = 1.f / (float)p.d;
  const int d = (int)p.d;
  // R rows at a time: their sums share the barrier and the shuffles' latency
  constexpr int R = kBlock && MAXB <= 512 ? 2 : 1;
  Rows<TX, V, NV, 2, kBlock, kShift> rows;
  rows.src[0] = static_cast<const TX*>(p.x);
  rows.src[1] = static_cast<const TX*>(p.dy);
  rows.d = p.d;
  rows.step = step;
  rows.T = p.T;
  rows.tid = tid;
  rows.tpr = tpr;
  rows.depth = p.depth;
  // gamma stays in registers when there is room
  constexpr bool kKeep = NV * V <= 16 && MAXB <= 640;
  Vec<float, V> gk[kKeep ? NV : 1];
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < NV; ++i) gk[i] = param<V, kShift>(p.gamma, 1.f, rows.vec(i) * V, d, p.vectors);
  }
  float dg[NV][V], db[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) dg[i][e] = db[i][e] = 0.f;
  rows.start(lead, dsm);
  const uint32_t stage = rows.slot + rows.bytes * (kBlock ? 1 : rows_at_once - (threadIdx.x >> 5)) +
                         (threadIdx.x >> 5) * kWarpOut;     // after all slots
  float mu_next[R], r_next[R];
  auto stats = [&](int64_t row) {
#pragma unroll
    for (int q = 0; q < R; ++q) {
      mu_next[q] = r_next[q] = 0.f;
      if (row + q * step < p.T) {
        mu_next[q] = ld_ahead(p.mean_in + row + q * step);
        r_next[q] = ld_ahead(p.rstd_in + row + q * step);
      }
    }
  };
  stats(lead);
  for (int64_t row = lead; row < p.T; row += R * step) {
    float mu[R], r[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      mu[q] = mu_next[q];
      r[q] = r_next[q];
    }
    stats(row + R * step);
    Vec<TX, V> v[R][2][NV];
    float sums[2 * R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      rows.get(row + q * step, v[q]);
      const bool there = row + q * step < p.T;
      F2 t1 = f2(0.f), t2 = f2(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = rows.vec(i) * V;
        if (c < d && there) {
          if constexpr (!kKeep) gk[0] = param<V, kShift>(p.gamma, 1.f, c, d, p.vectors);
          const Vec<float, V>& g = gk[kKeep ? i : 0];
          float fx[V], fw[V];
          widen(fx, v[q][0][i]);
          widen(fw, v[q][1][i]);
#pragma unroll
          for (int e = 0; e < V; e += 2) {
            const F2 h = mul2(add2(F2{fx[e], fx[e + 1]}, f2(-mu[q])), f2(r[q])), w = F2{fw[e], fw[e + 1]};
            const F2 a = mul2(w, F2{g.v[e], g.v[e + 1]});
            t1 = add2(t1, a);
            t2 = fma2(a, h, t2);
            const F2 x = fma2(w, h, F2{dg[i][e], dg[i][e + 1]}), z = add2(F2{db[i][e], db[i][e + 1]}, w);
            dg[i][e] = x.x;
            dg[i][e + 1] = x.y;
            db[i][e] = z.x;
            db[i][e + 1] = z.y;
          }
        }
      }
      sums[2 * q] = t1.x + t1.y;
      sums[2 * q + 1] = t2.x + t2.y;
    }
    row_sums<kBlock, 2 * R>(sums, red, slot);
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const int64_t at = row + q * step;
      if (at >= p.T) break;
      RowOut<TX, V, NV, kShift> out(static_cast<TX*>(p.y) + at * p.d, p.d, stage);
      // dX = r a - (r m1) - h (r m2): three constants of the row
      const float m1 = r[q] * (sums[2 * q] * inv_d), m2 = r[q] * (sums[2 * q + 1] * inv_d);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = rows.vec(i) * V;
        if (!kShift && c >= d) continue;
        Vec<TX, V> o;
        if (c < d) {
          if constexpr (!kKeep) gk[0] = param<V, kShift>(p.gamma, 1.f, c, d, p.vectors);
          const Vec<float, V>& g = gk[kKeep ? i : 0];
          float fx[V], fw[V], fo[V];
          widen(fx, v[q][0][i]);
          widen(fw, v[q][1][i]);
#pragma unroll
          for (int e = 0; e < V; e += 2) {
            const F2 h = mul2(add2(F2{fx[e], fx[e + 1]}, f2(-mu[q])), f2(r[q]));
            const F2 a = mul2(F2{fw[e], fw[e + 1]}, F2{g.v[e], g.v[e + 1]});
            const F2 x = fma2(h, f2(-m2), fma2(a, f2(r[q]), f2(-m1)));
            fo[e] = x.x;
            fo[e + 1] = x.y;
          }
          narrow(o, fo);
        }
        out.put(i, rows.vec(i), o);
      }
    }
  }
  if (!p.part) return;
  float* o = p.part + (int64_t)blockIdx.x * 2 * p.d;
  if constexpr (kBlock) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = rows.vec(i) * V;
      if constexpr (kShift) {
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (c + e < d) {
            o[c + e] = dg[i][e];
            o[p.d + c + e] = db[i][e];
          }
      } else if (c < d) {
        Vec<float, V> g, b;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          g.v[e] = dg[i][e];
          b.v[e] = db[i][e];
        }
        *reinterpret_cast<Vec<float, V>*>(o + c) = g;
        *reinterpret_cast<Vec<float, V>*>(o + p.d + c) = b;
      }
    }
  } else {
    // the warps' sums where their rows were, one line per column of a vector
    // (its length keeps both sides free of bank conflicts), then added in order
    constexpr int kLine = 32 + 32 / V, kWarp = 2 * NV * V * kLine;
    float* sum = reinterpret_cast<float*>(dsm);
    __syncthreads();
    float* mine = sum + (threadIdx.x >> 5) * kWarp + tid;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        mine[(i * V + e) * kLine] = dg[i][e];
        mine[(NV * V + i * V + e) * kLine] = db[i][e];
      }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * d; c += blockDim.x) {
      const int col = c < d ? c : c - d, vec = col / V;
      const float* at = sum + ((c < d ? 0 : NV * V) + vec / 32 * V + col % V) * kLine + vec % 32;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) v += at[w * kWarp];
      o[c] = v;
    }
  }
}

// Rows too long for a block's registers: the row is read again from memory
// (mostly from L2) for each reduction, and the partial weight gradients live
// in the block's row of the workspace, where only one thread ever touches a
// column.
template <typename TX>
__global__ void __launch_bounds__(1024) norm_long_kernel(const __grid_constant__ NormArgs p) {
  __shared__ float red[2][4][kMaxWarps];
  int slot = 0;
  const float inv_d = 1.f / (float)p.d;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const TX* x = static_cast<const TX*>(p.x) + row * p.d;
    TX* y = static_cast<TX*>(p.y) + row * p.d;
    float sum[1] = {0.f}, sq[1] = {0.f};
    for (int64_t c = threadIdx.x; c < p.d; c += blockDim.x) sum[0] += to_float(x[c]);
    row_sums<true, 1>(sum, red, slot);
    const float mu = sum[0] * inv_d;
    for (int64_t c = threadIdx.x; c < p.d; c += blockDim.x) {
      const float v = to_float(x[c]) - mu;
      sq[0] = fmaf(v, v, sq[0]);
    }
    row_sums<true, 1>(sq, red, slot);
    const float r = 1.f / sqrtf(sq[0] * inv_d + p.eps);
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[row] = mu;
      if (p.rstd) p.rstd[row] = r;
    }
    for (int64_t c = threadIdx.x; c < p.d; c += blockDim.x)
      y[c] = from_float<TX>(fmaf((to_float(x[c]) - mu) * r, p.gamma ? p.gamma[c] : 1.f,
                                 p.beta ? p.beta[c] : 0.f));
  }
}

template <typename TX>
__global__ void __launch_bounds__(1024) norm_grad_long_kernel(const __grid_constant__ NormArgs p) {
  __shared__ float red[2][4][kMaxWarps];
  int slot = 0;
  const float inv_d = 1.f / (float)p.d;
  float* o = p.part ? p.part + (int64_t)blockIdx.x * 2 * p.d : nullptr;
  if (o)
    for (int64_t c = threadIdx.x; c < p.d; c += blockDim.x) o[c] = o[p.d + c] = 0.f;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const TX* x = static_cast<const TX*>(p.x) + row * p.d;
    const TX* dy = static_cast<const TX*>(p.dy) + row * p.d;
    TX* dx = static_cast<TX*>(p.y) + row * p.d;
    const float mu = p.mean_in[row], r = p.rstd_in[row];
    float sums[2] = {0.f, 0.f};
    for (int64_t c = threadIdx.x; c < p.d; c += blockDim.x) {
      const float h = (to_float(x[c]) - mu) * r, d = to_float(dy[c]);
      const float a = d * (p.gamma ? p.gamma[c] : 1.f);
      sums[0] += a;
      sums[1] = fmaf(a, h, sums[1]);
      if (o) {
        o[c] = fmaf(d, h, o[c]);
        o[p.d + c] += d;
      }
    }
    row_sums<true, 2>(sums, red, slot);
    const float s1 = sums[0] * inv_d, s2 = sums[1] * inv_d;
    for (int64_t c = threadIdx.x; c < p.d; c += blockDim.x) {
      const float h = (to_float(x[c]) - mu) * r;
      const float a = to_float(dy[c]) * (p.gamma ? p.gamma[c] : 1.f);
      dx[c] = from_float<TX>(r * (a - s1 - h * s2));
    }
  }
}

// dgamma and dbeta: the sum over the partial rows.  A block takes 32 columns,
// its 16 warps every 16th row each, joined in shared memory in a fixed order.
__global__ void __launch_bounds__(512) norm_join_kernel(const float* __restrict__ part, int64_t rows,
                                                        int64_t d, float* __restrict__ dgamma,
                                                        float* __restrict__ dbeta) {
  __shared__ float red[16][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;      // over 2 d columns
  float v = 0.f;
  if (c < 2 * d) {
#pragma unroll 8
    for (int64_t r = warp; r < rows; r += 16) v += __ldcg(part + r * 2 * d + c);
  }
  red[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < 2 * d) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += red[w][lane];
    if (c < d) dgamma[c] = s;
    else dbeta[c - d] = s;
  }
}

// How a shape runs: vectors per thread, threads per row, and the rows in flight.
struct NormPlan {
  int nv;           // 0: the long-row kernels
  bool block;       // one block per row, else one warp
  bool shift;       // rows of any alignment
  int threads;      // of a block
  int depth, per_sm;
  size_t smem;
};

// Shared memory per SM that the rows in flight may take (of 228 KB), and one row.
constexpr size_t kRowBytes = 200 * 1024, kMaxRow = 224 * 1024;

NormPlan norm_plan(int64_t T, int64_t d, int dtype, bool aligned, int arrays) {
  NormPlan q = {};
  const int v = dtype == BAKRON_F32 ? 4 : 8;
  q.shift = !aligned || d % v != 0;
  const int64_t vecs = (d + v - 1) / v;
  const size_t extra = q.shift ? (size_t)arrays * 16 : 0, out = q.shift ? kWarpOut : 0;   // per warp
  // columns per thread: 32 forward, 16 backward (two sums per column live in
  // registers there), 32 once a block of 896 threads is too small for that
  const int most = arrays == 1 || vecs > 16 / v * 896 ? 32 / v : 16 / v;
  const bool few = T <= sm_count() && vecs > 32 && vecs <= 1024;
  if (vecs <= 32 * (32 / v) && !few) {        // 1024 columns: a warp per row
    q.threads = 256;
    q.nv = 32 / v;
    q.per_sm = arrays == 1 ? 4 : 2;
    q.depth = 3;
    q.smem = (size_t)8 * (q.depth * (arrays * q.nv * 32 * 16 + extra) + out);
    // (the warps' sums need 8 x 2 x 32 x (32 + 32 / v) floats, less than this)
    return q;
  }
  q.block = true;
  if (few) {
    // one row per block at most: its latency counts, which a vector per thread keeps
    // shortest (37 x 1111 fp32 forward: 2.9 us, 8 with eight vectors)
    q.nv = 1;
    q.threads = (int)std::max<int64_t>(256, (vecs + 31) / 32 * 32);
    q.per_sm = 1;
    q.depth = 1;
    q.smem = (size_t)arrays * q.threads * 16 + (extra + out) * (q.threads / 32);
    return q;
  }
  const int threads = (int)std::min<int64_t>(2048, ((vecs + most - 1) / most + 31) / 32 * 32);
  const size_t row = (size_t)arrays * most * threads * 16 + extra * (threads / 32);
  const size_t fixed = out * (threads / 32);
  if (threads > 1024 || row + fixed > kMaxRow) {
    q.threads = 1024;
    q.per_sm = 2;
    return q;
  }
  q.nv = most;
  q.threads = threads;
  // blocks per SM: what the registers allow (128 a thread), fewer for long rows; as many rows
  // ahead as fit beside that
  q.per_sm = std::max(1, std::min(arrays == 1 ? 8 : 4, 512 / q.threads));
  while (q.per_sm > 1 && (row * 2 + fixed) * q.per_sm > kRowBytes) --q.per_sm;
  q.depth = (int)std::max<size_t>(1, std::min<size_t>(4, (kRowBytes / q.per_sm - fixed) / row));
  // gamma is read from memory by blocks this large, and stays in the L1 cache beside
  // two rows, not three (2048 x 14336 fp16: 53 us, 57)
  if (arrays == 2 && q.threads > 640) q.depth = std::min(q.depth, 2);
  q.smem = row * q.depth + fixed;
  return q;
}

int64_t norm_blocks(const NormPlan& q, int64_t T) {
  const int rows = q.block ? 1 : q.threads / 32;
  return std::min<int64_t>((T + rows - 1) / rows, (int64_t)sm_count() * q.per_sm);
}

template <typename K>
cudaError_t launch_norm(K k, const NormPlan& q, const NormArgs& a, std::atomic<unsigned long long>& done,
                        cudaStream_t s, int64_t more_blocks = 0) {
  if (q.smem > 46 * 1024) {      // beyond the default of 48 KB with the static part
    const cudaError_t e = ensure_smem_limit((const void*)k, 226 * 1024, done);
    if (e != cudaSuccess) return e;
  }
  count_launch();
  k<<<(unsigned)(norm_blocks(q, a.T) + more_blocks), q.threads, q.smem, s>>>(a);
  return cudaGetLastError();
}

template <typename TX, int W, bool kShift>
cudaError_t run_fwd(const NormPlan& q, const NormArgs& a, cudaStream_t s) {
  constexpr int N = 32 / W;
  static std::atomic<unsigned long long> d[4];
  if (q.nv == 1) return launch_norm(norm_kernel<TX, W, 1, true, kShift, 1024>, q, a, d[3], s);
  if (!q.block) return launch_norm(norm_kernel<TX, W, N, false, kShift, 256>, q, a, d[0], s);
  if (q.threads <= 512) return launch_norm(norm_kernel<TX, W, N, true, kShift, 512>, q, a, d[1], s);
  return launch_norm(norm_kernel<TX, W, N, true, kShift, 1024>, q, a, d[2], s);
}
template <typename TX, int W>
cudaError_t run_fwd(const NormPlan& q, const NormArgs& a, cudaStream_t s) {
  static std::atomic<unsigned long long> d;
  if (q.nv == 0) return launch_norm(norm_long_kernel<TX>, q, a, d, s);
  return q.shift ? run_fwd<TX, W, true>(q, a, s) : run_fwd<TX, W, false>(q, a, s);
}
template <typename TX, int W, bool kShift>
cudaError_t run_grad(const NormPlan& q, const NormArgs& a, cudaStream_t s) {
  constexpr int N = 16 / W;
  static std::atomic<unsigned long long> d[7];
  if (q.nv == 1)
    return launch_norm(norm_grad_kernel<TX, W, 1, true, kShift, 1024>, q, a, d[5], s, a.dgamma ? (a.d + 31) / 32 : 0);
  if (!q.block) return launch_norm(norm_grad_kernel<TX, W, 2 * N, false, kShift, 256>, q, a, d[0], s);
  if (q.nv == 2 * N) return launch_norm(norm_grad_kernel<TX, W, 2 * N, true, kShift, 1024>, q, a, d[1], s);
  if (q.threads <= 256) return launch_norm(norm_grad_kernel<TX, W, N, true, kShift, 256>, q, a, d[2], s);
  if (q.threads <= 512) return launch_norm(norm_grad_kernel<TX, W, N, true, kShift, 512>, q, a, d[3], s);
  if (q.threads <= 640) return launch_norm(norm_grad_kernel<TX, W, N, true, kShift, 640>, q, a, d[6], s);
  return launch_norm(norm_grad_kernel<TX, W, N, true, kShift, 896>, q, a, d[4], s);
}
template <typename TX, int W>
cudaError_t run_grad(const NormPlan& q, const NormArgs& a, cudaStream_t s) {
  static std::atomic<unsigned long long> d;
  if (q.nv == 0) return launch_norm(norm_grad_long_kernel<TX>, q, a, d, s);
  return q.shift ? run_grad<TX, W, true>(q, a, s) : run_grad<TX, W, false>(q, a, s);
}

bool norm_args_ok(int64_t T, int64_t d, int dtype) {
  return dtype_ok(dtype) && T >= 0 && T <= (int64_t(1) << 31) && d >= 1 && d <= (int64_t(1) << 20);
}

bool floats_aligned(std::initializer_list<const float*> all) {
  return std::all_of(all.begin(), all.end(), [](const float* p) { return aligned_to(p, 4); });
}

// The alignment of the pointers and the type are not known to the size call.
size_t grad_bytes(int64_t T, int64_t d) {
  int64_t rows = 0;
  for (int dt : {BAKRON_F32, BAKRON_BF16})
    for (bool al : {false, true})
      for (int64_t t : {T, std::min<int64_t>(T, sm_count())})      // fewer rows may take more blocks
        rows = std::max(rows, norm_blocks(norm_plan(t, d, dt, al, 2), t));
  return (size_t)(rows * 2 * d) * sizeof(float);
}

}  // namespace
}  // namespace bakron

using namespace bakron;

extern "C" bakron_status bakron_layernorm(const void* X, int64_t T, int64_t d, int dtype,
                                          const float* gamma, const float* beta, float eps, void* Y,
                                          float* mean, float* rstd, void* stream) {
  if (!norm_args_ok(T, d, dtype) || !(eps >= 0.f)) return BAKRON_ERR_INVALID_ARG;
  if (T == 0) return BAKRON_OK;
  const size_t es = dtype_size(dtype);
  if (!X || !Y || !aligned_to(X, es) || !aligned_to(Y, es) || !floats_aligned({gamma, beta, mean, rstd}))
    return BAKRON_ERR_INVALID_ARG;
  NormArgs a = {};
  a.x = X;
  a.T = T;
  a.d = d;
  a.gamma = gamma;
  a.beta = beta;
  a.eps = eps;
  a.y = Y;
  a.mean = mean;
  a.rstd = rstd;
  const bool al = aligned_to(X, 16) && aligned_to(Y, 16) && aligned_to(gamma, 32) && aligned_to(beta, 32);
  const NormPlan q = norm_plan(T, d, dtype, al, 1);
  a.vectors = aligned_to(gamma, 32) && aligned_to(beta, 32);
  a.depth = q.depth;
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = dtype == BAKRON_F32    ? run_fwd<float, 4>(q, a, s)
                        : dtype == BAKRON_BF16 ? run_fwd<__nv_bfloat16, 8>(q, a, s)
                                               : run_fwd<__half, 8>(q, a, s);
  return launch_status(e);
}

extern "C" bakron_status bakron_layernorm_grad_workspace_size(int64_t T, int64_t d, size_t* bytes) {
  if (!bytes || !norm_args_ok(T, d, BAKRON_F32)) return BAKRON_ERR_INVALID_ARG;
  *bytes = grad_bytes(T, d);
  return BAKRON_OK;
}

extern "C" bakron_status bakron_layernorm_grad(const void* dY, const void* X, int64_t T, int64_t d,
                                               int dtype, const float* gamma, const float* mean,
                                               const float* rstd, void* dX, float* dgamma,
                                               float* dbeta, void* ws, size_t ws_bytes,
                                               void* stream) {
  if (!norm_args_ok(T, d, dtype) || (dgamma == nullptr) != (dbeta == nullptr))
    return BAKRON_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (T == 0) {
    if (dgamma && (cudaMemsetAsync(dgamma, 0, (size_t)d * 4, s) != cudaSuccess ||
                   cudaMemsetAsync(dbeta, 0, (size_t)d * 4, s) != cudaSuccess))
      return BAKRON_ERR_CUDA;
    return BAKRON_OK;
  }
  const size_t es = dtype_size(dtype);
  if (!X || !dY || !dX || !mean || !rstd || !aligned_to(X, es) || !aligned_to(dY, es) ||
      !aligned_to(dX, es) || !floats_aligned({gamma, mean, rstd, dgamma, dbeta}))
    return BAKRON_ERR_INVALID_ARG;
  if (dgamma && (!ws || !aligned_to(ws, 256) || ws_bytes < grad_bytes(T, d)))
    return BAKRON_ERR_INVALID_ARG;
  NormArgs a = {};
  a.x = X;
  a.dy = dY;
  a.T = T;
  a.d = d;
  a.gamma = gamma;
  a.y = dX;
  a.mean_in = mean;
  a.rstd_in = rstd;
  const bool al = aligned_to(X, 16) && aligned_to(dY, 16) && aligned_to(dX, 16) && aligned_to(gamma, 32);
  const NormPlan q = norm_plan(T, d, dtype, al, 2);
  a.vectors = aligned_to(gamma, 32);
  a.depth = q.depth;
  if (q.nv == 1) {
    a.dgamma = dgamma;
    a.dbeta = dbeta;
  } else if (dgamma) {
    a.part = static_cast<float*>(ws);
  }
  const cudaError_t e = dtype == BAKRON_F32    ? run_grad<float, 4>(q, a, s)
                        : dtype == BAKRON_BF16 ? run_grad<__nv_bfloat16, 8>(q, a, s)
                                               : run_grad<__half, 8>(q, a, s);
  if (e != cudaSuccess) return launch_status(e);
  if (a.part) {
    count_launch();
    norm_join_kernel<<<(unsigned)((2 * d + 31) / 32), 512, 0, s>>>(a.part, norm_blocks(q, T), d, dgamma,
                                                                     dbeta);
    if (cudaGetLastError() != cudaSuccess) return BAKRON_ERR_CUDA;
  }
  return BAKRON_OK;
}
