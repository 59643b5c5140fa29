// bakron_linear_grad: D[j][t] = sum_i V_ij dy_ti on the tcgen05 tensor cores.
//
// The weights are the M operand (128 columns j of V), the incoming gradients the
// N operand (N tokens t), the sum runs over the rows i.  The scale s_ig varies along the
// sum, so the operand holds the value s (u - z): rounded once to dY's type for 16-bit dY
// (the exact operands of the forward product would need a scaled copy of dY per
// group, and as much rounding of that), in three exact bf16 terms for fp32 dY (with
// three of dY; six products: the three left out are at most 2^-24 of the whole, as the
// terms are rounded; cut off they came to 2^-21, always towards zero).
//
// The packed words run along the columns, so the operand (rows along K) is their
// transpose: a thread takes 4 rows x 32 columns of codes; one byte permutation
// brings the same columns of two rows next to each other, and each column's 4
// rows leave as 8 bytes of a 128-byte line of the operand.  Two warps share a
// step of 64 rows (four with three terms), so that a stage is filled by them
// while the other weights' warps fill the next ones.
//
// 16-bit dY: the sum over 4096 rows (bf16: 32768) stays in TMEM, a chain of one addition
// per 16 rows that cuts off at most 2^-23 of the partial sum: 2^-15 (2^-12) in all, an eighth
// of the result's own rounding.  Longer sums are added from such chains in fp32, by way of
// the workspace (fp16, 1024 tokens of 14336 x 4096 in four chains 116 us, bf16 in one 107;
// 512 of 65536 x 4096 in 16 and 2 chains 483 and 441).  Two accumulators
// let the epilogue take one while the next is summed.  fp32 dY: the sum is cut after every 128 rows and
// added in fp32 registers, and the five small products have an accumulator of
// their own, so that the large one is cut off 8 times a unit instead of 48 (error
// of a 333 x 1000 x 1300 product against 64 bits: with one accumulator 1.3e-6).
//
// One block per SM, which takes output tiles in turn (or, when there are few, a
// part of the rows of one, joined over a cluster through distributed shared memory):
//   warp 0: TMA producer of dY;  warp 1: issues the tcgen05.mma (M 128, K 16);
//   warp 2: allocates and frees TMEM;  warps 4-11: weights;  warps 12-15: epilogue.
// The scales enter and leave by a power of two (operand_range), so that V may be of any
// size in any type.
//
// Measured: 2048 tokens of 4096 x 14336 bf16 in 204 us in a graph of one weight (1.18
// PFLOP/s) and 215 among calls on several, bound by the issuing warp's waits and by the
// warps that transpose; 333 tokens of 1000 x 1300 fp32 21 us and 1024 of 4096 x 4096 fp32
// 257 us (groups of 32: 280), bound by the warps that split each weight into its terms
// (with a branch for infinite weights there 27 and 443 us; code for them behind the
// sums, even where no call reached it, 272).
//
// Every mbarrier wait is bounded (clock64 budget); a block whose wait runs
// out records BAKRON_ERR_TIMEOUT in the device's status word, stops issuing,
// drains its copies and MMAs (bounded again), frees TMEM and returns.
#include <cooperative_groups.h>

#include <algorithm>
#include <cstdlib>
#include <type_traits>

#include "linear_tc.cuh"

namespace bakron {

namespace cg = cooperative_groups;
using namespace tc;

namespace {

constexpr int kThreads = 512;
constexpr uint32_t kABytes = 128 * 64 * 2;   // one plane of the weights' stage: 128 x 64
constexpr uint32_t kRing = 224 * 1024;       // shared memory for the stages
constexpr int kMaxStages = 8;

struct GradArgs {
  PackedView w;
  void* y;
  int64_t T;          // tokens
  int64_t plane;      // token rows per plane of dY's map
  int tiles_m;
  int64_t tiles;      // tiles of the output
  int steps;          // K steps of 64 rows
  int N;              // tokens per tile, a multiple of 32
  int stages;
  int most;           // no |c - z| is larger
  float* sums;        // [block][N][128]: 16-bit dY, chains before the last
  int* status;
};

__device__ __forceinline__ void sts64(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
// Two fp32 values as a pair of H, and back.
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __nv_bfloat16) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __half) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack2(uint32_t p, __nv_bfloat16) {
  return make_float2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t p, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&p));
}

// The power of two that the scales take on their way into the operand, and its
// inverse, which the sums take on their way out: V itself need not be in the
// range of the operand's type, or of fp32.  fp16: the largest weight comes next to
// the largest number, so that a weight keeps its 11 bits down to 2^-25 (2^-21 where
// |c - z| exceeds 15) of the largest scale.  bf16 (and its terms): a factor only
// where a weight could overflow or the last of three terms lose bits.
template <typename H>
__device__ __forceinline__ void operand_range(const GradArgs& a, float& in, float& out) {
  const float top = __ldg(a.w.largest);
  const int e = (int)(__float_as_uint(top) >> 23) - 127;
  int p = 0;
  if (top > 0.f) {
    if (std::is_same<H, __half>::value) p = max(-126, min(126, (a.most <= 15 ? 11 : 7) - e));
    else if (e > 119) p = 119 - e;
    else if (e < -90) p = -90 - e;
  }
  in = __uint_as_float((uint32_t)(127 + p) << 23);
  out = __uint_as_float((uint32_t)(127 - p) << 23);
}

// Two weights in three exact bf16 terms each, as pairs, the first two rounded to
// nearest (split3_near); operand_range keeps them below 2^127.
__device__ __forceinline__ void split_pair(float x, float y, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = pack2(x, y, __nv_bfloat16());
  const float2 h = unpack2(hi, __nv_bfloat16());
  const float rx = x - h.x, ry = y - h.y;
  mid = pack2(rx, ry, __nv_bfloat16());
  const float2 m = unpack2(mid, __nv_bfloat16());
  lo = __byte_perm(__float_as_uint(rx - m.x), __float_as_uint(ry - m.y), 0x7632);
}

struct Bars {
  unsigned long long full[kMaxStages], empty[kMaxStages];
  unsigned long long acc_full[2], acc_empty[2], done;
  uint32_t tmem;
  int abort;
};

// The block's work: output tiles tile, tile + step, ...; K steps [k0, k1) of each.
struct Work {
  int64_t tile, step;
  int k0, k1;
};

// Warps that fill a stage, and the 32-column parts that one of their threads takes.
// Splitting into terms is long, and three stages of such weights are all that fits:
// with two warps a stage, two of the eight had none (1024 x 4096 x 4096: 279 us, 332).
template <int TW>
constexpr int kStepWarps = TW == 1 ? 2 : 4;
template <int TW>
constexpr int kParts = TW == 1 ? 4 : 2;

// What a thread holds of a step: 4 rows x 32 (16) columns of codes and the rows'
// grid for the columns' groups (one group, or one per 32 columns).
template <int SN, int NS>
struct Codes {
  uint32_t q[4][SN];
  float4 sc[NS < SN ? NS : SN];
  uint32_t z[NS < SN ? NS : SN];
};

template <typename H, int TW, int NS>
__device__ __forceinline__ void weights(const GradArgs& a, const Work& k, Bars& bars, uint32_t ring,
                                        uint32_t stage_bytes, int warp, int lane) {
  const PackedView& w = a.w;
  constexpr int W = kStepWarps<TW>, SN = kParts<TW>, G = NS < SN ? NS : SN;
  const int group = warp / W, hh = (lane >> 3) & 1, rb = lane & 7;
  // word 4 t + s of a row: t by warp and lane, or t by warp and half of s by lane
  const int t = SN == 4 ? 2 * (warp & 1) + (lane >> 4) : warp & 3;
  const int s0 = SN == 4 ? 0 : 2 * (lane >> 4);
  const int turn = min(8 / W, a.stages);    // groups of warps at work: a wait tells a stage's
  if (group >= turn) return;                // uses apart by one bit, so none may be two ahead
  const uint32_t full = smem_u32(bars.full), empty = smem_u32(bars.empty);
  const int64_t nb = w.mp / 8;
  const int n = k.k1 - k.k0;
  auto load = [&](Codes<SN, NS>& c, int64_t tile, int m, int i) {
    const int64_t b = (int64_t)(k.k0 + i) * 8 + rb;
    const bool live = tile < a.tiles && b < nb;
    const uint8_t* src = w.codes + ((live ? b : 0) * w.nc + (live ? m : 0)) * kBlockBytes + hh * 256 + t * 16 + s0 * 4;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      for (int e = 0; e < SN; ++e) c.q[r][e] = 0;
      if (live) {
        if constexpr (SN == 4) {
          const uint4 u = ld_codes(src + r * 64);
          c.q[r][0] = u.x;
          c.q[r][1] = u.y;
          c.q[r][2] = u.z;
          c.q[r][3] = u.w;
        } else {
          asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(c.q[r][0]), "=r"(c.q[r][1]) : "l"(src + r * 64));
        }
      }
    }
#pragma unroll
    for (int s = 0; s < G; ++s) {
      c.sc[s] = make_float4(0.f, 0.f, 0.f, 0.f);
      c.z[s] = 0;
      if (live) {
        const int64_t at = grid_row(w, 0, b * 8 + hh * 4) + grid_group(w, (uint32_t)m * 128u + 32 * (s0 + s)) * 16;
        asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(c.sc[s].x), "=f"(c.sc[s].y), "=f"(c.sc[s].z), "=f"(c.sc[s].w)
                     : "l"(w.scale + at));
        if (w.zero) asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(c.z[s]) : "l"(w.zero + at));
      }
    }
  };
  // this group's steps over all tiles: every turn-th
  int64_t tile = k.tile;
  int m = (int)(tile % a.tiles_m), i = group;
  auto settle = [&]() {
    if (i < n) return;
    while (i >= n && tile < a.tiles) {
      i -= n;
      tile += k.step;
    }
    m = (int)(tile % a.tiles_m);
  };
  settle();
  Codes<SN, NS> c;
  load(c, tile, m, i);
  float range_in, range_out;
  operand_range<H>(a, range_in, range_out);
  Ring rg;
  rg.advance(group, a.stages);
  while (tile < a.tiles) {
    const Codes<SN, NS> now = c;
    i += turn;
    settle();
    load(c, tile, m, i);
    if (!__all_sync(0xffffffffu, rg.first || wait_or_abort(empty + 8u * (uint32_t)rg.s, rg.parity ^ 1u, &bars.abort, a.status)))
      return;
    const uint32_t sa = ring + (uint32_t)rg.s * stage_bytes + (uint32_t)hh * 8u;
    float sc[4];
    uint32_t off[2];
#pragma unroll
    for (int s = 0; s < SN; ++s) {
      if (s < G) {
        sc[0] = now.sc[s].x * range_in;
        sc[1] = now.sc[s].y * range_in;
        sc[2] = now.sc[s].z * range_in;
        sc[3] = now.sc[s].w * range_in;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const float z0 = w.zero ? (float)((now.z[s] >> (16 * p)) & 255u) : (float)w.zu;
          const float z1 = w.zero ? (float)((now.z[s] >> (16 * p + 8)) & 255u) : (float)w.zu;
          off[p] = pack2(Half2<H>::kBase + z0, Half2<H>::kBase + z1, H());
        }
      }
      uint32_t word[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) word[r] = now.q[r][s];
#pragma unroll
      for (int odd = 0; odd < 2; ++odd) {
        uint32_t tr[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) tr[p] = __byte_perm(word[2 * p], word[2 * p + 1], odd ? 0x7632 : 0x5410);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = 32 * (s0 + s) + 8 * t + 2 * e + odd;
          const uint32_t at = sa + (uint32_t)col * 128u + (uint32_t)((rb ^ (2 * e + odd)) << 4);
          uint32_t o[TW][2];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const uint32_t u = Half2<H>::sub(((tr[p] >> (4 * e)) & 0x000f000fu) | Half2<H>::kMagic, off[p]);
            float2 f = unpack2(u, H());
            f.x *= sc[2 * p];
            f.y *= sc[2 * p + 1];
            if constexpr (TW == 1) {
              o[0][p] = pack2(f.x, f.y, H());
            } else {
              split_pair(f.x, f.y, o[0][p], o[1][p], o[2][p]);
            }
          }
#pragma unroll
          for (int q = 0; q < TW; ++q) sts64(at + q * kABytes, o[q][0], o[q][1]);
        }
      }
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(full + 8u * (uint32_t)rg.s);
    rg.advance(turn, a.stages);
  }
}

// TX, TW: 16-bit terms of dY and of the weights (1 and 1: the sum is cut every grad_chain
// rows; else every 128); NS: groups per 128 columns.
template <typename TO, typename H, int TX, int TW, int NS>
__global__ void __launch_bounds__(kThreads, 1)
    linear_grad_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ GradArgs a) {
  constexpr bool kWhole = TW == 1;
  // K steps of an accumulator's chain
  constexpr int kChain = kWhole ? (int)(grad_chain(std::is_same<H, __half>::value ? BAKRON_F16 : BAKRON_BF16) / 64) : 2;
  constexpr int NC = 64;                     // columns in registers when the sum is cut
  extern __shared__ __align__(1024) unsigned char dsm[];
  __shared__ Bars bars;
  cg::cluster_group cluster = cg::this_cluster();
  const int S = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  // the shuffle tells the compiler that the warp's number, and so its role, is uniform
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t base_raw = smem_u32(dsm);
  const uint32_t ring = (base_raw + 1023u) & ~1023u;
  const uint32_t plane_b = (uint32_t)a.N * 128u;
  const uint32_t stage_bytes = TW * kABytes + TX * plane_b;
  Work k;
  k.tile = blockIdx.x / S;
  k.step = gridDim.x / S;
  // steps split in pairs, so that units of 128 rows do not straddle blocks
  const int pairs = (a.steps + 1) / 2;
  k.k0 = 2 * (int)((int64_t)pairs * rank / S);
  k.k1 = 2 * (int)((int64_t)pairs * (rank + 1) / S);
  const int steps = k.k1 - k.k0;                      // per tile; even
  const int units = (steps + kChain - 1) / kChain;
  // accumulators: two of N columns, each with one for the small products beside it
  const uint32_t acc_cols = (kWhole ? 1u : 2u) * (uint32_t)a.N;
  uint32_t cols = 32;
  while (cols < 2u * acc_cols) cols *= 2;

  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map) : "memory");
    bars.abort = 0;
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(smem_u32(&bars.full[s]), 1 + kStepWarps<TW>);     // the copies and the weights' warps
      mbar_init(smem_u32(&bars.empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&bars.acc_full[b]), 1);
      mbar_init(smem_u32(&bars.acc_empty[b]), 4);
    }
    mbar_init(smem_u32(&bars.done), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars.tmem)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars.tmem, 0);
  grid_dep_wait();
  grid_dep_launch();

  if (warp == 0) {
    // ---------------- incoming gradients
    const uint32_t full = smem_u32(bars.full), empty = smem_u32(bars.empty);
    int64_t issued = 0;
    Ring rg;
    bool go = true;
    for (int64_t tile = k.tile; tile < a.tiles && go; tile += k.step) {
      const int64_t t0 = tile / a.tiles_m * a.N;
      for (int i = k.k0; i < k.k1; ++i) {
        go = rg.first || wait_or_abort(empty + 8u * (uint32_t)rg.s, rg.parity ^ 1u, &bars.abort, a.status);
        go = __all_sync(0xffffffffu, go);
        if (!go) break;
        if (elect_one()) {
          const uint32_t fb = full + 8u * (uint32_t)rg.s;
          mbar_expect_tx(fb, TX * plane_b);
          const uint32_t sb = ring + (uint32_t)rg.s * stage_bytes + TW * kABytes;
#pragma unroll
          for (int q = 0; q < TX; ++q)
            tma_load_2d(sb + q * plane_b, &map, fb, i * 64, (int)(q * a.plane + t0));
        }
        rg.advance(1, a.stages);
        ++issued;
      }
    }
    __syncwarp();
    // every issued copy must have landed before the block may exit
    for (int64_t i = max((int64_t)0, issued - a.stages); i < issued; ++i) {
      const long long t0 = clock64();
      while (!mbar_try_wait(full + 8u * (uint32_t)(i % a.stages), (uint32_t)((i / a.stages) & 1))) {
        // after an abort the weights may never arrive; the copies still do
        if (*(volatile int*)&bars.abort && clock64() - t0 > kBudget / 8) break;
        if (clock64() - t0 > kBudget) {
          atomicCAS(a.status, 0, (int)BAKRON_ERR_TIMEOUT);
          break;
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer: the warp waits together, one lane issues
    const uint32_t idesc = idesc_f16<H>(a.N);
    const uint64_t desc_a0 = desc_sw128(ring), desc_b0 = desc_sw128(ring + TW * kABytes);
    const uint32_t stage16 = stage_bytes >> 4, plane16 = plane_b >> 4;
    const uint32_t full = smem_u32(bars.full), empty = smem_u32(bars.empty);
    const uint32_t af = smem_u32(&bars.acc_full[0]), ae = smem_u32(&bars.acc_empty[0]);
    uint32_t u = 0;                          // units begun
    bool go = true;
    Ring rg;
    for (int64_t tile = k.tile; tile < a.tiles && go; tile += k.step) {
      for (int i = 0; i < steps; ++i) {
        const bool begin = i % kChain == 0, end = i % kChain == kChain - 1 || i == steps - 1;
        if (begin) {
          // the accumulator's previous unit, u - 2, has been read
          if (u >= 2) go = wait_or_abort(ae + 8u * (u & 1), ((u >> 1) & 1) ^ 1u, &bars.abort, a.status);
          ++u;
        }
        go = go && wait_or_abort(full + 8u * (uint32_t)rg.s, rg.parity, &bars.abort, a.status);
        go = __all_sync(0xffffffffu, go);
        if (!go) break;
        fence_after_sync();
        const uint64_t da = desc_a0 + (uint32_t)rg.s * stage16, db = desc_b0 + (uint32_t)rg.s * stage16;
        const uint32_t buf = (u - 1) & 1, d = tmem + buf * acc_cols;
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int qw = 0; qw < TW; ++qw)
#pragma unroll
              for (int qx = 0; qx < TX; ++qx) {
                // together at most 2^-24 (1 + 2^-9) of the product; the last term of dY, which
                // holds its infinities, meets the first of the weights alone (split3_grad)
                if (qw + qx > 2) continue;
                const bool large = qw == 0 && qx == 0;
                mma_f16(large ? d : d + (uint32_t)a.N, da + (uint32_t)(qw * (kABytes >> 4) + j * 2),
                        db + (qx * plane16 + j * 2), idesc, begin && j == 0 && (large || (qw == 0 && qx == 1)) ? 0u : 1u);
              }
          mma_commit(empty + 8u * (uint32_t)rg.s);
          if (end) mma_commit(af + 8u * buf);
        }
        __syncwarp();
        rg.advance(1, a.stages);
      }
    }
    if (elect_one()) mma_commit(smem_u32(&bars.done));
    __syncwarp();
  } else if (warp >= 4 && warp < 12) {
    weights<H, TW, NS>(a, k, bars, ring, stage_bytes, warp - 4, lane);
    __syncwarp();
  } else if (warp >= 12) {
    // ---------------- epilogue
    const int quarter = warp & 3;
    const uint32_t af = smem_u32(&bars.acc_full[0]), ae = smem_u32(&bars.acc_empty[0]);
    float* part = reinterpret_cast<float*>(dsm + (ring - base_raw));   // S > 1: [column][row], in the idle ring
    float range_in, range_out;
    operand_range<H>(a, range_in, range_out);
    uint32_t u_all = 0;
    bool ok = true;
    for (int64_t tile = k.tile; tile < a.tiles && ok; tile += k.step) {
      const int64_t row = (tile % a.tiles_m) * 128 + quarter * 32 + lane;
      const int64_t t0 = tile / a.tiles_m * a.N;
      TO* y = static_cast<TO*>(a.y) + t0 * a.w.n + row;
      float acc[kWhole ? 1 : NC];
      if constexpr (!kWhole) {
#pragma unroll
        for (int t = 0; t < NC; ++t) acc[t] = 0.f;
      }
      for (int u = 0; u < units; ++u, ++u_all) {
        ok = wait_or_abort(af + 8u * (u_all & 1), (u_all >> 1) & 1, &bars.abort, a.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        fence_after_sync();
        const uint32_t ta = tmem + ((uint32_t)(quarter * 32) << 16) + (u_all & 1) * acc_cols;
        if constexpr (kWhole) {
          for (int g = 0; g < a.N; g += 32) {
            float v[32];
            tmem_ld32(ta + (uint32_t)g, v);
            if (units > 1) {
              // chains are added in fp32, rounded, by way of the workspace
              float* sum = a.sums + ((int64_t)blockIdx.x * a.N + g) * 128 + quarter * 32 + lane;
              if (u > 0) {
#pragma unroll
                for (int t = 0; t < 32; ++t) v[t] += sum[t * 128];
              }
              if (u < units - 1) {
#pragma unroll
                for (int t = 0; t < 32; ++t) sum[t * 128] = v[t];
                continue;
              }
            }
            if (S > 1) {
#pragma unroll
              for (int t = 0; t < 32; ++t) part[(g + t) * 128 + quarter * 32 + lane] = v[t];
            } else if (row < a.w.n) {
              // lane = output column: the 32 lanes write 32 consecutive elements
#pragma unroll
              for (int t = 0; t < 32; ++t)
                if (t0 + g + t < a.T) y[(int64_t)(g + t) * a.w.n] = from_float<TO>(v[t] * range_out);
            }
          }
        } else {
#pragma unroll
          for (int g = 0; g < NC / 16; ++g) {
            if (g * 16 < a.N) {
              uint32_t v[16], c[16];
              tmem_ld16(ta + g * 16, v);
              tmem_ld16(ta + (uint32_t)a.N + g * 16, c);
              tmem_ld_wait();
#pragma unroll
              for (int t = 0; t < 16; ++t) acc[g * 16 + t] += __uint_as_float(v[t]) + __uint_as_float(c[t]);
            }
          }
        }
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(ae + 8u * (u_all & 1));
      }
      if constexpr (!kWhole) {
#pragma unroll
        for (int t = 0; t < NC; ++t) {
          if (t < a.N) {
            if (S > 1) part[t * 128 + quarter * 32 + lane] = acc[t];
            else if (ok && row < a.w.n && t0 + t < a.T) y[(int64_t)t * a.w.n] = from_float<TO>(acc[t] * range_out);
          }
        }
      }
    }
  }
  __syncwarp();
  // the wait below begins when the roles have ended: its budget is for the last
  // products, not for all of the block's tiles
  __syncthreads();

  // all MMAs must have completed before TMEM is freed and the ring is reused
  if (warp == 2) {
    const long long t0 = clock64();
    bool done = true;
    while (!mbar_try_wait(smem_u32(&bars.done), 0u)) {
      if (clock64() - t0 > kBudget) { done = false; break; }
    }
    if (!__all_sync(0xffffffffu, done) && lane == 0) atomicCAS(a.status, 0, (int)BAKRON_ERR_TIMEOUT);
  }
  fence_before_sync();
  __syncthreads();
  if (warp == 2) {
    fence_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
  }
  if (S > 1) {
    // each block adds up and writes every S-th column
    float* part = reinterpret_cast<float*>(dsm + (ring - base_raw));
    float range_in, range_out;
    operand_range<H>(a, range_in, range_out);
    __syncwarp();
    cluster.sync();
    const int r = threadIdx.x & 127;
    const int64_t row = (k.tile % a.tiles_m) * 128 + r, t0 = k.tile / a.tiles_m * a.N;
    for (int c = rank + S * (threadIdx.x >> 7); c < a.N; c += S * (kThreads / 128)) {
      if (row >= a.w.n || t0 + c >= a.T) continue;
      float v = 0.f;
      for (int q = 0; q < S; ++q) v += cluster.map_shared_rank(part, q)[c * 128 + r];
      static_cast<TO*>(a.y)[(t0 + c) * a.w.n + row] = from_float<TO>(v * range_out);
    }
    __syncwarp();
    cluster.sync();   // no block leaves while its sums are read
  }
}

template <typename TO, typename H, int TX, int TW, int NS>
cudaError_t run(const LinearArgs& a, int N, cudaStream_t s) {
  auto k = linear_grad_kernel<TO, H, TX, TW, NS>;
  const int64_t K = a.w.m;
  GradArgs t = {};
  t.w = a.w;
  t.y = a.y;
  t.T = a.T;
  t.tiles_m = (int)((a.w.n + 127) / 128);
  t.tiles = (int64_t)t.tiles_m * ((a.T + N - 1) / N);
  t.steps = (int)((K + 63) / 64);
  t.N = N;
  t.most = a.w.zero ? 15 : std::max(std::abs(a.w.zu), std::abs(15 - a.w.zu));
  const uint32_t stage = TW * kABytes + TX * (uint32_t)N * 128u;
  t.stages = (int)std::min<uint32_t>(kMaxStages, kRing / stage);
  t.status = async_status_word();
  if (!t.status) return cudaErrorInvalidSymbol;
  // dY: as it is when TMA can read it, else as planes
  const void* x = a.x;
  int64_t ldx = K, rows = a.T;
  t.plane = a.T;
  if (TX != 1 || !aligned_to(a.x, 16) || K % 8 != 0) {
    const int64_t kp = (K + 127) / 128 * 128;
    const cudaError_t e = launch_planes(a.x, a.dtype, a.T, K, kp, a.ws, s, true);
    if (e != cudaSuccess) return e;
    x = a.ws;
    ldx = kp;
    rows = TX * a.T;
  }
  CUtensorMap map;
  if (!make_map16(&map, x, rows, ldx, N, std::is_same<H, __nv_bfloat16>::value)) return cudaErrorInvalidValue;
  // blocks per tile: as many as there are SMs without a tile, 256 rows each at
  // least
  int S = 1;
  while (S < 8 && t.tiles * 2 * S <= sm_count() && t.steps >= 8 * S) S *= 2;
  if (a.dtype != BAKRON_F32 && a.w.m > grad_chain(a.dtype)) t.sums = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + grad_planes_bytes(a));
  static std::atomic<unsigned long long> done;
  const size_t smem = (size_t)t.stages * stage + 1024;
  cudaError_t e = ensure_smem_limit((const void*)k, kRing + 1024, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(std::min<int64_t>(t.tiles, S > 1 ? t.tiles : sm_count()) * S));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)S;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  count_launch();
  return cudaLaunchKernelEx(&cfg, k, map, t);
}

template <typename TO, typename H, int TX, int TW>
cudaError_t by_groups(const LinearArgs& a, int N, cudaStream_t s) {
  return a.w.ng == 1 || a.w.g % 128 == 0 ? run<TO, H, TX, TW, 1>(a, N, s) : run<TO, H, TX, TW, 4>(a, N, s);
}

// Tokens per tile, a multiple of 32: the fewest tokens' worth of rounds, each
// with a cost of its own of about 64 tokens.
int tokens_per_tile(int64_t T, int64_t tiles_m, int most) {
  int best = most;
  double cost = 0.0;
  for (int n = most; n >= 64 || n == most; n -= 32) {
    const double rounds = (double)((tiles_m * ((T + n - 1) / n) + sm_count() - 1) / sm_count());
    const double c = rounds * (n + 64);
    if (cost == 0.0 || c < cost) {
      cost = c;
      best = n;
    }
  }
  return (int)std::min<int64_t>(best, (T + 31) / 32 * 32);
}

}  // namespace

cudaError_t launch_linear_grad(const LinearArgs& a, cudaStream_t s) {
  const int64_t tiles_m = (a.w.n + 127) / 128;
  switch (a.dtype) {
    case BAKRON_F32: return by_groups<float, __nv_bfloat16, 3, 3>(a, tokens_per_tile(a.T, tiles_m, 64), s);
    case BAKRON_BF16: return by_groups<__nv_bfloat16, __nv_bfloat16, 1, 1>(a, tokens_per_tile(a.T, tiles_m, kGradTokens), s);
    default: return by_groups<__half, __half, 1, 1>(a, tokens_per_tile(a.T, tiles_m, kGradTokens), s);
  }
}

}  // namespace bakron
