// bakron_linear for many tokens and bakron_linear_grad: products of the packed
// weights on the tcgen05 tensor cores.
//
//   forward   D[i][t] = sum_j V_ij x_tj        (128 rows i of V, N tokens t)
//   gradient  D[j][t] = sum_i V_ij dy_ti       (128 columns j of V, N tokens t)
//
// The weights are the M operand: they come from memory as 4-bit words, turn
// into 16-bit values in registers and go to shared memory in the operand's
// layout (K-major, 128-byte swizzle); the activations are the N operand and
// come through TMA.  With the weights on the M side an output row is a TMEM
// lane, so the forward scale of a group is one number per thread.
//
// Forward: the operand holds the exact integers u - z.  The sum over a group
// (or over 128 columns of a longer one) goes into a fresh TMEM buffer, which
// the epilogue warps read, scale in fp32 and add to their registers while
// the tensor core fills the other buffer: no rounding of the weights, and no
// long chain of the tensor core's additions, which cut off instead of
// rounding.
// Gradient: the scale varies along the sum, so the operand holds the value
// s (u - z): rounded once to dY's type for 16-bit dY, in three exact bf16 terms
// for fp32 (six products, those whose weight is at least 2^-16).  fp32
// activations are three exact bf16 terms in both directions.  The columns of
// the packed words are the rows of this operand: a thread takes 8 rows x 8
// columns of codes and transposes them with one byte permutation per two words.
//
// One block of 16 warps per 128 x N tile, K in steps of 64:
//   warp 0, one thread: TMA producer of the activations;
//   warp 1, one thread: issues the tcgen05.mma (M 128, K 16 each);
//   warp 2: allocates and frees TMEM;
//   DW warps: weights from memory to registers, PF chunks ahead, to shared
//     memory;
//   EW warps: epilogue, each 32 TMEM lanes x NC columns in fp32 registers.
// Few tiles leave SMs without one: then K is split over the blocks of a
// cluster, whose sums meet in distributed shared memory, added in rank order.
//
// Every mbarrier wait is bounded (clock64 budget); a block whose wait runs
// out records BAKRON_ERR_TIMEOUT in the device's status word, stops issuing,
// drains its copies and MMAs (bounded again), frees TMEM and returns.
#include <cooperative_groups.h>

#include <algorithm>

#include "linear.cuh"
#include "tc_common.cuh"

namespace bakron {

namespace cg = cooperative_groups;
using namespace tc;

namespace {

constexpr int kThreads = 512;
constexpr uint32_t kABytes = 128 * 64 * 2;   // one plane of the weights' stage: 128 x 64
constexpr uint32_t kRing = 200 * 1024;       // shared memory for the stages
constexpr int kMaxStages = 8;
// NC = 128 needs more than the 128 registers a thread of the launch has: the
// epilogue's two warpgroups take 176, the weights' keeps 104 and the control
// warps' 56 (4 x 128 in all); every role returns to 128 before the common end.

struct TcArgs {
  PackedView w;
  void* y;
  int64_t T;          // tokens
  int64_t ld;         // leading dimension of y: rows of the M side that exist
  int64_t plane;      // token rows per plane of the activations' map
  int tiles_m;
  int chunks;         // 128-wide K chunks
  int N;              // tokens per tile, a multiple of 32 per epilogue column part
  int stages;
  int* status;
};

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

// Two fp32 values as a pair of H.
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

// Registers back to what the launch gave.  The epilogue gives its surplus up
// first and the other roles ask only after a barrier of the block: a role
// that asked earlier (with one or two accumulator buffers the issuer can end
// before the epilogue has its registers) would take what the epilogue waits
// for.  PTX also wants the warps of a warpgroup to meet between two setmaxnreg.
__device__ __forceinline__ void role_end(bool epilogue, int warp) {
  __syncwarp();
  if (epilogue) {
    asm volatile("bar.sync %0, 128;" ::"r"(1 + (warp >> 2)) : "memory");
    asm volatile("setmaxnreg.dec.sync.aligned.u32 128;");
    asm volatile("bar.sync 5, 512;" ::: "memory");
  } else {
    asm volatile("bar.sync 5, 512;" ::: "memory");
    asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
  }
}

struct Bars {
  unsigned long long full[kMaxStages], empty[kMaxStages];
  unsigned long long acc_full[2], acc_empty[2], done;
  uint32_t tmem;
  int abort;
};

// State that the roles share.
struct Ctx {
  Bars* bars;
  uint32_t ring;       // first stage
  uint32_t stage_bytes;
  uint32_t full, empty;   // barriers of the stages, 8 bytes each
  uint32_t tmem;
  int steps;           // K steps of 64
  int64_t c0;          // first K chunk
  int tile_m;
  int64_t t0;
};

// Bounded wait; the clock is read only once the first try has failed.
__device__ __forceinline__ bool wait_or_abort(const TcArgs& a, const Ctx& x, uint32_t bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  volatile int* ab = &x.bars->abort;
  if (mbar_wait(bar, parity, ab)) return true;
  atomicCAS(a.status, 0, (int)BAKRON_ERR_TIMEOUT);
  *ab = 1;
  return false;
}
// Position in the ring of stages, advanced without divisions: stage s and the
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
// Wait until the stage may be written.
__device__ __forceinline__ bool wait_free(const TcArgs& a, const Ctx& x, const Ring& r) {
  return r.first || wait_or_abort(a, x, x.empty + 8u * (uint32_t)r.s, r.parity ^ 1u);
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

// Weights of the forward product: warp dw of DW takes 16 / DW blocks of 8
// rows.  A 16-byte load holds words s = 0..3 of a row: 8 columns each, of the
// chunk's first K step (s = 0, 1) and second (s = 2, 3).
template <typename H, int DW, int PF>
__device__ __forceinline__ void weights_forward(const TcArgs& a, const Ctx& x, int dw, int lane) {
  constexpr int RB = 16 / DW;
  // eight lanes of a store phase: four 16-byte pieces of rows r and r + 4, whose
  // swizzles place them on different banks
  const int slot = lane >> 2, r = (slot >> 1) | ((slot & 1) << 2), t = lane & 3;
  const PackedView& w = a.w;
  const int64_t block0 = (int64_t)x.tile_m * 16 + dw * RB;
  const uint8_t* src = w.codes + (block0 * w.nc + x.c0) * kBlockBytes + r * 64 + t * 16;
  const int64_t stride = w.nc * kBlockBytes;
  const bool narrow = w.ng > 1 && w.g % 128 != 0;
  const int chunks = x.steps / 2;
  uint4 q[PF][RB];
  uint32_t z[PF][RB];   // zero points of the four words of a row, a byte each
  auto load = [&](uint4 (&qq)[RB], uint32_t (&zz)[RB], int c) {
    if (c >= chunks) return;
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const bool live = (block0 + b) * 8 < w.mp;
      qq[b] = make_uint4(0, 0, 0, 0);
      zz[b] = 0;
      if (live) {
        qq[b] = ld_codes(src + b * stride + (int64_t)c * kBlockBytes);
        if (w.zero) {
          const uint8_t* zp = w.zero + grid_row(w, 0, (block0 + b) * 8 + r);
          const uint32_t k0 = (uint32_t)((x.c0 + c) * 128);
          if (!narrow) {
            const uint32_t v = ld_ahead(zp + grid_group(w, k0) * 16);
            zz[b] = v * 0x01010101u;
          } else {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              zz[b] |= ld_ahead(zp + grid_group(w, k0 + 32 * s) * 16) << (8 * s);
            }
          }
        }
      }
    }
  };
  const uint32_t off_const = Half2<H>::pair(Half2<H>::kBase + (float)w.zu);
#pragma unroll
  for (int p = 0; p < PF; ++p) load(q[p], z[p], p);
  Ring rg;
  for (int c = 0; c < chunks; c += PF) {
#pragma unroll
    for (int p = 0; p < PF; ++p) {
      if (c + p < chunks) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!wait_free(a, x, rg)) return;
          const uint32_t sa = x.ring + (uint32_t)rg.s * x.stage_bytes;
#pragma unroll
          for (int b = 0; b < RB; ++b) {
            const int row = (dw * RB + b) * 8 + r;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int s = 2 * h + e;
              const uint32_t word = s == 0 ? q[p][b].x : s == 1 ? q[p][b].y : s == 2 ? q[p][b].z : q[p][b].w;
              const uint32_t off =
                  w.zero ? Half2<H>::pair(Half2<H>::kBase + (float)((z[p][b] >> (8 * s)) & 255u)) : off_const;
              uint32_t v[4];
              unpack_word<H>(word, off, v);
              sts128(sa + (uint32_t)row * 128u + (uint32_t)(((e * 4 + t) ^ (row & 7)) << 4), v[0], v[1], v[2], v[3]);
            }
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(x.full + 8u * (uint32_t)rg.s);
          rg.advance(1, a.stages);
        }
        load(q[p], z[p], c + p + PF);
      }
    }
  }
}

// Weights of the gradient's product: the K steps (64 rows x 128 columns of
// codes) go round the warps, at most one warp per stage (a wait tells a stage's
// uses apart by one bit, so no warp may be two uses ahead).  A thread holds 8 rows (a block) x 32
// columns and writes, for each of its columns, the 8 rows as one 16-byte piece.
template <typename H, int TW, int DW>
__device__ __forceinline__ void weights_gradient(const TcArgs& a, const Ctx& x, int dw, int lane) {
  const PackedView& w = a.w;
  const int rb = lane & 7, t = lane >> 3;
  const int64_t nb = w.mp / 8;
  const uint8_t* src = w.codes + (int64_t)x.tile_m * kBlockBytes + t * 16;
  const bool narrow = w.ng > 1 && w.g % 128 != 0;
  const uint32_t j0 = (uint32_t)x.tile_m * 128u;
  const int64_t first = x.c0 * 16 + rb;     // 8-row block of step 0
  uint4 q[8];
  auto load = [&](int i) {
    const int64_t b = first + (int64_t)i * 8;
    const bool live = i < x.steps && b < nb;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      q[k] = make_uint4(0, 0, 0, 0);
      if (live) q[k] = ld_codes(src + b * w.nc * kBlockBytes + k * 64);
    }
  };
  const int turn = min(DW, a.stages);
  if (dw >= turn) return;
  load(dw);
  Ring rg;
  rg.advance(dw, a.stages);
  for (int i = dw; i < x.steps; i += turn) {
    const int64_t b = first + (int64_t)i * 8;
    const bool live = b < nb;
    float sc[8];
    uint32_t off[4];
    const uint32_t sa = x.ring + (uint32_t)rg.s * x.stage_bytes;
    bool waited = false;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s == 0 || narrow) {
        const int64_t at = live ? grid_row(w, 0, b * 8) + grid_group(w, j0 + 32 * s) * 16 : 0;
        float4 s0 = make_float4(0.f, 0.f, 0.f, 0.f), s1 = s0;
        if (live) {
          s0 = __ldg(reinterpret_cast<const float4*>(w.scale + at));
          s1 = __ldg(reinterpret_cast<const float4*>(w.scale + at + 4));
        }
        sc[0] = s0.x; sc[1] = s0.y; sc[2] = s0.z; sc[3] = s0.w;
        sc[4] = s1.x; sc[5] = s1.y; sc[6] = s1.z; sc[7] = s1.w;
        uint2 zz = make_uint2(0, 0);
        if (w.zero && live) zz = __ldg(reinterpret_cast<const uint2*>(w.zero + at));
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint32_t zw = p < 2 ? zz.x : zz.y;
          const float z0 = w.zero ? (float)((zw >> (16 * (p & 1))) & 255u) : (float)w.zu;
          const float z1 = w.zero ? (float)((zw >> (16 * (p & 1) + 8)) & 255u) : (float)w.zu;
          off[p] = pack2(Half2<H>::kBase + z0, Half2<H>::kBase + z1, H());
        }
      }
      uint32_t word[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) word[k] = s == 0 ? q[k].x : s == 1 ? q[k].y : s == 2 ? q[k].z : q[k].w;
      if (!waited) {
        if (!wait_free(a, x, rg)) return;
        waited = true;
      }
#pragma unroll
      for (int odd = 0; odd < 2; ++odd) {
        uint32_t tr[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) tr[p] = __byte_perm(word[2 * p], word[2 * p + 1], odd ? 0x7632 : 0x5410);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int col = 32 * s + 8 * t + 2 * k + odd;
          const uint32_t at = sa + (uint32_t)col * 128u + (uint32_t)((rb ^ (col & 7)) << 4);
          uint32_t o[TW][4];
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const uint32_t u = Half2<H>::sub(((tr[p] >> (4 * k)) & 0x000f000fu) | Half2<H>::kMagic, off[p]);
            float2 f = unpack2(u, H());
            f.x *= sc[2 * p];
            f.y *= sc[2 * p + 1];
            if constexpr (TW == 1) {
              o[0][p] = pack2(f.x, f.y, H());
            } else {
              float x3[3], y3[3];
              split3(f.x, x3[0], x3[1], x3[2]);
              split3(f.y, y3[0], y3[1], y3[2]);
#pragma unroll
              for (int e = 0; e < TW; ++e) o[e][p] = (uint32_t)bf16_bits(x3[e]) | (uint32_t)bf16_bits(y3[e]) << 16;
            }
          }
#pragma unroll
          for (int e = 0; e < TW; ++e) sts128(at + e * kABytes, o[e][0], o[e][1], o[e][2], o[e][3]);
        }
      }
    }
    load(i + turn);
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(x.full + 8u * (uint32_t)rg.s);
    rg.advance(turn, a.stages);
  }
}

// GRAD: direction; TX, TW: 16-bit terms of the activations and of the
// weights; NC: columns per epilogue warp; DW: weight warps (EW = 12 - DW);
// KU: accumulation unit in MMA steps of 16 (2, 4 or 8).
template <typename TO, typename H, bool GRAD, int TX, int TW, int NC, int DW, int KU>
__global__ void __launch_bounds__(kThreads, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ TcArgs a) {
  constexpr int EW = 12 - DW;
  constexpr int PARTS = EW / 4;              // column parts of the epilogue
  extern __shared__ __align__(1024) unsigned char dsm[];
  __shared__ Bars bars;
  cg::cluster_group cluster = cg::this_cluster();
  const int S = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  // the shuffle tells the compiler that the warp's number, and so its role, is uniform
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int64_t tile = blockIdx.x / S;
  Ctx x;
  x.bars = &bars;
  x.full = smem_u32(bars.full);
  x.empty = smem_u32(bars.empty);
  const uint32_t base_raw = smem_u32(dsm);
  x.ring = (base_raw + 1023u) & ~1023u;
  const uint32_t plane_b = (uint32_t)a.N * 128u;
  x.stage_bytes = TW * kABytes + TX * plane_b;
  x.tile_m = (int)(tile % a.tiles_m);
  x.t0 = tile / a.tiles_m * a.N;
  x.c0 = (int64_t)a.chunks * rank / S;
  x.steps = 2 * (int)((int64_t)a.chunks * (rank + 1) / S - x.c0);
  const int units = x.steps * 4 / KU;
  uint32_t cols = 32;
  while (cols < 2u * (uint32_t)a.N) cols *= 2;

  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map) : "memory");
    bars.abort = 0;
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(smem_u32(&bars.full[s]), 1 + (GRAD ? 1 : DW));   // the copies and the weights
      mbar_init(smem_u32(&bars.empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&bars.acc_full[b]), 1);
      mbar_init(smem_u32(&bars.acc_empty[b]), EW);
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
  x.tmem = __shfl_sync(0xffffffffu, bars.tmem, 0);
  grid_dep_wait();
  grid_dep_launch();

  const int ew = warp - 4 - DW;              // epilogue warp
  const int quarter = warp & 3;
  const int col0 = ew >= 0 ? (ew / 4) * (a.N / PARTS) : 0;
  const int ncols = a.N / PARTS;             // a multiple of 16, at most NC

  if (warp < 4) {
    if constexpr (NC == 128) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      // ---------------- activations
      int issued = 0;
      Ring rg;
      for (int i = 0; i < x.steps; ++i) {
        if (!__all_sync(0xffffffffu, wait_free(a, x, rg))) break;
        if (elect_one()) {
          const uint32_t fb = x.full + 8u * (uint32_t)rg.s;
          mbar_expect_tx(fb, TX * plane_b);
          const uint32_t sb = x.ring + (uint32_t)rg.s * x.stage_bytes + TW * kABytes;
#pragma unroll
          for (int q = 0; q < TX; ++q)
            tma_load_2d(sb + q * plane_b, &map, fb, (int)(x.c0 * 128) + i * 64, (int)(q * a.plane + x.t0));
        }
        rg.advance(1, a.stages);
        ++issued;
      }
      __syncwarp();
      // every issued copy must have landed before the block may exit
      for (int i = max(0, issued - a.stages); i < issued; ++i) {
        const long long t0 = clock64();
        while (!mbar_try_wait(x.full + 8u * (uint32_t)(i % a.stages), (uint32_t)((i / a.stages) & 1))) {
          if (clock64() - t0 > kBudget) {
            atomicCAS(a.status, 0, (int)BAKRON_ERR_TIMEOUT);
            break;
          }
        }
      }
    } else if (warp == 1) {
      // ---------------- MMA issuer: the warp waits together, one lane issues.
      // A single warp's dependent instructions, not the tensor core, bound
      // this loop when it is long, so everything is fixed per K chunk of two
      // stages: where units begin and end, and the descriptors' offsets.
      const uint32_t idesc = idesc_f16<H>(a.N);
      const uint64_t desc_a0 = desc_sw128(x.ring), desc_b0 = desc_sw128(x.ring + TW * kABytes);
      const uint32_t stage16 = x.stage_bytes >> 4, plane16 = plane_b >> 4;
      const uint32_t af = smem_u32(&bars.acc_full[0]), ae = smem_u32(&bars.acc_empty[0]);
      constexpr int UPS = KU >= 4 ? 1 : 2;    // units that a stage takes part in
      uint32_t u = 0;                         // units begun
      bool go = true;
      Ring rg;
      for (int c = 0; c < x.steps / 2 && go; ++c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (KU < 8 || h == 0) {
#pragma unroll
            for (int k = 0; k < UPS; ++k) {
              // the buffer's previous unit, u - 2, has been read
              if (u >= 2) go = go && wait_or_abort(a, x, ae + 8u * (u & 1), ((u >> 1) & 1) ^ 1u);
              ++u;
            }
          }
          go = go && wait_or_abort(a, x, x.full + 8u * (uint32_t)rg.s, rg.parity);
          go = __all_sync(0xffffffffu, go);
          if (!go) break;
          fence_after_sync();
          if (elect_one()) {
            const uint64_t da = desc_a0 + (uint32_t)rg.s * stage16, db = desc_b0 + (uint32_t)rg.s * stage16;
            const uint32_t first_u = u - UPS;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t buf = (first_u + (KU == 2 ? j / 2 : 0)) & 1;
              const uint32_t d = x.tmem + buf * (uint32_t)a.N;
              const bool begin = KU == 8 ? h == 0 && j == 0 : j % KU == 0;
              const bool end = KU == 8 ? h == 1 && j == 3 : j % KU == KU - 1;
              bool fresh = begin;
#pragma unroll
              for (int qw = 0; qw < TW; ++qw)
#pragma unroll
                for (int qx = 0; qx < TX; ++qx) {
                  if (qw + qx > 2) continue;   // below 2^-24 of the product
                  mma_f16(d, da + (uint32_t)(qw * (kABytes >> 4) + j * 2), db + (qx * plane16 + j * 2), idesc,
                          fresh ? 0u : 1u);
                  fresh = false;
                }
              if (end) mma_commit(af + 8u * buf);
            }
            mma_commit(x.empty + 8u * (uint32_t)rg.s);
          }
          __syncwarp();
          rg.advance(1, a.stages);
        }
      }
      if (elect_one()) mma_commit(smem_u32(&bars.done));
      __syncwarp();
    }
    if constexpr (NC == 128) role_end(false, warp);
  } else if (warp < 4 + DW) {
    // ---------------- weights
    if constexpr (NC == 128) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if constexpr (GRAD) weights_gradient<H, TW, DW>(a, x, warp - 4, lane);
    else weights_forward<H, DW, DW == 8 ? 4 : 2>(a, x, warp - 4, lane);
    if constexpr (NC == 128) role_end(false, warp);
  } else {
    // ---------------- epilogue: running fp32 sums
    if constexpr (NC == 128) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    float acc[NC];
    bool ok = true;
#pragma unroll
    for (int t = 0; t < NC; ++t) acc[t] = 0.f;
    const int64_t row = (int64_t)x.tile_m * 128 + quarter * 32 + lane;
    const bool live = !GRAD && row < a.w.mp;
    const float* scale_row = a.w.scale + (live ? grid_row(a.w, 0, row) : 0);
    auto scale_of = [&](int u) {
      if (!live || u >= units) return 0.f;
      const uint32_t k = (uint32_t)(x.c0 * 128) + (uint32_t)u * (KU * 16);
      return ld_ahead(scale_row + grid_group(a.w, k) * 16);
    };
    float s_next = scale_of(0);
    for (int u = 0; u < units; ++u) {
      const float s = GRAD ? 1.f : s_next;
      if constexpr (!GRAD) s_next = scale_of(u + 1);
      ok = wait_or_abort(a, x, smem_u32(&bars.acc_full[u & 1]), (uint32_t)((u >> 1) & 1));
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      fence_after_sync();
      const uint32_t ta = x.tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)((u & 1) * a.N + col0);
#pragma unroll
      for (int g = 0; g < NC / 16; ++g) {
        if (g * 16 < ncols) {
          uint32_t v[16];
          tmem_ld16(ta + g * 16, v);
          tmem_ld_wait();
#pragma unroll
          for (int t = 0; t < 16; ++t) acc[g * 16 + t] = fmaf(s, __uint_as_float(v[t]), acc[g * 16 + t]);
        }
      }
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.acc_empty[u & 1]));
    }
    if (S > 1) {
      // this block's sums [column][row] into the ring, idle once the last
      // accumulator has been read
      float* part = reinterpret_cast<float*>(dsm + (x.ring - base_raw));
#pragma unroll
      for (int t = 0; t < NC; ++t)
        if (t < ncols) part[(col0 + t) * 128 + quarter * 32 + lane] = acc[t];
    } else if (ok && row < a.ld) {
      // lane = output column: the 32 lanes write 32 consecutive elements
      TO* y = static_cast<TO*>(a.y) + (x.t0 + col0) * a.ld + row;
#pragma unroll
      for (int t = 0; t < NC; ++t)
        if (t < ncols && x.t0 + col0 + t < a.T) y[(int64_t)t * a.ld] = from_float<TO>(acc[t]);
    }
    if constexpr (NC == 128) role_end(true, warp);
  }
  __syncwarp();

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
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(x.tmem), "r"(cols) : "memory");
  }
  if (S > 1) {
    // each block adds up and writes every S-th column
    float* part = reinterpret_cast<float*>(dsm + (x.ring - base_raw));
    cluster.sync();
    const int r = threadIdx.x & 127;
    const int64_t row = (int64_t)x.tile_m * 128 + r;
    for (int c = rank + S * (threadIdx.x >> 7); c < a.N; c += S * (kThreads / 128)) {
      if (row >= a.ld || x.t0 + c >= a.T) continue;
      float v = 0.f;
      for (int k = 0; k < S; ++k) v += cluster.map_shared_rank(part, k)[c * 128 + r];
      static_cast<TO*>(a.y)[(x.t0 + c) * a.ld + row] = from_float<TO>(v);
    }
    __syncwarp();
    cluster.sync();   // no block leaves while its sums are read
  }
}

// x (T x K, any alignment) -> planes [TERMS][T][kp] of 16-bit terms, zeros
// past K: the activations as the tensor map wants them.
template <typename TX, int TERMS>
__global__ void __launch_bounds__(256) planes_kernel(const TX* __restrict__ x, int64_t T, int64_t K,
                                                     int64_t kp, uint16_t* __restrict__ out) {
  const int64_t per = kp / 8, total = T * per;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t t = i / per, k = (i - t * per) * 8;
    uint32_t h[TERMS][4];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t v[3] = {0, 0, 0};
      if (k + e < K) {
        const TX* p = x + t * K + k + e;
        if constexpr (TERMS == 1) {
          v[0] = *reinterpret_cast<const uint16_t*>(p);
        } else {
          float f[3];
          split3(to_float(*p), f[0], f[1], f[2]);
#pragma unroll
          for (int q = 0; q < 3; ++q) v[q] = bf16_bits(f[q]);
        }
      }
#pragma unroll
      for (int q = 0; q < TERMS; ++q) h[q][e >> 1] = (e & 1) ? (h[q][e >> 1] | v[q] << 16) : v[q];
    }
#pragma unroll
    for (int q = 0; q < TERMS; ++q)
      *reinterpret_cast<uint4*>(out + (q * T + t) * kp + k) = make_uint4(h[q][0], h[q][1], h[q][2], h[q][3]);
  }
}

int64_t k_padded(int64_t K) { return (K + 127) / 128 * 128; }

template <typename TO, typename H, bool GRAD, int TX, int TW, int NC, int DW, int KU>
cudaError_t run_unit(const LinearArgs& a, int N, cudaStream_t s) {
  auto k = linear_tc_kernel<TO, H, GRAD, TX, TW, NC, DW, KU>;
  const int64_t K = GRAD ? a.w.m : a.w.n, M = GRAD ? a.w.n : a.w.m;
  TcArgs t = {};
  t.w = a.w;
  t.y = a.y;
  t.T = a.T;
  t.ld = M;
  t.tiles_m = (int)((M + 127) / 128);
  t.chunks = (int)((K + 127) / 128);
  t.N = N;
  const uint32_t stage = TW * kABytes + TX * (uint32_t)N * 128u;
  t.stages = (int)std::min<uint32_t>(kMaxStages, kRing / stage);
  t.status = async_status_word();
  if (!t.status) return cudaErrorInvalidSymbol;
  // activations: as they are when TMA can read them, else as planes
  const void* x = a.x;
  int64_t ldx = K, rows = a.T;
  t.plane = a.T;
  if (TX != 1 || !aligned_to(a.x, 16) || K % 8 != 0) {
    const int64_t kp = k_padded(K);
    cudaError_t e = launch_planes(a.x, a.dtype, a.T, K, kp, a.ws, s);
    if (e != cudaSuccess) return e;
    x = a.ws;
    ldx = kp;
    rows = TX * a.T;
  }
  CUtensorMap map;
  if (!make_map16(&map, x, rows, ldx, N, std::is_same<H, __nv_bfloat16>::value)) return cudaErrorInvalidValue;
  const int64_t tiles = (int64_t)t.tiles_m * ((a.T + N - 1) / N);
  // blocks per tile: as many as there are SMs without a tile, at least two
  // chunks each
  int S = 1;
  while (S < 8 && tiles * 2 * S <= sm_count() && t.chunks >= 4 * S) S *= 2;
  static std::atomic<unsigned long long> done;
  const size_t smem = (size_t)t.stages * stage + 1024;
  cudaError_t e = ensure_smem_limit((const void*)k, kRing + 1024, done);
  if (e != cudaSuccess) return e;
  if (tiles * S > 0x7fffffff) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * S));
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

// A unit ends where a group does: 128, 64 or 32 columns.
template <typename TO, typename H, bool GRAD, int TX, int TW, int NC, int DW>
cudaError_t run(const LinearArgs& a, int N, cudaStream_t s) {
  if constexpr (!GRAD) {
    if (a.w.ng > 1 && a.w.g % 128 != 0)
      return a.w.g % 64 == 0 ? run_unit<TO, H, GRAD, TX, TW, NC, DW, 4>(a, N, s)
                             : run_unit<TO, H, GRAD, TX, TW, NC, DW, 2>(a, N, s);
  }
  return run_unit<TO, H, GRAD, TX, TW, NC, DW, 8>(a, N, s);
}

int tokens_per_tile(int64_t T, int most) {
  const int64_t n = (T + 31) / 32 * 32;
  return (int)std::min<int64_t>(n, most);
}

template <typename TO, bool GRAD>
cudaError_t run16(const LinearArgs& a, cudaStream_t s) {
  if (a.T <= 64) return run<TO, TO, GRAD, 1, 1, 64, 8>(a, tokens_per_tile(a.T, 64), s);
  return run<TO, TO, GRAD, 1, 1, 128, 4>(a, tokens_per_tile(a.T, 256), s);
}

}  // namespace

cudaError_t launch_planes(const void* x, int dtype, int64_t T, int64_t K, int64_t kp, void* out,
                          cudaStream_t s) {
  const int64_t total = T * kp / 8;
  const unsigned g = (unsigned)std::max<int64_t>(1, std::min<int64_t>((total + 255) / 256, (int64_t)sm_count() * 16));
  uint16_t* o = static_cast<uint16_t*>(out);
  count_launch();
  if (dtype == BAKRON_F32) planes_kernel<float, 3><<<g, 256, 0, s>>>(static_cast<const float*>(x), T, K, kp, o);
  else planes_kernel<uint16_t, 1><<<g, 256, 0, s>>>(static_cast<const uint16_t*>(x), T, K, kp, o);
  return cudaGetLastError();
}

size_t linear_tc_workspace(int64_t T, int64_t K, int dtype) {
  return (size_t)(dtype == BAKRON_F32 ? 3 : 1) * (size_t)T * (size_t)k_padded(K) * 2;
}

cudaError_t launch_linear_tc(const LinearArgs& a, bool grad, cudaStream_t s) {
  switch (a.dtype) {
    case BAKRON_F32:
      if (grad) return run<float, __nv_bfloat16, true, 3, 3, 64, 8>(a, tokens_per_tile(a.T, 64), s);
      return run<float, __nv_bfloat16, false, 3, 1, 64, 4>(a, tokens_per_tile(a.T, 128), s);
    case BAKRON_BF16:
      return grad ? run16<__nv_bfloat16, true>(a, s) : run16<__nv_bfloat16, false>(a, s);
    default:
      return grad ? run16<__half, true>(a, s) : run16<__half, false>(a, s);
  }
}

}  // namespace bakron
