// bakron_linear for many tokens: D[i][t] = sum_j V_ij x_tj on the tcgen05
// tensor cores.
//
// The weights are the M operand (128 rows i), the activations the N operand (N
// tokens t), so an output row is a TMEM lane and the scale of a group one number
// per thread.  The codes never reach shared memory as an operand: a warp whose lanes are 32
// rows turns a row's words into the exact integers u - z in registers and
// stores them to tensor memory, from which the tensor core takes its A operand.
// With A and B both in shared memory the products were bound by its bandwidth
// (A and B written and read: 96 KB a step of 64 columns and 256 tokens, 750 cycles
// of 128 bytes against 512 of the tensor core; measured 810).
//
// The sum over a group (or over 128 columns of a longer one) goes into a fresh
// accumulator, which the epilogue warps read, scale in fp32 and add to their
// registers while the tensor core fills the other one: no rounding of the weights,
// and no long chain of the tensor core's additions, which cut off instead of
// rounding.  fp32 activations are three exact bf16 terms; the products of the two
// small ones have an accumulator of their own.
//
// One block per SM, which takes output tiles in turn (or, when there are few, a
// part of the columns of one, joined over a cluster through distributed shared memory):
//   warp 0: TMA producer of the activations;
//   warp 1: issues the tcgen05.mma (M 128, K 16 each);
//   warp 2: allocates and frees TMEM;
//   warps 4-11: weights, two groups of four (32 rows each) that take the
//     128-column chunks in turn, codes copied asynchronously kAhead chunks ahead;
//   the rest: epilogue, each 32 TMEM lanes x NC columns in fp32 registers.
// A stage is a whole chunk, of weights (64 TMEM columns) and of activations: what the
// issuing warp waits and commits per stage costs it some 400 cycles, so stages of
// half a chunk kept the tensor core waiting for it.  TMEM: two accumulators of N
// columns, then four stages of weights (two where N is above 128).
//
// Measured: 2048 tokens of 8192 x 8192 bf16 in 206 us in a graph of one weight (1.34
// PFLOP/s) and 215 among calls on several; 48 tokens 25 us; fp32, 1024 tokens of 4096 x 4096 103 us
// and 2048 of 8192 x 8192 648 us (three products: 1.27 PFLOP/s).  A
// chunk takes 1270 cycles at 192 tokens, of which the tensor core works 768: the
// issuing warp's waits, one after the other, are the rest; few tokens do not make it
// shorter than 985, what eight warps need to turn a chunk's codes into
// operands.  With groups of 32 columns an accumulator goes to and fro every 32
// columns, 650 cycles each (1024 tokens of 4096 x 4096: 102 us, groups of 128: 44).  Tried and
// slower: one wait of three lanes on the three barriers (208 -> 260 us), the scales
// copied ahead to shared memory (208 -> 234).
//
// Every mbarrier wait is bounded (clock64 budget); a block whose wait runs
// out records BAKRON_ERR_TIMEOUT in the device's status word, stops issuing,
// drains its copies and MMAs (bounded again), frees TMEM and returns.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "linear_tc.cuh"

namespace bakron {

namespace cg = cooperative_groups;
using namespace tc;

namespace {

constexpr int kWStages = 4;                  // of weights in TMEM, 64 columns each, at most
constexpr int kMaxStages = 8;                // of activations in shared memory
constexpr int kSlots = 3;                    // chunks of codes per weights warp, in flight and at hand
constexpr uint32_t kSlotBytes = 32 * 64;     // 32 rows x 128 columns of codes
constexpr uint32_t kCodes = 8 * kSlots * kSlotBytes;
constexpr uint32_t kRing = 172 * 1024;       // shared memory for the activations' stages

struct FwdArgs {
  PackedView w;
  void* y;
  int64_t T;          // tokens
  int64_t plane;      // token rows per plane of the activations' map
  int tiles_m;
  int64_t tiles;      // tiles of the output
  int chunks;         // 128-wide K chunks
  int N;              // tokens per tile, a multiple of 32
  int stages;
  int wstages;        // 4 where TMEM has room, else 2: a power of two
  int* status;
};

__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc));
}
// 32 registers of each lane to 32 TMEM columns of its row.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// Two fp32 values with one instruction: of short groups, whose accumulators are
// read most often, these additions are what the epilogue is bound by.
__device__ __forceinline__ void add2(uint32_t& x, uint32_t& y, uint32_t a, uint32_t b) {
  asm("{\n .reg .b64 p, q;\n mov.b64 p, {%0, %1};\n mov.b64 q, {%2, %3};\n add.rn.f32x2 p, p, q;\n"
      " mov.b64 {%0, %1}, p;\n}\n"
      : "+r"(x), "+r"(y)
      : "r"(a), "r"(b));
}
__device__ __forceinline__ void fma2(float& x, float& y, float s, uint32_t a, uint32_t b) {
  asm("{\n .reg .b64 p, q, r;\n mov.b64 p, {%0, %1};\n mov.b64 q, {%2, %2};\n mov.b64 r, {%3, %4};\n"
      " fma.rn.f32x2 p, q, r, p;\n mov.b64 {%0, %1}, p;\n}\n"
      : "+f"(x), "+f"(y)
      : "f"(s), "r"(a), "r"(b));
}

struct Bars {
  unsigned long long full_b[kMaxStages], empty_b[kMaxStages], full_a[kWStages], empty_a[kWStages];
  unsigned long long acc_full[2], acc_empty[2], done;
  uint32_t tmem;
  int abort;
};

// The block's work: output tiles tile, tile + step, ...; K chunks [c0, c1) of each.
struct Work {
  int64_t tile, step;
  int c0, c1;
};

// Registers back to what the launch gave.  The epilogue gives its surplus up
// first and the other roles ask only after a barrier of the block: a role
// that asked earlier (with one or two accumulators the issuer can end before
// the epilogue has its registers) would take what the epilogue waits for.
// PTX also wants the warps of a warpgroup to meet between two setmaxnreg.
template <int THREADS, int REGS>
__device__ __forceinline__ void role_end(bool epilogue, int warp) {
  __syncwarp();
  if (epilogue) {
    asm volatile("bar.sync %0, 128;" ::"r"(1 + (warp >> 2)) : "memory");
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
    asm volatile("bar.sync 7, %0;" ::"n"(THREADS) : "memory");
  } else {
    asm volatile("bar.sync 7, %0;" ::"n"(THREADS) : "memory");
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
  }
}

// One chunk of codes at a time: 32 rows (a lane each) x 128 columns.
template <typename H>
__device__ __forceinline__ void weights(const FwdArgs& a, const Work& k, Bars& bars, uint32_t tmem_a,
                                        uint32_t codes, int group, int quarter, int lane) {
  const PackedView& w = a.w;
  const bool narrow = w.ng > 1 && w.g % 128 != 0;
  const uint32_t off_const = Half2<H>::pair(Half2<H>::kBase + (float)w.zu);
  const uint32_t full = smem_u32(bars.full_a), empty = smem_u32(bars.empty_a);
  // Copies: lane l brings 16 bytes of row 8 i + l / 4 of the warp's four blocks
  // i; a row's 16-byte pieces are rotated by the row so that reading a row per
  // lane meets all banks.
  const int copy_row = lane >> 2, copy_t = lane & 3;
  const uint32_t copy_at = codes + (uint32_t)copy_row * 64u + (uint32_t)(((copy_t + (copy_row >> 1)) & 3) << 4);
  const uint32_t read_at = codes + (uint32_t)lane * 64u;
  const int turn = (lane >> 1) & 3;
  // sequence of this group's chunks over all tiles: every other one
  int64_t tile_ahead = k.tile, tile_now = k.tile;
  int c_ahead = k.c0 + group, c_now = k.c0 + group;
  const int n = k.c1 - k.c0;
  int m_ahead = (int)(k.tile % a.tiles_m), m_now = m_ahead;      // the tile's row block
  auto settle = [&](int64_t& tile, int& c, int& m) {
    if (c < k.c1) return;
    while (c >= k.c1 && tile < a.tiles) {
      c -= n;
      tile += k.step;
    }
    m = (int)(tile % a.tiles_m);
  };
  settle(tile_ahead, c_ahead, m_ahead);
  settle(tile_now, c_now, m_now);
  uint32_t fill = 0, read = 0;
  auto copy = [&]() {
    if (tile_ahead < a.tiles) {
      const int64_t block = (int64_t)m_ahead * 16 + quarter * 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool live = (block + i) * 8 < w.mp;      // zeros below the last row
        const uint8_t* src = w.codes + ((live ? block + i : 0) * w.nc + c_ahead) * kBlockBytes + lane * 16;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(copy_at + fill + (uint32_t)i * 512u), "l"(src),
                     "r"(live ? 16u : 0u)
                     : "memory");
      }
      c_ahead += 2;
      settle(tile_ahead, c_ahead, m_ahead);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    fill = fill + kSlotBytes == kSlots * kSlotBytes ? 0 : fill + kSlotBytes;
  };
  // the row's zero points of a chunk, a byte per 32 columns
  auto zeros = [&](int64_t tile, int c, int m) -> uint32_t {
    if (w.zero == nullptr || tile >= a.tiles) return 0u;
    const int64_t row = (int64_t)m * 128 + quarter * 32 + lane;
    if (row >= w.mp) return 0u;
    const uint8_t* p = w.zero + grid_row(w, 0, row);
    if (!narrow) return ld_ahead(p + grid_group(w, (uint32_t)c * 128) * 16) * 0x01010101u;
    uint32_t z = 0;
#pragma unroll
    for (int s = 0; s < 4; ++s) z |= ld_ahead(p + grid_group(w, (uint32_t)c * 128 + 32 * s) * 16) << (8 * s);
    return z;
  };
#pragma unroll
  for (int p = 0; p < kSlots - 1; ++p) copy();
  uint32_t z = zeros(tile_now, c_now, m_now);
  uint32_t seq = (uint32_t)group;      // chunk of the block
  const uint32_t last_stage = (uint32_t)a.wstages - 1;
  const int log_stages = a.wstages == 4 ? 2 : 1;
  while (tile_now < a.tiles) {
    copy();
    asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory");
    __syncwarp();
    uint4 q[4];              // words (s, t): q[t] holds s = 0..3
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t at = read_at + read + (uint32_t)(((t + turn) & 3) << 4);
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(q[t].x), "=r"(q[t].y), "=r"(q[t].z), "=r"(q[t].w)
                   : "r"(at)
                   : "memory");
    }
    read = read + kSlotBytes == kSlots * kSlotBytes ? 0 : read + kSlotBytes;
    const uint32_t z_now = z;
    c_now += 2;
    settle(tile_now, c_now, m_now);
    z = zeros(tile_now, c_now, m_now);
    const uint32_t ws = seq & last_stage;        // (a fresh barrier passes the wait for its previous use)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t v[32];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int s = 2 * h + e;
        const uint32_t off =
            w.zero ? Half2<H>::pair(Half2<H>::kBase + (float)((z_now >> (8 * s)) & 255u)) : off_const;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t word = s == 0 ? q[t].x : s == 1 ? q[t].y : s == 2 ? q[t].z : q[t].w;
          uint32_t p[4];
          unpack_word<H>(word, off, p);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[e * 16 + t * 4 + i] = p[i];
        }
      }
      if (h == 0) {
        if (!__all_sync(0xffffffffu, wait_or_abort(empty + 8u * ws, ((seq >> log_stages) & 1) ^ 1u, &bars.abort, a.status))) goto out;
        fence_after_sync();
      }
      tmem_st32(tmem_a + ((uint32_t)(quarter * 32) << 16) + ws * 64u + (uint32_t)(h * 32), v);
    }
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
    fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(full + 8u * ws);
    seq += 2;
  }
out:
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// TX: 16-bit terms of the activations; NC: columns per epilogue warp; EW:
// epilogue warps; KU: accumulation unit in MMA steps of 16 (2, 4 or 8).
template <typename TO, typename H, int TX, int NC, int EW, int KU>
__global__ void __launch_bounds__(32 * (12 + EW), 1)
    linear_fwd_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ FwdArgs a) {
  constexpr int THREADS = 32 * (12 + EW);
  constexpr int PARTS = EW / 4;              // column parts of the epilogue
  // 640 threads start with 96 registers each; the roles share them out
  // (8 x 136 + 8 x 72 + 4 x 64 warps' worth of 20 x 96)
  constexpr bool kSplit = EW == 8;
  extern __shared__ __align__(1024) unsigned char dsm[];
  __shared__ Bars bars;
  cg::cluster_group cluster = cg::this_cluster();
  const int S = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  // the shuffle tells the compiler that the warp's number, and so its role, is uniform
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t base_raw = smem_u32(dsm);
  const uint32_t ring = (base_raw + 1023u) & ~1023u;
  const uint32_t plane_b = (uint32_t)a.N * 128u, half_bytes = TX * plane_b, stage_bytes = 2 * half_bytes;
  Work k;
  k.tile = blockIdx.x / S;
  k.step = gridDim.x / S;
  k.c0 = (int)((int64_t)a.chunks * rank / S);
  k.c1 = (int)((int64_t)a.chunks * (rank + 1) / S);
  const int units = (k.c1 - k.c0) * 8 / KU;   // per tile

  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map) : "memory");
    bars.abort = 0;
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(smem_u32(&bars.full_b[s]), 1);
      mbar_init(smem_u32(&bars.empty_b[s]), 1);
    }
    for (int s = 0; s < kWStages; ++s) {
      mbar_init(smem_u32(&bars.full_a[s]), 4);       // the warps of a group
      mbar_init(smem_u32(&bars.empty_a[s]), 1);
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
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t acc_cols = (TX == 1 ? 1u : 2u) * (uint32_t)a.N;
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars.tmem, 0), tmem_a = tmem + 2u * acc_cols;
  grid_dep_wait();
  grid_dep_launch();

  if (warp < 4) {
    if constexpr (kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0) {
      // ---------------- activations
      const uint32_t full = smem_u32(bars.full_b), empty = smem_u32(bars.empty_b);
      int64_t issued = 0;
      Ring rg;
      bool go = true;
      for (int64_t tile = k.tile; tile < a.tiles && go; tile += k.step) {
        const int64_t t0 = tile / a.tiles_m * a.N;
        for (int c = k.c0; c < k.c1; ++c) {
          go = rg.first || wait_or_abort(empty + 8u * (uint32_t)rg.s, rg.parity ^ 1u, &bars.abort, a.status);
          go = __all_sync(0xffffffffu, go);
          if (!go) break;
          if (elect_one()) {
            const uint32_t fb = full + 8u * (uint32_t)rg.s;
            mbar_expect_tx(fb, stage_bytes);
            const uint32_t sb = ring + (uint32_t)rg.s * stage_bytes;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int q = 0; q < TX; ++q)
                tma_load_2d(sb + h * half_bytes + q * plane_b, &map, fb, c * 128 + h * 64, (int)(q * a.plane + t0));
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
          if (clock64() - t0 > kBudget) {
            atomicCAS(a.status, 0, (int)BAKRON_ERR_TIMEOUT);
            break;
          }
        }
      }
    } else if (warp == 1) {
      // ---------------- MMA issuer: the warp waits together, one lane issues.
      // A single warp's dependent instructions, not the tensor core, bound
      // this loop when it is long, so everything is fixed per K chunk:
      // where units begin and end, and the descriptors' offsets.
      const uint32_t idesc = idesc_f16<H>(a.N);
      const uint64_t desc_b0 = desc_sw128(ring);
      const uint32_t stage16 = stage_bytes >> 4, half16 = half_bytes >> 4, plane16 = plane_b >> 4;
      const uint32_t fb = smem_u32(bars.full_b), eb = smem_u32(bars.empty_b);
      const uint32_t fa = smem_u32(bars.full_a), ea = smem_u32(bars.empty_a);
      const uint32_t af = smem_u32(&bars.acc_full[0]), ae = smem_u32(&bars.acc_empty[0]);
      constexpr int UPC = 8 / KU;             // units of a chunk
      uint32_t u = 0;                         // units begun
      uint32_t seq = 0;                       // chunks begun
      const uint32_t last_stage = (uint32_t)a.wstages - 1;
      const int log_stages = a.wstages == 4 ? 2 : 1;
      bool go = true;
      Ring rg;
      for (int64_t tile = k.tile; tile < a.tiles && go; tile += k.step) {
        for (int c = k.c0; c < k.c1; ++c) {
          const uint32_t ws = seq & last_stage;
          go = wait_or_abort(fb + 8u * (uint32_t)rg.s, rg.parity, &bars.abort, a.status) &&
               wait_or_abort(fa + 8u * ws, (seq >> log_stages) & 1, &bars.abort, a.status);
          fence_after_sync();
          const uint64_t db = desc_b0 + (uint32_t)rg.s * stage16;
          const uint32_t ta = tmem_a + ws * 64u;
#pragma unroll
          for (int i = 0; i < UPC; ++i) {
            const uint32_t v = u + i, buf = v & 1;
            // the accumulator: unit v - 2 has been read
            go = go && (v < 2 || wait_or_abort(ae + 8u * buf, ((v >> 1) & 1) ^ 1u, &bars.abort, a.status));
            go = __all_sync(0xffffffffu, go);
            if (!go) break;
            fence_after_sync();
            if (elect_one()) {
              const uint32_t d = tmem + buf * acc_cols;
#pragma unroll
              for (int j = i * KU; j < (i + 1) * KU; ++j)
#pragma unroll
                for (int q = 0; q < TX; ++q)
                  mma_f16_ts(q == 0 ? d : d + (uint32_t)a.N, ta + j * 8,
                             db + ((j / 4) * half16 + q * plane16 + (j % 4) * 2), idesc, j % KU == 0 && q <= 1 ? 0u : 1u);
              mma_commit(af + 8u * buf);
              if (i == UPC - 1) {
                mma_commit(eb + 8u * (uint32_t)rg.s);
                mma_commit(ea + 8u * ws);
              }
            }
            __syncwarp();
          }
          if (!go) break;
          u += UPC;
          ++seq;
          rg.advance(1, a.stages);
        }
      }
      if (elect_one()) mma_commit(smem_u32(&bars.done));
      __syncwarp();
    }
    if constexpr (kSplit) role_end<THREADS, 96>(false, warp);
  } else if (warp < 12) {
    // ---------------- weights
    if constexpr (kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const uint32_t codes = ring + (uint32_t)a.stages * stage_bytes + (uint32_t)(warp - 4) * (kSlots * kSlotBytes);
    weights<H>(a, k, bars, tmem_a, codes, (warp - 4) >> 2, warp & 3, lane);
    if constexpr (kSplit) role_end<THREADS, 96>(false, warp);
  } else {
    // ---------------- epilogue: running fp32 sums
    if constexpr (kSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
    const int quarter = warp & 3, ew = warp - 12;
    const int ncols = a.N / PARTS;           // a multiple of 16, at most NC
    const int col0 = (ew / 4) * ncols;
    const uint32_t af = smem_u32(&bars.acc_full[0]), ae = smem_u32(&bars.acc_empty[0]);
    uint32_t u_all = 0;
    bool ok = true;
    for (int64_t tile = k.tile; tile < a.tiles && ok; tile += k.step) {
      float acc[NC];
#pragma unroll
      for (int t = 0; t < NC; ++t) acc[t] = 0.f;
      const int64_t row = (tile % a.tiles_m) * 128 + quarter * 32 + lane;
      const int64_t t0 = tile / a.tiles_m * a.N + col0;
      const bool live = row < a.w.mp;
      const float* scale_row = a.w.scale + (live ? grid_row(a.w, 0, row) : 0);
      auto scale_of = [&](int u) {
        if (!live || u >= units) return 0.f;
        return ld_ahead(scale_row + grid_group(a.w, (uint32_t)(k.c0 * 128 + u * (KU * 16))) * 16);
      };
      float s_next = scale_of(0);
      for (int u = 0; u < units; ++u, ++u_all) {
        const float s = s_next;
        s_next = scale_of(u + 1);
        ok = wait_or_abort(af + 8u * (u_all & 1), (u_all >> 1) & 1, &bars.abort, a.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        fence_after_sync();
        const uint32_t ta = tmem + ((uint32_t)(quarter * 32) << 16) + (u_all & 1) * acc_cols + (uint32_t)col0;
        // 32 columns at a time where registers allow: fewer round trips to TMEM
        constexpr int LD = TX == 1 && NC <= 64 ? 32 : 16;
#pragma unroll
        for (int g = 0; g < NC / LD; ++g) {
          if (g * LD < ncols) {
            uint32_t v[LD];
            tmem_ld16(ta + g * LD, *reinterpret_cast<uint32_t(*)[16]>(v));
            if constexpr (LD == 32) tmem_ld16(ta + g * LD + 16, *reinterpret_cast<uint32_t(*)[16]>(v + 16));
            if constexpr (TX > 1) {
              uint32_t c[16];
              tmem_ld16(ta + (uint32_t)a.N + g * 16, c);
              tmem_ld_wait();
#pragma unroll
              for (int t = 0; t < 16; t += 2) add2(v[t], v[t + 1], c[t], c[t + 1]);
            } else {
              tmem_ld_wait();
            }
#pragma unroll
            for (int t = 0; t < LD; t += 2) fma2(acc[g * LD + t], acc[g * LD + t + 1], s, v[t], v[t + 1]);
          }
        }
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(ae + 8u * (u_all & 1));
      }
      if (S > 1) {
        // this block's sums [column][row] into the ring, idle once the last
        // accumulator has been read
        float* part = reinterpret_cast<float*>(dsm + (ring - base_raw));
#pragma unroll
        for (int t = 0; t < NC; ++t)
          if (t < ncols) part[(col0 + t) * 128 + quarter * 32 + lane] = acc[t];
      } else if (ok && row < a.w.m) {
        // lane = output column: the 32 lanes write 32 consecutive elements
        TO* y = static_cast<TO*>(a.y) + t0 * a.w.m + row;
#pragma unroll
        for (int t = 0; t < NC; ++t)
          if (t < ncols && t0 + t < a.T) y[(int64_t)t * a.w.m] = from_float<TO>(acc[t]);
      }
    }
    if constexpr (kSplit) role_end<THREADS, 96>(true, warp);
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
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
  if (S > 1) {
    // each block adds up and writes every S-th column
    float* part = reinterpret_cast<float*>(dsm + (ring - base_raw));
    __syncwarp();
    cluster.sync();
    const int r = threadIdx.x & 127;
    const int64_t row = (k.tile % a.tiles_m) * 128 + r, t0 = k.tile / a.tiles_m * a.N;
    for (int c = rank + S * (threadIdx.x >> 7); c < a.N; c += S * (THREADS / 128)) {
      if (row >= a.w.m || t0 + c >= a.T) continue;
      float v = 0.f;
      for (int q = 0; q < S; ++q) v += cluster.map_shared_rank(part, q)[c * 128 + r];
      static_cast<TO*>(a.y)[(t0 + c) * a.w.m + row] = from_float<TO>(v);
    }
    __syncwarp();
    cluster.sync();   // no block leaves while its sums are read
  }
}

// Blocks per tile: as many as there are SMs without a tile, two chunks each at
// least.
int blocks_per_tile(int64_t tiles, int64_t chunks) {
  int S = 1;
  while (S < 8 && tiles * 2 * S <= sm_count() && chunks >= 4 * S) S *= 2;
  return S;
}

template <typename TO, typename H, int TX, int NC, int EW, int KU>
cudaError_t run_unit(const LinearArgs& a, int N, cudaStream_t s) {
  auto k = linear_fwd_kernel<TO, H, TX, NC, EW, KU>;
  const int64_t K = a.w.n;
  FwdArgs t = {};
  t.w = a.w;
  t.y = a.y;
  t.T = a.T;
  t.tiles_m = (int)((a.w.m + 127) / 128);
  t.tiles = (int64_t)t.tiles_m * ((a.T + N - 1) / N);
  t.chunks = (int)a.w.nc;
  t.N = N;
  const uint32_t stage = TX * (uint32_t)N * 256u;
  t.stages = (int)std::min<uint32_t>(kMaxStages, kRing / stage);
  t.wstages = (TX == 1 ? 2 : 4) * N + 4 * 64 <= 512 ? 4 : 2;
  t.status = async_status_word();
  if (!t.status) return cudaErrorInvalidSymbol;
  // activations: as they are when TMA can read them, else as planes
  const void* x = a.x;
  int64_t ldx = K, rows = a.T;
  t.plane = a.T;
  if (TX != 1 || !aligned_to(a.x, 16) || K % 8 != 0) {
    const int64_t kp = (K + 127) / 128 * 128;
    const cudaError_t e = launch_planes(a.x, a.dtype, a.T, K, kp, a.ws, s);
    if (e != cudaSuccess) return e;
    x = a.ws;
    ldx = kp;
    rows = TX * a.T;
  }
  CUtensorMap map;
  if (!make_map16(&map, x, rows, ldx, N, std::is_same<H, __nv_bfloat16>::value)) return cudaErrorInvalidValue;
  const int S = blocks_per_tile(t.tiles, t.chunks);
  static std::atomic<unsigned long long> done;
  const size_t smem = (size_t)t.stages * stage + kCodes + 1024;
  cudaError_t e = ensure_smem_limit((const void*)k, kRing + kCodes + 1024, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(std::min<int64_t>(t.tiles, S > 1 ? t.tiles : sm_count()) * S));
  cfg.blockDim = dim3(32 * (12 + EW));
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
template <typename TO, typename H, int TX, int NC, int EW>
cudaError_t run_narrow(const LinearArgs& a, int N, cudaStream_t s) {
  return a.w.g % 64 == 0 ? run_unit<TO, H, TX, NC, EW, 4>(a, N, s) : run_unit<TO, H, TX, NC, EW, 2>(a, N, s);
}
bool narrow_groups(const LinearArgs& a) { return a.w.ng > 1 && a.w.g % 128 != 0; }

// Tokens per tile, a multiple of 32: a chunk costs about as much as 500 tokens
// besides its own (measured: 985 cycles at 64 tokens, 1270 at 192).
int tokens_per_tile(const LinearArgs& a, int most) {
  const int64_t tiles_m = (a.w.m + 127) / 128;
  int best = most;
  double cost = 0.0;
  for (int n = most; n >= 32; n -= 32) {
    if (n > a.T + 31 && n > 32) continue;
    const int64_t tiles = tiles_m * ((a.T + n - 1) / n);
    const int S = blocks_per_tile(tiles, a.w.nc);
    const double rounds = S > 1 ? 1.0 : (double)((tiles + sm_count() - 1) / sm_count());
    const double c = rounds * (n + 500) / S;
    if (cost == 0.0 || c < cost) {
      cost = c;
      best = n;
    }
  }
  return best;
}

template <typename TO>
cudaError_t run16(const LinearArgs& a, cudaStream_t s) {
  if (narrow_groups(a)) return run_narrow<TO, TO, 1, 64, 8>(a, tokens_per_tile(a, 128), s);
  return run_unit<TO, TO, 1, 96, 8, 8>(a, tokens_per_tile(a, 192), s);
}

}  // namespace

int64_t linear_fwd_steps(const LinearArgs& a) {
  const int N = tokens_per_tile(a, narrow_groups(a) ? 128 : 192);
  const int64_t tiles = (a.w.m + 127) / 128 * ((a.T + N - 1) / N);
  const int S = blocks_per_tile(tiles, a.w.nc);
  return S > 1 ? (a.w.nc + S - 1) / S : (tiles + sm_count() - 1) / sm_count() * a.w.nc;
}

cudaError_t launch_linear_fwd(const LinearArgs& a, cudaStream_t s) {
  switch (a.dtype) {
    case BAKRON_F32: {
      const int N = (int)std::min<int64_t>(64, (a.T + 31) / 32 * 32);
      if (narrow_groups(a)) return run_narrow<float, __nv_bfloat16, 3, 64, 4>(a, N, s);
      return run_unit<float, __nv_bfloat16, 3, 64, 4, 8>(a, N, s);
    }
    case BAKRON_BF16: return run16<__nv_bfloat16>(a, s);
    default: return run16<__half>(a, s);
  }
}

}  // namespace bakron
