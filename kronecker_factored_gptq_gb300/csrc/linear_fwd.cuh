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
// registers while the tensor core fills others: no rounding of the weights,
// and no long chain of the tensor core's additions, which cut off instead of
// rounding.  fp32 activations are three exact bf16 terms; the products of the two
// small ones have an accumulator of their own.
//
// The same kernel runs bakron_linear_act (its epilogue, see finish()) and bakron_experts, whose
// tiles are tokens of one expert each: a table of the experts' tiles is made from their offsets
// by every block (expert_tiles), so that nothing about them need be known on the host.
//
// One block per SM, which takes output tiles in turn (or, when there are few, a
// part of the columns of one, joined over a cluster through distributed shared memory):
//   warp 0: TMA producer of the activations;
//   warps 1 and 3: issue the tcgen05.mma (M 128, K 16 each), 128-column chunks in turn (warp 1
//     alone where short groups have one set of epilogue warps);
//   warp 2: allocates and frees TMEM;
//   warps 4-11: weights, two groups of four (32 rows each) that take the
//     chunks in turn, codes copied asynchronously kSlots - 1 of their chunks ahead;
//   the rest: epilogue, each 32 TMEM lanes x NC columns in fp32 registers.  Where units are short, two
//   sets of them may take the units in turn and add their sums at the end of a tile (cut_of).
// Activations come by whole chunks, weights pass on by halves of one (32 TMEM columns), so that the
// second half is unpacked while the first is multiplied.  TMEM: an accumulator for each issuer (two of them
// for short groups) of N columns, twice as many for fp32, then four stages of weights, 64 columns each, where
// the 512 columns have room for them, else two.
//
// Measured, in graphs: 2048 tokens of 8192 x 8192 bf16 in 174 us (two weights; 1.58 PFLOP/s, 1.62 at
// 4096 tokens); 48 tokens 22 us, of 14336 x 4096 19; fp32, 1024 tokens of 4096 x 4096 85 us and 2048 of
// 8192 x 8192 507 us (three products: 1.63 PFLOP/s); experts, 4096 rows over 8 of 28672 x 4096 740 to 763 us (1.26
// PFLOP/s: an expert's last tile is mostly not full), 256 rows over 32 of 1408 x 1024 25 us (fp32 26), 1024
// rows over 8 of 4096 x 4096 fp32 110.  A chunk takes
// 1040 cycles at 192 tokens, of which the tensor core works 816 (at cuBLAS's rate 950): with one issuing
// warp, whose waits and instructions follow one another, it took 1270 (206 us), with weights passed on
// by whole chunks 1100.  Few tokens do not make a chunk shorter than about 1000: a warp's instructions follow
// one another, five or six cycles each, the epilogue's of a unit some 100 and the weights' of a chunk
// some 300; twice as many weights warps changed nothing, more instructions in the epilogue (scales
// prefetched into L2, four units ahead, copied to shared memory) made it slower.  Short groups: 2048 tokens
// of 8192 x 8192 298 us in groups of 64 (312 with zero points), 555 in groups of 32; 1024 of 4096 x 4096 82 us in
// groups of 32, 50 in groups of 64, 38 in groups of 128 (fp32: 178, 109, 85).
//
// Every mbarrier wait is bounded (clock64 budget); a block whose wait runs
// out records BAKRON_ERR_TIMEOUT in the device's status word, stops issuing,
// drains its copies and MMAs (bounded again), frees TMEM and returns.
#pragma once

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
  int N;              // tokens per tile, a multiple of 32 (of 16: fp32, short groups, two sets)
  int stages;
  int wstages;        // 4 where TMEM has room, else 2: a power of two
  int log_acc;        // each issuer has 1 << log_acc accumulators
  uint32_t group_mul; // floor(2^31 / (g / 32)) + 1: (32 c) / g = (c group_mul) >> 31 for c, g / 32 <= 2^15
  int* status;
  Epilogue epi;       // kWithAct
  const int* offsets; // kExperts
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

// 16 registers of each lane to 16 TMEM columns of its row.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15, %16};" ::"r"(taddr),
      "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]), "f"(r[9]),
      "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15])
      : "memory");
}

constexpr int kFinish = 16;
// bakron_linear_act's epilogue for a warp's sums, 32 rows (a lane each) x n tokens, that lie in
// TMEM: kFinish tokens at a time in a loop whose code stays small.  (Unrolled over all 96 tokens that a
// thread's registers hold, the code did not fit the instruction cache: 2048 tokens of 8192 x 8192
// 344 us with an activation alone, 500 with residuals, loaded one by one; now 200 and 216, the product
// alone 174: 6000 and 10000 cycles a tile in which the tensor core mostly waits.)  The residuals of the next ones
// are on their way while these are finished.
template <typename TO>
__device__ __forceinline__ void finish(const FwdArgs& a, uint32_t ta, int n, int64_t y0, int64_t row) {
  const bool live = row < a.w.m;
  const float bias = a.epi.bias && live ? __ldg(a.epi.bias + row) : 0.f;
  const TO* res = static_cast<const TO*>(a.epi.residual) + y0;
  TO* pre = static_cast<TO*>(a.epi.pre) + y0;
  TO* y = static_cast<TO*>(a.y) + y0;
  const bool with_res = a.epi.residual != nullptr, with_pre = a.epi.pre != nullptr;
  const int mine = live ? n : 0;
  by_act(a.epi.act, [&](auto A) {
    TO r[kFinish], next[kFinish] = {};
    auto fetch = [&](int g) {
      if (!with_res) return;
#pragma unroll
      for (int t = 0; t < kFinish; ++t) {
        if (g + t < mine) next[t] = __ldg(res);
        res += a.w.m;
      }
    };
    fetch(0);
#pragma unroll 1
    for (int g = 0; g < n; g += kFinish) {
      uint32_t v[kFinish];
      tmem_ld16(ta + (uint32_t)g, v);
#pragma unroll
      for (int t = 0; t < kFinish; ++t) r[t] = next[t];
      fetch(g + kFinish);
      tmem_ld_wait();
      // values first, then the stores: a condition around each would line them up
      TO z[kFinish], o[kFinish];
#pragma unroll
      for (int t = 0; t < kFinish; ++t) {
        const float f = __uint_as_float(v[t]) + bias;
        z[t] = from_float<TO>(f);
        float q = activate<TO, A>(f);
        if (with_res) q += to_float(r[t]);
        o[t] = from_float<TO>(q);
      }
      if (with_pre) {
#pragma unroll
        for (int t = 0; t < kFinish; ++t) {
          if (g + t < mine) *pre = z[t];
          pre += a.w.m;
        }
      }
#pragma unroll
      for (int t = 0; t < kFinish; ++t) {
        if (g + t < mine) *y = o[t];
        y += a.w.m;
      }
    }
  });
}

constexpr int kMaxAcc = 4;                   // accumulators

struct Bars {
  unsigned long long full_b[kMaxStages], empty_b[kMaxStages], full_a[2 * kWStages], empty_a[2 * kWStages];
  unsigned long long acc_full[kMaxAcc], acc_empty[kMaxAcc], turn[2], done;
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
__device__ __forceinline__ void role_end(bool epilogue, int warpgroup = 0) {
  __syncwarp();
  if (epilogue) {
    asm volatile("bar.sync %0, 128;" ::"r"(1 + warpgroup) : "memory");
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
    asm volatile("bar.sync 7, %0;" ::"n"(THREADS) : "memory");
  } else {
    asm volatile("bar.sync 7, %0;" ::"n"(THREADS) : "memory");
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
  }
}

// One chunk of codes at a time: 32 rows (a lane each) x 128 columns.
template <typename H, Product P>
__device__ __forceinline__ void weights(const FwdArgs& a, const Work& k, const Tiles<P, FwdArgs>& tiles, Bars& bars,
                                        uint32_t tmem_a, uint32_t codes, int group, int quarter, int lane) {
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
  // the tile's row block and expert
  int m_ahead = 0, e_ahead = 0;
  if (k.tile < tiles.count()) {
    const Place p = tiles.at(k.tile);
    m_ahead = p.m;
    e_ahead = p.e;
  }
  int m_now = m_ahead, e_now = e_ahead;
  auto settle = [&](int64_t& tile, int& c, int& m, int& e) {
    if (c < k.c1) return;
    while (c >= k.c1 && tile < tiles.count()) {
      c -= n;
      tile += k.step;
    }
    if (P == kExperts && tile >= tiles.count()) return;
    const Place p = tiles.at(tile);
    m = p.m;
    e = p.e;
  };
  settle(tile_ahead, c_ahead, m_ahead, e_ahead);
  settle(tile_now, c_now, m_now, e_now);
  uint32_t fill = 0, read = 0;
  auto copy = [&]() {
    if (tile_ahead < tiles.count()) {
      const int64_t block = (int64_t)m_ahead * 16 + quarter * 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool live = (block + i) * 8 < w.mp;      // zeros below the last row
        const uint8_t* src =
            w.codes + ((e_ahead * (w.mp / 8) + (live ? block + i : 0)) * w.nc + c_ahead) * kBlockBytes + lane * 16;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(copy_at + fill + (uint32_t)i * 512u), "l"(src),
                     "r"(live ? 16u : 0u)
                     : "memory");
      }
      c_ahead += 2;
      settle(tile_ahead, c_ahead, m_ahead, e_ahead);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    fill = fill + kSlotBytes == kSlots * kSlotBytes ? 0 : fill + kSlotBytes;
  };
  // the row's zero points of a chunk, a byte per 32 columns
  auto zeros = [&](int64_t tile, int c, int m, int e) -> uint32_t {
    if (w.zero == nullptr || tile >= tiles.count()) return 0u;
    const int64_t row = (int64_t)m * 128 + quarter * 32 + lane;
    if (row >= w.mp) return 0u;
    const uint8_t* p = w.zero + grid_row(w, e, row);
    if (!narrow) return ld_ahead(p + grid_group(w, (uint32_t)c * 128) * 16) * 0x01010101u;
    uint32_t z = 0;
#pragma unroll
    for (int s = 0; s < 4; ++s) z |= ld_ahead(p + grid_group(w, (uint32_t)c * 128 + 32 * s) * 16) << (8 * s);
    return z;
  };
#pragma unroll
  for (int p = 0; p < kSlots - 1; ++p) copy();
  uint32_t z = zeros(tile_now, c_now, m_now, e_now);
  uint32_t seq = (uint32_t)group;      // chunk of the block
  const uint32_t last_stage = (uint32_t)a.wstages - 1;
  const int log_stages = a.wstages == 4 ? 2 : 1;
  while (tile_now < tiles.count()) {
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
    settle(tile_now, c_now, m_now, e_now);
    z = zeros(tile_now, c_now, m_now, e_now);
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
      if (!__all_sync(0xffffffffu, wait_or_abort(empty + 8u * (2 * ws + h), ((seq >> log_stages) & 1) ^ 1u, &bars.abort, a.status)))
        goto out;
      fence_after_sync();
      tmem_st32(tmem_a + ((uint32_t)(quarter * 32) << 16) + ws * 64u + (uint32_t)(h * 32), v);
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(full + 8u * (2 * ws + h));
    }
    seq += 2;
  }
out:
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Barriers of the epilogue's 256 threads; the second returns whether all of them say so.
__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 8, 256;" ::: "memory"); }
__device__ __forceinline__ bool epilogue_all(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.and.pred q, 8, 256, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(all)
      : "r"((uint32_t)ok)
      : "memory");
  return all != 0;
}

// Warps that issue the products.  Units shorter than a chunk that one set of epilogue warps takes need
// two accumulators that follow each other within a chunk: one issuer has both.
constexpr int issuers(int KU, int SETS) { return SETS == 1 && KU < 8 ? 1 : 2; }

// TX: 16-bit terms of the activations; NC: columns per epilogue warp; EW:
// epilogue warps; KU: accumulation unit in MMA steps of 16 (2, 4 or 8); SETS: sets of
// epilogue warps that take the units in turn.
template <typename TO, typename H, int TX, int NC, int EW, int KU, int SETS, Product P>
__global__ void __launch_bounds__(32 * (12 + EW), 1)
    linear_fwd_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ FwdArgs a) {
  constexpr int THREADS = 32 * (12 + EW);
  constexpr int PARTS = EW / 4 / SETS;       // column parts of the epilogue
  constexpr int ISSUERS = issuers(KU, SETS);
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
    for (int s = 0; s < 2 * kWStages; ++s) {         // halves
      mbar_init(smem_u32(&bars.full_a[s]), 4);       // the warps of a group
      mbar_init(smem_u32(&bars.empty_a[s]), 1);
    }
    for (int b = 0; b < kMaxAcc; ++b) {
      mbar_init(smem_u32(&bars.acc_full[b]), 1);
      mbar_init(smem_u32(&bars.acc_empty[b]), EW / SETS);
    }
    for (int b = 0; b < 2; ++b) mbar_init(smem_u32(&bars.turn[b]), 1);
    mbar_init(smem_u32(&bars.done), ISSUERS);
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
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars.tmem, 0), tmem_a = tmem + ((uint32_t)ISSUERS << a.log_acc) * acc_cols;
  grid_dep_wait();
  grid_dep_launch();
  Tiles<P, FwdArgs> tiles = {a, 0, nullptr, nullptr, 0};
  if constexpr (P == kExperts) {
    __shared__ int sums[2][kTileThreads / 32];
    int* table = reinterpret_cast<int*>(dsm + (ring - base_raw) + (uint32_t)a.stages * stage_bytes + kCodes);
    tiles.E = (int)a.w.count;
    tiles.bounds = table;
    tiles.first = table + tiles.E + 1;
    tiles.own = (int64_t)a.tiles_m * expert_tiles(a.offsets, tiles.E, (int)a.T, a.N, table, table + tiles.E + 1, sums);
  }

  if (warp < 4) {
    if constexpr (kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0) {
      // ---------------- activations
      const uint32_t full = smem_u32(bars.full_b), empty = smem_u32(bars.empty_b);
      int64_t issued = 0;
      Ring rg;
      bool go = true;
      for (int64_t tile = k.tile; tile < tiles.count() && go; tile += k.step) {
        const int64_t t0 = tiles.at(tile).t0;
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
    } else if (warp == 1 || (ISSUERS == 2 && warp == 3)) {
      // ---------------- MMA issuers, which take the chunks in turn: a warp waits together, one lane
      // issues.  Their own instructions, not the tensor core, bounded a single issuer: what it
      // waited for and issued one after the other.  Each has its accumulators and its stages of
      // weights; the stages of activations are waited for in the order of the chunks (`turn`), so that
      // a use of a stage is never mistaken for the one before.
      const int me = ISSUERS == 2 ? warp >> 1 : 0;
      const uint32_t idesc = idesc_f16<H>(a.N);
      const uint64_t desc_b0 = desc_sw128(ring);
      const uint32_t stage16 = stage_bytes >> 4, half16 = half_bytes >> 4, plane16 = plane_b >> 4;
      const uint32_t fb = smem_u32(bars.full_b), eb = smem_u32(bars.empty_b);
      const uint32_t fa = smem_u32(bars.full_a), ea = smem_u32(bars.empty_a);
      const uint32_t my_turn = smem_u32(&bars.turn[me]), other_turn = smem_u32(&bars.turn[me ^ 1]);
      const uint32_t af = smem_u32(&bars.acc_full[me << a.log_acc]), ae = smem_u32(&bars.acc_empty[me << a.log_acc]);
      const uint32_t tmem_me = tmem + ((uint32_t)me << a.log_acc) * acc_cols;
      uint32_t u = 0;                         // units begun
      const uint32_t last_stage = (uint32_t)a.wstages - 1, last_acc = (1u << a.log_acc) - 1;
      const int log_stages = a.wstages == 4 ? 2 : 1;
      const int64_t chunks = k.tile < tiles.count() ? ((tiles.count() - 1 - k.tile) / k.step + 1) * (k.c1 - k.c0) : 0;
      uint32_t turns = 0;
      Ring rg;
      rg.advance(me, a.stages);
      for (int64_t seq = me; seq < chunks; seq += ISSUERS) {
        const uint32_t ws = (uint32_t)seq & last_stage;
        bool go = ISSUERS == 1 || seq == 0 || wait_or_abort(my_turn, (turns + (uint32_t)me + 1) & 1, &bars.abort, a.status);
        ++turns;
        go = go && wait_or_abort(fb + 8u * (uint32_t)rg.s, rg.parity, &bars.abort, a.status);
        go = __all_sync(0xffffffffu, go);
        if (!go) break;
        if (ISSUERS == 2 && lane == 0) mbar_arrive(other_turn);
        const uint64_t db = desc_b0 + (uint32_t)rg.s * stage16;
        const uint32_t ta = tmem_a + ws * 64u;
        // halves of the chunk, each as soon as its weights are there; J steps at a time
        constexpr int J = KU < 4 ? KU : 4;
#pragma unroll
        for (int j0 = 0; j0 < 8; j0 += J) {
          const int h = j0 / 4;
          const uint32_t buf = u & last_acc, use = u >> a.log_acc;
          if (j0 % 4 == 0)
            go = go && wait_or_abort(fa + 8u * (2 * ws + h), (uint32_t)(seq >> log_stages) & 1, &bars.abort, a.status);
          // the accumulator: its previous unit has been read
          if (j0 % KU == 0) go = go && (use == 0 || wait_or_abort(ae + 8u * buf, (use & 1) ^ 1u, &bars.abort, a.status));
          go = __all_sync(0xffffffffu, go);
          if (!go) break;
          fence_after_sync();
          if (elect_one()) {
            const uint32_t d = tmem_me + buf * acc_cols;
#pragma unroll
            for (int j = j0; j < j0 + J; ++j)
#pragma unroll
              for (int q = 0; q < TX; ++q)
                mma_f16_ts(q == 0 ? d : d + (uint32_t)a.N, ta + j * 8,
                           db + ((j / 4) * half16 + q * plane16 + (j % 4) * 2), idesc, j % KU == 0 && q <= 1 ? 0u : 1u);
            if ((j0 + J) % KU == 0) mma_commit(af + 8u * buf);
            if ((j0 + J) % 4 == 0) mma_commit(ea + 8u * (2 * ws + h));
            if (j0 + J == 8) mma_commit(eb + 8u * (uint32_t)rg.s);
          }
          __syncwarp();
          if ((j0 + J) % KU == 0) ++u;
        }
        if (!go) break;
        rg.advance(ISSUERS, a.stages);
      }
      if (elect_one()) mma_commit(smem_u32(&bars.done));
      __syncwarp();
    }
    if constexpr (kSplit) role_end<THREADS, 96>(false);
  } else if (warp < 12) {
    // ---------------- weights
    if constexpr (kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const uint32_t codes = ring + (uint32_t)a.stages * stage_bytes + (uint32_t)(warp - 4) * (kSlots * kSlotBytes);
    weights<H, P>(a, k, tiles, bars, tmem_a, codes, (warp - 4) >> 2, warp & 3, lane);
    if constexpr (kSplit) role_end<THREADS, 96>(false);
  } else {
    // ---------------- epilogue: running fp32 sums
    if constexpr (kSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
    const int quarter = warp & 3, ew = warp - 12;
    const int ncols = a.N / PARTS;           // a multiple of 16, at most NC
    const int set = SETS == 2 ? ew / 4 : 0, col0 = SETS == 2 ? 0 : (ew / 4) * ncols;
    const uint32_t af = smem_u32(&bars.acc_full[0]), ae = smem_u32(&bars.acc_empty[0]);
    // A warp's instructions follow one another, several cycles each, and the time of a unit is their
    // number: so where an accumulator is and which of its uses follows from the count alone.
    uint32_t count = 0;
    const uint32_t tmem_ep = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)set * acc_cols + (uint32_t)col0;
    const uint32_t af_ep = af + 8u * (uint32_t)set, ae_ep = ae + 8u * (uint32_t)set;
    static_assert(SETS == 1 || KU < 8);
    bool ok = true;
    for (int64_t tile = k.tile; tile < tiles.count() && ok; tile += k.step) {
      const Place at = tiles.at(tile);
      float acc[NC];
#pragma unroll
      for (int t = 0; t < NC; ++t) acc[t] = 0.f;
      const int64_t row = (int64_t)at.m * 128 + quarter * 32 + lane;
      const int64_t t0 = at.t0 + col0;
      const bool live = row < a.w.mp;
      const float* scale_row = a.w.scale + (live ? grid_row(a.w, at.e, row) : 0);
      // (past the last unit the last group's; rows past the matrix take another row's)
      auto scale_of = [&](int u) {
        const uint32_t col32 = (uint32_t)(k.c0 * 4 + u * (KU / 2));
        return ld_ahead(scale_row + min(__umulhi(2 * col32, a.group_mul), (uint32_t)a.w.ng - 1) * 16);
      };
      if (P == kWithAct && S == 1 && a.epi.residual) {
        // the residuals of the tile on their way into L2: a lane per token, 32 rows' bytes
        const int64_t first = row - lane, last = min(first + 31, a.w.m - 1);
        for (int t = lane; first < a.w.m && t < ncols && t0 + t < at.end; t += 32) {
          const TO* p = static_cast<const TO*>(a.epi.residual) + (t0 + t) * a.w.m;
          for (int64_t c = first; c <= last; c += 32 / sizeof(TO))
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p + c));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(p + last));
        }
      }
      uint32_t slot = 0;           // of the accumulator at hand
      auto unit = [&](int u, float s) {
        // two sets: issuer 0's and 1's chunks in turn, a set's units of a chunk one after the other; one
        // set: the two accumulators in turn
        constexpr bool kPairs = SETS == 2 && KU == 2;
        const uint32_t turn = kPairs ? count >> 1 : count, use = kPairs ? count : count >> 1;
        slot = SETS * (turn & 1);
        ++count;
        ok = wait_or_abort(af_ep + 8u * slot, use & 1, &bars.abort, a.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        fence_after_sync();
        const uint32_t ta = tmem_ep + slot * acc_cols;
        // 32 columns at a time where registers allow: fewer round trips to TMEM
        constexpr int LD = TX == 1 ? 32 : 16;
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
        // (the accumulator that was read last may still be needed)
        if ((SETS == 1 && (P != kWithAct || S > 1)) || u < units - SETS) {
          fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(ae_ep + 8u * slot);
        }
      };
      // this set's units: every SETS-th
      float s0 = scale_of(set);
      if constexpr (SETS == 1 && !(TX > 1 && KU == 2)) {
        // scales two units ahead, each in a register of its own (moved, it would be waited for;
        // for two sets, and for fp32 units of 32 columns, the longer code costs more than it saves)
        float s1 = scale_of(1);
        for (int u = 0; u < units && ok; u += 2) {
          unit(u, s0);
          s0 = scale_of(u + 2);
          if (u + 1 >= units || !ok) break;
          unit(u + 1, s1);
          s1 = scale_of(u + 3);
        }
      } else {
        for (int u = set; u < units && ok; u += SETS) {
          const float s = s0;
          s0 = scale_of(u + SETS);
          unit(u, s);
        }
      }
      const uint32_t ta = tmem_ep + slot * acc_cols;
      const int n = (int)max((int64_t)0, min((int64_t)ncols, at.end - t0));      // tokens of this warp
      if constexpr (SETS == 2) {
        // the second set's sums pass to the first through the accumulator that it read last
        if (set == 1 && ok) {
#pragma unroll
          for (int g = 0; g < NC; g += 16)
            if (g < ncols) tmem_st16(ta + g, acc + g);
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          fence_before_sync();
        }
        ok = epilogue_all(ok);
        if (!ok) break;
        fence_after_sync();
        if (set == 0) {
#pragma unroll
          for (int g = 0; g < NC; g += 16) {
            if (g < ncols) {
              uint32_t v[16];
              tmem_ld16(ta + acc_cols + g, v);
              tmem_ld_wait();
#pragma unroll
              for (int t = 0; t < 16; ++t) acc[g + t] += __uint_as_float(v[t]);
            }
          }
        }
      }
      if (S > 1) {
        // this block's sums [column][row] into the ring, idle once the last
        // accumulator has been read
        float* part = reinterpret_cast<float*>(dsm + (ring - base_raw));
        if (set == 0) {
#pragma unroll
          for (int t = 0; t < NC; ++t)
            if (t < ncols) part[(col0 + t) * 128 + quarter * 32 + lane] = acc[t];
        }
      } else if (P == kWithAct) {
        if (!ok) break;
        // the sums pass through the accumulator that was read last
        if (set == 0) {
#pragma unroll
          for (int g = 0; g < NC; g += 16)
            if (g < ncols) tmem_st16(ta + g, acc + g);
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        }
        const int64_t y0 = t0 * a.w.m + row;
        if constexpr (SETS == 2) {
          // each set finishes half of the tokens
          fence_before_sync();
          epilogue_sync();
          fence_after_sync();
          const int half = min(n, (ncols / 2 + kFinish - 1) / kFinish * kFinish);
          if (set == 0) finish<TO>(a, ta, half, y0, row);
          else finish<TO>(a, ta - acc_cols + half, n - half, y0 + (int64_t)half * a.w.m, row);
        } else {
          finish<TO>(a, ta, n, y0, row);
        }
      } else if (ok && set == 0 && row < a.w.m) {
        // lane = output column: the 32 lanes write 32 consecutive elements
        TO* y = static_cast<TO*>(a.y) + t0 * a.w.m + row;
#pragma unroll
        for (int t = 0; t < NC; ++t)
          if (t < n) y[(int64_t)t * a.w.m] = from_float<TO>(acc[t]);
      }
      if (SETS == 2 || (P == kWithAct && S == 1)) {
        fence_before_sync();
        __syncwarp();
        if constexpr (SETS == 2) epilogue_sync();       // both sets have read both accumulators
        if (lane == 0) mbar_arrive(ae_ep + 8u * slot);
      }
    }
    if constexpr (kSplit) role_end<THREADS, 96>(true, ew >> 2);
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
    Place at = {};
    if (k.tile < tiles.count()) at = tiles.at(k.tile);
    const int64_t row = (int64_t)at.m * 128 + r;
    for (int c = rank + S * (threadIdx.x >> 7); c < a.N; c += S * (THREADS / 128)) {
      if (row >= a.w.m || at.t0 + c >= at.end) continue;
      float v = 0.f;
      for (int q = 0; q < S; ++q) v += cluster.map_shared_rank(part, q)[c * 128 + r];
      const int64_t i = (at.t0 + c) * a.w.m + row;
      put<TO, P == kWithAct>(static_cast<TO*>(a.y) + i, a.epi, i, row, v);
    }
    __syncwarp();
    cluster.sync();   // no block leaves while its sums are read
  }
}

// Blocks per tile: as many as there are SMs without a tile, two chunks each at least; eight
// only where as many clusters of eight fit at once (128 x 16384 bf16, 96 tokens, one tile 14 us, in clusters
// of four 21; 1792 x 8192, 32 tokens, 14 tiles 10 and 12.5; 2048 x 8192, 16 of which one waits, 22 and 14).
int blocks_per_tile(int64_t tiles, int64_t chunks) {
  int S = 1;
  while (S < 4 && tiles * 2 * S <= sm_count() && chunks >= 4 * S) S *= 2;
  if (S == 4 && chunks >= 16 && tiles <= linear_fwd_eights()) S = 8;
  return S;
}

template <typename TO, typename H, int TX, int NC, int EW, int KU, int SETS, Product P>
cudaError_t run_unit(const LinearArgs& a, int N, cudaStream_t s) {
  auto k = linear_fwd_kernel<TO, H, TX, NC, EW, KU, SETS, P>;
  const uint32_t table = P == kExperts ? 8u * (uint32_t)(a.w.count + 1) : 0u;    // the experts'
  const int64_t K = a.w.n;
  FwdArgs t = {};
  t.w = a.w;
  t.y = a.y;
  t.T = a.T;
  t.tiles_m = (int)((a.w.m + 127) / 128);
  t.tiles = t.tiles_m * token_tiles(a, N);
  t.chunks = (int)a.w.nc;
  t.N = N;
  const uint32_t stage = TX * (uint32_t)N * 256u;
  t.stages = (int)std::min<uint32_t>(kMaxStages, (kRing - table) / stage);
  // Short groups change accumulators within a chunk: two for each issuer.
  t.log_acc = KU < 8 ? 1 : 0;
  t.group_mul = (uint32_t)((uint64_t(1) << 31) / (uint64_t)(a.w.g / 32) + 1);
  t.wstages = (issuers(KU, SETS) << t.log_acc) * (TX == 1 ? 1 : 2) * N + 4 * 64 <= 512 ? 4 : 2;
  t.epi = a.epi;
  t.offsets = a.offsets;
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
  const size_t smem = (size_t)t.stages * stage + kCodes + 1024 + table;
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

bool narrow_groups(const LinearArgs& a) { return a.w.ng > 1 && a.w.g % 128 != 0; }

// How a product is cut: tokens per tile, and the sets of epilogue warps.
struct Cut {
  int N, sets;
};

// The cut that takes the least time: rounds of tiles times a tile's chunks.  A chunk costs about as much as
// 500 tokens besides its own.  Short groups: a third of a token each besides a fixed cost, and one set of epilogue
// warps more than two.  But one set leaves TMEM for tiles of 128 tokens (fp32: 64) where two end at 96
// (48), and ends a tile sooner: it is faster where it saves a round, lets more blocks share a tile, or a tile
// is short.  Groups of 64 with zero points, two sets and one: 2048 tokens of 8192 x 8192 412 and 312 us, 65
// 29.7 and 30.1, 512 of 4096 x 4096 45 and 26.5, 128 of 1024 x 1024 8.1 and 6.9; fp32, 1024 of 4096 x 4096 108 and 124.
Cut cut_of(const LinearArgs& a) {
  const bool f32 = a.dtype == BAKRON_F32, narrow = narrow_groups(a);
  const int64_t tiles_m = (a.w.m + 127) / 128;
  Cut best = {};
  double cost = 0.0;
  for (int sets = narrow ? 2 : 1; sets >= 1; --sets) {
    const int most = !narrow ? (f32 ? 64 : 192) : sets == 2 ? (f32 ? 48 : 96) : (f32 ? 64 : 128);
    const int step = f32 && sets == 2 ? 16 : 32;
    for (int n = most; n >= step; n -= step) {
      if (n > a.T + step - 1 && n > step) continue;
      const int64_t tiles = tiles_m * likely_tiles(a, n);
      const int S = blocks_per_tile(tiles_m * token_tiles(a, n), a.w.nc);
      const double rounds = S > 1 ? 1.0 : (double)((tiles + sm_count() - 1) / sm_count());
      double c;
      if (!narrow) c = rounds * (n + 500) / S;
      else if (sets == 2) c = rounds * ((double)((a.w.nc + S - 1) / S) * (n + 333) + (f32 ? 0 : 333));
      else c = rounds * (double)((a.w.nc + S - 1) / S) * (n + 333) * (f32 ? 1.2 : 1.08);
      if (best.N == 0 || c < cost) {
        cost = c;
        best = {n, sets};
      }
    }
  }
  return best;
}

// A unit ends where a group does: 128, 64 or 32 columns.
template <typename TO, typename H, int TX, Product P>
cudaError_t run(const LinearArgs& a, cudaStream_t s) {
  const Cut c = cut_of(a);
  constexpr int EW = TX == 1 ? 8 : 4;        // epilogue warps of one set
  if (!narrow_groups(a)) return run_unit<TO, H, TX, TX == 1 ? 96 : 64, EW, 8, 1, P>(a, c.N, s);
  const bool half = a.w.g % 64 == 0;
  if (c.sets == 1)
    return half ? run_unit<TO, H, TX, 64, EW, 4, 1, P>(a, c.N, s) : run_unit<TO, H, TX, 64, EW, 2, 1, P>(a, c.N, s);
  constexpr int NC = TX == 1 ? 96 : 48;
  return half ? run_unit<TO, H, TX, NC, 8, 4, 2, P>(a, c.N, s) : run_unit<TO, H, TX, NC, 8, 2, 2, P>(a, c.N, s);
}

template <Product P>
cudaError_t forward(const LinearArgs& a, cudaStream_t s) {
  switch (a.dtype) {
    case BAKRON_F32: return run<float, __nv_bfloat16, 3, P>(a, s);     // three terms
    case BAKRON_BF16: return run<__nv_bfloat16, __nv_bfloat16, 1, P>(a, s);
    default: return run<__half, __half, 1, P>(a, s);
  }
}

}  // namespace
}  // namespace bakron
