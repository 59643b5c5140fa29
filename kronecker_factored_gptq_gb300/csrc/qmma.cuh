// Products of packed 4-bit rows with a few columns of activations on the
// warp-level matrix instructions (m16n8k16): the device code shared by the
// few-token linear layer and the mixture-of-experts layer.
//
// These products are bound by the weights' bytes: a 16 x 128 block of codes
// is 1 KB and meets at most a few dozen tokens.  What matters is that enough
// of them are in flight and that few instructions stand between memory and the
// matrix instructions: asynchronous copies bring whole blocks (8 rows x 128
// columns) to shared memory several chunks ahead, and a thread's 16 bytes of
// them are already the A fragments of 8 matrix instructions (packed.cuh).  The k slots
// of an instruction are any 16 columns as long as both operands agree: slots
// (2 t, 2 t + 1) and (2 t + 8, 2 t + 9) of thread t are four consecutive
// columns, and the thread's eight columns of a step are one 16-byte read of
// the activations.
//
// A is the exact integer u - z; the group's sum comes out of the tensor core
// in fp32 (at most 128 products, so no long chain of its additions) and is
// scaled and added to the running sum with fp32 FMAs.  fp32 activations are
// three bf16 terms whose sum is exact (split3); the products of the two small
// ones have a group sum of their own (chunk_product).
#pragma once

#include "packed.cuh"

namespace bakron {
namespace qm {

// c = A B + c, or c = A B when fresh (a constant at each use).
template <typename H>
__device__ __forceinline__ void mma16816(float (&c)[4], bool fresh, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], bool fresh, uint32_t a0, uint32_t a1,
                                                        uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(fresh ? 0.f : c[0]), "f"(fresh ? 0.f : c[1]),
        "f"(fresh ? 0.f : c[2]), "f"(fresh ? 0.f : c[3]));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], bool fresh, uint32_t a0, uint32_t a1,
                                                        uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(fresh ? 0.f : c[0]), "f"(fresh ? 0.f : c[1]),
        "f"(fresh ? 0.f : c[2]), "f"(fresh ? 0.f : c[3]));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

// What one 128-column chunk of a 16-row tile needs, per thread: rows lane / 4
// and lane / 4 + 8.  NS scales per row: 1 when the group is a multiple of 128
// columns, else one per 32 columns.
template <int NS>
struct Chunk16 {
  uint4 w[2];
  float s[2][NS];
  uint32_t z[2][NS];
};

// A thread's part of RT 16-row tiles: the codes of its rows (at its 16 bytes of
// the first chunk), their zero points, and the scale of the one row it fetches
// for the warp (row lane of the 16 RT rows).
template <int RT>
struct TileRef {
  const uint8_t* codes[RT][2];
  const uint8_t* zero[RT][2];
  const float* scale;
};

// Tile r holds rows row0[r] .. + 15 of matrix e; rows past the padding repeat
// its last row (their products are dropped by the caller).
template <int RT>
__device__ __forceinline__ void tile_ref(TileRef<RT>& t, const PackedView& w, int64_t e,
                                         const int64_t (&row0)[RT], int lane) {
#pragma unroll
  for (int r = 0; r < RT; ++r) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t row = min(row0[r] + (lane >> 2) + 8 * i, w.mp - 1);
      t.codes[r][i] = w.codes + (e * (w.mp / 8) + row / 8) * w.nc * kBlockBytes + (row & 7) * 64 + (lane & 3) * 16;
      t.zero[r][i] = w.zero ? w.zero + grid_row(w, e, row) : nullptr;
    }
  }
  const int mine = RT == 1 ? 0 : lane >> 4;
  t.scale = w.scale + grid_row(w, e, min(row0[mine] + (lane & 15), w.mp - 1));
}

// Chunks c and c + 1 into L2, ahead of the wait for the kernel before: only a
// hint, so it may run while that kernel still writes.
template <int RT>
__device__ __forceinline__ void prefetch_codes(const TileRef<RT>& t, int c, int lane) {
  // a lane in eight per row block and 128 bytes of its two chunks (codes[r][i]
  // is at row lane / 4, 16 (lane % 4) bytes: 512 bytes per row block and chunk)
  if (lane % 8 == 0) {
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(t.codes[r][i] + (int64_t)(c + h) * kBlockBytes));
  }
}

// A warp's codes in flight: D slots in shared memory of two chunks each (two, so
// that the addresses and counters of a step are paid once per 256 columns),
// filled by asynchronous copies D - 1 slots ahead.  A thread copies the 16 bytes
// of codes that it reads itself, so they need no synchronisation; only the
// scales, one row per thread, pass between the lanes of the warp.
template <int RT, int NS, int D>
struct Pipe {
  static constexpr uint32_t kHalf = RT * 2 * 512 + NS * 128;   // one chunk
  static constexpr uint32_t kSlot = 2 * kHalf;
  static constexpr uint32_t kBytes = D * kSlot;                // per warp
  uint32_t base;                                               // of the warp
  uint32_t fill = 0, read = 0;                                 // byte offsets of slots

  static __device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  }
  static __device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
  }
  // Start chunks c .. c + n - 1 (n 0, 1 or 2) of the tiles; n 0 keeps the count.
  __device__ __forceinline__ void issue(const PackedView& w, const TileRef<RT>& t, int c, int n, int lane) {
    const uint32_t slot = base + fill;
    const int64_t at = (int64_t)c * kBlockBytes;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h < n) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            copy16(slot + h * kHalf + (uint32_t)((r * 2 + i) * 512 + lane * 16), t.codes[r][i] + at + h * kBlockBytes);
        if (lane < 16 * RT) {
#pragma unroll
          for (int s = 0; s < NS; ++s)
            copy4(slot + h * kHalf + RT * 1024 + (uint32_t)(s * 128 + lane * 4),
                  t.scale + grid_group(w, (uint32_t)((c + h) * 128 + 32 * s)) * 16);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    fill = fill + kSlot == kBytes ? 0 : fill + kSlot;
  }
  // Wait for the oldest slot.
  __device__ __forceinline__ void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
    __syncwarp();
  }
  // Its chunk h (0 or 1).
  __device__ __forceinline__ void take(Chunk16<NS> (&f)[RT], int h, int lane) const {
    const uint32_t slot = base + read + h * kHalf;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f[r].w[i] = lds128(slot + (uint32_t)((r * 2 + i) * 512 + lane * 16));
#pragma unroll
        for (int s = 0; s < NS; ++s)
          asm volatile("ld.shared.f32 %0, [%1];"
                       : "=f"(f[r].s[i][s])
                       : "r"(slot + RT * 1024 + (uint32_t)(s * 128 + (r * 16 + i * 8 + (lane >> 2)) * 4)));
      }
  }
  // The slot may be filled again.
  __device__ __forceinline__ void release() {
    read = read + kSlot == kBytes ? 0 : read + kSlot;
    __syncwarp();     // its scales have been read by every lane
  }
};

// Zero points of chunk c, where the grid has them.
template <int RT, int NS>
__device__ __forceinline__ void load_zeros(uint32_t (&z)[RT][2][NS], const PackedView& w, const TileRef<RT>& t,
                                           int64_t c) {
  if (w.zero == nullptr) return;
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const uint32_t g = grid_group(w, (uint32_t)(c * 128 + 32 * s)) * 16;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int i = 0; i < 2; ++i) z[r][i][s] = ld_ahead(t.zero[r][i] + g);
  }
}
template <int RT, int NS>
__device__ __forceinline__ void set_zeros(Chunk16<NS> (&f)[RT], const uint32_t (&z)[RT][2][NS]) {
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int s = 0; s < NS; ++s) f[r].z[i][s] = z[r][i][s];
}

// tot[r][j] += products of the chunk of row tile r with column tile j.  fetch(j, q, s): this thread's 8 columns 32 s + 8 t .. of
// term q of its activation row in column tile j.  A warp's instructions, not the
// matrix pipe, are what a chunk costs, so two row tiles share a fetch where they can.
// Three terms are fp32 activations: the matrix instructions cut their sums off instead
// of rounding, so the two small terms have a sum of their own and the large one
// is cut off a third as often.
template <typename H, int TERMS, int RT, int NT, int NS, typename Fetch>
__device__ __forceinline__ void chunk_product(float (&tot)[RT][NT][4], const Chunk16<NS> (&f)[RT],
                                              bool has_zero, int zu, Fetch fetch) {
  constexpr bool kApart = TERMS == 3;
  float acc[RT][NT][4], low[kApart ? RT : 1][kApart ? NT : 1][4];
  uint32_t off[RT][2];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    uint32_t a[RT][4], b[RT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      if (s < NS) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          off[r][i] = Half2<H>::pair(Half2<H>::kBase + (float)(has_zero ? (int)f[r].z[i][s] : zu));
      }
      const uint4 w0 = f[r].w[0], w1 = f[r].w[1];
      unpack_word<H>(s == 0 ? w0.x : s == 1 ? w0.y : s == 2 ? w0.z : w0.w, off[r][0], a[r]);
      unpack_word<H>(s == 0 ? w1.x : s == 1 ? w1.y : s == 2 ? w1.z : w1.w, off[r][1], b[r]);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int q = 0; q < TERMS; ++q) {
        const uint4 x = fetch(j, q, s);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          float(&to)[4] = kApart && q > 0 ? low[kApart ? r : 0][kApart ? j : 0] : acc[r][j];
          const bool first = q <= (kApart ? 1 : 0) && (s == 0 || NS == 4);
          mma16816<H>(to, first, a[r][0], b[r][0], a[r][1], b[r][1], x.x, x.y);
          mma16816<H>(to, false, a[r][2], b[r][2], a[r][3], b[r][3], x.z, x.w);
        }
      }
    }
    if (NS == 4 || s == 3) {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float s0 = f[r].s[0][NS == 4 ? s : 0], s1 = f[r].s[1][NS == 4 ? s : 0];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if constexpr (kApart) {
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][j][i] += low[r][j][i];
          }
          tot[r][j][0] = fmaf(s0, acc[r][j][0], tot[r][j][0]);
          tot[r][j][1] = fmaf(s0, acc[r][j][1], tot[r][j][1]);
          tot[r][j][2] = fmaf(s1, acc[r][j][2], tot[r][j][2]);
          tot[r][j][3] = fmaf(s1, acc[r][j][3], tot[r][j][3]);
        }
      }
    }
  }
}

// Bytes between two columns' rows in shared memory: an odd multiple of 64, so
// that the 16-byte reads of two neighbouring columns fall on different banks.
__host__ __device__ __forceinline__ uint32_t x_pitch(int chunks) { return (uint32_t)chunks * 256u + 64u; }

// Stage `rows` rows of x (row r at x + idx(r) * ld), columns [k0, k0 + 128
// chunks) with zeros past n, as TERMS planes of 16-bit values.  All threads
// of the block take part; the caller synchronises.
template <typename TX, int TERMS, typename Idx>
__device__ __forceinline__ void stage_x(uint8_t* xs, uint32_t xplane, uint32_t xpitch, const TX* x,
                                        int64_t ld, int rows, Idx idx, int64_t k0, int chunks,
                                        int64_t n, bool vec_ok) {
  const int per = chunks * 16;     // 8-column pieces of a row
  for (int i = threadIdx.x; i < rows * per; i += blockDim.x) {
    const int r = i / per, p = i - r * per;
    const int64_t c = k0 + 8 * p;
    const TX* src = x + idx(r) * ld + c;
    uint8_t* dst = xs + (uint32_t)r * xpitch + (uint32_t)p * 16;
    if constexpr (sizeof(TX) == 2) {
      uint4 v;
      if (vec_ok && c + 8 <= n) {
        v = *reinterpret_cast<const uint4*>(src);
      } else {
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          h[e] = c + e < n ? (uint32_t) * reinterpret_cast<const uint16_t*>(src + e) : 0u;
        v = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
      }
      if constexpr (TERMS == 1) *reinterpret_cast<uint4*>(dst) = v;
    } else {
      float f[8];
      if (vec_ok && c + 8 <= n) {
        const float4 a = *reinterpret_cast<const float4*>(src);
        const float4 b = *reinterpret_cast<const float4*>(src + 4);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = c + e < n ? to_float(src[e]) : 0.f;
      }
      uint32_t h[3][4];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float t[3];
        split3(f[e], t[0], t[1], t[2]);
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          const uint32_t b = bf16_bits(t[q]);
          h[q][e >> 1] = (e & 1) ? (h[q][e >> 1] | b << 16) : b;
        }
      }
#pragma unroll
      for (int q = 0; q < TERMS; ++q)
        *reinterpret_cast<uint4*>(dst + q * xplane) = make_uint4(h[q][0], h[q][1], h[q][2], h[q][3]);
    }
  }
}

}  // namespace qm
}  // namespace bakron
