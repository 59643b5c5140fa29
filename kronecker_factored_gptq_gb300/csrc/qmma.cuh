// Products of packed 4-bit rows with a few columns of activations on the
// warp-level matrix instructions (m16n8k16): the device code shared by the
// few-token linear layer and the mixture-of-experts layer.
//
// These products are bound by the weights' bytes: a 16 x 128 block of codes
// is 1 KB and meets at most a few dozen tokens.  What matters is that the
// codes go from memory to the operand registers with few instructions and
// nothing in between: a warp's 16-byte loads are two whole blocks (8 rows x
// 128 columns) and already hold the A fragments of 8 matrix instructions
// (packed.cuh), so the codes never pass through shared memory.  The k slots
// of an instruction are any 16 columns as long as both operands agree: slots
// (2 t, 2 t + 1) and (2 t + 8, 2 t + 9) of thread t are four consecutive
// columns, and the thread's eight columns of a step are one 16-byte read of
// the activations.
//
// A is the exact integer u - z; the group's sum comes out of the tensor core
// in fp32 (at most 128 products, so no long chain of its additions) and is
// scaled and added to the running sum with fp32 FMAs.  fp32 activations are
// three bf16 terms whose sum is exact (split3); their products go into the
// same group sum.
#pragma once

#include "packed.cuh"

namespace bakron {
namespace qm {

template <typename H>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], uint32_t a0, uint32_t a1,
                                                        uint32_t a2, uint32_t a3, uint32_t b0,
                                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], uint32_t a0, uint32_t a1,
                                                 uint32_t a2, uint32_t a3, uint32_t b0,
                                                 uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// What one 128-column chunk of a 16-row tile needs from memory, per thread:
// rows lane / 4 and lane / 4 + 8.  NS scales per row: 1 when the group is a
// multiple of 128 columns, else one per 32 columns.
template <int NS>
struct Chunk16 {
  uint4 w[2];
  float s[2][NS];
  uint32_t z[2][NS];
};

// A thread's two rows of a 16-row tile: codes (at the thread's 16 bytes of
// the first chunk) and grid.
struct TileRef {
  const uint8_t* codes[2];
  const float* scale[2];    // + k mp
  const uint8_t* zero[2];   // likewise; NULL when every zero point is the same
};

// Rows row0 + lane / 4 and + 8 of matrix e; rows past the padding repeat its
// last row (their products are dropped by the caller).
__device__ __forceinline__ TileRef tile_ref(const PackedView& w, int64_t e, int64_t row0, int lane) {
  TileRef t;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t r = min(row0 + (lane >> 2) + 8 * i, w.mp - 1);
    t.codes[i] = w.codes + (e * (w.mp / 8) + r / 8) * w.nc * kBlockBytes + (r & 7) * 64 + (lane & 3) * 16;
    t.scale[i] = w.scale + e * w.ng * w.mp + r;
    t.zero[i] = w.zero ? w.zero + e * w.ng * w.mp + r : nullptr;
  }
  return t;
}

template <int NS>
__device__ __forceinline__ void load_chunk(Chunk16<NS>& f, const PackedView& w, const TileRef& t,
                                           int64_t c) {
  f.w[0] = ld_codes(t.codes[0] + c * kBlockBytes);
  f.w[1] = ld_codes(t.codes[1] + c * kBlockBytes);
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    int64_t k = 0;
    if (w.ng > 1) {
      k = (int64_t)((uint32_t)(c * 128 + 32 * s) / (uint32_t)w.g);
      if (k > w.ng - 1) k = w.ng - 1;
    }
    k *= w.mp;
    f.s[0][s] = ld_ahead(t.scale[0] + k);
    f.s[1][s] = ld_ahead(t.scale[1] + k);
    if (w.zero) {
      f.z[0][s] = ld_ahead(t.zero[0] + k);
      f.z[1][s] = ld_ahead(t.zero[1] + k);
    }
  }
}

// tot[r][j] += products of the chunk of row tile r with column tile j, for j <
// live (uniform).  fetch(j, q, s): this thread's 8 columns 32 s + 8 t .. of
// term q of its activation row in column tile j.
template <typename H, int TERMS, int RT, int NT, int NS, typename Fetch>
__device__ __forceinline__ void chunk_product(float (&tot)[RT][NT][4], const Chunk16<NS> (&f)[RT],
                                              bool has_zero, int zu, int live, Fetch fetch) {
  float acc[RT][NT][4];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[r][j][i] = 0.f;
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
      if (j < live) {
#pragma unroll
        for (int q = 0; q < TERMS; ++q) {
          const uint4 x = fetch(j, q, s);
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            mma16816<H>(acc[r][j], a[r][0], b[r][0], a[r][1], b[r][1], x.x, x.y);
            mma16816<H>(acc[r][j], a[r][2], b[r][2], a[r][3], b[r][3], x.z, x.w);
          }
        }
      }
    }
    if (NS == 4 || s == 3) {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float s0 = f[r].s[0][NS == 4 ? s : 0], s1 = f[r].s[1][NS == 4 ? s : 0];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          tot[r][j][0] = fmaf(s0, acc[r][j][0], tot[r][j][0]);
          tot[r][j][1] = fmaf(s0, acc[r][j][1], tot[r][j][1]);
          tot[r][j][2] = fmaf(s1, acc[r][j][2], tot[r][j][2]);
          tot[r][j][3] = fmaf(s1, acc[r][j][3], tot[r][j][3]);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][j][i] = 0.f;
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
