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

// Address of a 16-row tile: codes of its first 8-row block, scales, zeros.
struct TileRef {
  const uint8_t* codes;   // block row of rows 0..7; rows 8..15 are nc blocks further
  const float* scale;     // + k mp
  const uint8_t* zero;
};

__device__ __forceinline__ TileRef tile_ref(const PackedView& w, int64_t e, int64_t row0) {
  TileRef t;
  t.codes = w.codes + (e * (w.mp / 8) + row0 / 8) * w.nc * kBlockBytes;
  t.scale = w.scale + e * w.ng * w.mp + row0;
  t.zero = w.zero ? w.zero + e * w.ng * w.mp + row0 : nullptr;
  return t;
}

template <int NS>
__device__ __forceinline__ void load_chunk(Chunk16<NS>& f, const PackedView& w, const TileRef& t,
                                           int64_t c, int lane) {
  const uint8_t* p = t.codes + c * kBlockBytes + lane * 16;
  f.w[0] = __ldg(reinterpret_cast<const uint4*>(p));
  f.w[1] = __ldg(reinterpret_cast<const uint4*>(p + w.nc * kBlockBytes));
  const int r = lane >> 2;
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    int64_t k = 0;
    if (w.ng > 1) {
      k = (int64_t)((uint32_t)(c * 128 + 32 * s) / (uint32_t)w.g);
      if (k > w.ng - 1) k = w.ng - 1;
    }
    k *= w.mp;
    f.s[0][s] = __ldg(t.scale + k + r);
    f.s[1][s] = __ldg(t.scale + k + r + 8);
    if (t.zero) {
      f.z[0][s] = __ldg(t.zero + k + r);
      f.z[1][s] = __ldg(t.zero + k + r + 8);
    }
  }
}

// tot += the chunk's products with the activations of NT x 8 columns.
// xs: shared memory, TERMS planes of xplane bytes, a column's row of xpitch
// bytes, the chunk's first column at xs; col[j]: this thread's column of
// column tile j.
template <typename H, int TERMS, int NT, int NS>
__device__ __forceinline__ void chunk_product(float (&tot)[NT][4], const Chunk16<NS>& f, bool has_zero,
                                              int zu, const uint8_t* xs, uint32_t xplane,
                                              uint32_t xpitch, const int (&col)[NT], int lane) {
  const int t = lane & 3;
  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
  uint32_t off0 = 0, off1 = 0;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if (s < NS) {
      const int z0 = has_zero ? (int)f.z[0][s] : zu, z1 = has_zero ? (int)f.z[1][s] : zu;
      off0 = Half2<H>::pair(Half2<H>::kBase + (float)z0);
      off1 = Half2<H>::pair(Half2<H>::kBase + (float)z1);
    }
    const uint32_t wa = s == 0 ? f.w[0].x : s == 1 ? f.w[0].y : s == 2 ? f.w[0].z : f.w[0].w;
    const uint32_t wb = s == 0 ? f.w[1].x : s == 1 ? f.w[1].y : s == 2 ? f.w[1].z : f.w[1].w;
    uint32_t a[4], b[4];
    unpack_word<H>(wa, off0, a);
    unpack_word<H>(wb, off1, b);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int q = 0; q < TERMS; ++q) {
        const uint4 x = *reinterpret_cast<const uint4*>(xs + q * xplane + (uint32_t)col[j] * xpitch +
                                                        s * 64 + t * 16);
        mma16816<H>(acc[j], a[0], b[0], a[1], b[1], x.x, x.y);
        mma16816<H>(acc[j], a[2], b[2], a[3], b[3], x.z, x.w);
      }
    }
    if (NS == 4 || s == 3) {
      const float s0 = f.s[0][NS == 4 ? s : 0], s1 = f.s[1][NS == 4 ? s : 0];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        tot[j][0] = fmaf(s0, acc[j][0], tot[j][0]);
        tot[j][1] = fmaf(s0, acc[j][1], tot[j][1]);
        tot[j][2] = fmaf(s1, acc[j][2], tot[j][2]);
        tot[j][3] = fmaf(s1, acc[j][3], tot[j][3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
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
