// Packed 4-bit weights: the layout bakron_pack writes, and the device code
// that turns its words into matrix operands.
//
// Layout (bakron.h, bakron_pack).  A 32-bit word holds 8 consecutive columns
// of a row, the even ones in its low half and the odd ones in its high half,
// so that (w >> 4 k) & 0x000f000f is the pair of columns (2 k, 2 k + 1) in the
// two halves of a register: one logic instruction per pair also sets the
// exponent, and one subtraction of 16-bit pairs removes the offset and the
// zero point.  Inside a row's 128 columns word (s, t) sits at 4 t + s: a
// 16-byte load of thread t of a quad then brings the columns 32 s + 8 t .. + 7
// for s = 0..3, and each step s of a quad covers 32 consecutive columns, the
// smallest group.  Blocks of 8 rows x 128 columns are contiguous, so a warp's
// 16-byte loads take 512 contiguous bytes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.cuh"

namespace bakron {

constexpr size_t kPackHeader = 256;
constexpr size_t kPackLargest = 128;  // in the header: the largest scale
constexpr int kBlockBytes = 512;      // 8 rows x 128 columns
constexpr int64_t kMaxPackedDim = int64_t(1) << 20;
constexpr int64_t kMaxPackedCodes = int64_t(1) << 38;

struct PackLayout {
  int64_t mp, np, nc, ng, g;   // padded sizes, 128-column blocks, groups, group size
  size_t codes, scale, zero, total;
};

// Sizes and offsets of a packed buffer; false when they are not acceptable.
inline bool pack_layout(int64_t count, int64_t m, int64_t n, int64_t group, int has_zero,
                        PackLayout* L) {
  if (count < 1 || m < 1 || n < 1 || count > kMaxPackedDim || m > kMaxPackedDim ||
      n > kMaxPackedDim || group < 0 || (has_zero != 0 && has_zero != 1))
    return false;
  if (group > 0 && group < n && group % 32 != 0) return false;
  L->mp = (m + 15) / 16 * 16;
  L->np = (n + 127) / 128 * 128;
  if (L->mp * L->np > kMaxPackedCodes / count) return false;
  L->nc = L->np / 128;
  // one group per row spans the padding too, so that a padded column's group
  // index (clamped to ng - 1 for finer groups) is always one that exists
  L->g = (group == 0 || group >= n) ? L->np : group;
  L->ng = (n + L->g - 1) / L->g;
  size_t off = kPackHeader;
  L->codes = off;
  off += (size_t)(count * L->mp * L->np / 2);
  L->scale = off;
  off += (size_t)(count * L->ng * L->mp) * 4;
  L->zero = off;
  if (has_zero) off += ((size_t)(count * L->ng * L->mp) + 15) / 16 * 16;
  L->total = off;
  return true;
}

// A packed matrix as the kernels see it.
struct PackedView {
  const uint8_t* codes;   // [count][mp / 8][nc][512]
  const float* scale;     // [count][mp / 16][ng][16]
  const uint8_t* zero;    // likewise, or NULL: every zero point is `zu`
  int zu;                 // -qmin
  const float* largest;   // the largest scale of all (0: not known)
  int64_t count, m, n, mp, nc, ng, g;
  uint64_t g_mul;         // floor(2^40 / g) + 1: k / g = (k g_mul) >> 40 for k, g <= 2^20
};

// The view of a caller's descriptor, checked; false when it is not usable.
inline bool packed_view(const bakron_packed* w, PackedView* v) {
  PackLayout L;
  if (!w || !w->data || !pack_layout(w->count, w->m, w->n, w->group, w->has_zero, &L)) return false;
  if ((reinterpret_cast<uintptr_t>(w->data) & 15) != 0 || w->bytes < L.total) return false;
  if (w->qmin < -128 || w->qmin > 127) return false;
  const uint8_t* p = static_cast<const uint8_t*>(w->data);
  v->codes = p + L.codes;
  v->scale = reinterpret_cast<const float*>(p + L.scale);
  v->zero = w->has_zero ? p + L.zero : nullptr;
  v->zu = -w->qmin;
  v->largest = reinterpret_cast<const float*>(p + kPackLargest);
  v->count = w->count;
  v->m = w->m;
  v->n = w->n;
  v->mp = L.mp;
  v->nc = L.nc;
  v->ng = L.ng;
  v->g = L.g;
  v->g_mul = (uint64_t(1) << 40) / (uint64_t)L.g + 1;
  return true;
}

// Offset of row r's grid entry of its first group; a group is 16 entries further.
__host__ __device__ __forceinline__ int64_t grid_row(const PackedView& w, int64_t e, int64_t r) {
  return ((e * (w.mp / 16) + r / 16) * w.ng) * 16 + r % 16;
}
// Group of column k; a padded column belongs to the last one.
__device__ __forceinline__ uint32_t grid_group(const PackedView& w, uint32_t k) {
  return min((uint32_t)(((uint64_t)k * w.g_mul) >> 40), (uint32_t)w.ng - 1);
}

inline bool dtype_ok(int dtype) {
  return dtype == BAKRON_F32 || dtype == BAKRON_BF16 || dtype == BAKRON_F16;
}
inline size_t dtype_size(int dtype) { return dtype == BAKRON_F32 ? 4 : 2; }
inline bool aligned_to(const void* p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// The status of a launch; a failed one leaves no error behind for the next call.
inline bakron_status launch_status(cudaError_t e) {
  if (e == cudaSuccess) return BAKRON_OK;
  (void)cudaGetLastError();
  return BAKRON_ERR_CUDA;
}

// Device word of the current device that keeps the first error of the
// enqueue-only calls (bakron_async_status); NULL when it cannot be resolved.
int* async_status_word();

// ------------------------------------------------------------ device code

// Loads ahead of their use.  The compiler may move an ordinary read-only load
// down to its use, past the barriers in between, which would expose its latency;
// these stay where they are written.  The codes are read once: past L1.
__device__ __forceinline__ uint4 ld_codes(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ float ld_ahead(const float* p) {
  float v;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld_ahead(const uint8_t* p) {
  uint32_t v;
  asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

// The 16-bit operand type of the products: exact for integers up to 256
// (bf16) or 2048 (fp16), so u - z never rounds.
template <typename H>
struct Half2;
template <>
struct Half2<__nv_bfloat16> {
  static constexpr uint32_t kMagic = 0x43004300u;   // 128 in both halves; ulp 1
  static constexpr float kBase = 128.f;
  static __device__ __forceinline__ uint32_t pair(float x) {
    const __nv_bfloat162 v = __float2bfloat162_rn(x);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                     *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};
template <>
struct Half2<__half> {
  static constexpr uint32_t kMagic = 0x64006400u;   // 1024 in both halves; ulp 1
  static constexpr float kBase = 1024.f;
  static __device__ __forceinline__ uint32_t pair(float x) {
    const __half2 v = __float2half2_rn(x);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a),
                              *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};

// The 8 columns of a word as 4 pairs of exact integers u - z; off is the
// pair (base + z, base + z).
template <typename H>
__device__ __forceinline__ void unpack_word(uint32_t w, uint32_t off, uint32_t (&p)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t v;
    // (w >> 4 k) & 0x000f000f | magic
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;"
        : "=r"(v)
        : "r"(w >> (4 * k)), "n"(0x000f000f), "r"(Half2<H>::kMagic));
    p[k] = Half2<H>::sub(v, off);
  }
}

// x = hi + mid + lo exactly, each a bf16 (8 significant bits, cut off rather
// than rounded, so hi never overflows); Inf and NaN are kept in hi alone.
__device__ __forceinline__ void split3(float x, float& hi, float& mid, float& lo) {
  const uint32_t u = __float_as_uint(x);
  hi = __uint_as_float(u & 0xffff0000u);
  if ((u & 0x7f800000u) == 0x7f800000u) {
    if (x != x) hi = __uint_as_float(0x7fc00000u);
    mid = lo = 0.f;
    return;
  }
  const float r = x - hi;
  mid = __uint_as_float(__float_as_uint(r) & 0xffff0000u);
  lo = r - mid;
}

// The same sum with hi and mid rounded to nearest instead of cut off: mid is at
// most 2^-8 and lo 2^-17 of the power of two below |x| (cut off: 2^-7 and 2^-15),
// where products of small terms are left out.  Cut where rounding would overflow.
__device__ __forceinline__ void split3_near(float x, float& hi, float& mid, float& lo) {
  if ((__float_as_uint(x) & 0x7fffffffu) >= 0x7f7f8000u) return split3(x, hi, mid, lo);
  hi = __bfloat162float(__float2bfloat16_rn(x));
  const float r = x - hi;
  mid = __bfloat162float(__float2bfloat16_rn(r));
  lo = r - mid;
}

// split3_near for the gradient's dY, whose last term is multiplied with the weights'
// first terms only: there an infinity or NaN meets what the formula has, zero where the
// weight is, and not the exact zeros that the weights' other terms often are.
__device__ __forceinline__ void split3_grad(float x, float& hi, float& mid, float& lo) {
  split3_near(x, hi, mid, lo);
  if ((__float_as_uint(x) & 0x7f800000u) == 0x7f800000u) {
    lo = hi;
    hi = 0.f;
  }
}

// The top half of a float that is a bf16.
__device__ __forceinline__ uint16_t bf16_bits(float x) {
  return (uint16_t)(__float_as_uint(x) >> 16);
}

template <typename TX>
__device__ __forceinline__ float to_float(TX x);
template <>
__device__ __forceinline__ float to_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_float<__half>(__half x) { return __half2float(x); }
template <typename TX>
__device__ __forceinline__ TX from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }

}  // namespace bakron
