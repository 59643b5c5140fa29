// bakron_pack / bakron_unpack: 4-bit codes into the layout of the products
// (packed.cuh) and back to values.  Both run once per layer and were left
// simple: eight one-byte loads (stores of four bytes) a thread.  A call that
// ends with its status read back: 8192 x 8192 144 to 158 us to pack (the bytes at 6.68 TB/s:
// 15), 210 to 216 to unpack (45).
#include <algorithm>

#include "packed.cuh"

namespace bakron {

namespace {

__device__ int g_async_status = 0;

// One thread per 32-bit word of the codes: 8 codes of a row (zero on the
// padding), range-checked, in the bit order of the layout.
__global__ void pack_codes_kernel(const int8_t* __restrict__ codes, int64_t count, int64_t m,
                                  int64_t n, int64_t mp, int64_t nc, int qmin, int qmax,
                                  uint32_t* __restrict__ out, DevStatus* st) {
  const int64_t total = count * mp * nc * 16;
  bool bad = false;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int word = (int)(i & 15), row = (int)(i >> 4) & 7;
    const int64_t block = i >> 7;                     // over count x (mp / 8) x nc
    const int64_t c = block % nc, rb = block / nc;
    const int64_t e = rb / (mp / 8), r = (rb - e * (mp / 8)) * 8 + row;
    const int t = word >> 2, s = word & 3;
    const int64_t j0 = c * 128 + 32 * s + 8 * t;
    uint32_t w = 0;
    if (r < m) {
      const int8_t* src = codes + (e * m + r) * n + j0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (j0 + k < n) {
          const int v = src[k];
          bad |= v < qmin || v > qmax;
          const uint32_t u = (uint32_t)(v - qmin) & 15u;
          w |= u << (4 * (k >> 1) + 16 * (k & 1));
        }
      }
    }
    out[i] = w;
  }
  if (__any_sync(0xffffffffu, bad) && (threadIdx.x & 31) == 0) set_status(st, BAKRON_ERR_CODE_RANGE);
}

// scale[e][i][k] -> [e][i / 16][k][i % 16], 0 on the padding rows; zero points likewise
// as bytes z - qmin.  The bits of positive floats are ordered as they are, so the largest
// scale is a maximum of whole numbers, whatever the order.
__global__ void pack_grid_kernel(const float* __restrict__ scale, const float* __restrict__ zero,
                                 int64_t count, int64_t m, int64_t mp, int64_t ng, float qmin,
                                 float qmax, float* __restrict__ so, uint8_t* __restrict__ zo,
                                 unsigned* __restrict__ largest, DevStatus* st) {
  const int64_t total = count * ng * mp;
  bool bad = false, badz = false;
  unsigned top = 0;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t b = i / 16, k = b % ng, r = (b / ng) % (mp / 16) * 16 + i % 16, e = i / (mp * ng);
    float s = 0.f;
    uint8_t z = 0;
    if (r < m) {
      const int64_t at = (e * m + r) * ng + k;
      s = scale[at];
      if (s > 0.f && isfinite(s)) top = max(top, __float_as_uint(s));
      else bad = true;
      if (zero) {
        const float v = zero[at];
        const bool wrong = !(v >= qmin && v <= qmax) || rintf(v) != v;
        badz |= wrong;
        if (!wrong) z = (uint8_t)(int)(v - qmin);
      }
    }
    so[i] = s;
    if (zero) zo[i] = z;
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) atomicMax(largest, top);
  if (__any_sync(0xffffffffu, bad) && (threadIdx.x & 31) == 0) set_status(st, BAKRON_ERR_NONFINITE);
  if (__any_sync(0xffffffffu, badz) && (threadIdx.x & 31) == 0) set_status(st, BAKRON_ERR_CODE_RANGE);
}

// V = s (c - z), one thread per word.
__global__ void unpack_kernel(const PackedView w, float* __restrict__ V) {
  const int64_t total = w.count * w.mp * w.nc * 16;
  const uint32_t* words = reinterpret_cast<const uint32_t*>(w.codes);
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int word = (int)(i & 15), row = (int)(i >> 4) & 7;
    const int64_t block = i >> 7;
    const int64_t c = block % w.nc, rb = block / w.nc;
    const int64_t e = rb / (w.mp / 8), r = (rb - e * (w.mp / 8)) * 8 + row;
    const int t = word >> 2, s = word & 3;
    const int64_t j0 = c * 128 + 32 * s + 8 * t;
    if (r >= w.m || j0 >= w.n) continue;
    const int64_t at = grid_row(w, e, r) + j0 / w.g * 16;
    const float sc = w.scale[at];
    const int z = w.zero ? w.zero[at] : w.zu;
    const uint32_t v = words[i];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int u = (int)(v >> (4 * (k >> 1) + 16 * (k & 1))) & 15;
      // a row of one group whose size is no multiple of 8 ends inside a word
      if (j0 + k < w.n) V[(e * w.m + r) * w.n + j0 + k] = sc * (float)(u - z);
    }
  }
}

unsigned grid_words(int64_t total) {
  return (unsigned)std::max<int64_t>(1, std::min<int64_t>((total + 255) / 256, (int64_t)sm_count() * 32));
}

}  // namespace

int* async_status_word() {
  static std::atomic<int*> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  int* p = cached[dev].load(std::memory_order_acquire);
  if (p) return p;
  void* v = nullptr;
  if (cudaGetSymbolAddress(&v, g_async_status) != cudaSuccess) return nullptr;
  cached[dev].store(static_cast<int*>(v), std::memory_order_release);
  return static_cast<int*>(v);
}

}  // namespace bakron

using namespace bakron;

extern "C" bakron_status bakron_async_status(void* stream) {
  cudaStream_t s = (cudaStream_t)stream;
  int* word = async_status_word();
  int st = 0;
  if (!word) return BAKRON_ERR_CUDA;
  if (cudaMemcpyAsync(&st, word, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaMemsetAsync(word, 0, sizeof(int), s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return BAKRON_ERR_CUDA;
  return (bakron_status)st;
}

extern "C" bakron_status bakron_pack_size(int64_t count, int64_t m, int64_t n, int64_t group,
                                          int has_zero, size_t* bytes) {
  PackLayout L;
  if (!bytes || !pack_layout(count, m, n, group, has_zero, &L)) return BAKRON_ERR_INVALID_ARG;
  *bytes = L.total;
  return BAKRON_OK;
}

extern "C" bakron_status bakron_pack(const int8_t* codes, const float* scale, const float* zero,
                                     int64_t count, int64_t m, int64_t n, int64_t group, int qmin,
                                     int qmax, void* data, size_t data_bytes, void* stream) {
  PackLayout L;
  if (!codes || !scale || !data || !pack_layout(count, m, n, group, zero != nullptr, &L))
    return BAKRON_ERR_INVALID_ARG;
  if (qmin < -128 || qmin > qmax || qmax > 127 || qmax - qmin > 15) return BAKRON_ERR_INVALID_ARG;
  if (!aligned_to(data, 16) || data_bytes < L.total || !aligned_to(scale, 4) || !aligned_to(zero, 4))
    return BAKRON_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  uint8_t* p = static_cast<uint8_t*>(data);
  DevStatus* st = reinterpret_cast<DevStatus*>(p);
  if (cudaMemsetAsync(st, 0, kPackHeader, s) != cudaSuccess) return BAKRON_ERR_CUDA;
  count_launch(2);
  pack_codes_kernel<<<grid_words(count * L.mp * L.nc * 16), 256, 0, s>>>(
      codes, count, m, n, L.mp, L.nc, qmin, qmax, reinterpret_cast<uint32_t*>(p + L.codes), st);
  pack_grid_kernel<<<grid_words(count * L.ng * L.mp), 256, 0, s>>>(
      scale, zero, count, m, L.mp, L.ng, (float)qmin, (float)qmax,
      reinterpret_cast<float*>(p + L.scale), zero ? p + L.zero : nullptr,
      reinterpret_cast<unsigned*>(p + kPackLargest), st);
  if (cudaGetLastError() != cudaSuccess) return BAKRON_ERR_CUDA;
  DevStatus host;
  if (cudaMemcpyAsync(&host, st, sizeof(host), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return BAKRON_ERR_CUDA;
  return (bakron_status)host.status;
}

extern "C" bakron_status bakron_unpack(const bakron_packed* w, float* V, void* stream) {
  PackedView v;
  if (!V || !aligned_to(V, 4) || !packed_view(w, &v)) return BAKRON_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  count_launch();
  unpack_kernel<<<grid_words(v.count * v.mp * v.nc * 16), 256, 0, s>>>(v, V);
  if (cudaGetLastError() != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess)
    return BAKRON_ERR_CUDA;
  return BAKRON_OK;
}
