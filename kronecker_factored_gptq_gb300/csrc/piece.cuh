// Consecutive elements of a row as one access of up to 16 bytes, kept as the words that were
// loaded: as an array of bf16 elements the compiler takes them apart half by half (32 registers more
// for 16 elements, and spills).
#pragma once

#include <type_traits>

#include "packed.cuh"

namespace bakron {

template <int VB>
struct PieceWords {
  using type = uint16_t;
  static constexpr int n = 1;
};
template <>
struct PieceWords<4> {
  using type = uint32_t;
  static constexpr int n = 1;
};
template <>
struct PieceWords<8> {
  using type = uint32_t;
  static constexpr int n = 2;
};
template <>
struct PieceWords<16> {
  using type = uint32_t;
  static constexpr int n = 4;
};

// VB bytes: V elements of T.
template <typename T, int VB>
struct alignas(VB) Piece {
  static constexpr int V = VB / (int)sizeof(T), W = PieceWords<VB>::n;
  typename PieceWords<VB>::type w[W];

  // element e as a float; e is a constant after unrolling
  __device__ __forceinline__ float get(int e) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[e]);
    } else if constexpr (VB == 2) {
      return to_float(*reinterpret_cast<const T*>(&w[0]));
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      const uint32_t u = w[e >> 1];
      return __uint_as_float(e & 1 ? u & 0xffff0000u : u << 16);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[e >> 1]));
      return e & 1 ? f.y : f.x;
    }
  }
  __device__ __forceinline__ void set(const float (&f)[V]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < V; ++e) w[e] = __float_as_uint(f[e]);
    } else if constexpr (VB == 2) {
      const T t = from_float<T>(f[0]);
      w[0] = *reinterpret_cast<const uint16_t*>(&t);
    } else {
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
          const __nv_bfloat162 p = __floats2bfloat162_rn(f[e], f[e + 1]);
          w[e >> 1] = *reinterpret_cast<const uint32_t*>(&p);
        } else {
          const __half2 p = __floats2half2_rn(f[e], f[e + 1]);
          w[e >> 1] = *reinterpret_cast<const uint32_t*>(&p);
        }
      }
    }
  }
};

}  // namespace bakron
