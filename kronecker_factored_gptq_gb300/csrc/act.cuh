// Activations and what a fused product does with its sums.
//
// silu and the tanh form of gelu are both z / (1 + exp(-z q)), q = 1 or c1 + c3 z^2: 0.5 (1 + tanh u)
// is 1 / (1 + exp(-2 u)).  gelu is z erfc(-z / sqrt 2) / 2: the form with 1 + erf would
// cancel for negative z.
#pragma once

#include <type_traits>

#include "packed.cuh"

namespace bakron {

constexpr float kTanh1 = 1.5957691216057308f, kTanh3 = 0.07135481627260025f;   // 2 sqrt(2 / pi), 0.044715 of it
constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

// s = 1 / (1 + exp(-x)) and 1 - s, from exp(-|x|): nothing overflows, and the small one of the two
// keeps its bits.  Results of 16 bits take the fast exponential and quotient (relative error about 2^-20
// where it matters), fp32 CUDA's own.
template <typename T>
__device__ __forceinline__ void sigmoid(float x, float& s, float& rest) {
  float e, r;
  if constexpr (sizeof(T) == 2) {
    e = __expf(-fabsf(x));
    r = __fdividef(1.f, 1.f + e);
  } else {
    e = expf(-fabsf(x));
    r = 1.f / (1.f + e);
  }
  const bool up = x >= 0.f;
  s = up ? r : e * r;
  rest = up ? e * r : r;
}
template <typename T>
__device__ __forceinline__ float exp_for(float x) {
  if constexpr (sizeof(T) == 2) return __expf(x);
  else return expf(x);
}

inline bool act_ok(int act) { return act >= BAKRON_ACT_NONE && act <= BAKRON_ACT_SILU; }

// Calls f with the activation as a constant: the choice is made once for many values.
template <typename F>
__device__ __forceinline__ void by_act(int act, F f) {
  switch (act) {
    case BAKRON_ACT_NONE: return f(std::integral_constant<int, BAKRON_ACT_NONE>());
    case BAKRON_ACT_RELU: return f(std::integral_constant<int, BAKRON_ACT_RELU>());
    case BAKRON_ACT_GELU: return f(std::integral_constant<int, BAKRON_ACT_GELU>());
    case BAKRON_ACT_GELU_TANH: return f(std::integral_constant<int, BAKRON_ACT_GELU_TANH>());
    default: return f(std::integral_constant<int, BAKRON_ACT_SILU>());
  }
}

// a(z), for a result of type T.
template <typename T, int A>
__device__ __forceinline__ float activate(float z) {
  if constexpr (A == BAKRON_ACT_NONE) {
    return z;
  } else if constexpr (A == BAKRON_ACT_RELU) {
    return z < 0.f ? 0.f : z;                                 // NaN stays
  } else if constexpr (A == BAKRON_ACT_GELU) {
    return 0.5f * z * erfcf(-kSqrtHalf * z);
  } else {
    float p, rest;
    sigmoid<T>(A == BAKRON_ACT_GELU_TANH ? z * fmaf(kTanh3, z * z, kTanh1) : z, p, rest);
    return z * p;
  }
}

// a(z) and a'(z).  The values of finite z are finite: z^2 is kept below what would meet a
// factor of zero as infinity.
template <typename T, int A>
__device__ __forceinline__ void activate_slope(float z, float& a, float& slope) {
  if constexpr (A == BAKRON_ACT_NONE) {
    a = z;
    slope = 1.f;
  } else if constexpr (A == BAKRON_ACT_RELU) {
    a = z < 0.f ? 0.f : z;
    slope = z > 0.f ? 1.f : z <= 0.f ? 0.f : z;               // NaN stays
  } else if constexpr (A == BAKRON_ACT_GELU) {
    const float p = 0.5f * erfcf(-kSqrtHalf * z);
    a = z * p;
    slope = fmaf(z * exp_for<T>(-0.5f * z * z), kInvSqrt2Pi, p);
  } else {
    float s, rest;
    if constexpr (A == BAKRON_ACT_GELU_TANH) {
      const float zz = fminf(z * z, 1e30f);
      sigmoid<T>(z * fmaf(kTanh3, zz, kTanh1), s, rest);
      a = z * s;
      slope = fmaf(a * rest, fmaf(3.f * kTanh3, zz, kTanh1), s);
    } else {
      sigmoid<T>(z, s, rest);
      a = z * s;
      slope = fmaf(a, rest, s);
    }
  }
}

// What a product does with a sum v on its way out: z = v + bias, kept in `pre`;
// y = residual + a(z).
struct Epilogue {
  const float* bias;      // per column of y, nullable
  const void* residual;   // of y's shape and type, nullable
  void* pre;              // likewise, nullable
  int act;
};

// Stores the sum of an element of y, the `at`-th, of column `col`; with kAct false as it is.
template <typename T, bool kAct>
__device__ __forceinline__ void put(T* y, const Epilogue& e, int64_t at, int64_t col, float v) {
  if constexpr (kAct) {
    if (e.bias) v += __ldg(e.bias + col);
    if (e.pre) static_cast<T*>(e.pre)[at] = from_float<T>(v);
    by_act(e.act, [&](auto A) { v = activate<T, A>(v); });
    if (e.residual) v += to_float(static_cast<const T*>(e.residual)[at]);
  }
  *y = from_float<T>(v);
}

}  // namespace bakron
