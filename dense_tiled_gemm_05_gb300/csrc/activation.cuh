// activation.cuh -- element types, 16-byte row pieces and activation functions shared by the
// feed-forward operators' kernels (products with an epilogue, the gated pair, layer norm).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "gemm.h"

// Runs a statement with T naming the element type of a gemm_dtype_t.
#define FF_TYPED(dt, T, ...)                                  \
  switch (dt) {                                               \
    case GEMM_F32: { using T = float; __VA_ARGS__; break; }   \
    case GEMM_F16: { using T = __half; __VA_ARGS__; break; }  \
    default: { using T = __nv_bfloat16; __VA_ARGS__; break; } \
  }

namespace gemm_gb300 {
namespace ff {

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Element i of a vector whose type is known at run time (biases and norm weights, which are
// read once a column and may be wider than the rows they apply to).
__device__ __forceinline__ float load_any(const void *p, int dtype, int64_t i) {
  if (dtype == GEMM_F32) return static_cast<const float *>(p)[i];
  if (dtype == GEMM_F16) return __half2float(static_cast<const __half *>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}
__device__ __forceinline__ void store_any(void *p, int dtype, int64_t i, float v) {
  if (dtype == GEMM_F32) static_cast<float *>(p)[i] = v;
  else if (dtype == GEMM_F16) static_cast<__half *>(p)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

// VEC consecutive values of a row from column j0, as fp32; columns past n read as 0. With
// VECTOR (the row starts on a multiple of the piece's size, up to 16 bytes) a whole piece is
// read in 16-byte loads (8 for a piece of four 16-bit values).
template <typename T, int VEC, bool VECTOR>
__device__ __forceinline__ void load_piece(const T *row, int64_t j0, int64_t n, float (&v)[VEC]) {
  if (VECTOR && j0 + VEC <= n) {
    constexpr int BYTES = VEC * static_cast<int>(sizeof(T));
    static_assert(BYTES % 16 == 0 || BYTES == 8, "piece size");
    alignas(16) T e[VEC];
    if (BYTES == 8) {
      *reinterpret_cast<uint2 *>(e) = *reinterpret_cast<const uint2 *>(row + j0);
    } else {
#pragma unroll
      for (int w = 0; w < BYTES / 16; ++w)
        reinterpret_cast<uint4 *>(e)[w] = reinterpret_cast<const uint4 *>(row + j0)[w];
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = to_f32(e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = j0 + i < n ? to_f32(row[j0 + i]) : 0.0f;
  }
}

template <typename T, int VEC, bool VECTOR>
__device__ __forceinline__ void store_piece(T *row, int64_t j0, int64_t n, const float (&v)[VEC]) {
  if (VECTOR && j0 + VEC <= n) {
    constexpr int BYTES = VEC * static_cast<int>(sizeof(T));
    static_assert(BYTES % 16 == 0 || BYTES == 8, "piece size");
    alignas(16) T e[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) e[i] = from_f32<T>(v[i]);
    if (BYTES == 8) {
      *reinterpret_cast<uint2 *>(row + j0) = *reinterpret_cast<const uint2 *>(e);
    } else {
#pragma unroll
      for (int w = 0; w < BYTES / 16; ++w)
        reinterpret_cast<uint4 *>(row + j0)[w] = reinterpret_cast<const uint4 *>(e)[w];
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (j0 + i < n) row[j0 + i] = from_f32<T>(v[i]);
  }
}

constexpr int VEC = 8;  // columns a thread takes of a row

// A thread's eight columns among the 8 T from `first` on. VECTOR (rows start on 16-byte
// boundaries, and so do N and the parameters): eight consecutive ones, in 16-byte accesses.
// Otherwise every T-th one, so that the lanes of a warp read neighbours.
template <int T, bool VECTOR>
struct Columns {
  int64_t first, n;
  int t;
  __device__ __forceinline__ int64_t at(int i) const {
    return VECTOR ? first + t * VEC + i : first + i * T + t;
  }
  __device__ __forceinline__ bool in(int i) const { return at(VECTOR ? 0 : i) < n; }

  template <typename E>
  __device__ __forceinline__ void load(const E *row, E (&e)[VEC]) const {
    if (VECTOR) {
      constexpr int W = VEC * sizeof(E) / 16;
#pragma unroll
      for (int w = 0; w < W; ++w)
        reinterpret_cast<uint4 *>(e)[w] =
            in(0) ? reinterpret_cast<const uint4 *>(row + at(0))[w] : uint4{0, 0, 0, 0};
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) e[i] = in(i) ? row[at(i)] : from_f32<E>(0.0f);
    }
  }
  template <typename E>
  __device__ __forceinline__ void store(E *row, const float (&v)[VEC]) const {
    if (VECTOR) {
      constexpr int W = VEC * sizeof(E) / 16;
      alignas(16) E e[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) e[i] = from_f32<E>(v[i]);
      if (in(0)) {
#pragma unroll
        for (int w = 0; w < W; ++w)
          reinterpret_cast<uint4 *>(row + at(0))[w] = reinterpret_cast<const uint4 *>(e)[w];
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (in(i)) row[at(i)] = from_f32<E>(v[i]);
    }
  }
  template <typename E>
  __device__ __forceinline__ void load_f32(const E *row, float (&v)[VEC]) const {
    alignas(16) E e[VEC];
    load(row, e);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = to_f32(e[i]);
  }
  __device__ __forceinline__ void store(void *base, int dtype, int64_t offset,
                                        const float (&v)[VEC]) const {
    FF_TYPED(dtype, E, { store(static_cast<E *>(base) + offset, v); })
  }
  // A parameter vector (1 or 0 for every column where there is none).
  __device__ __forceinline__ void params(const void *p, int dtype, float missing,
                                         float (&v)[VEC]) const {
    if (!p) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = missing;
      return;
    }
    FF_TYPED(dtype, E, { load_f32(static_cast<const E *>(p), v); })
  }
};

__device__ __forceinline__ void prefetch_l2(const void *p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// Two fp32 values in one register pair: Blackwell's packed add, multiply and multiply-add round
// each half as the scalar instruction does and take one issue slot for both.
struct F2 {
  uint64_t v;
  __device__ __forceinline__ F2() : v(0) {}
  __device__ __forceinline__ F2(float lo, float hi) {
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  }
  __device__ __forceinline__ float2 get() const {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
  }
};
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 c;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(c.v) : "l"(a.v), "l"(b.v));
  return c;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 c;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(c.v) : "l"(a.v), "l"(b.v));
  return c;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return d;
}

constexpr float kSqrtHalf = 0.70710678118654752440f;
constexpr float kSqrt2OverPi = 0.79788456080286535588f;   // sqrt(2 / pi)
constexpr float kInvSqrt2Pi = 0.39894228040143267794f;    // 1 / sqrt(2 pi)
constexpr float kGeluCubic = 0.044715f;                   // of the tanh form of gelu

constexpr float kLog2e = 1.44269504088896340736f;

// Full accuracy, for fp32 inputs. Where the sigmoid has saturated, s (1 - s) is 0 and the
// second term of a slope is left out: its other factor may be infinite there.
__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }

// Argument of the logistic form of tanh-gelu: (1 + tanh t) / 2 = sigmoid(2 t).
__device__ __forceinline__ float gelu_tanh_arg(float z) {
  return 2.0f * kSqrt2OverPi * z * fmaf(kGeluCubic * z, z, 1.0f);
}

__device__ __forceinline__ float relu(float z) { return z > 0.0f ? z : z != z ? z : 0.0f; }  // NaN stays
__device__ __forceinline__ float relu_slope(float z) { return z > 0.0f ? 1.0f : z != z ? z : 0.0f; }

// The normal distribution function is (1 + erf(z / sqrt 2)) / 2, by erfc of the negated
// argument, which keeps the lower tail's relative accuracy.
__device__ __forceinline__ float normal_cdf(float z) { return 0.5f * erfcf(-z * kSqrtHalf); }

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case GEMM_ACT_RELU: return relu(z);
    case GEMM_ACT_GELU: return z * normal_cdf(z);
    case GEMM_ACT_GELU_TANH: return z * sigmoid(gelu_tanh_arg(z));
    case GEMM_ACT_SILU: return z * sigmoid(z);
    case GEMM_ACT_SIGMOID: return sigmoid(z);
    default: return z;
  }
}

// act(z) and act'(z) together (they share their exponential).
__device__ __forceinline__ void activate_slope(float z, int act, float &a, float &d) {
  switch (act) {
    case GEMM_ACT_RELU:
      a = relu(z);
      d = relu_slope(z);
      return;
    case GEMM_ACT_GELU: {
      const float p = normal_cdf(z), e = expf(-0.5f * z * z);
      a = z * p;
      d = p + (e > 0.0f ? z * kInvSqrt2Pi * e : 0.0f);
      return;
    }
    case GEMM_ACT_GELU_TANH: {
      const float s = sigmoid(gelu_tanh_arg(z)), t = s * (1.0f - s);
      a = z * s;
      d = s + (t > 0.0f ? z * t * (2.0f * kSqrt2OverPi) * fmaf(3.0f * kGeluCubic * z, z, 1.0f) : 0.0f);
      return;
    }
    case GEMM_ACT_SILU: {
      const float s = sigmoid(z), t = s * (1.0f - s);
      a = z * s;
      d = s + (t > 0.0f ? z * t : 0.0f);
      return;
    }
    case GEMM_ACT_SIGMOID:
      a = sigmoid(z);
      d = a * (1.0f - a);
      return;
    default:
      a = z;
      d = 1.0f;
      return;
  }
}

// The same for kernels whose inputs are 16-bit, two elements at a time: products and sums in
// packed fp32, exponentials and reciprocals by the hardware's approximations with subnormals
// flushed (a few fp32 ulps, against the 2^-9 of the inputs' rounding; both saturate to exactly
// 0 and 1). It is for the slopes kernels, which have six bytes of HBM traffic an element to hide
// the arithmetic under: bias gradient alone, 4096 x 4096 bf16 on one GB300, against unpacked
// __expf, __fdividef and erff: gelu 20 us (32), its tanh form 16 (22), silu 15 (19). The
// products' epilogues run it too, at the same speed as before.
__device__ __forceinline__ F2 exp2_fast(F2 x) {
  float2 f = x.get();
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(f.x));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(f.y));
  return {f.x, f.y};
}
__device__ __forceinline__ F2 reciprocal_fast(F2 x) {
  float2 f = x.get();
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(f.x));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(f.y));
  return {f.x, f.y};
}
__device__ __forceinline__ F2 both(float v) { return {v, v}; }
// 1 / (1 + 2^x): sigmoid of -x ln 2.
__device__ __forceinline__ F2 logistic2(F2 x) { return reciprocal_fast(exp2_fast(x) + both(1.0f)); }
// base + z t w where t > 0, base elsewhere (w may be infinite where t is 0).
__device__ __forceinline__ F2 slope_sum(F2 base, F2 t, F2 zw) {
  const float2 b = base.get(), q = t.get(), r = fma2(t, zw, base).get();
  return {q.x > 0.0f ? r.x : b.x, q.y > 0.0f ? r.y : b.y};
}

// The normal distribution function Phi(z) and e = exp(-z^2 / 2). With t = 1 / (1 + 0.33 |z|),
// Phi(-|z|) = e t q(t): q, of degree 8, is a least-maximum fit of the ratio's relative error by
// linear programming over 0 <= |z| <= 14, where e has vanished: 6e-8, and 3.0e-7 in fp32
// arithmetic. (Degree 6, with 1.2e-6, showed in fp32 outputs.)
__device__ __forceinline__ F2 normal_cdf_fast(F2 z, F2 &e) {
  const float2 f = z.get();
  const F2 t = reciprocal_fast(fma2({fabsf(f.x), fabsf(f.y)}, both(0.33f), both(1.0f)));
  e = exp2_fast(z * z * both(-0.5f * kLog2e));
  F2 q = fma2(both(-0.0208073501f), t, both(0.123078719f));
  q = fma2(q, t, both(-0.267183691f));
  q = fma2(q, t, both(0.224627852f));
  q = fma2(q, t, both(-0.0565249808f));
  q = fma2(q, t, both(0.121818528f));
  q = fma2(q, t, both(0.111066021f));
  q = fma2(q, t, both(0.132302761f));
  q = fma2(q, t, both(0.131622165f));
  const float2 h = (q * t * e).get();
  return {f.x > 0.0f ? 1.0f - h.x : h.x, f.y > 0.0f ? 1.0f - h.y : h.y};
}

__device__ __forceinline__ F2 activate_fast(F2 z, int act) {
  const float2 f = z.get();
  switch (act) {
    case GEMM_ACT_RELU: return {relu(f.x), relu(f.y)};
    case GEMM_ACT_GELU: {
      F2 e;
      return z * normal_cdf_fast(z, e);
    }
    case GEMM_ACT_GELU_TANH: {
      constexpr float c = -2.0f * kSqrt2OverPi * kLog2e;
      return z * logistic2(z * fma2(z * z, both(c * kGeluCubic), both(c)));
    }
    case GEMM_ACT_SILU: return z * logistic2(z * both(-kLog2e));
    case GEMM_ACT_SIGMOID: return logistic2(z * both(-kLog2e));
    default: return z;
  }
}

__device__ __forceinline__ void activate_slope_fast(F2 z, int act, F2 &a, F2 &d) {
  const float2 f = z.get();
  switch (act) {
    case GEMM_ACT_RELU:
      a = {relu(f.x), relu(f.y)};
      d = {relu_slope(f.x), relu_slope(f.y)};
      return;
    case GEMM_ACT_GELU: {
      F2 e;
      const F2 p = normal_cdf_fast(z, e);
      a = z * p;
      d = slope_sum(p, e, z * both(kInvSqrt2Pi));
      return;
    }
    case GEMM_ACT_GELU_TANH: {
      constexpr float c = -2.0f * kSqrt2OverPi * kLog2e, k = 2.0f * kSqrt2OverPi;
      const F2 q = z * z;
      const F2 s = logistic2(z * fma2(q, both(c * kGeluCubic), both(c)));
      a = z * s;
      d = slope_sum(s, fma2(s * both(-1.0f), s, s), z * fma2(q, both(3.0f * k * kGeluCubic), both(k)));
      return;
    }
    case GEMM_ACT_SILU: {
      const F2 s = logistic2(z * both(-kLog2e));
      a = z * s;
      d = slope_sum(s, fma2(s * both(-1.0f), s, s), z);
      return;
    }
    case GEMM_ACT_SIGMOID:
      a = logistic2(z * both(-kLog2e));
      d = fma2(a * both(-1.0f), a, a);
      return;
    default:
      a = z;
      d = both(1.0f);
      return;
  }
}

// One element, in the arithmetic of its kernel's input type.
template <bool FAST>
__device__ __forceinline__ float activate_one(float z, int act) {
  return FAST ? activate_fast(both(z), act).get().x : activate(z, act);
}

// A piece at a time, with one branch on the activation for all of it (a branch per element
// would keep the elements' exponentials from overlapping).
#define FF_EACH_ACT(X)      \
  X(GEMM_ACT_RELU)          \
  X(GEMM_ACT_GELU)          \
  X(GEMM_ACT_GELU_TANH)     \
  X(GEMM_ACT_SILU)          \
  X(GEMM_ACT_SIGMOID)

template <bool FAST, int N>
__device__ __forceinline__ void activate_all(float (&v)[N], int act) {
  static_assert(!FAST || N % 2 == 0, "pairs");
  switch (act) {
#define FF_ONE(A)                                                                   \
  case A: {                                                                         \
    if constexpr (FAST) {                                                           \
      _Pragma("unroll") for (int i = 0; i < N; i += 2) {                            \
        const float2 y = activate_fast({v[i], v[i + 1]}, A).get();                  \
        v[i] = y.x, v[i + 1] = y.y;                                                 \
      }                                                                             \
    } else {                                                                        \
      _Pragma("unroll") for (int i = 0; i < N; ++i) v[i] = activate(v[i], A);       \
    }                                                                               \
    return;                                                                         \
  }
    FF_EACH_ACT(FF_ONE)
#undef FF_ONE
    default: return;
  }
}

template <bool FAST, int N>
__device__ __forceinline__ void activate_slope_all(const float (&z)[N], int act, float (&a)[N],
                                                   float (&d)[N]) {
  static_assert(!FAST || N % 2 == 0, "pairs");
  switch (act) {
#define FF_ONE(A)                                                                              \
  case A: {                                                                                    \
    if constexpr (FAST) {                                                                      \
      _Pragma("unroll") for (int i = 0; i < N; i += 2) {                                       \
        F2 a2, d2;                                                                             \
        activate_slope_fast({z[i], z[i + 1]}, A, a2, d2);                                      \
        a[i] = a2.get().x, a[i + 1] = a2.get().y;                                              \
        d[i] = d2.get().x, d[i + 1] = d2.get().y;                                              \
      }                                                                                        \
    } else {                                                                                   \
      _Pragma("unroll") for (int i = 0; i < N; ++i) activate_slope(z[i], A, a[i], d[i]);       \
    }                                                                                          \
    return;                                                                                    \
  }
    FF_EACH_ACT(FF_ONE)
#undef FF_ONE
    default: {
#pragma unroll
      for (int i = 0; i < N; ++i) a[i] = z[i], d[i] = 1.0f;
      return;
    }
  }
}
#undef FF_EACH_ACT

}  // namespace ff
}  // namespace gemm_gb300
