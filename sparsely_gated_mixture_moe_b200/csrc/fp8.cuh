// The 8-bit format of the library's fp8 operators: e4m3 values with one fp32 scale for each
// block of 128 consecutive values of a row (activations) or 128 x 128 values (weights).
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {

constexpr int kScaleBlock = 128;
constexpr float kE4m3Max = 448.0f;
// A block's largest magnitude is taken as at least this: its scale is then a normal fp32
// number, and a block of zeros gives q = 0.
constexpr float kAmaxFloor = 448.0f * 1.17549435e-38f;  // 448 * 2^-126

// Maximum that keeps a NaN from either side: a NaN anywhere in a block reaches its scale.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// max(|a|, |b|, |c|), keeping a NaN.
__device__ __forceinline__ float amax3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// GELU of 2 N values in place, z Phi(z) = max(z, 0) - a Phi(-a) with a = |z|, and Phi(-a) =
// exp(-a^2 / 2) P(a): P = Phi(-a) exp(a^2 / 2) falls smoothly from 1/2 and is a polynomial of
// degree 9 here, fitted on [0, 6] so that the largest error of a exp(-a^2 / 2) P(a) is least (a
// linear program over Chebyshev polynomials).  |error| <= 4.6e-7, and 1.2e-5 |z|, below the
// e4m3 rounding that follows at any scale.  One exponential a value and no reciprocal: with
// the rational form of gelu2_as7126 (two special-function operations a value) the special
// functions alone took as long as the products of an up-projection 1024 deep.  The N pairs go
// through each step together, so that their chains of dependent operations overlap.  a is held at 8 for P (from there exp(-a^2 / 2) < 2e-14 leaves
// nothing); the exponential's argument is not, so that a NaN stays one.
template <int N>
__device__ __forceinline__ void gelu_poly(float (&v)[2 * N]) {
  static_assert(N <= 9, "one exponential pair a step");
  constexpr float kC[10] = {-0.49998804926872253f, 0.39874154329299927f,   -0.24880152940750122f,
                            0.12939025461673737f,  -0.05621607229113579f,  0.019581008702516556f,
                            -0.005101285874843597f, 0.0009078671573661268f, -9.652071457821876e-05f,
                            4.564738446788397e-06f};  // -P
  uint64_t a[N], p[N], e[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    a[i] = f2_pack(fminf(fabsf(v[2 * i]), 8.0f), fminf(fabsf(v[2 * i + 1]), 8.0f));
    p[i] = f2_splat(kC[9]);
    const uint64_t z = f2_pack(v[2 * i], v[2 * i + 1]);
    e[i] = f2_mul(z, f2_mul(z, f2_splat(-0.72134752044448170f)));  // -(z^2 / 2) log2(e)
  }
#pragma unroll
  for (int c = 8; c >= 0; --c) {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = f2_fma(p[i], a[i], f2_splat(kC[c]));
    if (c >= 9 - N) {  // an exponential pair between two steps
      float q0, q1;
      f2_unpack(e[c - (9 - N)], q0, q1);
      e[c - (9 - N)] = f2_pack(ex2_ftz(q0), ex2_ftz(q1));
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) p[i] = f2_mul(p[i], e[i]);
#pragma unroll
  for (int i = 0; i < N; ++i)
    f2_unpack(f2_fma(a[i], p[i], f2_pack(fmaxf(v[2 * i], 0.0f), fmaxf(v[2 * i + 1], 0.0f))), v[2 * i],
              v[2 * i + 1]);
}

// Scale of a block whose largest magnitude is amax (already floored).
__device__ __forceinline__ float block_scale(float amax) { return amax / kE4m3Max; }

// Two / four values, already divided by their scale, as e4m3 (nearest even, saturated at
// +-448; NaN stays NaN); the first value in the lowest byte.
__device__ __forceinline__ uint32_t pack_e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  return pack_e4m3x2(a, b) | (pack_e4m3x2(c, d) << 16);
}

// 448 v / amax with a correctly rounded quotient.  7/8 = 448/512 keeps a 16-bit v exact and
// cannot overflow; the 512 is a power of two.  A 16-bit value over a 16-bit maximum often
// lies exactly midway between two e4m3 values, and a product with the rounded reciprocal
// would tip such a tie either way.
__device__ __forceinline__ float exact_quotient(float v, float amax) {
  return __fdiv_rn(v * 0.875f, amax) * 512.0f;
}

// Eight consecutive values of a row of T as fp32, and back (one rounding for bf16).
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// Largest magnitude over the 16 lanes that hold one block of 128 (8 values a lane).  Every
// lane of the warp must call it.
__device__ __forceinline__ float amax_half_warp(float m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

}  // namespace moe
