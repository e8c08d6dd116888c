// epilogue.h -- bias, activation, gate and residual applied to a product
// before its single rounding.
//
//   plain:  y = act(z + b) + residual                 z has d_out columns, y too
//   gated:  y = act(g + b_g) * (u + b_u) + residual   z = [g; u], y has d_out / 2 columns
//
// All of it in fp32 on the accumulators; only y is rounded.
//
// A gated product needs feature f's gate row f and up row d_out / 2 + f in one
// lane. The kernels therefore walk W in virtual rows: blocks of 32 hold 16
// features, their gate rows first, then their up rows. In the 32x32 MFMA
// result layout (register v of a lane is row 8 (v / 4) + 4 (lane / 32) + v % 4)
// registers v and v + 8 of a lane are then one feature's pair, and in the 16x16
// layout two consecutive row blocks are.
#pragma once
#include "../../include/mlora.h"
#include "common.h"

namespace mlora {

// What follows the product. Bias and residual are in the element type; the
// residual has y's shape and may be y itself (each element is read by the
// thread that writes it, before it does).
struct EpiView {
  const void* bias;       // [d_out] or null
  const void* residual;   // [rows of y, columns of y] or null
  int act;                // MLORA_ACT_* without the gate flag
};

// Virtual rows of a gated product over d_out rows of W (whole blocks of 32).
__host__ __device__ __forceinline__ int gated_rows(int d_out) { return (d_out / 2 + 15) / 16 * 32; }

// Feature of virtual row v, and its row of W (features past the last one are
// clamped to it; they are never stored).
__device__ __forceinline__ int gated_feature(int v) { return (v >> 5) * 16 + (v & 15); }
__device__ __forceinline__ int gated_wrow(int v, int d_out) {
  const int F = d_out / 2;
  return ((v >> 4) & 1) * F + min(gated_feature(v), F - 1);
}
template <bool GATED>
__device__ __forceinline__ int wrow_of(int v, int d_out) {
  return GATED ? gated_wrow(v, d_out) : min(v, d_out - 1);
}

// Activations. FAST (bf16 outputs): the hardware exponential and reciprocal. The
// exponential's argument is rounded once as it is scaled by log2(e), so the result
// is off by about (|t| + 4) 2^-24 relative, t the argument: below 2^-17 up to 88
// (bf16's half step is 2^-8). Past t = -88 (and where the reciprocal's result
// would be subnormal) it is 0 in place of less than 1e-35. fp32 outputs take the
// library's exponential and a full division. tanh(u) is written through the
// exponential: (1 + tanh u) / 2 = 1 / (1 + exp(-2 u)), and 1 + erf(a) as erfc(-a):
// the sums cancel where z is far below 0 (1 + erf was 4% off at z = -5 and 0 from
// -5.6 on, in fp32). NaN passes through.
template <bool FAST>
__device__ __forceinline__ float sigmoid_times(float z, float t) {   // z / (1 + exp(-t))
  if constexpr (FAST) {
    return z * __builtin_amdgcn_rcpf(1.0f + __expf(-t));
  } else {
    return z / (1.0f + expf(-t));
  }
}
// gelu, z Phi(z) with Phi the normal distribution. FAST: Phi(-x) = exp(-x^2 / 2) R(x)
// for x = |z|, and R, which falls smoothly from 1/2 towards 1 / (x sqrt(2 pi)), as
// t P(t) with t = 1 / (1 + 0.265 x): a least-maximum fit of P, within 6.5e-7 of R
// everywhere (about 11 roundings of fp32; the library's erfcf in its place: 975 ->
// 1767 us, 4096 tokens, 4096 -> 2 x 14336 gated).
template <bool FAST>
__device__ __forceinline__ float gelu(float z) {
  if constexpr (FAST) {
    const float x = fabsf(z), t = __builtin_amdgcn_rcpf(fmaf(0.265f, x, 1.0f));
    float p = -0.0677952636f;
    p = fmaf(p, t, 0.195301499f);
    p = fmaf(p, t, -0.066401835f);
    p = fmaf(p, t, 0.142520221f);
    p = fmaf(p, t, 0.0829368182f);
    p = fmaf(p, t, 0.107838527f);
    p = fmaf(p, t, 0.105599717f);
    const float q = p * t * __builtin_amdgcn_exp2f(-0.72134752f * x * x);   // (log2(e) / 2)
    return z * (z < 0.f ? q : 1.0f - q);
  } else {
    return 0.5f * z * erfcf(z * -0.70710678118654752f);
  }
}
template <bool FAST>
__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {   // uniform
    case MLORA_ACT_RELU: return z < 0.f ? 0.f : z;
    case MLORA_ACT_SILU: return sigmoid_times<FAST>(z, z);
    case MLORA_ACT_GELU: return gelu<FAST>(z);
    case MLORA_ACT_GELU_TANH: return sigmoid_times<FAST>(z, 1.5957691216057308f * fmaf(0.044715f * z * z, z, z));
    default: return z;
  }
}

// The activation of N values, chosen once for all of them.
template <bool FAST, int N>
__device__ __forceinline__ void activate_n(float (&z)[N], int act) {
  if (act == MLORA_ACT_NONE) return;   // uniform
  if (act == MLORA_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = activate<FAST>(z[i], MLORA_ACT_SILU);
  } else if (act == MLORA_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = activate<FAST>(z[i], MLORA_ACT_RELU);
  } else if (act == MLORA_ACT_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = activate<FAST>(z[i], MLORA_ACT_GELU_TANH);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = activate<FAST>(z[i], MLORA_ACT_GELU);
  }
}

// Vectors of bf16 or fp32 elements at any element's address: rows of y need not
// start on a 16-byte boundary (a width that is no multiple of 8), and global
// memory takes wide accesses at any address (2087 tokens, 1072 -> 13740 with a
// residual: 158 us, 214 by single elements).
typedef u32x4_t u32x4_any __attribute__((aligned(2)));
typedef u32x2_t u32x2_any __attribute__((aligned(2)));
typedef f32x4_t f32x4_any __attribute__((aligned(4)));

// One element of bias or residual.
template <typename E>
__device__ __forceinline__ float elem_f32(const void* p, long long i);
template <>
__device__ __forceinline__ float elem_f32<uint16_t>(const void* p, long long i) {
  return bf16_bits_to_f32(((const uint16_t*)p)[i]);
}
template <>
__device__ __forceinline__ float elem_f32<float>(const void* p, long long i) {
  return ((const float*)p)[i];
}

}  // namespace mlora
