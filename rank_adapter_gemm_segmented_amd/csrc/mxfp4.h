// mxfp4.h -- microscaled 4-bit floating point: codes, scales and their layout.
//
// A row of d columns (a multiple of 32) is cut into blocks of 32. A block has 32
// E2M1 codes (sign, 2 exponent bits, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6),
// two to a byte with the even column in the low half, and one scale byte s that
// stands for 2^(s - 127) (255: NaN). A value has two significant bits, so it is
// exact in bf16 with its scale in (s <= 252; beyond bf16's range it is infinite).
//
// Codes are [rows, d / 2]. Scales are [ceil(d / 128), rows, 4]: plane p holds one
// dword per row, the scales of columns 128 p .. 128 p + 127, consecutive rows side
// by side. Tiles read scales of many rows at a few columns: 32 rows of a plane are
// one 128-byte line, and [rows, d / 32] would be 32 lines.
#pragma once
#include "../../include/mlora.h"
#include "common.h"

namespace mlora {

constexpr int kMxBlock = 32;     // columns per scale
constexpr int kMxPlane = 128;    // columns per plane of scales

__host__ __device__ __forceinline__ int mx_planes(int d) { return (d + kMxPlane - 1) / kMxPlane; }

// A scale byte as the float whose exponent it is, which the conversions and their
// hardware take (0 for 2^-127 and infinity for NaN included: they look at the
// exponent field alone; checked on all 256 bytes).
__device__ __forceinline__ float mx_scale(uint32_t s) { return __uint_as_float(s << 23); }
// Byte i of a dword of scales, as such a float.
__device__ __forceinline__ float mx_scale_at(uint32_t w, int i) { return __uint_as_float(((w >> (8 * i)) & 0xffu) << 23); }

// Eight codes (a dword) times their scale -> eight bf16, exact.
__device__ __forceinline__ u32x4_t mx_bf16x8(uint32_t w, float scale) {
  u32x4_t r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  return r;
}

// Products of codes with codes. Lane l of the wave supplies 32 columns of row l %
// 32 (16x16: l % 16), one block with one scale: byte SA of sa, byte SB of sb. The
// block of lane group l / 32 (l / 16) is whichever both operands agree on. Results
// as those of the bf16 products of the same shape; products are exact, sums fp32.
typedef int i32x8_t __attribute__((ext_vector_type(8)));
__device__ __forceinline__ i32x8_t mx_operand(u32x4_t c) {
  return i32x8_t{(int)c.x, (int)c.y, (int)c.z, (int)c.w, 0, 0, 0, 0};   // (a 4-bit operand is its first four)
}
template <int SA, int SB>
__device__ __forceinline__ f32x16_t mfma32mx(u32x4_t a, uint32_t sa, u32x4_t b, uint32_t sb, f32x16_t c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(a), mx_operand(b), c, 4, 4, SA, (int)sa, SB, (int)sb);
}
// (scales in byte 0)
__device__ __forceinline__ f32x4_t mfma16mx(u32x4_t a, uint32_t sa, u32x4_t b, uint32_t sb, f32x4_t c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(a), mx_operand(b), c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// ---- quantisation (kernels_mxfp4.hip) -------------------------------------------
struct QuantArgs {
  const void* x;        // [batch, rows, d] bf16 or fp32
  uint8_t* codes;       // [batch, rows, d / 2]
  uint8_t* scale;       // [batch, planes, rows, 4]
  int batch, rows, d;
};
void launch_quantize(const QuantArgs& a, bool bf16, hipStream_t st);
struct DequantArgs {
  const uint8_t* codes;
  const uint8_t* scale;
  void* y;
  int batch, rows, d;
};
void launch_dequantize(const DequantArgs& a, bool bf16, hipStream_t st);

}  // namespace mlora
