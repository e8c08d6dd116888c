// kernels_mxfp4.hip -- matrices to microscaled 4-bit floating point and back.
//
// A block of 32 columns with largest magnitude m: scale 2^e with e = floor(log2 m)
// - 2, the exponent of m less that of E2M1's largest value (at least -127), codes
// x / 2^e rounded to nearest even, magnitudes past 6 to 6 (the conversion of the
// hardware rounds and saturates so; both checked on ties, subnormals and past the
// ends). A block that holds a NaN or an infinity has scale 255 and codes 0: all of
// it stands for NaN.
//
// Bound by bytes: 2 or 4 read and 17 / 32 written per value. A 14336 x 4096 fp32 matrix
// takes 57 us there (4.7 TB/s), 87 back, as long as a copy of the matrix, which writes as
// much, and 139 for both in turn, with four sets of operands (123 with one, of which the
// caches keep a part); in bf16 33.5, 33.7 (a copy 45) and 61. 64 x 4096 in bf16 2.5 us each.
// (With nontemporal loads and stores 184 us for both in fp32: a row's 32 bytes per lane
// leave by two stores, and the mark writes half lines.)
#include "mxfp4.h"

namespace mlora {

// 16 lanes take the 128 columns of a plane of one row, 8 columns each: four lanes
// hold a block. A workgroup takes 16 rows, so that the scales it writes per plane
// are 64 bytes side by side, and the planes blockIdx.y, + gridDim.y, ...
constexpr int kQThreads = 256, kQRows = kQThreads / 16;

__device__ __forceinline__ uint32_t max_of_4_lanes(uint32_t v) {   // quad_perm
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0xb1, 0xf, 0xf, false));
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x4e, 0xf, 0xf, false));
}

template <typename E>
__global__ __launch_bounds__(kQThreads) void k_quantize(QuantArgs a) {
  const int tid = threadIdx.x, c16 = tid % 16;
  const int row = blockIdx.x * kQRows + tid / 16;
  const bool row_ok = row < a.rows;
  const int planes = mx_planes(a.d);
  const long long r = (long long)blockIdx.z * a.rows + min(row, a.rows - 1);
  for (int p = blockIdx.y; p < planes; p += gridDim.y) {   // uniform
    const int col = p * kMxPlane + 8 * c16;
    const bool in = col < a.d;
    const E* src = (const E*)a.x + r * a.d + (in ? col : 0);
    float v[8];
    uint32_t m = 0u;
    if constexpr (sizeof(E) == 2) {
      const u32x4_t w = ld16(src);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float((i & 1) ? (w[i / 2] & 0xffff0000u) : (w[i / 2] << 16));
    } else {
      const f32x4_t lo = *(const f32x4_t*)src, hi = *(const f32x4_t*)(src + 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < 4 ? lo[i] : hi[i - 4];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    m = max_of_4_lanes(m);
    const uint32_t e = m >> 23;                            // biased exponent (0: zero or subnormal)
    const bool bad = e == 255u;
    uint32_t s = bad ? 255u : e > 2u ? e - 2u : 0u;
    const float sc = mx_scale(s);
    uint32_t q = 0u;
    if (!bad) {
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], sc, 0);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], sc, 1);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], sc, 2);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], sc, 3);
    }
    if (!in) s = 127u;                                     // (behind the last block)
    // the row's four scales meet in its lane 0
    uint32_t w = s << (8 * (c16 / 4));
    w |= (uint32_t)__shfl_xor((int)w, 4, kWave);
    w |= (uint32_t)__shfl_xor((int)w, 8, kWave);
    if (row_ok) {
      if (in) *(uint32_t*)(a.codes + (r * a.d + col) / 2) = q;
      if (c16 == 0) *(uint32_t*)(a.scale + 4 * (((long long)blockIdx.z * planes + p) * a.rows + row)) = w;
    }
  }
}

// The same cut: 8 codes to 8 values per lane.
template <typename E>
__global__ __launch_bounds__(kQThreads) void k_dequantize(DequantArgs a) {
  const int tid = threadIdx.x, c16 = tid % 16;
  const int row = blockIdx.x * kQRows + tid / 16;
  if (row >= a.rows) return;
  const int planes = mx_planes(a.d);
  const long long r = (long long)blockIdx.z * a.rows + row;
  for (int p = blockIdx.y; p < planes; p += gridDim.y) {
    const int col = p * kMxPlane + 8 * c16;
    if (col >= a.d) continue;
    const uint32_t q = *(const uint32_t*)(a.codes + (r * a.d + col) / 2);
    const uint32_t w = *(const uint32_t*)(a.scale + 4 * (((long long)blockIdx.z * planes + p) * a.rows + row));
    const float sc = mx_scale_at(w, c16 / 4);
    if constexpr (sizeof(E) == 2) {
      *(u32x4_t*)((uint16_t*)a.y + r * a.d + col) = mx_bf16x8(q, sc);
    } else {
      typedef float f32x2v_t __attribute__((ext_vector_type(2)));
      const f32x2v_t v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, sc, 0), v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, sc, 1),
                     v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, sc, 2), v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, sc, 3);
      float* y = (float*)a.y + r * a.d + col;
      *(f32x4_t*)y = f32x4_t{v0.x, v0.y, v1.x, v1.y};
      *(f32x4_t*)(y + 4) = f32x4_t{v2.x, v2.y, v3.x, v3.y};
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// Workgroups along the planes: one plane each while that fills the card, then
// several.
static dim3 quant_grid(int batch, int rows, int d) {
  const int rg = (rows + kQRows - 1) / kQRows, planes = mx_planes(d);
  const long long all = (long long)rg * planes * batch;
  const int per = all > 8192 ? 4 : 1;
  return dim3(rg, (planes + per - 1) / per, batch);
}

void launch_quantize(const QuantArgs& a, bool bf16, hipStream_t st) {
  const dim3 grid = quant_grid(a.batch, a.rows, a.d);
  if (bf16) hipLaunchKernelGGL(k_quantize<uint16_t>, grid, dim3(kQThreads), 0, st, a);
  else hipLaunchKernelGGL(k_quantize<float>, grid, dim3(kQThreads), 0, st, a);
}

void launch_dequantize(const DequantArgs& a, bool bf16, hipStream_t st) {
  const dim3 grid = quant_grid(a.batch, a.rows, a.d);
  if (bf16) hipLaunchKernelGGL(k_dequantize<uint16_t>, grid, dim3(kQThreads), 0, st, a);
  else hipLaunchKernelGGL(k_dequantize<float>, grid, dim3(kQThreads), 0, st, a);
}

}  // namespace mlora
