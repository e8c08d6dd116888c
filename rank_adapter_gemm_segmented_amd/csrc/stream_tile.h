// stream_tile.h -- rows of W times a few tokens, W streamed from memory straight
// into MFMA operand registers.
//
// MFMA 16x16 layouts: lane l supplies row l % 16 of either operand; result
// register v of lane l is row 4 (l / 16) + v, column l % 16. Rows are W rows,
// columns tokens.
#pragma once
#include "common.h"

namespace mlora {

__device__ __forceinline__ f32x4_t mfma16e(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
}

constexpr int kXBf16 = 0, kXFp8w = 1, kXF32 = 2;   // element types: bf16, bf16 with an FP8 W, fp32

// acc[r][t] = this wave's part of rows 16 r .. 16 r + 15 times tokens 16 t .. 16 t
// + 15: NW waves take a contiguous part of d_in each, in units of 128 bytes of a
// W row.
//
// A unit is two 16-byte loads per row block: lane group g = l / 16 takes bytes
// 16 g and 64 + 16 g, so a row's 128-byte line is whole within the unit. bf16:
// a load is one 32-column MFMA operand; FP8: 16 columns, two operands (columns
// 16 g and 16 g + 8 of the 64); fp32: 4 columns, four 16x16x4 products.
//
//
// Bound by W's bytes. One unit per wave is in flight, refilled as it is
// consumed: the waves resident on a CU keep over 200 KB requested, and a second
// unit per wave cost as much occupancy as it gave (121 against 113 us, 64 tokens
// over 64 FP8 experts of 4096 -> 2 x 1024). W is loaded without the nontemporal
// mark: a line's two halves come by two loads, and the mark lost the first
// half's line (128 against 113 us). Registers are occupancy here, and occupancy
// is bytes in flight, so W has a uniform base and a 32-bit offset per lane and
// row block (a 64-bit address each: 108 registers, 127 us).
//
// wbase: the first row of W; gated: row blocks alternate between gate and up
// rows, `up` bytes further. wo[]: byte offsets of the lane's row of each (gated:
// pair of) row block, with 16 g; xp[]: the lane's rows of x, at group g's columns.
template <int TYPE, int NR, int NTB, int NW, bool GATED>
__device__ __forceinline__ void stream_product(const char* wbase, long long up, const uint32_t* wo, const char* const* xp,
                                               int d_in, int wave, int g, f32x4_t (&acc)[NR][NTB]) {
  constexpr int EB = TYPE == kXFp8w ? 1 : TYPE == kXF32 ? 4 : 2;   // bytes per W element
  constexpr int XB = TYPE == kXF32 ? 4 : 2;                        // and per x element
  constexpr int UC = 128 / EB;                                     // columns per unit
  constexpr int XL = XB / EB;                                      // x loads per W load
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int t = 0; t < NTB; ++t) acc[r][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  u32x4_t w[2][NR], x[2][XL][NTB];
  auto load = [&](int u) {                                         // unit u, whole
    const char* wu = wbase + (long long)u * 128;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int r = 0; r < NR; ++r) w[h][r] = ld16((GATED && (r & 1) ? wu + up : wu) + wo[GATED ? r / 2 : r] + 64 * h);
#pragma unroll
      for (int i = 0; i < XL; ++i)
#pragma unroll
        for (int t = 0; t < NTB; ++t) x[h][i][t] = ld16(xp[t] + (long long)u * (UC * XB) + h * (UC / 2 * XB) + 16 * i);
    }
  };
  auto multiply = [&]() {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int t = 0; t < NTB; ++t) {
          if constexpr (TYPE == kXBf16) {
            acc[r][t] = mfma16e(w[h][r], x[h][0][t], acc[r][t]);
          } else if constexpr (TYPE == kXFp8w) {
            acc[r][t] = mfma16e(e4m3x8_bf16(w[h][r].x, w[h][r].y), x[h][0][t], acc[r][t]);
            acc[r][t] = mfma16e(e4m3x8_bf16(w[h][r].z, w[h][r].w), x[h][XL - 1][t], acc[r][t]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[h][r][i]), __uint_as_float(x[h][0][t][i]),
                                                               acc[r][t], 0, 0, 0);
          }
        }
  };
  const int nu = d_in / UC;                                        // whole units
  const int ub = nu * wave / NW, ue = nu * (wave + 1) / NW;        // this wave's
  if (ub < ue) {   // uniform
    load(ub);
    for (int u = ub; u + 1 < ue; ++u) {
      multiply();
      load(u + 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    multiply();
  }
  if (nu * UC < d_in && wave == NW - 1) {   // uniform: the columns behind the last whole unit
    const char* wu = wbase + (long long)nu * 128;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = nu * UC + h * UC / 2 + 16 / EB * g < d_in;   // (d_in is a multiple of 16 bytes of W)
#pragma unroll
      for (int r = 0; r < NR; ++r)
        w[h][r] = in ? ld16((GATED && (r & 1) ? wu + up : wu) + wo[GATED ? r / 2 : r] + 64 * h) : zero_u32x4();
#pragma unroll
      for (int i = 0; i < XL; ++i)
#pragma unroll
        for (int t = 0; t < NTB; ++t)
          x[h][i][t] = in ? ld16(xp[t] + (long long)nu * (UC * XB) + h * (UC / 2 * XB) + 16 * i) : zero_u32x4();
    }
    multiply();
  }
}

}  // namespace mlora
