// kernels_experts.hip -- products of routed rows with their experts' weights
// (experts_kernels.h) in bf16, fp32 and FP8, and the weighted way back: the fp32
// products of every sorted position followed by k_combine, out[t] = residual[t] + sum_j
// w[t][j] z[position[t][j]].
#include "experts_kernels.h"

namespace mlora {

// ---------------------------------------------------------------------------
// Way back: a token's rows weighted, summed in slot order and added to the
// residual, in fp32, one rounding. A thread takes 4 columns of one token.
//
// The products stay in fp32 between the two kernels: with bf16 rows a token's sum
// would carry top_k more roundings. A prefill batch (8192 rows of 4096) moves 200
// MB here, 37 to 47 us from run to run (5.4 to 4.3 TB/s), of about 900 in all; a
// decode batch 6 to 7 us, mostly the launch.
// ---------------------------------------------------------------------------
template <typename E_>
__global__ __launch_bounds__(256) void k_combine(CombineArgs a) {
  const int t = blockIdx.x, c = 4 * (blockIdx.y * 256 + threadIdx.x);
  if (c >= a.d_out) return;
  const bool whole = c + 4 <= a.d_out;
  float o[4] = {0.f, 0.f, 0.f, 0.f};
  const long long at = (long long)t * a.d_out + c;
  const int pitch = f32_pitch(a.d_out);
  for (int j = 0; j < a.k; ++j) {
    const int p = a.position[(long long)t * a.k + j];
    const float w = a.weight[(long long)t * a.k + j];
    if (p < 0 || p >= a.n_pos) continue;   // uniform: no expert in this slot
    const f32x4_t v = *(const f32x4_t*)(a.part + (long long)p * pitch + c);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = fmaf(w, v[i], o[i]);
  }
  float r[4] = {0.f, 0.f, 0.f, 0.f};
  if (a.residual) {
    if (!whole) {
      #pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < a.d_out) r[i] = elem_f32<E_>(a.residual, at + i);
    } else if constexpr (sizeof(E_) == 2) {
      const u32x2_t v = *(const u32x2_any*)((const uint16_t*)a.residual + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = __uint_as_float((i & 1) ? (v[i / 2] & 0xffff0000u) : (v[i / 2] << 16));
    } else {
      const f32x4_t v = *(const f32x4_any*)((const float*)a.residual + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = v[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] += r[i];
  }
  if (whole) {
    if constexpr (sizeof(E_) == 2)
      *(u32x2_any*)((uint16_t*)a.out + at) = u32x2_t{cvt_pk_bf16(o[0], o[1]), cvt_pk_bf16(o[2], o[3])};
    else *(f32x4_any*)((float*)a.out + at) = f32x4_t{o[0], o[1], o[2], o[3]};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < a.d_out) {
        if constexpr (sizeof(E_) == 2) ((uint16_t*)a.out)[at + i] = f32_to_bf16_bits(o[i]);
        else ((float*)a.out)[at + i] = o[i];
      }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// Shape of the streaming form. Few items (a token or two): 32 rows and 8 waves
// each, so that the card is full (one token, two of eight experts of 4096 -> 2
// x 14336: 79.5 us against 85.6 with 64 rows and 4 waves); so too with more
// positions where the items are fewer than the CUs (75 tokens, four of eight
// experts, 4864 -> 2 x 305: 27.2 us against 36.3; 102 tokens of five experts, 4720
// -> 335: 17.1 against 26.0; with 256 items, 24 tokens of eight experts, 4096 ->
// 2048, 29.9 against 27.5). Otherwise 64 rows and 4 waves (64 tokens, 64 FP8
// experts: 113 us against 134). Positions per item by the mean per expert, with
// room for uneven ones; FP8 keeps to 16 longer, its x operands taking twice the
// registers per byte of W.
template <int TYPE>
static void launch_stream(const ExpertsArgs& a, hipStream_t st) {
  const long long active = std::min(a.E, a.n_pos);
  const long long row_tiles = ((a.gated ? gated_rows(a.d_out) : a.d_out) + 63) / 64;
  const double mean = (double)a.n_pos / active;
  const int nt = mean <= (TYPE == kXFp8w ? 10 : 4) ? 1 : mean <= 24 ? 2 : 4;   // blocks of 16 positions
  const long long items = row_tiles * std::max(active, a.n_pos / (16 * nt) + active / 2);
  if (items < 256 || (row_tiles * active < 2048 && mean <= 4)) {
    if (nt == 1) launch_stream_n<TYPE, 2, 1, 8>(a, st);
    else if (nt == 2) launch_stream_n<TYPE, 2, 2, 8>(a, st);
    else launch_stream_n<TYPE, 2, 4, 8>(a, st);
  } else {
    if (nt == 1) launch_stream_n<TYPE, 4, 1, 4>(a, st);
    else if (nt == 2) launch_stream_n<TYPE, 4, 2, 4>(a, st);
    else launch_stream_n<TYPE, 4, 4, 4>(a, st);
  }
}

template <bool W8> using Tile128 = GCfg<128, 128, 64, 32, 3, W8 ? 128 : 64, W8 ? 2 : 3, W8 ? kWFp8 : kWBf16>;
template <bool W8> using Tile64 = GCfg<128, 64, 32, 32, 4, W8 ? 128 : 64, 4, W8 ? kWFp8 : kWBf16>;
typedef GCfg<128, 32, 32, 32, 5, 64, 5> Tile32;

// Form by the rows per expert. Up to two (FP8: twenty), the streaming form; it
// also takes fp32 and what has too few tiles for the card: fewer than 256 of 32
// positions (24 tokens, two of eight experts, 4096 -> 2048, 128 tiles: 27.6 us
// streamed, 33.8 tiled), fewer than 64 of more (FP8,
// 100 tokens over 4 experts, 32 tiles: 12.8 us streamed, 20.7 tiled; two of eight
// experts, 100 tokens, 4096 -> 1024, 64 tiles: 22.4 and 24.1; 400 tokens, 4096 -> 2 x
// 512, 80 tiles: 43.1 and 35.1). Then tiles of 32, 64,
// 128 and 256 positions, the smallest that holds most experts' rows: W, which
// decides the time up to about 100 rows, is then read once, and the tile's
// rings keep more of it requested than registers can. Two of eight experts,
// 4096 -> 2 x 14336, bf16, us: 16 tokens 316 with 32 positions, 337 streamed; 64
// tokens 322 with 64, 390 streamed; 128 tokens 342 with 64, 360 with 128; 256
// tokens 378 with 128, 451 with 64; 512 tokens 532 with 256, 557 with 128. FP8
// halves W, not the tile's work: 64 tokens 201 streamed, 222 with 64 positions;
// 128 tokens 230 with 64, 284 streamed. (FP8 stages are 128 columns deep: 237
// with 64.)
template <bool W8>
static void launch_bf16(const ExpertsArgs& a, hipStream_t st) {
  const long long active = std::min(a.E, a.n_pos);
  const double mean = (double)a.n_pos / active;
  const int rows = a.gated ? gated_rows(a.d_out) : a.d_out;
  // the largest tile addresses x and its rows of W by 32-bit offsets
  const bool near = 2ll * a.n_rows * a.d_in < (1ll << 32) && (a.gated ? 1ll * a.d_out : 512ll) * a.d_in < (1ll << 31);
  const long long tiles256 = (rows + 255) / 256 * (a.n_pos / 256 + active / 2);   // of about this many
  const int bt = mean <= 8 ? 32 : mean <= 48 ? 64 : 128;
  const long long tiles = (rows + 127) / 128 * std::max(active, a.n_pos / bt + active / 2);
  if (mean <= (W8 ? 20 : 2) || tiles < (mean <= 8 ? 256 : 64)) return launch_stream<W8 ? kXFp8w : kXBf16>(a, st);
  if constexpr (!W8) {
    if (mean <= 8) return launch_tile<Tile32>(a, st);
    if (near && (mean >= 192 || (mean >= 112 && tiles256 >= 1024))) return launch_tile256<kWBf16>(a, st);
  }
  if (mean <= 48) launch_tile<Tile64<W8>>(a, st);
  else launch_tile<Tile128<W8>>(a, st);
}

void launch_experts(const ExpertsArgs& a, bool bf16, hipStream_t st) {
  if (a.n_pos <= 0) return;
  if (!bf16) launch_stream<kXF32>(a, st);
  else if (a.w_mx) launch_experts_mx(a, st);
  else if (a.w_scale) launch_bf16<true>(a, st);
  else launch_bf16<false>(a, st);
}

void launch_combine(const CombineArgs& a, bool bf16, hipStream_t st) {
  const dim3 grid(a.T, (a.d_out + 1023) / 1024);
  if (bf16) hipLaunchKernelGGL(k_combine<uint16_t>, grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL(k_combine<float>, grid, dim3(256), 0, st, a);
}

}  // namespace mlora
