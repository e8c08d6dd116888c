// kernels_experts_mx.hip -- products of routed rows with their experts' weights in
// MXFP4 (experts_kernels.h), the rows in bf16 or in MXFP4 too.
#include "experts_kernels.h"

namespace mlora {

// MXFP4: W alone, and the rows of x too
template <bool XMX> using Mx32 = GCfg<128, 32, 32, 32, 4, XMX ? 256 : 128, 4, XMX ? kWMxX : kWMx>;
template <bool XMX> using Mx64 = GCfg<128, 64, 32, 32, 4, XMX ? 256 : 128, 4, XMX ? kWMxX : kWMx>;
typedef GCfg<256, 64, 64, 32, 3, 128, 3, kWMx> Mx64Tall;
typedef GCfg<128, 128, 64, 32, 3, 256, 3, kWMxX> Mx128;

// MXFP4: W's bytes are a quarter, so what a form spends per byte of W decides sooner.
// Streamed, x in bf16 costs a load per 8 columns of 16 rows against W's one per 32:
// 64 or 128 rows per item share them (one token, two of eight experts, 4096 -> 2 x
// 14336: 28.7 us with 64 rows and 4 waves, 35.8 with 32 and 8; 64 tokens, 8 of 64
// experts, 4096 -> 2 x 1024: 58.1 with 128 rows, 62.1 with 64; few items: 32 rows and 2
// waves, 8.2 against 8.7, 32 tokens over 16 experts of 2048 -> 1408). Rows of codes
// cost what W does: 32 rows and 8 waves on long rows, 64 and 4 on short ones (us, with 8 waves
// and with 4, a row per expert: 64 experts of 2048 -> 2 x 1024 34.2 and 28.2, eight of 1024
// -> 2 x 14336 39.8 and 27.4). Long rows gain where few experts have any (two of eight, 4096 ->
// 2 x 14336 27.0 and 28.0; eight of 64, 7168 -> 2 x 1024 17.1 and 21.2; two of eight, 14336 ->
// 28672 not gated 78.1 and 90.9) and lose where all have (eight, 4096 -> 2 x 14336 92.2 and
// 85.9, 4096 -> 28672 not gated 100.7 and 86.5; 64, 8192 -> 2 x 4096 392 and 382).
// Tiles, x in bf16: a wave converts each of its W fragments for its own positions,
// and reads a position fragment per product and row block. Tiles of 256 rows by 64
// positions in waves of 64 x 32 halve the reads (mean 32 rows, 8 experts of 4096 -> 2
// x 14336: 160 us, 175 with 128 rows in waves of 32 x 32; mean 128: 346 and 411, 415
// with 128 positions), where they are enough for the card (16 experts of 2048 -> 1408,
// 96 tiles: 19.2 against 13.9).
// Tiles by rows per expert, us at 8 experts of 4096 -> 2 x 14336: mean 8, 99 streamed, 116
// with 32 positions; 16, 119 with 32, 131 streamed; codes on both sides: 8, 92 streamed and 94;
// 16, 97 with 32, 101 with 64; 32, 104 with 64, 120 with 32; 64, 132 with 128, 136 with 64.
template <bool XMX>
static void launch_mx_t(const ExpertsArgs& a, hipStream_t st) {
  const long long active = std::min(a.E, a.n_pos);
  const double mean = (double)a.n_pos / active;
  const int rows = a.gated ? gated_rows(a.d_out) : a.d_out;
  const bool near = 2ll * a.n_rows * a.d_in < (1ll << 32) && (a.gated ? 1ll * a.d_out : 512ll) * a.d_in < (1ll << 31);
  auto tiles = [&](int br, int bt) { return (long long)(rows + br - 1) / br * std::max(active, a.n_pos / bt + active / 2); };
  if (mean <= 12 || tiles(128, 64) < 64) {
    constexpr int TYPE = XMX ? kXMxX : kXMx;
    if (mean > 12) launch_stream_n<TYPE, 2, 4, 4>(a, st);
    else if (XMX && mean <= 4 && a.d_in >= 4096) launch_stream_n<TYPE, 2, 1, 8>(a, st);
    else if (tiles(64, 16) < 512) launch_stream_n<TYPE, 2, 1, 2>(a, st);
    else if (XMX || mean <= 5 || a.d_in <= 2048) launch_stream_n<TYPE, 4, 1, 4>(a, st);
    else launch_stream_n<TYPE, 8, 1, 4>(a, st);
  } else if (mean <= 20) {
    launch_tile<Mx32<XMX>>(a, st);
  } else if (near && (mean >= 192 || (mean >= 112 && tiles(256, 256) >= 1024))) {
    launch_tile256<XMX ? kWMxX : kWMx>(a, st);
  } else if constexpr (XMX) {
    if (mean <= 48) launch_tile<Mx64<true>>(a, st);
    else launch_tile<Mx128>(a, st);
  } else {
    if (tiles(256, 64) >= 192) launch_tile<Mx64Tall>(a, st);
    else launch_tile<Mx64<false>>(a, st);
  }
}

void launch_experts_mx(const ExpertsArgs& a, hipStream_t st) {
  if (a.x_mx) launch_mx_t<true>(a, st);
  else launch_mx_t<false>(a, st);
}

}  // namespace mlora
