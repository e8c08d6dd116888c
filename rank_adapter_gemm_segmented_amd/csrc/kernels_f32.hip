// kernels_f32.hip -- fp32 multi-LoRA linear on the gfx950 vector ALUs.
//
// Same layer as the bf16 path (the LoRA forward of "Multi-LoRA Serving in
// Practice", section "Core Principle", per adapter segment), computed and
// stored in fp32. It serves small fp32 layers; the large configurations are
// bf16 and run on MFMA.
#include "common.h"
#include "launch.h"

namespace mlora {

// v of sorted position p for rank rows j0 .. j0 + kF32Rows - 1 below r, by one wave:
// the 64 lanes split d_in (16-byte loads, lane l at k = 4l + 256 i), every load of
// the group in flight; each row's partial sums are added across the wave with
// xor shuffles (a fixed order).
constexpr int kF32Rows = 8;
__device__ __forceinline__ void shrink_rows(const LinearArgs& a, int p, const float* __restrict__ Aa, int j0, int r) {
  const int lane = threadIdx.x % kWave, d_in = a.d_in;   // d_in: a multiple of 4
  int row = a.sv.token_index ? a.sv.token_index[p] : p;
  row = min(max(row, 0), a.T - 1);
  const float* xr = (const float*)a.x + (long long)row * d_in;
  float acc[kF32Rows];
#pragma unroll
  for (int i = 0; i < kF32Rows; ++i) acc[i] = 0.f;
  for (int k = 4 * lane; k < d_in; k += 4 * kWave) {
    const f32x4_t xv = *(const f32x4_t*)(xr + k);
    f32x4_t av[kF32Rows];
#pragma unroll
    for (int i = 0; i < kF32Rows; ++i) av[i] = *(const f32x4_t*)(Aa + (long long)min(j0 + i, r - 1) * d_in + k);
#pragma unroll
    for (int i = 0; i < kF32Rows; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[i] = fmaf(av[i][c], xv[c], acc[i]);
  }
#pragma unroll
  for (int i = 0; i < kF32Rows; ++i) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) acc[i] += __shfl_xor(acc[i], off, kWave);
  }
  if (lane < kF32Rows && j0 + lane < r) {
    float v = acc[0];
#pragma unroll
    for (int i = 1; i < kF32Rows; ++i) v = lane == i ? acc[i] : v;
    a.v_part[(long long)p * a.r_ws + j0 + lane] = v;
  }
}

// v_part[0][p][j] = sum_k A_a[j,k] x[row(p),k]; one workgroup per segment,
// which also writes its positions' entries of the position table.
// Wave w takes positions ps + w, ps + w + 4, ...
__global__ __launch_bounds__(256) void k_shrink_f32(LinearArgs a) {
  const int s = blockIdx.x;
  const SegView& sv = a.sv;
  const int S = seg_count(sv);
  if (s >= S) return;
  const int ps = max(sv.seg_start[s], 0);
  const int pe = min(sv.seg_start[s + 1], a.T);
  if (pe <= ps) return;
  int r;
  const int ad = seg_adapter_checked(sv, a.pv, s, &r);
  // the position table: {segment, adapter or -1, rank, scale bits}
  for (int p = ps + (int)threadIdx.x; p < pe; p += 256)
    a.pos_info[p] = make_int4(s, ad, ad >= 0 ? r : 0, __float_as_int(ad >= 0 ? sv.seg_scale[s] : 0.f));
  if (ad < 0) return;
  const int wave = threadIdx.x / kWave;
  const float* __restrict__ Aa = (const float*)a.pv.base + (long long)ad * a.pv.slot_elems;
  for (int p = ps + wave; p < pe; p += 4)
    for (int j0 = 0; j0 < r; j0 += kF32Rows) shrink_rows(a, p, Aa, j0, r);
}

// The same by position, for calls with an epilogue: a wave per position and group
// of rank rows, which finds its segment itself, so that a long segment spreads
// over the card. v has the bits of k_shrink_f32.
__global__ __launch_bounds__(256) void k_shrink_f32_wide(LinearArgs a) {
  const SegView& sv = a.sv;
  const int p = blockIdx.x * 4 + threadIdx.x / kWave, j0 = blockIdx.y * kF32Rows;
  if (p >= a.T) return;   // (no barrier)
  const int S = seg_count(sv);
  const int s = S > 0 ? min(max(find_segment(sv.seg_start, S, p), 0), S - 1) : 0;
  int r = 0, ad = -1;
  if (S > 0 && sv.seg_start[s] <= p && p < sv.seg_start[s + 1]) ad = seg_adapter_checked(sv, a.pv, s, &r);
  if (j0 == 0 && threadIdx.x % kWave == 0)
    a.pos_info[p] = make_int4(s, ad, ad >= 0 ? r : 0, __float_as_int(ad >= 0 ? sv.seg_scale[s] : 0.f));
  if (ad < 0 || j0 >= r) return;
  shrink_rows(a, p, (const float*)a.pv.base + (long long)ad * a.pv.slot_elems, j0, r);
}

// Tile: 16 output features x 16 sorted positions, one output per thread
// (tx = feature, ty = position), so a small layer spreads over many
// workgroups: the 256-wide layer of 16 tokens runs 16 of them (64-feature
// tiles ran 4, each issuing ~5000 LDS reads per wave: 10 us). d_in is walked
// in chunks of kF32KB columns with the next chunk's loads in flight in
// registers while the current one is multiplied from LDS; the chunk is wide
// (4 W and 4 x loads of 16 bytes per thread, all in flight at once), so a
// small layer loads everything in one round trip.
constexpr int kF32KB = 256;
constexpr int kF32Feat = 16;
constexpr int kF32FusedRank = 16;   // largest rank of the fused shrink (two groups of 8)

// EPI: what follows the layer. Gated: the 16 rows are 8 features' gate rows,
// then their up rows, so thread tx + 8 holds the up value of thread tx.
// FUSED: the shrink runs here too (no k_shrink_f32, no table): the 16 threads of
// a position split each chunk's columns among them and keep partial dot
// products with the position's rank rows, 4 loads of 16 bytes a row. Every
// feature tile repeats it.
template <int EPI, bool FUSED>
__global__ __launch_bounds__(256) void k_gemm_f32(LinearArgs a) {
  constexpr bool GATED = EPI == kEpiGated;
  __shared__ float Ws[kF32Feat][kF32KB + 1];
  __shared__ float Xs[16][kF32KB + 1];
  const int tid = threadIdx.x;
  const int tx = tid % kF32Feat, ty = tid / kF32Feat;
  const int n0 = blockIdx.x * kF32Feat, p0 = blockIdx.y * 16;
  const int T = a.T, d_in = a.d_in, d_out = a.d_out;
  // row of W of the tile's row i; rows past the last one are clamped to it
  auto wrow = [&](int i) {
    return GATED ? (i >> 3) * (d_out / 2) + min(n0 / 2 + (i & 7), d_out / 2 - 1) : min(n0 + i, d_out - 1);
  };
  const float* __restrict__ x = (const float*)a.x;
  const float* __restrict__ W = (const float*)a.W;
  float acc = 0.f;
  // loader: W chunk 16 x 256 and x chunk 16 x 256, 1024 float4 each (4 per
  // thread); absent rows or columns load zeros
  constexpr int N4 = 16 * kF32KB / 4 / 256;
  const float* wsrc[N4];
  const float* xsrc[N4];
  int lr_[N4], lc_[N4];
#pragma unroll
  for (int i = 0; i < N4; ++i) {
    const int q = tid + 256 * i;
    lr_[i] = q / (kF32KB / 4);
    lc_[i] = 4 * (q % (kF32KB / 4));
    wsrc[i] = W + (long long)wrow(lr_[i]) * d_in + lc_[i];
    int xrow = min(p0 + lr_[i], T - 1);
    if (a.sv.token_index) xrow = min(max(a.sv.token_index[xrow], 0), T - 1);
    xsrc[i] = x + (long long)xrow * d_in + lc_[i];
  }
  // this position's adapter entry, requested with the first chunk (the
  // epilogue's B and v loads then need no further round trip)
  const int p = p0 + ty;
  const int4 pe4 = !FUSED && a.lora_on ? a.pos_info[min(p, T - 1)] : make_int4(0, -1, 0, 0);
  f32x4_t wreg[N4], xreg[N4];
  auto load = [&](int kb) {
#pragma unroll
    for (int i = 0; i < N4; ++i) {
      const bool wok = (GATED || n0 + lr_[i] < d_out) && kb + lc_[i] < d_in;
      wreg[i] = wok ? *(const f32x4_t*)(wsrc[i] + kb) : f32x4_t{0.f, 0.f, 0.f, 0.f};
      const bool xok = p0 + lr_[i] < T && kb + lc_[i] < d_in;
      xreg[i] = xok ? *(const f32x4_t*)(xsrc[i] + kb) : f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
  };
  // FUSED: the position's segment, adapter and rank rows. The rows to read are
  // the segment's own, clamped into the slot; the registered rank only masks v.
  // Loads are unconditional, at clamped places, and the first one leads W and x.
  constexpr int RG = 8;                                   // rank rows loaded together
  const SegView& sg = a.sv;
  const int f_S = FUSED ? seg_count(sg) : 0, pc = min(p, T - 1);
  int f_st = 0;
  if constexpr (FUSED) f_st = sg.seg_start[min(tx, f_S)];
  load(0);
  int f_ad = -1, f_r = 0, f_rows = 0;
  float f_sc = 0.f, vacc[FUSED ? kF32FusedRank : 1];
  const float* f_A = (const float*)a.pv.zeros;
  if constexpr (FUSED) {
    int s = 0;
    if (f_S <= 16) {   // uniform: the starts are in the position's 16 threads
      const unsigned long long m = __ballot(tx < f_S && f_st <= pc) >> (16 * (ty % 4));
      s = max(__popcll(m & 0xffffull) - 1, 0);
    } else {
      s = find_segment(sg.seg_start, f_S, pc);
    }
    const int sc = min(s, max(f_S - 1, 0));
    int beg = sg.seg_start[sc], end = sg.seg_start[sc + 1], ad = sg.seg_adapter[sc], rk = sg.seg_rank[sc];
    f_sc = sg.seg_scale[sc];
    asm volatile("" : "+v"(beg), "+v"(end), "+v"(ad), "+v"(rk), "+v"(f_sc));   // (all in flight together)
    if (f_S > 0 && beg <= pc && pc < end && ad >= 0 && ad < a.pv.capacity && rk > 0) {
      f_ad = ad;
      f_rows = min(rk, a.pv.max_rank);
      f_A = (const float*)a.pv.base + (long long)ad * a.pv.slot_elems;
    }
    f_r = a.pv.rank[max(f_ad, 0)];                        // (used behind the products)
#pragma unroll
    for (int j = 0; j < kF32FusedRank; ++j) vacc[j] = 0.f;
  }
  // rank rows j0 .. j0 + RG - 1 at the thread's columns of chunk kb (absent rows
  // repeat the last, without an adapter they are zeros)
  auto load_a = [&](int kb, int j0, f32x4_t (&av)[RG][kF32KB / 64]) {
#pragma unroll
    for (int j = 0; j < RG; ++j)
#pragma unroll
      for (int i = 0; i < kF32KB / 64; ++i)
        av[j][i] = *(const f32x4_t*)(f_A + (f_rows > 0 ? (long long)min(j0 + j, f_rows - 1) * d_in + min(kb + 64 * i + 4 * tx, d_in - 4) : 0));
  };
  // the row of B, in groups of 4 columns below the rank rounded up to 8 (the
  // rows' pitch; columns past the rank are zero)
  f32x4_t bq[kF32FusedRank / 4];
  auto load_b = [&]() {
    f_r = f_ad >= 0 ? max(min(f_rows, f_r), 0) : 0;
    const int nb = GATED ? wrow(tx) : min(n0 + tx, d_out - 1);
    const float* bn = f_A + (f_r > 0 ? a.pv.b_offset + (long long)nb * round_up8(f_r) : 0);
#pragma unroll
    for (int g = 0; g < kF32FusedRank / 4; ++g) bq[g] = *(const f32x4_t*)(4 * g < f_r ? bn + 4 * g : (const float*)a.pv.zeros);
  };
  auto dot_a = [&](int j0, const f32x4_t (&av)[RG][kF32KB / 64]) {
#pragma unroll
    for (int i = 0; i < kF32KB / 64; ++i)                 // (columns past d_in: x is zero in LDS)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float xv = Xs[ty][64 * i + 4 * tx + e];
#pragma unroll
        for (int j = 0; j < RG; ++j) vacc[j0 + j] = fmaf(av[j][i][e], xv, vacc[j0 + j]);
      }
  };
  for (int kb = 0; kb < d_in; kb += kF32KB) {
#pragma unroll
    for (int i = 0; i < N4; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        Ws[lr_[i]][lc_[i] + c] = wreg[i][c];
        Xs[lr_[i]][lc_[i] + c] = xreg[i][c];
      }
    __syncthreads();
    if (kb + kF32KB < d_in) load(kb + kF32KB);   // uniform
    f32x4_t av[RG][kF32KB / 64];
    if constexpr (FUSED) {
      load_a(kb, 0, av);                                  // in flight during the base product
      if (kb == 0) load_b();
    }
#pragma unroll 16
    for (int kk = 0; kk < kF32KB; ++kk) acc = fmaf(Ws[tx][kk], Xs[ty][kk], acc);
    if constexpr (FUSED) {
      dot_a(0, av);
      if (a.pv.max_rank > RG) {                           // uniform
        load_a(kb, RG, av);
        dot_a(RG, av);
      }
    }
    __syncthreads();
  }
  if constexpr (FUSED) {
#pragma unroll
    for (int j = 0; j < kF32FusedRank; ++j)
#pragma unroll
      for (int off = 1; off < 16; off <<= 1) vacc[j] += __shfl_xor(vacc[j], off, 16);
  }
  const int n = GATED ? wrow(tx) : n0 + tx;
  if (!GATED && (n >= d_out || p >= T)) return;
  const SegView& sv = a.sv;
  float val = acc;
  const int ad = FUSED ? f_ad : pe4.y, r = min(FUSED ? f_r : pe4.z, a.pv.max_rank);
  if (a.lora_on && ad >= 0 && ad < a.pv.capacity && r > 0) {
    const float* Bb = (const float*)a.pv.base + (long long)ad * a.pv.slot_elems + a.pv.b_offset;
    const float* bn = Bb + (long long)n * round_up8(r);
    const float* vp = a.v_part + (long long)(GATED ? min(p, T - 1) : p) * a.r_ws;
    float lora = 0.f;
    if constexpr (FUSED) {
#pragma unroll
      for (int j = 0; j < kF32FusedRank; ++j) lora = fmaf(bq[j / 4][j % 4], j < r ? vacc[j] : 0.f, lora);
      val = fmaf(f_sc, lora, val);
    } else {
      for (int j = 0; j < r; ++j) lora = fmaf(bn[j], vp[j], lora);
      val = fmaf(__int_as_float(pe4.w), lora, val);
    }
  }
  int f = n, d_y = d_out;                 // y's column and width
  if constexpr (EPI != kEpiNone) {
    if (a.epi.bias) val += elem_f32<float>(a.epi.bias, n);
    if constexpr (GATED) {
      const float up = __shfl(val, (threadIdx.x % kWave) + 8, kWave);   // (tx >= 8: unused)
      d_y = d_out / 2;
      f = n0 / 2 + tx;
      if (tx >= 8 || f >= d_y || p >= T) return;
      val = activate<false>(val, a.epi.act) * up;
    } else {
      val = activate<false>(val, a.epi.act);
    }
  }
  int row = sv.token_index ? sv.token_index[p] : p;
  row = min(max(row, 0), T - 1);
  const long long at = (long long)row * d_y + f;
  if constexpr (EPI != kEpiNone) {
    if (a.epi.residual) val += elem_f32<float>(a.epi.residual, at);
  }
  ((float*)a.y)[at] = val;
}

// With an epilogue the shrink is the wide one (512 -> 512, rank 16, 1024 tokens of
// 16 segments: 228 us with a workgroup per segment, 47 with it; 408 -> 101, rank
// 64, 100 tokens of 4 segments: 188 and 20), or fused where one chunk holds d_in,
// ranks are low and the tiles are at most one per CU, since each repeats it (256
// -> 256, rank 8: 16 tokens 10.0 us fused, 11.3 in two launches; 1024 tokens 38 and
// 19; 512 -> 512, 16 tokens: 19.0 and 14.2).
void launch_linear_f32(const LinearArgs& a, hipStream_t st) {
  const bool lora = a.lora_on && a.seg_grid > 0;
  const int rows = a.epi_kind == kEpiGated ? gated_rows(a.d_out) : a.d_out;
  const dim3 grid((rows + kF32Feat - 1) / kF32Feat, (a.T + 15) / 16);
  const bool fused = lora && a.epi_kind != kEpiNone && a.pv.max_rank <= kF32FusedRank && a.d_in <= kF32KB && grid.x * grid.y <= 256;
  if (lora && !fused) {
    if (a.epi_kind == kEpiNone) hipLaunchKernelGGL(k_shrink_f32, dim3(a.seg_grid), dim3(256), 0, st, a);
    else hipLaunchKernelGGL(k_shrink_f32_wide, dim3((a.T + 3) / 4, (a.pv.max_rank + kF32Rows - 1) / kF32Rows), dim3(256), 0, st, a);
  }
  if (a.epi_kind == kEpiGated) {
    if (fused) hipLaunchKernelGGL((k_gemm_f32<kEpiGated, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_gemm_f32<kEpiGated, false>), grid, dim3(256), 0, st, a);
  } else if (a.epi_kind == kEpiPlain) {
    if (fused) hipLaunchKernelGGL((k_gemm_f32<kEpiPlain, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_gemm_f32<kEpiPlain, false>), grid, dim3(256), 0, st, a);
  } else {
    hipLaunchKernelGGL((k_gemm_f32<kEpiNone, false>), grid, dim3(256), 0, st, a);
  }
}

}  // namespace mlora
