// kernels_experts.hip -- products of routed rows with their experts' weights.
//
//   y[p] = act(W_e x[row(p)] + b_e)      p in [seg_start[e], seg_start[e + 1])
//
// and, for the way back, the fp32 products of every sorted position followed
// by k_combine: out[t] = residual[t] + sum_j w[t][j] z[position[t][j]].
//
// MFMA 16x16 layouts: lane l supplies row l % 16 of either operand; result
// register v of lane l is row 4 (l / 16) + v, column l % 16. Rows are W rows,
// columns positions.
#include <algorithm>

#include "../../include/mlora.h"
#include "experts.h"
#include "gemm_tile.h"
#include "stream_tile.h"

namespace mlora {

__device__ __attribute__((aligned(16))) uint32_t expert_zeros[64];   // read past d_in

// ---------------------------------------------------------------------------
// Streaming form, every type: an item is 16 NR (virtual) rows of one expert by
// up to 16 NTB of its positions, over the whole of d_in. The NW waves take a
// contiguous part of d_in each, in units of 128 bytes of a W row, load W and x
// straight into MFMA operand registers, and their sums are added in wave order
// through LDS. W is read once where an expert has at most 16 NTB rows.
//
// Bound by W's bytes (stream_tile.h). Neighbouring workgroups take neighbouring
// row tiles, so the card streams W in order (an order that put an expert's runs
// side by side on an XCD: 119 us against 113).
// ---------------------------------------------------------------------------
constexpr int kGridY = 32768;   // runs per grid row (y is limited; z takes the rest)

template <int TYPE, int NR, int NTB, int NW, bool GATED>
__global__ __launch_bounds__(NW * kWave) void k_experts_stream(ExpertsArgs a) {
  constexpr int EB = TYPE == kXFp8w ? 1 : TYPE == kXF32 ? 4 : 2;   // bytes per W element
  constexpr int XB = TYPE == kXF32 ? 4 : 2;                        // and per x element
  constexpr int UC = 128 / EB;                                     // columns per unit
  constexpr int XL = XB / EB;                                      // x loads per W load
  __shared__ f32x4_t red[NW][NR * NTB][kWave];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave), lane = tid % kWave;
  const int l16 = lane % 16, g = lane / 16;
  const int rt = blockIdx.x;
  int p0, p1;
  const int e = find_expert(scan_runs(a.seg_start, a.E, a.n_pos, 16 * NTB, 0), a.seg_start, a.E, a.n_pos, 16 * NTB,
                            (int)(blockIdx.y + blockIdx.z * kGridY), &p0, &p1);
  if (e < 0) return;   // uniform: past the last item
  const int d_in = a.d_in, d_out = a.d_out;
  const int v0 = rt * 16 * NR;                                     // first (virtual) row
  auto wrow = [&](int v) { return (long long)e * d_out + wrow_of<GATED>(v, d_out); };

  // W: a uniform base and 32-bit offsets; rows past the last are clamped to it
  constexpr int NO = GATED ? NR / 2 : NR;                          // distinct row blocks
  const int f0 = GATED ? v0 / 2 : v0, nf = GATED ? d_out / 2 : d_out;
  const char* wbase = (const char*)a.W + ((long long)e * d_out + f0) * d_in * EB;
  const long long up = (long long)nf * d_in * EB;                  // gated: from a gate row to its up row
  uint32_t wo[NO];
#pragma unroll
  for (int r = 0; r < NO; ++r) wo[r] = (uint32_t)min(16 * r + l16, nf - 1 - f0) * (uint32_t)(d_in * EB) + 16 * g;
  const char* xp[NTB];
#pragma unroll
  for (int t = 0; t < NTB; ++t) {
    const int p = min(p0 + 16 * t + l16, p1 - 1);                  // (absent positions repeat the last)
    const int row = a.token_index ? a.token_index[p] : p;
    xp[t] = (const char*)a.x + (long long)min(max(row, 0), a.n_rows - 1) * d_in * XB + 16 * XL * g;
  }

  f32x4_t acc[NR][NTB];
  stream_product<TYPE, NR, NTB, NW, GATED>(wbase, up, wo, xp, d_in, wave, g, acc);
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int t = 0; t < NTB; ++t) red[wave][r * NTB + t][lane] = acc[r][t];
  __syncthreads();

  // sums in wave order, then the epilogue: a thread takes 4 consecutive rows
  // of one position (gated: the gate rows and the up rows of 4 features)
  constexpr int NB = GATED ? NR / 2 : NR;                          // row blocks of features
  const int d_y = GATED ? d_out / 2 : d_out;
  for (int q = tid; q < NB * NTB * kWave; q += NW * kWave) {
    const int ql = q % kWave, t = (q / kWave) % NTB, b = q / kWave / NTB;
    const int p = p0 + 16 * t + ql % 16;
    const int f = (GATED ? v0 / 2 : v0) + 16 * b + 4 * (ql / 16);  // first feature
    if (p >= p1 || f >= d_y) continue;
    auto sum = [&](int r, float* z) {                              // row block r
      f32x4_t s = red[0][r * NTB + t][ql];
#pragma unroll
      for (int w = 1; w < NW; ++w)
#pragma unroll
        for (int v = 0; v < 4; ++v) s[v] += red[w][r * NTB + t][ql][v];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const long long n = wrow(v0 + 16 * r + 4 * (ql / 16) + v);
        z[v] = s[v];
        if constexpr (TYPE == kXFp8w) z[v] *= a.w_scale[n];
        if (a.epi.bias) z[v] += TYPE == kXF32 ? elem_f32<float>(a.epi.bias, n) : elem_f32<uint16_t>(a.epi.bias, n);
      }
    };
    float o[4];
    sum(GATED ? 2 * b : b, o);
    activate_n<TYPE != kXF32>(o, a.epi.act);
    if constexpr (GATED) {
      float u[4];
      sum(2 * b + 1, u);
#pragma unroll
      for (int v = 0; v < 4; ++v) o[v] *= u[v];
    }
    const bool whole = f + 4 <= d_y;
    if (TYPE == kXF32 || a.f32_out) {
      float* y = (float*)a.y + (long long)p * (a.f32_out ? f32_pitch(d_y) : d_y) + f;
      if (whole || a.f32_out) *(f32x4_any*)y = f32x4_t{o[0], o[1], o[2], o[3]};
      else
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (f + v < d_y) y[v] = o[v];
    } else {
      uint16_t* y = (uint16_t*)a.y + (long long)p * d_y + f;
      if (whole)
        *(u32x2_any*)y = u32x2_t{(uint32_t)f32_to_bf16_bits(o[0]) | ((uint32_t)f32_to_bf16_bits(o[1]) << 16),
                                 (uint32_t)f32_to_bf16_bits(o[2]) | ((uint32_t)f32_to_bf16_bits(o[3]) << 16)};
      else
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (f + v < d_y) y[v] = f32_to_bf16_bits(o[v]);
    }
  }
}

// ---------------------------------------------------------------------------
// Tiled form (more rows per expert): a workgroup takes BR (virtual) rows of one
// expert by a run of up to BT of its positions over the whole of d_in.
//
// Order of the tiles: block b runs on XCD b % 8, which takes row tiles xcd, xcd +
// 8, ... : group of runs by group, in a group row tile by row tile, its runs side
// by side, so the XCDs read neighbouring rows of W at the same time (an eighth of
// the row tiles in a row for each XCD: 1167 us against 1072, way back of a prefill
// batch). The last n_rt % 8 row tiles go round the XCDs run by run.
//
// Where experts have several runs, a group is of one expert's, at most 8: the
// runs in flight on an XCD share its L2's copy of the expert's rows of W, which is
// read from memory once per group, and the row tiles in flight share the rows of
// x (prefill batch, 8 experts of about 1024 rows: 1828 us, 1856 with groups of 4,
// 1893 with groups of 16 runs whatever their expert; 512 tokens: 521 against 553).
// Where hardly an expert has two, W's bytes decide, and groups of 4 runs of
// several experts read W from several places at a time (64 tokens, two of eight
// experts: 326 us against 351 expert by expert; 256 tokens: 379 against 392).
// ---------------------------------------------------------------------------
constexpr int kExpertGroup = 8, kRunGroup = 4;

// Tiles of XCD x among `runs` runs by n_rt row tiles, and the j-th of them: its
// expert (or -1), positions [*p0, *p1) and row tile.
__host__ __device__ __forceinline__ int xcd_tiles(int x, int runs, int n_rt) {
  return n_rt / 8 * runs + (n_rt % 8 * runs - x + 7) / 8;
}
__device__ __forceinline__ int xcd_tile(const ExpertsArgs& a, const RunScan& first, int BT, bool by_expert, int j, int x,
                                        int runs, int n_rt, int* rt, int* p0, int* p1) {
  const int n8 = n_rt / 8;
  int run;
  if (j >= n8 * runs) {
    const int k = (j - n8 * runs) * 8 + x;
    *rt = n8 * 8 + k / runs;
    run = k % runs;
  } else if (by_expert) {   // uniform
    int s0, s1, mine, before;
    if (find_run(first, a.seg_start, a.E, a.n_pos, BT, j / n8, &s0, &s1, &mine, &before) < 0) return -1;
    const int k = j - n8 * before, c = k / (n8 * kExpertGroup), kc = k - c * n8 * kExpertGroup;
    const int gs = max(min(kExpertGroup, mine - c * kExpertGroup), 1);
    *rt = min(kc / gs, n8 - 1) * 8 + x;
    run = before + c * kExpertGroup + kc % gs;
  } else {
    const int group = j / (n8 * kRunGroup), k = j - group * n8 * kRunGroup, gs = min(kRunGroup, runs - group * kRunGroup);
    *rt = k / gs * 8 + x;
    run = group * kRunGroup + k % gs;
  }
  const int e = find_expert(first, a.seg_start, a.E, a.n_pos, BT, run, p0, p1);
  return e >= 0 && *p0 < *p1 ? e : -1;
}

// One tile: rows r0 .. r0 + BR - 1 by positions p0 .. min(p0 + BT, p1) - 1.
// OUT: 0 bf16 rows, 1 bf16 rows of a gated product, 2 fp32 rows (no activation)
template <class C, int OUT, bool PIPE>
__device__ __forceinline__ void expert_tile(const ExpertsArgs& a, int e, int p0, int p1, int r0, char* lds) {
  constexpr bool GATED = OUT == 1;
  constexpr int WB = C::kW8 ? 1 : 2;                     // bytes per W element
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave), lane = tid % kWave;
  const int d_in = a.d_in, d_out = a.d_out;
  const char* __restrict__ W = (const char*)a.W + (long long)e * d_out * d_in * WB;
  const uint16_t* __restrict__ x = (const uint16_t*)a.x;
  auto row_of = [&](int r) {
    const int p = min(p0 + r, p1 - 1);                   // (absent positions repeat the last)
    const int row = a.token_index ? a.token_index[p] : p;
    return min(max(row, 0), a.n_rows - 1);
  };
  f32x16_t acc[C::MR][C::MT];
#pragma unroll
  for (int m = 0; m < C::MR; ++m)
#pragma unroll
    for (int n = 0; n < C::MT; ++n)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[m][n][v] = 0.f;
  if constexpr (PIPE) {
    // W offsets from the tile's first row (gated: its first gate row; the up
    // rows lie d_out / 2 rows further)
    const int w0 = wrow_of<GATED>(r0, d_out);
    PipeSrc<C> src;
    src.set(wave, lane, W + (long long)w0 * d_in * 2, x,
            [&](int r) { return (uint32_t)(wrow_of<GATED>(r0 + r, d_out) - w0) * (uint32_t)(2 * d_in); },
            [&](int r) { return (uint32_t)row_of(r) * (uint32_t)(2 * d_in); });
    pipe_mainloop<C>(src, d_in, expert_zeros, lds, wave, lane, acc);
  } else {
    TileSrc<C> src;
    src.set(wave, lane, [&](int r) { return W + (long long)wrow_of<GATED>(r0 + r, d_out) * d_in * WB; },
            [&](int r) { return x + (long long)row_of(r) * d_in; });
    ring_mainloop<C>(src, d_in, expert_zeros, lds, wave, lane, acc);
  }

  const int wr = wave / C::NWT, wt = wave % C::NWT;
  const int v0 = r0 + wr * C::kWR, pw = p0 + wt * C::kWT;
  EpiView epi = a.epi;
  if (epi.bias) epi.bias = (const uint16_t*)epi.bias + (long long)e * d_out;
  const float* ws = C::kW8 ? a.w_scale + (long long)e * d_out : nullptr;
  if constexpr (OUT == 2) {
    store_f32<C>(acc, lds, wave, lane, v0, pw, p1, d_out, (const uint16_t*)epi.bias, ws, (float*)a.y, f32_pitch(d_out));
  } else {
    store_epilogue<C, GATED>(acc, lds, wave, lane, v0, pw, p1, d_out, epi, ws, a.y, [](int p) { return p; });
  }
}

template <class C, int OUT>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(C::NW / 4, C::NW / 4)))
void k_experts_tile(ExpertsArgs a, int n_rt, int max_runs, bool by_expert) {
  __shared__ __attribute__((aligned(1024))) char lds[C::TILE_BYTES];
  const int x = blockIdx.x & 7, j = blockIdx.x >> 3;
  if (j >= xcd_tiles(x, max_runs, n_rt)) return;   // uniform
  int rt, p0, p1;
  // (of the most runs there can be: the rest find no expert)
  const RunScan first = scan_runs(a.seg_start, a.E, a.n_pos, C::kBT, 0);
  const int e = xcd_tile(a, first, C::kBT, by_expert, j, x, max_runs, n_rt, &rt, &p0, &p1);
  if (e < 0) return;   // uniform
  expert_tile<C, OUT, false>(a, e, p0, p1, rt * C::kBR, lds);
}

// The largest tile, 256 x 256, and what it leaves. An XCD's 32 CUs take its
// tiles in rounds of 32; those of a last round that would keep a quarter or a
// half of them busy are cut into four (128 x 128) or two (256 x 128) for all of
// them (the way back of a prefill batch, 72 tiles per XCD: 1072 -> 1007 us). A run
// of at most 128 positions takes the 256 x 128 form too.
typedef GCfg<256, 256, 128, 128, 3, 64, 2> Tile256;
typedef GCfg<256, 128, 128, 64, 3, 64, 3> Tile256Half;
typedef GCfg<128, 128, 64, 64, 4, 64, 4> Tile256Quarter;
constexpr int kXcdCus = 32;

template <int OUT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1)))
void k_experts_tile256(ExpertsArgs a, int n_rt, int max_runs) {
  __shared__ __attribute__((aligned(1024))) char lds[160 * 1024];
  static_assert(Tile256::TILE_BYTES <= sizeof(lds) && Tile256Half::TILE_BYTES <= sizeof(lds) && Tile256Quarter::TILE_BYTES <= sizeof(lds), "one LDS block");
  const RunScan first = scan_runs(a.seg_start, a.E, a.n_pos, 256, 0);
  const int runs = min(count_runs(first, a.seg_start, a.E, a.n_pos, 256), max_runs);   // (more: overlapping segments)
  const int x = blockIdx.x & 7, j = blockIdx.x >> 3;
  const int mine = xcd_tiles(x, runs, n_rt);
  const int whole = mine / kXcdCus * kXcdCus, rem = mine - whole;
  const int cut = rem <= kXcdCus / 4 ? 4 : rem <= kXcdCus / 2 ? 2 : 1;
  if (j >= whole + rem * cut) return;   // uniform: past the XCD's last tile
  const int i = j < whole ? j : whole + (j - whole) / cut, piece = j < whole ? 0 : (j - whole) % cut;
  const int parts = j < whole ? 1 : cut;
  int rt, p0, p1;
  const int e = xcd_tile(a, first, 256, true, i, x, runs, n_rt, &rt, &p0, &p1);
  if (e < 0) return;
  // (parts 4: piece & 1 the row half, piece >> 1 the position half; parts 2: the position half)
  const int ph = parts == 4 ? piece >> 1 : piece;
  const int q0 = p0 + 128 * ph;
  if (q0 >= p1) return;
  if (parts == 4) expert_tile<Tile256Quarter, OUT, true>(a, e, q0, min(p1, q0 + 128), rt * 256 + 128 * (piece & 1), lds);
  else if (parts == 2 || p1 - p0 <= 128) expert_tile<Tile256Half, OUT, true>(a, e, q0, min(p1, q0 + 128), rt * 256, lds);
  else expert_tile<Tile256, OUT, true>(a, e, p0, p1, rt * 256, lds);
}

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
// Items of a batch cut into runs of BT positions per expert, at most.
static long long run_bound(const ExpertsArgs& a, int BT) {
  return (long long)a.n_pos / BT + (a.E < a.n_pos ? a.E : a.n_pos);
}

template <int TYPE, int NR, int NTB, int NW>
static void launch_stream_n(const ExpertsArgs& a, hipStream_t st) {
  const int rows = a.gated ? gated_rows(a.d_out) : a.d_out;
  const long long runs = run_bound(a, 16 * NTB);
  const dim3 grid((rows + 16 * NR - 1) / (16 * NR), (unsigned)std::min<long long>(runs, kGridY), (unsigned)((runs + kGridY - 1) / kGridY));
  if (a.gated) hipLaunchKernelGGL((k_experts_stream<TYPE, NR, NTB, NW, true>), grid, dim3(NW * kWave), 0, st, a);
  else hipLaunchKernelGGL((k_experts_stream<TYPE, NR, NTB, NW, false>), grid, dim3(NW * kWave), 0, st, a);
}

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

template <class C>
static void launch_tile(const ExpertsArgs& a, hipStream_t st) {
  const int rows = a.gated ? gated_rows(a.d_out) : a.d_out;
  const int n_rt = (rows + C::kBR - 1) / C::kBR;
  const int max_runs = (int)run_bound(a, C::kBT);
  const bool by_expert = 4ll * a.n_pos >= 3ll * C::kBT * std::min(a.E, a.n_pos);   // a mean of three quarters of a run
  const dim3 grid(8 * xcd_tiles(0, max_runs, n_rt)), block(C::NT);
  if (a.f32_out) hipLaunchKernelGGL((k_experts_tile<C, 2>), grid, block, 0, st, a, n_rt, max_runs, by_expert);
  else if (a.gated) hipLaunchKernelGGL((k_experts_tile<C, 1>), grid, block, 0, st, a, n_rt, max_runs, by_expert);
  else hipLaunchKernelGGL((k_experts_tile<C, 0>), grid, block, 0, st, a, n_rt, max_runs, by_expert);
}

static void launch_tile256(const ExpertsArgs& a, hipStream_t st) {
  const int rows = a.gated ? gated_rows(a.d_out) : a.d_out;
  const int n_rt = (rows + 255) / 256;
  // per XCD at most its share of the tiles and, where the last ones are cut,
  // 24 pieces more
  const int max_runs = (int)run_bound(a, 256);
  const dim3 grid(8 * (xcd_tiles(0, max_runs, n_rt) + 24)), block(256);
  if (a.f32_out) hipLaunchKernelGGL(k_experts_tile256<2>, grid, block, 0, st, a, n_rt, max_runs);
  else if (a.gated) hipLaunchKernelGGL(k_experts_tile256<1>, grid, block, 0, st, a, n_rt, max_runs);
  else hipLaunchKernelGGL(k_experts_tile256<0>, grid, block, 0, st, a, n_rt, max_runs);
}

template <bool W8> using Tile128 = GCfg<128, 128, 64, 32, 3, W8 ? 128 : 64, W8 ? 2 : 3, W8>;
template <bool W8> using Tile64 = GCfg<128, 64, 32, 32, 4, W8 ? 128 : 64, 4, W8>;
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
    if (near && (mean >= 192 || (mean >= 112 && tiles256 >= 1024))) return launch_tile256(a, st);
  }
  if (mean <= 48) launch_tile<Tile64<W8>>(a, st);
  else launch_tile<Tile128<W8>>(a, st);
}

void launch_experts(const ExpertsArgs& a, bool bf16, hipStream_t st) {
  if (a.n_pos <= 0) return;
  if (!bf16) launch_stream<kXF32>(a, st);
  else if (a.w_scale) launch_bf16<true>(a, st);
  else launch_bf16<false>(a, st);
}

void launch_combine(const CombineArgs& a, bool bf16, hipStream_t st) {
  const dim3 grid(a.T, (a.d_out + 1023) / 1024);
  if (bf16) hipLaunchKernelGGL(k_combine<uint16_t>, grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL(k_combine<float>, grid, dim3(256), 0, st, a);
}

}  // namespace mlora
