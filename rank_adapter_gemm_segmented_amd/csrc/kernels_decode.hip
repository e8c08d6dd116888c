// kernels_decode.hip -- bf16 multi-LoRA linear for small token counts (T <= 64).
//
// y_i = W x_i + scale_s * B_a (A_a x_i) ("Multi-LoRA Serving in Practice",
// section "Core Principle", displayed formula), per adapter segment
// ("InvisibleLoRA" abstract). At decode the layer is HBM-bound: W (and each
// touched adapter) must be streamed once, and with T <= 64 a CU that covered
// the whole of d_in would re-read all of x from L2 (4x the bytes of its W
// rows). So d_in is split into chunks across CUs, and the layer runs in two
// launches with no inter-workgroup synchronization:
//
//  k_stream  one-shot items (n-tile of 64 W rows, d_in chunk c). An item loads
//            its x chunk into LDS and its W rows straight into MFMA operand
//            registers, every load in flight at once, then runs
//            v_mfma_f32_16x16x32_bf16. The shrink v = A_a x is folded in per
//            segment: item (c, tile) takes segments tile, tile + n_tiles, ...
//            and multiplies their A rows (restricted to chunk c) against the
//            same x chunk in LDS. Outputs: fp32 partial tiles of W x and of
//            v, one slot per chunk (deterministic, no atomics).
//  k_finish  y = sum_c partial_c + scale_s * B_a (sum_c v_c), summed in chunk
//            order, the expand on the vector ALUs in fp32, one bf16 store.
//
// MFMA 16x16x32 bf16 lane layout: lane l holds row l%16, k-slots
// 8*(l/16)..+7 of each operand; result register v of lane l is row
// 4*(l/16)+v, column l%16.
#include "common.h"
#include "gemm_tile.h"
#include "launch.h"
#include "stream_tile.h"

namespace mlora {

__device__ __forceinline__ f32x4_t mfma16d(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
}

constexpr int kDecThreads = 512;                   // 8 waves
constexpr int kDecWaves = kDecThreads / kWave;
constexpr int kDecRows = 64;                       // W rows per item (4 blocks of 16)
constexpr int kDecXPitch = kDecMaxKc + 8;          // LDS row pitch of the x chunk (bf16)
constexpr int kDecWSteps = kDecMaxKc / 2 / 32;     // 32-wide k-steps per wave (16)
constexpr int kDecWPre = 8;                        // W k-steps requested before the x barrier
constexpr int kDecASteps = kDecMaxKc / 8 / 32;     // shrink k-steps per wave per row block (4)

template <int TT>
struct DecSmem {
  uint16_t xs[TT * kDecXPitch];
  float red[4][kWave][4 * (TT / 16)];              // second-half partials of the W rows
};

// Partial tile layout (fragment-major): for chunk c, n-tile i, row block rb,
// token block tb: 256 floats ordered [lane][4].
__device__ __forceinline__ long long part_off(int c, int i, int rb, int tb, int n_tiles, int ntb) {
  return ((((long long)c * n_tiles + i) * 4 + rb) * ntb + tb) * 256;
}

// WQ = kWFp8: W holds FP8 e4m3 codes (one byte per element, a float32 scale per row
// applied by k_finish). A lane's 16-byte load then covers 16 columns, which
// serve two consecutive k-steps: lane group g = l / 16 of the step pair
// (2q, 2q + 1) starting at column C takes columns C + 16 g .. + 7 in step 2q
// and C + 16 g + 8 .. + 15 in step 2q + 1, and reads x at the same columns.
// WQ = kWMx: MXFP4 codes, 32 columns to a 16-byte load, one block with its scale:
// lane group g of four k-steps starting at column C takes columns C + 32 g + 8 q
// .. + 7 in step q (chunks are whole planes of scales).
// GATED: the items' rows are virtual rows (epilogue.h). NT: W loads marked
// nontemporal. With an epilogue they are not, but for 64 tokens on a long d_in:
// a row's 128-byte line comes by two loads, and the mark loses it in between
// (64 tokens, 4096 -> 4096: 18.2 us marked, 17.0 not; one token, gate|up in FP8:
// 40.6 and 38.6; 64 tokens, 14336 -> 4096: 51.1 and 53.5).
template <int TT, int WQ, bool GATED, bool NT>
__global__ __launch_bounds__(kDecThreads) void k_stream_bf16(DecodeArgs a) {
  constexpr bool W8 = WQ == kWFp8, MX = WQ == kWMx;
  constexpr int NTB = TT / 16;
  constexpr int XP = kDecXPitch;
  constexpr int XCH = TT * (kDecMaxKc / 8) / kDecThreads;  // 16-byte x pieces per thread
  __shared__ __attribute__((aligned(16))) DecSmem<TT> sm;

  const int item = blockIdx.x;
  const int c = item / a.n_tiles;
  const int tile = item % a.n_tiles;
  const int tid = threadIdx.x;
  const int wave = tid / kWave, lane = tid % kWave;
  const int l16 = lane % 16, kq = 8 * (lane / 16);
  const int T = a.T, d_in = a.d_in, d_out = a.d_out;
  const int k0 = c * a.kc;
  const int kc = min(a.kc, d_in - k0);          // this chunk's width (multiple of 8)
  const int nks = (kc + 31) / 32;
  const uint16_t* __restrict__ x = (const uint16_t*)a.x;
  const uint16_t* __restrict__ W = (const uint16_t*)a.W;
  const bool lora = a.lora_on != 0;

  // ---- 0. this item's shrink units -----------------------------------------
  // A unit is ur = a.unit_rows (4, 8 or 16) consecutive rank rows of one
  // segment: unit u = s * nq + q holds rows [q ur, (q + 1) ur) of segment s,
  // nq = ceil(max_rank / ur). Lane l of every wave holds unit tile + l * n_tiles
  // (at most 64 per item, which the host guarantees). The lane's segment
  // metadata loads go first in the queue, from clamped indices (without LoRA
  // they read the pool's zero block), so the waits for them never wait for the
  // x and W loads issued after them.
  // The device segment count, when there is one, is read the same way: the
  // offset vz is zero, but held in a vector register, so the load is a vector
  // load (ordered with the others) rather than a scalar one, whose wait would
  // come at once.
  int vz;
  asm volatile("v_mov_b32 %0, 0" : "=v"(vz));
  const int32_t* zi = (const int32_t*)a.pv.zeros;
  const bool nsd_on = lora && a.sv.n_seg_dev != nullptr;
  const int nsd = *((nsd_on ? a.sv.n_seg_dev : zi) + vz);
  const int ur = a.unit_rows;
  const int nq = (a.pv.max_rank + ur - 1) / ur;
  const int u_l = tile + lane * a.n_tiles;
  const int s_l = u_l / nq, j0_l = (u_l - s_l * nq) * ur;   // segment, first rank row
  const int si = lora ? min(s_l, max(a.sv.n_seg - 1, 0)) : 0;
  const int m_st0 = *(lora ? a.sv.seg_start + si : zi);
  const int m_st1 = *(lora ? a.sv.seg_start + si + 1 : zi);
  const int m_ad = *(lora ? a.sv.seg_adapter + si : zi);
  const int m_rk = *(lora ? a.sv.seg_rank + si : zi);
  const float m_sc = *(lora ? a.sv.seg_scale + si : (const float*)zi);

  // ---- 1. x chunk -> registers ---------------------------------------------
  // thread's pieces: token t_i = tid/128 + 4 i, 16-byte column tid % 128
  const int kc8 = kc / 8;
  const int xcol = tid % (kDecMaxKc / 8);
  const bool xcol_ok = xcol < kc8;
  const int xk = k0 + (xcol_ok ? xcol : 0) * 8;
  int xrow[XCH];
#pragma unroll
  for (int i = 0; i < XCH; ++i) xrow[i] = min(tid / (kDecMaxKc / 8) + (kDecThreads / (kDecMaxKc / 8)) * i, T - 1);
  if (a.sv.token_index) {  // uniform: gather rows of the sorted positions
#pragma unroll
    for (int i = 0; i < XCH; ++i) xrow[i] = min(max(a.sv.token_index[xrow[i]], 0), T - 1);
  }
  u32x4_t xr[XCH];
#pragma unroll
  for (int i = 0; i < XCH; ++i) {
    const int t = tid / (kDecMaxKc / 8) + (kDecThreads / (kDecMaxKc / 8)) * i;
    // absent tokens and columns past the chunk read the zero block (an
    // address select: a select on the loaded value would wait for it here)
    xr[i] = ld16(t < T && xcol_ok ? x + (long long)xrow[i] * d_in + xk : (const uint16_t*)a.pv.zeros);
  }

  // ---- 2. W rows -> MFMA A-operand registers --------------------------------
  // wave w: row block rb = w % 4, k-half kh = w / 4 of the chunk. Its first
  // kDecWPre k-steps are requested right behind the x loads, the rest inside
  // the MFMA loop, kDecWPre steps ahead of the step being multiplied: x's
  // requests lead every CU's queue, and HBM streams W while x lands (the
  // barrier below waits for LDS only, not for these loads). Requesting all of
  // the wave's W up front measured slower: x then lands later. Addresses past the chunk or d_out are clamped
  // into the row: their products meet zero x columns or land in discarded
  // rows; steps that belong to the other k-half read zeros. No select on a
  // loaded value.
  const int rb = wave & 3, kh = wave >> 2;
  const int nrow = tile * kDecRows + rb * 16 + l16;
  // (FP8: the first half ends on an even step, so no step pair straddles the halves)
  // (and MXFP4: on a whole group of four)
  const int half_steps = MX ? (((nks + 1) / 2 + 3) & ~3) : W8 ? (((nks + 1) / 2 + 1) & ~1) : (nks + 1) / 2;
  const int ks_begin = kh ? half_steps : 0;
  const int ks_end = kh ? nks : half_steps;
  const uint16_t* wrow = W + (long long)wrow_of<GATED>(nrow, d_out) * d_in + k0;
  const uint8_t* wrow8 = (const uint8_t*)a.W + (long long)wrow_of<GATED>(nrow, d_out) * d_in + k0;
  const uint8_t* wrow4 = (const uint8_t*)a.W + ((long long)wrow_of<GATED>(nrow, d_out) * d_in + k0) / 2;
  const uint8_t* wsc4 = MX ? a.w_mx + 4 * ((long long)(k0 / kMxPlane) * d_out + wrow_of<GATED>(nrow, d_out)) : nullptr;
  u32x4_t wr[kDecWSteps];
  uint32_t ws[MX ? kDecWSteps / 4 : 1];            // MXFP4: the load's dword of scales
  auto ld_w = [](const void* p) { return NT ? ld_nt16(p) : ld16(p); };
  auto load_w = [&](int s) {
    // steps of the other k-half read the pool's zero block (address select)
    if constexpr (MX) {   // slot s holds steps 4 s .. 4 s + 3
      const int k = min((ks_begin + 4 * s) * 32 + 4 * kq, kc - 32);
      const bool in = ks_begin + 4 * s < ks_end;
      wr[s] = ld_w(in ? (const void*)(wrow4 + k / 2) : (const void*)((const uint16_t*)a.pv.zeros + kq));
      // (the block's byte, shifted down where it is used)
      ws[s] = *(const uint32_t*)(in ? (const void*)(wsc4 + 4ll * (k / kMxPlane) * d_out) : (const void*)zi);
    } else if constexpr (W8) {   // slot s holds step pair (2s, 2s + 1)
      const int k = (ks_begin + 2 * s) * 32 + 2 * kq;
      wr[s] = ld_w(ks_begin + 2 * s < ks_end ? (const void*)(wrow8 + min(k, kc - 16))
                                                : (const void*)((const uint16_t*)a.pv.zeros + kq));
    } else {
      const int k = (ks_begin + s) * 32 + kq;
      wr[s] = ld_w(ks_begin + s < ks_end ? wrow + min(k, kc - 8) : (const uint16_t*)a.pv.zeros + kq);
    }
  };
  // FP8: the 16 steps are 8 loads; half of them are requested ahead of the
  // x barrier, as for the bf16 weight (8 ahead: 16.7 us LoRA-on, 4: 16.2 us,
  // 2: 16.5 us on the decode batch)
  constexpr int kWLoads = MX ? kDecWSteps / 4 : W8 ? kDecWSteps / 2 : kDecWSteps;
  constexpr int kWPre = MX ? kWLoads : W8 ? kWLoads / 2 : kDecWPre;
#pragma unroll
  for (int s = 0; s < kWPre; ++s) load_w(s);
  // nothing below is hoisted between these loads (it would wait for the
  // metadata before the last of them are issued)
  __builtin_amdgcn_sched_barrier(0);

  // ---- 3. rows to shrink per unit -------------------------------------------
  // the segment's rank capped by the slot size (the registered rank is applied
  // by the position table, which k_finish reads), cut to the unit's rows
  const int nseg = !lora ? 0 : nsd_on ? min(max(nsd, 0), a.sv.n_seg) : a.sv.n_seg;
  const bool s_ok = s_l < nseg;
  const int ps_l = max(m_st0, 0), pe_l = min(m_st1, T);
  const bool live_l = s_ok && pe_l > ps_l && m_ad >= 0 && m_ad < a.pv.capacity && m_rk > 0;
  const int rr_l = live_l ? min(m_rk, a.pv.max_rank) : 0;
  const int rows_l = min(max(rr_l - j0_l, 0), ur);
  const unsigned long long umask = __ballot(rows_l > 0);   // wave-uniform

  // ---- 4. x registers -> LDS -----------------------------------------------
#pragma unroll
  for (int i = 0; i < XCH; ++i) {
    const int t = tid / (kDecMaxKc / 8) + (kDecThreads / (kDecMaxKc / 8)) * i;
    *(u32x4_t*)&sm.xs[t * XP + xcol * 8] = xr[i];
  }
  // registered rank of the lane's adapter, for the position table written by
  // wave 0 of the chunk-0 items, lanes of a segment's first unit (the others
  // read the zero block)
  const bool pos_item = lora && c == 0 && wave == 0;
  const bool pos_lane = s_l < nseg && j0_l == 0;
  const int reg_r = *(pos_item && pos_lane && live_l ? a.pv.rank + m_ad : zi);
  lds_barrier();

  // ---- 5. shrink units, visited in lane order -------------------------------
  // The A rows of the first two are requested now, so they stream in under the
  // W MFMAs. An absent row reads the pool's zero block; k past the chunk reads
  // a clamped in-row address whose product meets zero x in LDS.
  auto next_unit = [&](int i) {
    const unsigned long long rest = i >= kWave - 1 ? 0ull : umask & (~0ull << (i + 1));
    return rest ? (int)__builtin_ctzll(rest) : kWave;
  };
  u32x4_t ar[2][kDecASteps];
  auto load_a = [&](int i, u32x4_t* dst) {
    const int ii = i < kWave ? i : 0;
    const int rows = i < kWave ? __builtin_amdgcn_readlane(rows_l, ii) : 0;
    const int j0 = __builtin_amdgcn_readlane(j0_l, ii);
    const int ad = __builtin_amdgcn_readlane(m_ad, ii);
    const bool rok = l16 < rows;
    const uint16_t* arow = rok ? (const uint16_t*)a.pv.base + (long long)ad * a.pv.slot_elems +
                                     (long long)(j0 + l16) * d_in + k0
                               : (const uint16_t*)a.pv.zeros;
    const int klim = rok ? kc - 8 : kZeroBlockElems - 8;
#pragma unroll
    for (int st = 0; st < kDecASteps; ++st) {
      const int k = (wave + 8 * st) * 32 + kq;
      dst[st] = ld16(arow + min(k, klim));
    }
  };
  int bi = umask ? (int)__builtin_ctzll(umask) : kWave;   // unit in ar[0]
  int ni = next_unit(bi);                                 // unit in ar[1]
  // issued unconditionally (absent units read zeros): a branch here would
  // make the compiler's waits for the W loads below conservative
  load_a(bi, ar[0]);
  load_a(ni, ar[1]);

  // ---- 6. base MFMAs --------------------------------------------------------
  f32x4_t acc[NTB];
#pragma unroll
  for (int tb = 0; tb < NTB; ++tb) acc[tb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < kDecWSteps; ++s) {
    if constexpr (MX) {   // (all requested)
    } else if constexpr (W8) {
      if ((s & 1) == 0 && s / 2 + kWPre < kWLoads) load_w(s / 2 + kWPre);
    } else {
      if (s + kDecWPre < kDecWSteps) load_w(s + kDecWPre);
    }
    // x columns past ks_end (past the chunk) are zero in LDS; k-steps past
    // the LDS chunk are clamped onto such columns
    int xc;
    u32x4_t wop;
    if constexpr (MX) {
      const int kp = min(ks_begin + (s & ~3), kDecMaxKc / 32 - 4);   // the group's first step
      xc = kp * 32 + 4 * kq + 8 * (s & 3);
      // (a block past the chunk is the chunk's last, against zero x)
      const int blk = min(kp * 32 + 4 * kq, kc - 32) / kMxBlock;
      wop = mx_bf16x8(wr[s / 4][s & 3], mx_scale_at(ws[s / 4], blk & 3));
    } else if constexpr (W8) {
      const int kp = min(ks_begin + (s & ~1), kDecMaxKc / 32 - 2);   // the step pair's first step
      xc = kp * 32 + 2 * kq + 8 * (s & 1);
      const u32x4_t raw = wr[s / 2];
      wop = (s & 1) ? e4m3x8_bf16(raw.z, raw.w) : e4m3x8_bf16(raw.x, raw.y);
    } else {
      xc = min(ks_begin + s, kDecMaxKc / 32 - 1) * 32 + kq;
      wop = wr[s];
    }
#pragma unroll
    for (int tb = 0; tb < NTB; ++tb) {
      const u32x4_t xo = *(const u32x4_t*)&sm.xs[(tb * 16 + l16) * XP + xc];
      acc[tb] = mfma16d(wop, xo, acc[tb]);
    }
    __builtin_amdgcn_sched_barrier(0);   // keep each step's load next to its MFMAs
  }
  // fixed-order sum of the two k-halves, then one coalesced fragment store
  if (kh == 1) {
#pragma unroll
    for (int tb = 0; tb < NTB; ++tb)
#pragma unroll
      for (int v = 0; v < 4; ++v) sm.red[rb][lane][tb * 4 + v] = acc[tb][v];
  }
  __syncthreads();
  if (kh == 0) {
#pragma unroll
    for (int tb = 0; tb < NTB; ++tb) {
      f32x4_t o;
#pragma unroll
      for (int v = 0; v < 4; ++v) o[v] = acc[tb][v] + sm.red[rb][lane][tb * 4 + v];
      // (nontemporal: the finish kernel reads it once, from another XCD)
      __builtin_nontemporal_store(o, (f32x4_t*)(a.ypart + part_off(c, tile, rb, tb, a.n_tiles, NTB) + lane * 4));
    }
  }

  // ---- 7. position table for k_finish --------------------------------------
  // Every sorted position's entry {adapter or -1, rank, scale bits}: the rank
  // is the segment's capped by the registered one, so a lying rank never reads
  // past the registered adapter and an emptied slot drops out. The lane of a
  // segment's first unit writes the segment's positions.
  if (pos_item) {   // uniform
    const int r = live_l ? min(rr_l, reg_r) : 0;
    const int ad = r > 0 ? m_ad : -1;
    const int4 e = make_int4(ad, ad >= 0 ? r : 0, __float_as_int(ad >= 0 ? m_sc : 0.f), 0);
    if (pos_lane)
      for (int t = ps_l; t < pe_l; ++t) a.pos[t] = e;
  }

  // ---- 8. shrink units -------------------------------------------------------
  // Each wave writes its own k-slice of the unit straight to
  // v_part[c][wave][t][j] (k_finish sums the 8 * n_chunks slices in a fixed
  // order): no barrier after the W MFMAs.
  float* vp = a.v_part + ((long long)c * kDecWaves + wave) * T * a.r_ws;
  auto shrink_unit = [&](u32x4_t* cur) {
    const int rows = __builtin_amdgcn_readlane(rows_l, bi);
    const int j0 = __builtin_amdgcn_readlane(j0_l, bi);
    const int ps = __builtin_amdgcn_readlane(ps_l, bi), pe = __builtin_amdgcn_readlane(pe_l, bi);
    const int tb_lo = ps / 16, tb_hi = (pe - 1) / 16;
    f32x4_t vacc[NTB];
#pragma unroll
    for (int tb = 0; tb < NTB; ++tb) vacc[tb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int st = 0; st < kDecASteps; ++st) {
      const int ks = wave + 8 * st;   // always < 32; operands past the chunk are zero
#pragma unroll
      for (int tb = 0; tb < NTB; ++tb) {
        if (tb < tb_lo || tb > tb_hi) continue;
        const u32x4_t xo = *(const u32x4_t*)&sm.xs[(tb * 16 + l16) * XP + ks * 32 + kq];
        vacc[tb] = mfma16d(cur[st], xo, vacc[tb]);
      }
    }
    // refill this buffer with the unit after next
    const int n2 = next_unit(ni);
    if (n2 < kWave) load_a(n2, cur);
#pragma unroll
    for (int tb = 0; tb < NTB; ++tb) {
      if (tb < tb_lo || tb > tb_hi) continue;
      const int t = tb * 16 + l16;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int jr = 4 * (lane / 16) + v;
        if (jr < rows && t >= ps && t < pe) __builtin_nontemporal_store(vacc[tb][v], vp + (long long)t * a.r_ws + j0 + jr);
      }
    }
    bi = ni;
    ni = n2;
  };
  while (bi < kWave) {   // uniform
    shrink_unit(ar[0]);
    if (bi >= kWave) break;
    shrink_unit(ar[1]);
  }
}

// ---------------------------------------------------------------------------
// stream, whole d_in: for a few tokens on wide layers (with an epilogue). A
// workgroup takes 16 NR (virtual) rows of W over the whole of d_in, its NW waves a
// part of d_in each (stream_tile.h), and adds their sums in wave order: no split
// of d_in over workgroups, one partial tile per row tile for k_finish.
// The first blocks are the shrink units, 16 rank rows of one segment each, which
// leave eight partials of v and the position table, as k_stream does.
//
// 32 rows and 8 waves; MXFP4 64 rows and 4 waves, which read x half as often per byte
// of W (one token, 4096 -> 2 x 14336 gated: 14.2 us, 16.0 with 32 rows and 8 waves).
// WQ = kWMxX (the base product of codes with codes, 32 rows and 8 waves): every batch that
// this path takes, of up to 64 tokens, in NTB blocks of 16; its x is as few bytes as W, and
// LDS would have to hold both forms of it, the shrink's being bf16. A shrink unit then
// takes its segment's blocks one after another and reads A for each, so few long segments
// on a long d_in take longer than the products (64 tokens of codes, quantised in the call,
// 14336 -> 4096, rank 16: 34 us without adapters, 57 with 32 segments, 111 with one).
// ---------------------------------------------------------------------------
template <int WQ, bool GATED, int NR, int NW, int NTB>
__global__ __launch_bounds__(NW * kWave) void k_stream_wide(DecodeArgs a, int n_units) {
  constexpr int TYPE = WQ == kWMxX ? kXMxX : WQ == kWMx ? kXMx : WQ == kWFp8 ? kXFp8w : kXBf16;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave), lane = tid % kWave;
  const int l16 = lane % 16, g = lane / 16;
  const int T = a.T, d_in = a.d_in, d_out = a.d_out;
  // the lane's tokens (absent ones repeat the last)
  int row[NTB];
#pragma unroll
  for (int t = 0; t < NTB; ++t) {
    row[t] = min(16 * t + l16, T - 1);
    if (a.sv.token_index) row[t] = min(max(a.sv.token_index[row[t]], 0), T - 1);   // uniform
  }
  const int b = blockIdx.x;
  if (b < n_units) {   // uniform: a shrink unit
    const SegView& sv = a.sv;
    const int nq = (a.pv.max_rank + 15) / 16, s = b / nq, j0 = b % nq * 16;
    if (s >= seg_count(sv)) return;
    const int ps = max(sv.seg_start[s], 0), pe = min(sv.seg_start[s + 1], T);
    const int ad0 = sv.seg_adapter[s], rk = sv.seg_rank[s];
    const bool live = pe > ps && ad0 >= 0 && ad0 < a.pv.capacity && rk > 0;
    const int rr = live ? min(rk, a.pv.max_rank) : 0;
    if (j0 == 0) {   // the rank the expand applies: capped by the registered one
      const int r = live ? min(rr, a.pv.rank[ad0]) : 0;
      const int ad = r > 0 ? ad0 : -1;
      for (int t = ps + tid; t < pe; t += NW * kWave)
        a.pos[t] = make_int4(ad, ad >= 0 ? r : 0, __float_as_int(ad >= 0 ? sv.seg_scale[s] : 0.f), 0);
    }
    const int rows = min(rr - j0, 16);
    if (rows <= 0) return;
    const char* A = (const char*)a.pv.base + ((long long)ad0 * a.pv.slot_elems + (long long)j0 * d_in) * 2;
    const uint32_t ao[1] = {(uint32_t)min(l16, rows - 1) * (uint32_t)(d_in * 2) + 16 * g};
#pragma unroll
    for (int tb = 0; tb < NTB; ++tb) {
      if (16 * tb + 16 <= ps || 16 * tb >= pe) continue;   // uniform
      const char* xp[1] = {(const char*)a.x + (long long)row[tb] * d_in * 2 + 16 * g};
      const int t = 16 * tb + l16;
      for (int w = wave; w < kDecWaves; w += NW) {
        f32x4_t v[1][1];
        stream_product<kXBf16, 1, 1, kDecWaves, false>(A, 0, ao, xp, d_in, w, g, v);
        float* vp = a.v_part + ((long long)w * T + t) * a.r_ws + j0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = 4 * g + i;
          if (j < rows && t >= ps && t < pe) vp[j] = v[0][0][i];
        }
      }
    }
    return;
  }
  __shared__ f32x4_t red[NW][NR * NTB][kWave];
  const long long wrb = w_row_bytes<TYPE>(d_in);
  const int v0 = 16 * NR * (b - n_units);
  const int f0 = GATED ? v0 / 2 : v0, nf = GATED ? d_out / 2 : d_out, fb = min(f0, nf - 1);
  constexpr int NO = GATED ? NR / 2 : NR;
  const char* wbase = (const char*)a.W + fb * wrb;
  uint32_t wo[NO], so[NO];
#pragma unroll
  for (int r = 0; r < NO; ++r) {
    const uint32_t f = (uint32_t)max(min(16 * r + l16, nf - 1 - f0), 0);
    wo[r] = f * (uint32_t)wrb + 16 * g;
    so[r] = 4 * f;
  }
  const long long xrb = x_row_bytes<TYPE>(d_in);
  auto xrow = [&](int t) {
    return (const char*)(TYPE == kXMxX ? (const void*)a.x_codes : a.x) + row[t] * xrb + x_group_bytes<TYPE>() * g;
  };
  f32x4_t acc[NR][NTB];
  if constexpr (TYPE >= kXMx) {
    const MxScales ms{(const char*)a.w_mx + 4ll * fb, 4ll * nf, 4ll * d_out, 4ll * T};
    stream_product_mx<TYPE, NR, NTB, NW, GATED>(wbase, nf * wrb, wo, ms, so, xrow, [&](int t) { return (const char*)a.x_mx + 4ll * row[t]; },
                                                d_in, wave, g, acc);
  } else {
    const char* xp[1] = {xrow(0)};
    stream_product<TYPE, NR, 1, NW, GATED>(wbase, nf * wrb, wo, xp, d_in, wave, g, acc);
  }
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int t = 0; t < NTB; ++t) red[wave][r * NTB + t][lane] = acc[r][t];
  __syncthreads();
  for (int q = wave; q < NR * NTB; q += NW) {
    f32x4_t sum = red[0][q][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] += red[w][q][lane][i];
    *(f32x4_t*)(a.ypart + part_off(0, v0 / 64, v0 / 16 % 4 + q / NTB, q % NTB, a.n_tiles, NTB) + lane * 4) = sum;
  }
}

// ---------------------------------------------------------------------------
// finish: one workgroup per (n-tile, 16-token block); wave w = row block w.
// Every load that does not depend on the adapter id is issued first (chunk
// partials, v partials, the position table, token_index); the B rows follow
// once the lane's adapter is known.
// ---------------------------------------------------------------------------
constexpr int kFinUnroll = 8;

// SL: the pool holds fused adapters over stacked projections (expand only
// the tile's slice window; a template flag, so plain pools keep a loop that
// starts at column 0: a run-time start measured 1 us slower)
// EPI: what follows the layer (kEpiNone: nothing; kEpiPlain, kEpiGated: a.epi).
template <int TT, bool W8, bool SL, int EPI>
__global__ __launch_bounds__(256) void k_finish_bf16(DecodeArgs a) {
  constexpr bool GATED = EPI == kEpiGated;
  constexpr int NTB = TT / 16;
  constexpr int kPre = 2;                // B column groups of 8 prefetched (ranks <= 16)
  const int tile = blockIdx.x / NTB, tb = blockIdx.x % NTB;
  const int tid = threadIdx.x;
  const int wave = tid / kWave, lane = tid % kWave;
  const int T = a.T, d_out = a.d_out;
  const int rb = wave;
  const bool lora = a.lora_on != 0;
  __shared__ float vs[16][kMaxRankWs + 4];
  __shared__ f32x4_t vgrp[4][256];

  const int t = tb * 16 + (lane % 16);   // this lane's token (sorted position)
  const int tc = min(t, T - 1);
  const int nv = tile * kDecRows + rb * 16 + 4 * (lane / 16);   // the lane's 4 rows (virtual when gated)
  // as rows of W (gated: a run of 4 virtual rows is one of W; runs past the
  // last feature are not stored)
  const int n = GATED ? ((nv >> 4) & 1) * (d_out / 2) + gated_feature(nv) : nv;
  int row = a.sv.token_index ? a.sv.token_index[tc] : tc;
  const int4 pe = lora ? a.pos[tc] : make_int4(-1, 0, 0, 0);

  // the chunk partials, all loads in flight (nontemporal, as they were
  // written: each is read once; measured 0.6 us faster per LoRA-on call on
  // the decode batch, same bits)
  const float* pbase = a.ypart + part_off(0, tile, rb, tb, a.n_tiles, NTB) + lane * 4;
  const long long cstride = (long long)a.n_tiles * 4 * NTB * 256;
  f32x4_t p[kFinUnroll];
#pragma unroll
  for (int u = 0; u < kFinUnroll; ++u)
    p[u] = __builtin_nontemporal_load((const f32x4_t*)(pbase + min(u, a.n_chunks - 1) * cstride));
  // FP8 weight: the row scales of the lane's 4 rows
  float wsc[4] = {1.f, 1.f, 1.f, 1.f};
  if constexpr (W8) {
#pragma unroll
    for (int v = 0; v < 4; ++v) wsc[v] = a.w_scale[min(n + v, d_out - 1)];
  }

  // v of the 16 tokens: sum of the stream kernel's slices [c][w]. A 16-byte
  // quad of one token is element e; G groups of threads each sum every G-th
  // slice of an element, then the groups are added in group order. The first
  // batch of slice loads is issued here, with the partials still in flight.
  // Rank quads summed and staged: all of them; for a fused pool only quads
  // [q0, q0 + nqv), the union over the block's 16 tokens of their windows in
  // this tile's slice, widened to multiples of 8 columns (the expand reads
  // v in groups of 8 from the window start rounded down to 8). Every wave
  // holds the same 16 tokens, so the union is the same in every wave.
  int q0 = 0, nqv = a.r_ws / 4;
  if constexpr (SL) {
    const int ad_ = pe.x, r_ = min(pe.y, a.pv.max_rank);
    const bool live_ = lora && ad_ >= 0 && ad_ < a.pv.capacity && r_ > 0 && t < T;
    int w0 = 0, w1 = r_;
    if (live_ && !GATED) slice_window(a.pv, tile * kDecRows, min(tile * kDecRows + kDecRows, d_out), r_, &w0, &w1);
    int lo = live_ ? (w0 & ~7) : 0x7fffffff, hi = live_ ? min(w1, r_) : 0;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
      lo = min(lo, __shfl_xor(lo, off, kWave));
      hi = max(hi, __shfl_xor(hi, off, kWave));
    }
    q0 = hi > lo ? lo / 4 : 0;
    nqv = hi > lo ? round_up8(hi) / 4 - q0 : 1;
  }
  const int E = 16 * nqv;
  const int G = E >= 256 ? 1 : E >= 128 ? 2 : 4;
  const int nsl = a.n_chunks * kDecWaves;
  const long long vstride = (long long)T * a.r_ws;
  auto vptr = [&](int e0) {
    const int e = min(e0 + tid / G, E - 1);
    return a.v_part + (long long)min(tb * 16 + e / nqv, T - 1) * a.r_ws + 4 * (q0 + e % nqv);
  };
  f32x4_t vq[kFinUnroll];
  {
    // without LoRA every lane reads the pool's zero block (an address select
    // keeps the loads unconditional)
    const float* vp = vptr(0);
#pragma unroll
    for (int u = 0; u < kFinUnroll; ++u)
      vq[u] = *(const f32x4_t*)(lora ? vp + min(tid % G + u * G, nsl - 1) * vstride : (const float*)a.pv.zeros);
  }
  // the slice loads stay ahead of the B loads, which wait for the position
  // entry: the v sums below then wait for them alone
  __builtin_amdgcn_sched_barrier(0);


  // B rows of the lane's adapter (first 16 rank columns), as soon as the
  // position entry is in
  const int ad = pe.x, r = min(pe.y, a.pv.max_rank);
  const bool live = lora && ad >= 0 && ad < a.pv.capacity && r > 0 && t < T;
  const uint16_t* Bb = (const uint16_t*)(live ? a.pv.base : a.pv.zeros) +
                       (live ? (long long)ad * a.pv.slot_elems + a.pv.b_offset : 0);
  const int bld = live ? round_up8(r) : 0;
  // a fused adapter over stacked projections: only the tile's slice window
  // of rank columns can be nonzero in its rows (from column jb, a multiple of 8)
  int jb = 0, je = r;
  if constexpr (SL) {
    int w0 = 0, w1 = r;
    if (live && !GATED) slice_window(a.pv, tile * kDecRows, min(tile * kDecRows + kDecRows, d_out), r, &w0, &w1);
    jb = w0 & ~7;
    je = min(w1, r);
  }
  u32x4_t b8[kPre][4];
#pragma unroll
  for (int g = 0; g < kPre; ++g)
#pragma unroll
    for (int v = 0; v < 4; ++v)
      b8[g][v] = ld16(Bb + (live ? bblk_off(min(n + v, d_out - 1), min(jb + 8 * g, bld - 8), d_out) : 0));

  // chunk partials summed in chunk order
  f32x4_t acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int u = 0; u < kFinUnroll; ++u)
    if (u < a.n_chunks) {
      acc[0] += p[u][0];
      acc[1] += p[u][1];
      acc[2] += p[u][2];
      acc[3] += p[u][3];
    }
  for (int c0 = kFinUnroll; c0 < a.n_chunks; c0 += kFinUnroll) {
#pragma unroll
    for (int u = 0; u < kFinUnroll; ++u)
      p[u] = __builtin_nontemporal_load((const f32x4_t*)(pbase + min(c0 + u, a.n_chunks - 1) * cstride));
#pragma unroll
    for (int u = 0; u < kFinUnroll; ++u)
      if (c0 + u < a.n_chunks) {
        acc[0] += p[u][0];
        acc[1] += p[u][1];
        acc[2] += p[u][2];
        acc[3] += p[u][3];
      }
  }

  if constexpr (W8) {
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] *= wsc[v];
  }

  if (lora) {
    for (int e0 = 0; e0 < E; e0 += 256 / G) {
      const int g = tid % G;
      const float* vp = vptr(e0);
      f32x4_t sum = f32x4_t{0.f, 0.f, 0.f, 0.f};
      for (int s0 = g; s0 < nsl; s0 += G * kFinUnroll) {
        if (e0 > 0 || s0 > g) {
#pragma unroll
          for (int u = 0; u < kFinUnroll; ++u) vq[u] = *(const f32x4_t*)(vp + min(s0 + u * G, nsl - 1) * vstride);
        }
#pragma unroll
        for (int u = 0; u < kFinUnroll; ++u)
          if (s0 + u * G < nsl) {
            sum[0] += vq[u][0];
            sum[1] += vq[u][1];
            sum[2] += vq[u][2];
            sum[3] += vq[u][3];
          }
      }
      vgrp[g][tid / G] = sum;
      lds_barrier();   // LDS only: the B loads stay in flight
      if (tid < 256 / G && e0 + tid < E) {
        f32x4_t tot = vgrp[0][tid];
        for (int gg = 1; gg < G; ++gg) {
          tot[0] += vgrp[gg][tid][0];
          tot[1] += vgrp[gg][tid][1];
          tot[2] += vgrp[gg][tid][2];
          tot[3] += vgrp[gg][tid][3];
        }
        const int ee = e0 + tid;
        *(f32x4_t*)&vs[ee / nqv][4 * (q0 + ee % nqv)] = tot;
      }
      lds_barrier();
    }
    if (live) {
      const float* vv = vs[lane % 16];
      float lsum[4] = {0.f, 0.f, 0.f, 0.f};
      for (int j0 = jb; j0 < je; j0 += 8) {
        u32x4_t bq[4];
        if (j0 - jb < 8 * kPre) {
#pragma unroll
          for (int v = 0; v < 4; ++v) bq[v] = b8[j0 - jb < 8 ? 0 : kPre - 1][v];
        } else {
#pragma unroll
          for (int v = 0; v < 4; ++v) bq[v] = ld16(Bb + bblk_off(min(n + v, d_out - 1), j0, d_out));
        }
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t wd = bq[v][e / 2];
            const float bv = bf16_bits_to_f32((uint16_t)((e & 1) ? (wd >> 16) : (wd & 0xffffu)));
            // columns j >= r of B are zero in the pool; v there is unused
            lsum[v] = fmaf(bv, j0 + e < r ? vv[j0 + e] : 0.f, lsum[v]);
          }
      }
      const float sc = __int_as_float(pe.z);
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[v] += sc * lsum[v];
    }
  }

  if constexpr (EPI != kEpiNone) {
    // bias, activation, gate and residual in fp32, one rounding. Gated: a
    // feature's gate row is in an even row block and its up row in the next
    // one, whose wave hands its sums over through LDS.
    __shared__ f32x4_t zup[2][kWave];
    const int d_y = GATED ? d_out / 2 : d_out;
    const int f = GATED ? gated_feature(nv) : n;         // first of the lane's features
    if (a.epi.bias) {
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[v] += elem_f32<uint16_t>(a.epi.bias, min(n + v, d_out - 1));
    }
    if constexpr (GATED) {
      if (rb & 1) zup[rb / 2][lane] = acc;
      __syncthreads();
      if (rb & 1) return;
    }
    if (t >= T) return;
    float o[4] = {acc[0], acc[1], acc[2], acc[3]};
    activate_n<true>(o, a.epi.act);
    row = min(max(row, 0), T - 1);
    const long long at = (long long)row * d_y + f;
    uint16_t* y = (uint16_t*)a.y;
    const uint16_t* res = (const uint16_t*)a.epi.residual;
    const bool vec = f + 4 <= d_y;
    float r4[4] = {0.f, 0.f, 0.f, 0.f};
    if (res) {
      if (vec) {
        const u32x2_t r = *(const u32x2_any*)(res + at);
#pragma unroll
        for (int v = 0; v < 4; ++v) r4[v] = __uint_as_float((v & 1) ? (r[v / 2] & 0xffff0000u) : (r[v / 2] << 16));
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v) r4[v] = f + v < d_y ? bf16_bits_to_f32(res[at + v]) : 0.f;
      }
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      if constexpr (GATED) o[v] *= zup[rb / 2][lane][v];
      if (res) o[v] += r4[v];
    }
    if (vec) {
      *(u32x2_any*)(y + at) = u32x2_t{(uint32_t)f32_to_bf16_bits(o[0]) | ((uint32_t)f32_to_bf16_bits(o[1]) << 16),
                                    (uint32_t)f32_to_bf16_bits(o[2]) | ((uint32_t)f32_to_bf16_bits(o[3]) << 16)};
    } else {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (f + v < d_y) y[at + v] = f32_to_bf16_bits(o[v]);
    }
    return;
  }
  if (t >= T) return;
  row = min(max(row, 0), T - 1);
  uint16_t* yr = (uint16_t*)a.y + (long long)row * d_out;
  if (n + 3 < d_out && (d_out & 3) == 0) {
    u32x2_t pk;
    pk.x = (uint32_t)f32_to_bf16_bits(acc[0]) | ((uint32_t)f32_to_bf16_bits(acc[1]) << 16);
    pk.y = (uint32_t)f32_to_bf16_bits(acc[2]) | ((uint32_t)f32_to_bf16_bits(acc[3]) << 16);
    *(u32x2_t*)(yr + n) = pk;
  } else {
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (n + v < d_out) yr[n + v] = f32_to_bf16_bits(acc[v]);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
bool decode_supported(int T, int n_seg_bound, int d_out, int max_rank) {
  // k_stream gives each item at most one wave's worth (64) of shrink units
  const long long n_tiles = (d_out + kDecRows - 1) / kDecRows;
  const long long units16 = (long long)n_seg_bound * ((max_rank + 15) / 16);
  return T >= 1 && T <= 64 && n_seg_bound <= kDecMaxSeg && units16 <= kWave * n_tiles;
}

// Rows per shrink unit: the smallest of 4, 8, 16 whose units (one per segment
// and row group) fit one per item of a chunk, so the A rows spread over as
// many items as possible; 16 when none does.
int decode_unit_rows(int n_seg_bound, int max_rank, int n_tiles) {
  for (int ur = 4; ur < 16; ur *= 2)
    if ((long long)n_seg_bound * ((max_rank + ur - 1) / ur) <= n_tiles) return ur;
  return 16;
}

// d_in chunk: a multiple of `unit` (at most the LDS x chunk), small enough that
// n_tiles * n_chunks covers the 256 CUs.
void decode_plan(int d_in, int d_out, int* n_tiles, int* kc, int* n_chunks, int unit) {
  *n_tiles = (d_out + kDecRows - 1) / kDecRows;
  int chunks = (d_in + kDecMaxKc - 1) / kDecMaxKc;
  while (*n_tiles * chunks < 256 && d_in / (chunks + 1) >= 256) ++chunks;
  int k = (d_in + chunks - 1) / chunks;
  k = (k + unit - 1) / unit * unit;
  if (k > kDecMaxKc) k = kDecMaxKc;
  *kc = k;
  *n_chunks = (d_in + k - 1) / k;
}

// Whole-d_in streaming with an epilogue: up to 8 tokens on layers of at least
// this many tiles of 64 rows. Both kernels, 4096 -> 2 x 14336 gated: one token
// 53.0 us against 59.5 with d_in split over workgroups (FP8 33.0 against 38.6),
// 4 tokens 54.5 against 62.8, 16 tokens 63.5 against 59.7; 4096 -> 8192: one token
// 22.0 against 19.0.
constexpr int kWideTiles = 256, kWideTokens = 8;

template <int TT, int WQ, int EPI>
static void launch_decode_epi(DecodeArgs a, hipStream_t st) {
  constexpr bool GATED = EPI == kEpiGated;
  const dim3 items(a.n_tiles * a.n_chunks);
  const int units = a.lora_on ? a.sv.n_seg * ((a.pv.max_rank + 15) / 16) : 0;   // of k_stream_wide
  if constexpr (WQ == kWMxX) {
    a.n_chunks = 1;   // what k_finish adds up
    hipLaunchKernelGGL((k_stream_wide<WQ, GATED, 2, 8, TT / 16>), dim3(units + 2 * a.n_tiles), dim3(8 * kWave), 0, st, a, units);
  } else if constexpr (EPI == kEpiNone) {
    hipLaunchKernelGGL((k_stream_bf16<TT, WQ, false, true>), items, dim3(kDecThreads), 0, st, a);
  } else {
    bool done = false;
    if constexpr (TT == 16) {
      if (a.T <= kWideTokens && a.n_tiles >= kWideTiles) {
        a.n_chunks = 1;   // what k_finish adds up
        constexpr int NR = WQ == kWMx ? 4 : 2, NW = WQ == kWMx ? 4 : 8;
        hipLaunchKernelGGL((k_stream_wide<WQ, GATED, NR, NW, 1>), dim3(units + 4 / NR * a.n_tiles), dim3(NW * kWave), 0, st, a, units);
        done = true;
      }
    }
    if constexpr (TT == 64) {
      if (a.d_in > 8192) {
        hipLaunchKernelGGL((k_stream_bf16<TT, WQ, GATED, true>), items, dim3(kDecThreads), 0, st, a);
        done = true;
      }
    }
    if (!done) hipLaunchKernelGGL((k_stream_bf16<TT, WQ, GATED, false>), items, dim3(kDecThreads), 0, st, a);
  }
  if (a.lora_on && a.pv.n_slices > 0)
    hipLaunchKernelGGL((k_finish_bf16<TT, WQ == kWFp8, true, EPI>), dim3(a.n_tiles * (TT / 16)), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((k_finish_bf16<TT, WQ == kWFp8, false, EPI>), dim3(a.n_tiles * (TT / 16)), dim3(256), 0, st, a);
}

template <int TT, int WQ>
static void launch_decode_tt(const DecodeArgs& a, hipStream_t st) {
  if (a.epi_kind == kEpiGated) launch_decode_epi<TT, WQ, kEpiGated>(a, st);
  else if (a.epi_kind == kEpiPlain) launch_decode_epi<TT, WQ, kEpiPlain>(a, st);
  else launch_decode_epi<TT, WQ, kEpiNone>(a, st);
}

template <int TT>
static void launch_decode_wq(const DecodeArgs& a, hipStream_t st) {
  if (a.x_mx) launch_decode_tt<TT, kWMxX>(a, st);
  else if (a.w_mx) launch_decode_tt<TT, kWMx>(a, st);
  else if (a.w_scale) launch_decode_tt<TT, kWFp8>(a, st);
  else launch_decode_tt<TT, kWBf16>(a, st);
}

void launch_decode_bf16(const DecodeArgs& a, hipStream_t st) {
  if (a.T <= 16) launch_decode_wq<16>(a, st);
  else if (a.T <= 32) launch_decode_wq<32>(a, st);
  else launch_decode_wq<64>(a, st);
}

}  // namespace mlora
