// gemm_tile.h -- tiles of the bf16 GEMM kernels: LDS rings fed by direct global
// -> LDS loads, their layout, and the main loop of the largest tile.
#pragma once
#include "common.h"
#include "epilogue.h"

namespace mlora {

__device__ __forceinline__ f32x16_t mfma32g(u32x4_t a, u32x4_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
}

// LDS address (byte offset in the workgroup's LDS) of a pointer into __shared__ memory
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

// Direct global -> LDS load (gfx950 LDS DMA): the wave's 64 lanes each fetch
// 16 bytes from their own global address and the data lands in LDS, lane l at
// byte m0 + 16 l, without passing through registers. Issued as inline
// assembly so that the compiler, which would otherwise wait for every
// outstanding DMA before any LDS read, leaves the waits to the stage ring
// below. One wait state separates the M0 write from its use.
__device__ __forceinline__ void dma16(const void* g, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(g), "s"(m0)
               : "memory", "m0");
}

// Wait until at most N of this wave's vector memory operations are in flight,
// then a workgroup barrier (LDS and scalar counters drained too; nothing else).
// The same load marked nontemporal, for W rows that the launch reads once
// (at most two position tiles, which run in the same round): measured on the
// verify and heterogeneous batches, their LoRA-off passes took 1-2 us less
// (45.2-46.3 against 47.3-47.8 us, 38.0 against 39.1 us). Where more position
// tiles re-read a W panel in later rounds (prefill) the mark lost about 10%
// (gate/up), and the positions' rows, re-read by every row tile, lost 5-18%.
__device__ __forceinline__ void dma16_nt(const void* g, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off nt" ::"v"(g), "s"(m0)
               : "memory", "m0");
}

template <int N>
__device__ __forceinline__ void vm_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// KB: k per stage (32 or 64). A stage is the tile's BR W rows and its BT
// positions over KB columns. The stages reach LDS by direct loads into two
// rings, one for the W rows (NB slots, NB - 1 stages in flight while one is
// multiplied) and one for the positions (NX slots, NX - 1 in flight). Rows
// are 2 KB bytes (KB bf16), unpadded, and 16-byte chunk c of row r sits in slot
// c ^ gswz(r) of the row, so the rows read together by one fragment load fall
// in distinct LDS banks.
template <int BR, int BT, int WR, int WT, int NB, int KB, int NX>
struct GCfg {
  static constexpr int NWR = BR / WR, NWT = BT / WT;
  static constexpr int NW = NWR * NWT;
  static constexpr int NT = NW * kWave;
  static constexpr int MR = WR / 32, MT = WT / 32;        // 32x32 blocks per wave
  static constexpr int RB = 2 * KB;                        // bytes per LDS row
  static constexpr int WSTAGE_B = BR * RB, XSTAGE_B = BT * RB;   // ring slots
  static constexpr int DPW_W = BR * 2 * KB / 1024 / NW;    // 1 KB loads per wave per stage: W rows
  static constexpr int DPW_X = BT * 2 * KB / 1024 / NW;    // and positions
  static constexpr int DPW = DPW_W + DPW_X;
  static constexpr int XRING = NB * WSTAGE_B;              // byte offset of the position ring
  static constexpr int MAIN_BYTES = NB * WSTAGE_B + NX * XSTAGE_B;
  // DMAs a wave has issued after stage st's position DMAs when stage st is
  // multiplied (its W DMAs were issued earlier still)
  static constexpr int VMC = (NX - 2) * DPW;
  // small row tiles get extra LDS so the epilogue stages many segment runs at
  // once; the y tile of the store passes through the same LDS
  static constexpr int YT_BYTES = NW * WT * (2 * WR + 16);
  static constexpr int LDS_BYTES0 = MAIN_BYTES > 96 * 1024 ? MAIN_BYTES : 96 * 1024;
  static constexpr int LDS_BYTES = LDS_BYTES0 > YT_BYTES ? LDS_BYTES0 : YT_BYTES;
  static_assert(KB == 32 || KB == 64, "stage depth");
  static_assert((BR * 2 * KB) % (1024 * NW) == 0 && (BT * 2 * KB) % (1024 * NW) == 0,
                "each ring's stage splits into whole loads per wave");
  static_assert(NB >= 2 && NX >= 2 && NB >= NX && VMC <= 63, "ring depths and vmcnt range");
};

// Slot permutation of row r (depends on r mod 16 only). A fragment read has
// lane l take row l % 32 at one chunk. gfx950 serves a 16-byte LDS read 16
// lanes (256 bytes) at a time, so the 16 rows of a lane group must land on
// 16 distinct 16-byte bank groups modulo 256 bytes. KB = 64: two rows per
// 256 bytes; rows of equal parity take distinct slots through r >> 1, and
// the parity flips the slot's top bit. KB = 32: four rows per 256 bytes,
// separated through r >> 2. Both were checked with the LDS bank-conflict
// counter on a read-pattern probe (no conflicts), where the plain r & 7 and
// (r >> 1) & 3 permutations conflicted two ways.
template <int KB>
__device__ __forceinline__ int gswz(int r) {
  return KB == 64 ? (((r >> 1) ^ ((r & 1) << 2)) & 7) : ((r >> 2) & 3);
}

// Scheduling hint for one k-step: the R fragment reads of the next k-step
// spread over the M MFMAs of this one (one read, then its share of MFMAs).
template <int R, int M, int J = 0>
__device__ __forceinline__ void sched_reads_over_mfma() {
  if constexpr (J < R) {
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                          // DS read
    __builtin_amdgcn_sched_group_barrier(0x008, M * (J + 1) / R - M * J / R, 0);  // MFMA
    sched_reads_over_mfma<R, M, J + 1>();
  }
}

// Store of a wave's accumulators with an epilogue: rows v0 .. v0 + WR - 1
// (virtual rows when gated; v0 is a multiple of 32) by positions p0 .. p0 +
// WT - 1, of which those below p_end are stored to row row_of(p) of y. 32
// positions and half of the wave's row blocks at a time pass through a
// wave-private fp32 LDS tile [position][row], so that each lane ends with 8
// consecutive features of one position (and, gated, both their rows): the bias
// of its features is loaded once, the residual is one 16-byte load, y is
// rounded once and stored as 16 bytes, consecutive lanes covering a row.
template <class C, bool GATED, class RowOf>
__device__ __forceinline__ void store_epilogue(f32x16_t (&acc)[C::MR][C::MT], char* lds, int wave, int lane, int v0,
                                               int p0, int p_end, int d_out, const EpiView& epi, void* y_,
                                               RowOf row_of) {
  constexpr int MC = C::MR >= 2 ? C::MR / 2 : 1;        // row blocks per pass
  constexpr int NF = MC * (GATED ? 16 : 32);            // features per pass
  constexpr int PITCH = MC * 128 + 16;                  // tile row (bytes)
  constexpr int CPR = NF / 8, PPP = kWave / CPR;        // lanes per position, positions per step
  static_assert(C::NW * 32 * PITCH <= C::LDS_BYTES, "epilogue tile fits the LDS");
  const int l32 = lane % 32, h = lane / 32, c = lane % CPR;
  const int d_y = GATED ? d_out / 2 : d_out;
  char* tile = lds + wave * 32 * PITCH;
  uint16_t* y = (uint16_t*)y_;
  const uint16_t* res = (const uint16_t*)epi.residual;
  const bool vec = d_y % 8 == 0;
  const int lr = GATED ? (c / 2) * 32 + (c % 2) * 8 : 8 * c;   // the lane's rows in the tile (gated: + 16 the up rows)
#pragma unroll
  for (int m0 = 0; m0 < C::MR; m0 += MC) {
    const int vr = v0 + m0 * 32;
    const int col = (GATED ? vr / 2 : vr) + 8 * c;
    float b[8], bu[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      b[e] = epi.bias ? elem_f32<uint16_t>(epi.bias, wrow_of<GATED>(vr + lr + e, d_out)) : 0.f;
      bu[e] = GATED && epi.bias ? elem_f32<uint16_t>(epi.bias, wrow_of<GATED>(vr + lr + 16 + e, d_out)) : 0.f;
    }
#pragma unroll
    for (int n = 0; n < C::MT; ++n) {
#pragma unroll
      for (int m = 0; m < MC; ++m)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *(f32x4_t*)(tile + l32 * PITCH + (m * 32 + 8 * q + 4 * h) * 4) =
              f32x4_t{acc[m0 + m][n][4 * q], acc[m0 + m][n][4 * q + 1], acc[m0 + m][n][4 * q + 2], acc[m0 + m][n][4 * q + 3]};
      // (wave-private tile: the wave's own LDS writes are ordered before its reads)
#pragma unroll 1
      for (int tb = 0; tb < 32; tb += PPP) {
        const int tl = tb + lane / CPR;
        const int p = p0 + n * 32 + tl;
        if (p >= p_end || col >= d_y) continue;
        const long long at = (long long)row_of(p) * d_y + col;
        float r8[8], o[8];
        if (res && vec) {   // uniform (col + 8 <= d_y then)
          const u32x4_t r = *(const u32x4_t*)(res + at);
#pragma unroll
          for (int e = 0; e < 8; ++e) r8[e] = __uint_as_float((e & 1) ? (r[e / 2] & 0xffff0000u) : (r[e / 2] << 16));
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) r8[e] = res && col + e < d_y ? bf16_bits_to_f32(res[at + e]) : 0.f;
        }
        const char* tr = tile + tl * PITCH + lr * 4;
        const f32x4_t z0 = *(const f32x4_t*)tr, z1 = *(const f32x4_t*)(tr + 16);
        f32x4_t u0 = z0, u1 = z1;
        if constexpr (GATED) {
          u0 = *(const f32x4_t*)(tr + 64);
          u1 = *(const f32x4_t*)(tr + 80);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = (e < 4 ? z0[e] : z1[e - 4]) + b[e];
        activate_n<true>(o, epi.act);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if constexpr (GATED) o[e] *= (e < 4 ? u0[e] : u1[e - 4]) + bu[e];
          if (res) o[e] += r8[e];
        }
        if (vec) {
          *(u32x4_t*)(y + at) = __builtin_bit_cast(u32x4_t, pack_bf16x8(o));
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (col + e < d_y) y[at + e] = f32_to_bf16_bits(o[e]);
        }
      }
    }
  }
}

}  // namespace mlora
