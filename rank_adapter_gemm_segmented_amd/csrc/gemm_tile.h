// gemm_tile.h -- tiles of the bf16 GEMM kernels: LDS rings fed by direct global
// -> LDS loads, their layout, and the main loop of the largest tile.
#pragma once
#include <utility>

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

// The same with a uniform base and a 32-bit byte offset per lane.
__device__ __forceinline__ void dma16_off(const void* base, uint32_t off, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(m0)
               : "memory", "m0");
}

// Wait until at most N of this wave's vector memory operations are in flight,
// then a workgroup barrier (LDS and scalar counters drained too; nothing else).
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
// W8: the W rows are FP8 codes of KB bytes (one per column), in the same ring.
template <int BR, int BT, int WR, int WT, int NB, int KB, int NX, bool W8 = false>
struct GCfg {
  static constexpr bool kW8 = W8;
  static constexpr int WRB = W8 ? KB : 2 * KB;             // bytes per LDS row of W
  static constexpr int kBR = BR, kBT = BT, kWR = WR, kWT = WT, kNB = NB, kKB = KB, kNX = NX;
  static constexpr int NWR = BR / WR, NWT = BT / WT;
  static constexpr int NW = NWR * NWT;
  static constexpr int NT = NW * kWave;
  static constexpr int MR = WR / 32, MT = WT / 32;        // 32x32 blocks per wave
  static constexpr int RB = 2 * KB;                        // bytes per LDS row of positions
  static constexpr int WSTAGE_B = BR * WRB, XSTAGE_B = BT * RB;   // ring slots
  static constexpr int DPW_W = BR * WRB / 1024 / NW;    // 1 KB loads per wave per stage: W rows
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
  // epilogue stores (store_epilogue, store_f32): 32 positions by half of the
  // wave's row blocks, fp32, per wave; LDS of a kernel with no other use for it
  static constexpr int EPI_MC = MR >= 2 ? MR / 2 : 1;
  static constexpr int EPI_BYTES = NW * 32 * (EPI_MC * 128 + 16);
  static constexpr int TILE_BYTES = MAIN_BYTES > EPI_BYTES ? MAIN_BYTES : EPI_BYTES;
  static_assert(KB == 32 || KB == 64 || (W8 && KB == 128), "stage depth");
  static_assert((BR * WRB) % (1024 * NW) == 0 && (BT * 2 * KB) % (1024 * NW) == 0,
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
  return KB == 128 ? r & 15 : KB == 64 ? (((r >> 1) ^ ((r & 1) << 2)) & 7) : ((r >> 2) & 3);
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

// The rows a wave loads: per stage DPW_W loads of the W ring and DPW_X of the
// position ring. Load i < DPW_W of wave w fills the W slot's 1 KB chunk
// J = i NW + w, load DPW_W + i the position slot's chunk J; lane l writes byte
// 1024 J + 16 l of the slot, i.e. one 16-byte slot of a row r, and so fetches
// chunk (slot ^ swizzle of r) of that row. wrow(r) and xrow(r) give the address
// of the tile's r-th W row and position.
template <class C>
struct TileSrc {
  static constexpr int kWSw = C::WRB / 2;                 // (gswz goes by the row's bytes)
  const char* src[C::DPW];
  int scol[C::DPW];                                       // first column of the lane's chunk
  template <class WRow, class XRow>
  __device__ __forceinline__ void set(int wave, int lane, WRow wrow, XRow xrow) {
#pragma unroll
    for (int i = 0; i < C::DPW; ++i) {
      const bool isx = i >= C::DPW_W;
      const int at = ((isx ? i - C::DPW_W : i) * C::NW + wave) * 64 + lane;   // 16-byte slot of the ring slot
      if (isx) {
        const int r = at / (C::RB / 16), c = (at % (C::RB / 16)) ^ gswz<C::kKB>(r);
        src[i] = (const char*)xrow(r) + 16 * c;
        scol[i] = 8 * c;
      } else {
        const int r = at / (C::WRB / 16), c = (at % (C::WRB / 16)) ^ gswz<kWSw>(r);
        src[i] = (const char*)wrow(r) + 16 * c;
        scol[i] = (C::kW8 ? 16 : 8) * c;
      }
    }
  }
  // load I of stage st (W rows for I < DPW_W, else positions) into the ring;
  // columns past d_in read `zeros`, so that every stage has the same count
  template <int I>
  __device__ __forceinline__ void issue(int st, uint32_t lds0, int wave, int d_in, const void* zeros) const {
    constexpr bool isx = I >= C::DPW_W;
    constexpr int j = isx ? I - C::DPW_W : I;
    const uint32_t slot = isx ? lds0 + C::XRING + (uint32_t)(st % C::kNX) * C::XSTAGE_B
                              : lds0 + (uint32_t)(st % C::kNB) * C::WSTAGE_B;
    const int k0 = st * C::kKB;
    dma16(sel_addr(k0 + scol[I] < d_in, src[I] + k0 * (isx || !C::kW8 ? 2 : 1), zeros),
          slot + (uint32_t)(j * C::NW + wave) * 1024);
  }
};

// The rows of the largest tile (below): as TileSrc, but a uniform base each for
// W and x and a 32-bit byte offset per lane and load, so that a load in the main
// loop costs no vector instruction but itself. (With a 64-bit address and a
// select against `zeros` per load, 7 to 9 instructions between two MFMAs, the
// wave fell behind its MFMAs: 1990 to 2095 us for the largest case.)
// The caller keeps W's tile and all of x within 4 GB of their bases.
template <class C>
struct PipeSrc {
  static_assert(C::NW == 4 && C::kNB >= C::kNX && !C::kW8, "one chunk column per lane");
  static constexpr int RPC = 1024 / C::RB, CPR = C::RB / 16;   // rows of a 1 KB chunk, 16-byte chunks of a row
  const char* wb;
  const char* xb;
  uint32_t off[C::DPW];
  int scol;                                               // first column of the lane's chunk, of every load
  template <class WOff, class XOff>
  __device__ __forceinline__ void set(int wave, int lane, const void* w, const void* x, WOff woff, XOff xoff) {
    wb = (const char*)w;
    xb = (const char*)x;
    // row r = RPC J + lane / CPR of chunk J = 4 j + wave: r mod 16 and with it the
    // swizzle do not go by j
    const int c = (lane % CPR) ^ gswz<C::kKB>(wave * RPC + lane / CPR);
    scol = 8 * c;
#pragma unroll
    for (int i = 0; i < C::DPW; ++i) {
      const bool isx = i < C::DPW_X;
      const int r = ((isx ? i : i - C::DPW_X) * C::NW + wave) * RPC + lane / CPR;
      off[i] = (isx ? xoff(r) : woff(r)) + 16 * c;
    }
  }
  // load I of iteration t, positions (stage t + NX) before W rows (stage t + NB);
  // WHOLE: the stages lie inside d_in
  template <int I, bool WHOLE>
  __device__ __forceinline__ void issue(int t, uint32_t lds0, int wave, int d_in, const void* zeros) const {
    constexpr bool isx = I < C::DPW_X;
    constexpr int j = isx ? I : I - C::DPW_X;
    const int st = t + (isx ? C::kNX : C::kNB);
    if (isx && C::kNB > C::kNX && st < 0) return;          // (before the first position stage)
    const uint32_t at = (isx ? lds0 + C::XRING + (uint32_t)(st % C::kNX) * C::XSTAGE_B
                             : lds0 + (uint32_t)(st % C::kNB) * C::WSTAGE_B) + (uint32_t)(j * C::NW + wave) * 1024;
    const char* base = (isx ? xb : wb) + (long long)st * (2 * C::kKB);
    if constexpr (WHOLE) dma16_off(base, off[I], at);
    else dma16(sel_addr(st * C::kKB + scol < d_in, base + off[I], zeros), at);
  }
};

// Main loop of the largest tile: 4 waves, one per SIMD, each 128 x 128 of a 256
// x 256 tile. A SIMD then has no second wave to cover a barrier or an LDS read
// with, so the loop is laid out by hand: MFMA by MFMA, with the reads of the
// next k-step's fragments and the loads of later stages placed between them.
//
// Why so large: a wave tile of 128 x 64 reads 6 KB of fragments for 8 MFMAs of
// 32 cycles, which with the ring's writes is the CU's 128 bytes of LDS per
// cycle; 128 x 128 reads 8 KB for 16, three quarters of it.
//
// The stage boundary lies inside a k-step: when the last k-step's first H MFMAs
// have issued, every fragment of the stage is in registers, the wave waits
// for its own loads of the next stage, and past the barrier the next stage is
// whole and this one's slots are free. The first fragments of the next stage
// are read under the remaining MFMAs.
template <class C>
__device__ __forceinline__ void pipe_mainloop(const PipeSrc<C>& s, int d_in, const void* zeros, char* lds,
                                              int wave, int lane, f32x16_t (&acc)[C::MR][C::MT]) {
  constexpr int KB = C::kKB, NB = C::kNB, NX = C::kNX, KS = KB / 16;
  constexpr int MR = C::MR, MT = C::MT, NM = MR * MT, NF = MR + MT;
  constexpr int H = NM / 4;
  // loads that may still be in flight at the boundary before stage s: those
  // requested after its positions' (with a deeper W ring also the W rows behind
  // them, whose stage comes later; its own W rows were requested before)
  constexpr int LATER = NB > NX ? C::DPW_W : 0, VMC = (NX - 2) * C::DPW + LATER;
  static_assert(KS % 2 == 0, "fragment sets alternate within a stage");
  static_assert(NF <= NM, "a read per MFMA at most");
  const int wr = wave / C::NWT, wt = wave % C::NWT, l32 = lane % 32, kh = lane / 32;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(lds));
  int fcol[KS];
#pragma unroll
  for (int kk = 0; kk < KS; ++kk) fcol[kk] = ((kk * 2 + kh) ^ gswz<KB>(l32)) * 16;
  const int wbase = (wr * C::kWR + l32) * C::RB, xbase = C::XRING + (wt * C::kWT + l32) * C::RB;

  u32x4_t fa[2][MR], fb[2][MT];
  // fragment f of k-step kk: the first MFMAs' operands first (W 0, positions 0 .. MT - 1, W 1 ..)
  auto frag = [&](int st, int kk, int set, int f) {
    if (f == 0 || f > MT) {
      const int m = f == 0 ? 0 : f - MT;
      fa[set][m] = *(const u32x4_t*)(lds + (st % NB) * C::WSTAGE_B + wbase + m * 32 * C::RB + fcol[kk]);
    } else {
      fb[set][f - 1] = *(const u32x4_t*)(lds + (st % NX) * C::XSTAGE_B + xbase + (f - 1) * 32 * C::RB + fcol[kk]);
    }
  };
  auto mfma = [&](int set, int i) {
    acc[i / MT][i % MT] = mfma32g(fa[set][i / MT], fb[set][i % MT], acc[i / MT][i % MT]);
    __builtin_amdgcn_sched_barrier(0);
  };

  // Iteration t of the loop requests position stage t + NX and W stage t + NB
  // into the slots that stage t has freed, one load per few MFMAs over three
  // quarters of a stage: a burst of them holds up the wave at issue, later ones
  // land too late. The first D1 go under the rest of stage t's last k-step, the
  // others under stage t + 1 before its own boundary. Prefill batch of 8 experts,
  // W ring of 3 and x ring of 2 stages: 1707 us, 1732 over half a stage, 1718 over
  // all of it; 2 + 2 stages: 1804 over half, 1885 over a quarter; stages of 32
  // columns (rows of half lines) in rings of 4: 1869.
  constexpr int NS = KS * NM;                            // MFMAs of a stage
  constexpr int SP = NS * 3 / 4;                         // over which its requests are spread
  auto upto = [](int i) constexpr { return i >= SP ? C::DPW : i * C::DPW / SP; };
  constexpr int D1 = upto(NM - H);
  auto request = [&]<bool WHOLE, int L0, int N>(std::bool_constant<WHOLE>, int t, std::integral_constant<int, L0>,
                                                std::integral_constant<int, N>) {
    [&]<int... J>(std::integer_sequence<int, J...>) { (s.template issue<L0 + J, WHOLE>(t, lds0, wave, d_in, zeros), ...); }
    (std::make_integer_sequence<int, N>{});
    if constexpr (N > 0) __builtin_amdgcn_sched_barrier(0);
  };
  // what is requested after MFMA I of a stage (counted from the boundary before it)
  auto request_at = [&]<int I>(auto whole, int t, std::integral_constant<int, I>) {
    constexpr int L0 = upto(I), L1 = upto(I + 1);
    request(whole, t, std::integral_constant<int, L0>{}, std::integral_constant<int, L1 - L0>{});
  };
  auto each = []<int... I>(std::integer_sequence<int, I...>, auto f) { (f(std::integral_constant<int, I>{}), ...); };
  auto stage = [&](auto whole, int st) {
    each(std::make_integer_sequence<int, (KS - 1) * NM>{}, [&](auto ic) {
      constexpr int I = ic.value, kk = I / NM, i = I % NM;
      mfma(kk & 1, i);
      if constexpr (i * NF / NM != (i + 1) * NF / NM) {   // NF reads spread over NM MFMAs
        frag(st, kk + 1, (kk + 1) & 1, i * NF / NM);
        __builtin_amdgcn_sched_barrier(0);
      }
      request_at(whole, st - 1, std::integral_constant<int, NM - H + I>{});
    });
    constexpr int LS = (KS - 1) & 1;
    each(std::make_integer_sequence<int, H>{}, [&](auto ic) {
      mfma(LS, ic.value);
      request_at(whole, st - 1, std::integral_constant<int, NS - H + ic.value>{});
    });
    vm_barrier<VMC>();
    __builtin_amdgcn_sched_barrier(0);
    each(std::make_integer_sequence<int, NM - H>{}, [&](auto ic) {
      constexpr int I = ic.value;
      mfma(LS, H + I);
      // a read per MFMA, or more where the fragments outnumber them (64 x 64 per wave)
      constexpr int F0 = NF <= NM - H ? (I < NF ? I : NF) : I * NF / (NM - H);
      constexpr int F1 = NF <= NM - H ? (I + 1 < NF ? I + 1 : NF) : (I + 1) * NF / (NM - H);
#pragma unroll
      for (int f = F0; f < F1; ++f) frag(st + 1, 0, 0, f);
      __builtin_amdgcn_sched_barrier(0);
      request_at(whole, st, ic);
    });
  };

  const int nst = (d_in + KB - 1) / KB, nwhole = d_in / KB;
  constexpr std::false_type part{};
  // the iterations before the first, the last of them its first part only
#pragma unroll
  for (int t = -NB; t < -1; ++t) request(part, t, std::integral_constant<int, 0>{}, std::integral_constant<int, C::DPW>{});
  request(part, -1, std::integral_constant<int, 0>{}, std::integral_constant<int, D1>{});
  vm_barrier<VMC + D1>();
#pragma unroll
  for (int f = 0; f < NF; ++f) frag(0, 0, 0, f);
  int st = 0;
  for (; st + NB < nwhole; ++st) stage(std::true_type{}, st);   // every request is a whole stage
  for (; st < nst; ++st) stage(part, st);
  vm_barrier<0>();   // the ring's last loads (zeros) land before the LDS is reused
}

// Main loop of the smaller tiles (two waves per SIMD): a barrier per stage, the
// fragments of k-step kk + 1 read while k-step kk is multiplied.
//
// FP8 W: a lane reads 16 codes at once, two k-steps' worth, and converts 8 of
// them per step (e4m3 is exact in bf16). Lane half h's codes are columns 32 q +
// 16 h .. + 15 of step pair q, so the position fragments of steps 2 q and 2 q + 1
// are columns 32 q + 16 h .. + 7 and + 8 .. + 15: which column sits in which k slot
// of an MFMA does not matter as long as both operands agree.
template <class C>
__device__ __forceinline__ void ring_mainloop(const TileSrc<C>& s, int d_in, const void* zeros, char* lds,
                                              int wave, int lane, f32x16_t (&acc)[C::MR][C::MT]) {
  constexpr int KB = C::kKB, NB = C::kNB, NX = C::kNX, KS = KB / 16;
  const int wr = wave / C::NWT, wt = wave % C::NWT, l32 = lane % 32, kh = lane / 32;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(lds));
  int fx[KS], fw[KS];                                     // byte of the lane's chunk in its row
#pragma unroll
  for (int kk = 0; kk < KS; ++kk) {
    fx[kk] = ((C::kW8 ? (kk >> 1) * 4 + 2 * kh + (kk & 1) : kk * 2 + kh) ^ gswz<KB>(l32)) * 16;
    fw[kk] = ((C::kW8 ? (kk >> 1) * 2 + kh : kk * 2 + kh) ^ gswz<TileSrc<C>::kWSw>(l32)) * 16;
  }
  auto load_w = [&](int st) {
    [&]<int... I>(std::integer_sequence<int, I...>) { (s.template issue<I>(st, lds0, wave, d_in, zeros), ...); }
    (std::make_integer_sequence<int, C::DPW_W>{});
  };
  auto load_x = [&](int st) {
    [&]<int... I>(std::integer_sequence<int, I...>) { (s.template issue<C::DPW_W + I>(st, lds0, wave, d_in, zeros), ...); }
    (std::make_integer_sequence<int, C::DPW_X>{});
  };
#pragma unroll
  for (int t = 0; t < NB - 1; ++t) {
    load_w(t);
    if (t >= NB - NX) load_x(t - (NB - NX));
  }
  const int nst = (d_in + KB - 1) / KB;
  for (int st = 0; st < nst; ++st) {
    vm_barrier<C::VMC>();
    load_w(st + NB - 1);
    load_x(st + NX - 1);
    const char* Lw = lds + (st % NB) * C::WSTAGE_B + (wr * C::kWR + l32) * C::WRB;
    const char* Lx = lds + C::XRING + (st % NX) * C::XSTAGE_B + (wt * C::kWT + l32) * C::RB;
    u32x4_t fa[2][C::MR], fb[2][C::MT];                   // (FP8: fa by step pair)
    auto frag = [&](int kk) {
      if (!C::kW8 || kk % 2 == 0) {
#pragma unroll
        for (int m = 0; m < C::MR; ++m)
          fa[C::kW8 ? (kk >> 1) & 1 : kk & 1][m] = *(const u32x4_t*)(Lw + m * 32 * C::WRB + fw[kk]);
      }
#pragma unroll
      for (int n = 0; n < C::MT; ++n) fb[kk & 1][n] = *(const u32x4_t*)(Lx + n * 32 * C::RB + fx[kk]);
    };
    frag(0);
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      if (kk + 1 < KS) frag(kk + 1);
#pragma unroll
      for (int m = 0; m < C::MR; ++m) {
        u32x4_t wa;
        if constexpr (C::kW8) {
          const u32x4_t raw = fa[(kk >> 1) & 1][m];
          wa = (kk & 1) ? e4m3x8_bf16(raw.z, raw.w) : e4m3x8_bf16(raw.x, raw.y);
        } else {
          wa = fa[kk & 1][m];
        }
#pragma unroll
        for (int n = 0; n < C::MT; ++n) acc[m][n] = mfma32g(wa, fb[kk & 1][n], acc[m][n]);
      }
    }
    if constexpr (!C::kW8) {
      __builtin_amdgcn_sched_group_barrier(0x100, C::MR + C::MT, 0);
#pragma unroll
      for (int kk = 0; kk + 1 < KS; ++kk) sched_reads_over_mfma<C::MR + C::MT, C::MR * C::MT>();
      __builtin_amdgcn_sched_group_barrier(0x008, C::MR * C::MT, 0);
    }
  }
  vm_barrier<0>();
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
                                               int p0, int p_end, int d_out, const EpiView& epi, const float* w_scale,
                                               void* y_, RowOf row_of) {
  constexpr int MC = C::EPI_MC;                         // row blocks per pass
  constexpr int NF = MC * (GATED ? 16 : 32);            // features per pass
  constexpr int PITCH = MC * 128 + 16;                  // tile row (bytes)
  constexpr int CPR = NF / 8, PPP = kWave / CPR;        // lanes per position, positions per step
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
    float sc[8], su[8];                                       // (FP8 W)
    if constexpr (C::kW8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sc[e] = w_scale[wrow_of<GATED>(vr + lr + e, d_out)];
        su[e] = GATED ? w_scale[wrow_of<GATED>(vr + lr + 16 + e, d_out)] : 0.f;
      }
    }
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
      auto finish = [&](auto plain) {   // plain: whole 16-byte pieces, no residual
        constexpr bool PLAIN = decltype(plain)::value;
#pragma unroll 2
        for (int tb = 0; tb < 32; tb += PPP) {
          const int tl = tb + lane / CPR;
          const int p = p0 + n * 32 + tl;
          if (p >= p_end || col >= d_y) continue;
          const long long at = (long long)row_of(p) * d_y + col;
          float r8[8], o[8];
          const bool whole = PLAIN || col + 8 <= d_y;
          if constexpr (!PLAIN) {
            if (res && whole) {
              const u32x4_t r = *(const u32x4_any*)(res + at);
#pragma unroll
              for (int e = 0; e < 8; ++e) r8[e] = __uint_as_float((e & 1) ? (r[e / 2] & 0xffff0000u) : (r[e / 2] << 16));
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e) r8[e] = res && col + e < d_y ? bf16_bits_to_f32(res[at + e]) : 0.f;
            }
          }
          const char* tr = tile + tl * PITCH + lr * 4;
          const f32x4_t z0 = *(const f32x4_t*)tr, z1 = *(const f32x4_t*)(tr + 16);
          f32x4_t u0 = z0, u1 = z1;
          if constexpr (GATED) {
            u0 = *(const f32x4_t*)(tr + 64);
            u1 = *(const f32x4_t*)(tr + 80);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float z = e < 4 ? z0[e] : z1[e - 4];
            o[e] = C::kW8 ? fmaf(z, sc[e], b[e]) : z + b[e];
          }
          activate_n<true>(o, epi.act);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float u = e < 4 ? u0[e] : u1[e - 4];
            if constexpr (GATED) o[e] *= C::kW8 ? fmaf(u, su[e], bu[e]) : u + bu[e];
            if constexpr (!PLAIN) {
              if (res) o[e] += r8[e];
            }
          }
          if (whole) {
            *(u32x4_any*)(y + at) = u32x4_t{cvt_pk_bf16(o[0], o[1]), cvt_pk_bf16(o[2], o[3]), cvt_pk_bf16(o[4], o[5]), cvt_pk_bf16(o[6], o[7])};
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (col + e < d_y) y[at + e] = f32_to_bf16_bits(o[e]);
          }
        }
      };
      if (vec && !res) finish(std::true_type{});   // uniform
      else finish(std::false_type{});
    }
  }
}

// Store of a wave's accumulators in fp32, rows v0 .. v0 + WR - 1 by positions
// p0 .. p0 + WT - 1 below p_end, position p to row p of y (pitch: d_out rounded up
// to a multiple of 4, so that every store is whole), bias added.
template <class C>
__device__ __forceinline__ void store_f32(f32x16_t (&acc)[C::MR][C::MT], char* lds, int wave, int lane, int v0, int p0,
                                          int p_end, int d_out, const uint16_t* bias, const float* w_scale, float* y, int pitch) {
  constexpr int MC = C::EPI_MC;   // row blocks per pass through the LDS tile, as store_epilogue
  constexpr int PITCH = MC * 128 + 16, CPR = MC * 8, PPP = kWave / CPR;
  const int l32 = lane % 32, h = lane / 32, c = lane % CPR;
  char* tile = lds + wave * 32 * PITCH;
#pragma unroll
  for (int m0 = 0; m0 < C::MR; m0 += MC) {
    const int col = v0 + m0 * 32 + 4 * c;
    float b[4], sc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      b[i] = bias ? elem_f32<uint16_t>(bias, min(col + i, d_out - 1)) : 0.f;
      sc[i] = C::kW8 ? w_scale[min(col + i, d_out - 1)] : 1.f;
    }
#pragma unroll
    for (int n = 0; n < C::MT; ++n) {
#pragma unroll
      for (int m = 0; m < MC; ++m)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *(f32x4_t*)(tile + l32 * PITCH + (m * 32 + 8 * q + 4 * h) * 4) =
              f32x4_t{acc[m0 + m][n][4 * q], acc[m0 + m][n][4 * q + 1], acc[m0 + m][n][4 * q + 2], acc[m0 + m][n][4 * q + 3]};
#pragma unroll 4
      for (int tb = 0; tb < 32; tb += PPP) {
        const int tl = tb + lane / CPR, p = p0 + n * 32 + tl;
        if (p >= p_end || col >= d_out) continue;
        f32x4_t z = *(const f32x4_t*)(tile + tl * PITCH + 16 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = C::kW8 ? fmaf(z[i], sc[i], b[i]) : z[i] + b[i];
        *(f32x4_t*)(y + (long long)p * pitch + col) = z;
      }
    }
  }
}

}  // namespace mlora
