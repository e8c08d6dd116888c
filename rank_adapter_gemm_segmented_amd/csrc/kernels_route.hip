// kernels_route.hip -- top-k expert choice of a batch and its segments.
//
// A token's weights are w_j = exp(l_j - m) / sum exp(l_i - m) at its k largest
// logits (m the largest, the sum over all experts or over the chosen ones),
// and the chosen (token, j) slots are grouped by expert, slots of one expert
// in slot order, as mlora_build_segments groups tokens by adapter.
//
// Bound by latency: a prefill batch of 4096 tokens over 64 experts reads 1 MB
// and writes 0.5 MB, a fraction of a microsecond of bandwidth. So the work is
// one launch where one workgroup holds the batch, else two: the choice with
// each block's count per expert, then the grouping, in which every block adds
// up the counts of the blocks before it by itself. No atomics on global memory
// and no order that depends on timing: the result is unique. Measured: 64
// tokens over 128 experts, top 8, 8.2 us; 4096 tokens over 64 experts, top 8, 4.6
// us for the choice and 5.5 for the grouping.
#include "../../include/mlora.h"
#include "experts.h"

namespace mlora {

constexpr int kRtThreads = 1024, kRtWaves = kRtThreads / kWave;
constexpr int kRtMaxBlocks = 256;   // blocks of the grouping (each reads all their counts)
constexpr int kRtMinTokens = 32;    // tokens per block at least

// Wave reductions on the vector ALUs (row shifts, then the row broadcasts),
// the result in every lane. Six steps of a lane exchange through LDS took three
// times as long, and a choice is k of these in a row.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t old, uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {   // (0 is neutral)
  v = max(v, dpp<0x111, 0xf>(0u, v));   // row_shr 1, 2, 4, 8
  v = max(v, dpp<0x112, 0xf>(0u, v));
  v = max(v, dpp<0x114, 0xf>(0u, v));
  v = max(v, dpp<0x118, 0xf>(0u, v));
  v = max(v, dpp<0x142, 0xa>(0u, v));   // row_bcast 15, 31
  v = max(v, dpp<0x143, 0xc>(0u, v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, kWave - 1);
}
__device__ __forceinline__ float wave_sum(float f) {
  auto add = [](float x, uint32_t y) { return x + __uint_as_float(y); };
  f = add(f, dpp<0x111, 0xf>(0u, __float_as_uint(f)));
  f = add(f, dpp<0x112, 0xf>(0u, __float_as_uint(f)));
  f = add(f, dpp<0x114, 0xf>(0u, __float_as_uint(f)));
  f = add(f, dpp<0x118, 0xf>(0u, __float_as_uint(f)));
  f = add(f, dpp<0x142, 0xa>(0u, __float_as_uint(f)));
  f = add(f, dpp<0x143, 0xc>(0u, __float_as_uint(f)));
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(f), kWave - 1));
}

// The same in 64 bits: the two halves of each lane's addend shift separately.
__device__ __forceinline__ double wave_sum64(double f) {
  auto add = [](double x, auto shift) {
    const unsigned long long u = __double_as_longlong(x);
    const uint32_t lo = shift((uint32_t)u), hi = shift((uint32_t)(u >> 32));
    return x + __longlong_as_double((long long)(((unsigned long long)hi << 32) | lo));
  };
  f = add(f, [](uint32_t v) { return dpp<0x111, 0xf>(0u, v); });
  f = add(f, [](uint32_t v) { return dpp<0x112, 0xf>(0u, v); });
  f = add(f, [](uint32_t v) { return dpp<0x114, 0xf>(0u, v); });
  f = add(f, [](uint32_t v) { return dpp<0x118, 0xf>(0u, v); });
  f = add(f, [](uint32_t v) { return dpp<0x142, 0xa>(0u, v); });
  f = add(f, [](uint32_t v) { return dpp<0x143, 0xc>(0u, v); });
  const unsigned long long u = __double_as_longlong(f);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, kWave - 1);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), kWave - 1);
  return __longlong_as_double((long long)(((unsigned long long)hi << 32) | lo));
}

// Order of a logit: larger is better, ties go to the lowest expert. NaN and
// -inf get 0 and are never chosen.
__device__ __forceinline__ uint32_t logit_key(float l) {
  if (!(l > -INFINITY)) return 0u;
  const uint32_t u = l == 0.f ? 0u : __float_as_uint(l);   // (-0 ties with 0)
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// exp(l - m) with inf - inf counted as 0 (equal infinite logits share the weight)
__device__ __forceinline__ float exp_from(float l, float m) { return l == m ? 1.0f : expf(l - m); }

// Choice of one token by one wave (many experts or choices): NV experts per lane
// (expert lane + 64 i). k rounds of a wave-wide maximum; the lowest expert that
// holds it is found with a ballot per i and drops out. Lane j keeps choice j.
template <typename E_, int NV>
__device__ __forceinline__ void choose1(const RouteArgs& a, int t, int lane, int* id, float* w) {
  uint32_t key[NV], lv[NV], my_key = 0u, top = 0u;
  const E_* __restrict__ row = (const E_*)a.logits + (long long)t * a.E;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + kWave * i;
    const float l = elem_f32<E_>(row, min(e, a.E - 1));
    lv[i] = key[i] = e < a.E ? logit_key(l) : 0u;
  }
  int my_id = -1;
  for (int j = 0; j < a.k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) best = max(best, key[i]);
    const uint32_t m = wave_max(best);                 // uniform
    if (m == 0u) break;                                // nothing left to choose
    int win = -1;                                      // uniform
#pragma unroll
    for (int i = NV - 1; i >= 0; --i) {
      const unsigned long long h = __ballot(key[i] == m);
      if (h) win = kWave * i + (int)__builtin_ctzll(h);
    }
    if (j == 0) top = m;
    if (lane == j) {
      my_id = win;
      my_key = m;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (win == lane + kWave * i) key[i] = 0u;
  }
  const float m = key_logit(top);
  const float mine = my_id >= 0 ? exp_from(key_logit(my_key), m) : 0.f;
  float sum = mine;
  if (!a.renorm) {   // uniform
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lv[i] != 0u) sum += exp_from(key_logit(lv[i]), m);
  }
  sum = wave_sum(sum);
  *id = my_id;
  *w = my_id >= 0 ? mine / sum : 0.f;
}

// Choice of four tokens by one wave, 16 lanes each (up to 256 experts, up to 16
// choices): expert l + 16 i in lane l. A round is the lane's own best, then a
// maximum and a minimum over 16 lanes by row rotations (both may count a lane
// twice), with all four tokens in every instruction: about 90 instructions per
// token against 240 with a wave per token, on a workgroup that is bound by
// issuing them. Lane j keeps choice j.
template <typename E_, int NV>
__device__ __forceinline__ void choose4(const RouteArgs& a, int t, bool there, int l, int* id, float* w) {
  auto ror_max = [](uint32_t v) {
    v = max(v, dpp<0x128, 0xf>(v, v));   // row_ror 8, 4, 2, 1
    v = max(v, dpp<0x124, 0xf>(v, v));
    v = max(v, dpp<0x122, 0xf>(v, v));
    return max(v, dpp<0x121, 0xf>(v, v));
  };
  const E_* __restrict__ row = (const E_*)a.logits + (long long)t * a.E;
  float lg[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) lg[i] = elem_f32<E_>(row, min(l + 16 * i, a.E - 1));
  uint32_t key[NV], lv[NV], my_key = 0u, top = 0u;
#pragma unroll
  for (int i = 0; i < NV; ++i) lv[i] = key[i] = there && l + 16 * i < a.E ? logit_key(lg[i]) : 0u;
  int my_id = -1;
  for (int j = 0; j < a.k; ++j) {
    uint32_t bk = key[0];
    int bi = 0;
#pragma unroll
    for (int i = 1; i < NV; ++i) {
      const bool gt = key[i] > bk;       // (ties: the lowest index)
      bk = gt ? key[i] : bk;
      bi = gt ? i : bi;
    }
    const uint32_t m = ror_max(bk);
    // the lowest expert among the lanes that hold m, as the largest complement
    const int e = l + 16 * bi;
    const int win = 0xffff - (int)ror_max(bk == m ? (uint32_t)(0xffff - e) : 0u);
    const bool any = m != 0u;
    if (j == 0) top = m;
    if (any && l == j) {
      my_id = win;
      my_key = m;
    }
    const int wi = win == e ? bi : -1;   // this lane's entry drops out
#pragma unroll
    for (int i = 0; i < NV; ++i) key[i] = wi == i ? 0u : key[i];
  }
  const float m = key_logit(top);
  const float mine = my_id >= 0 ? exp_from(key_logit(my_key), m) : 0.f;
  float sum = mine;
  if (!a.renorm) {   // uniform
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lv[i] != 0u) sum += exp_from(key_logit(lv[i]), m);
  }
  auto add = [](float x, uint32_t y) { return x + __uint_as_float(y); };
  sum = add(sum, dpp<0x128, 0xf>(0u, __float_as_uint(sum)));
  sum = add(sum, dpp<0x124, 0xf>(0u, __float_as_uint(sum)));
  sum = add(sum, dpp<0x122, 0xf>(0u, __float_as_uint(sum)));
  sum = add(sum, dpp<0x121, 0xf>(0u, __float_as_uint(sum)));
  *id = my_id;
  *w = my_id >= 0 ? mine / sum : 0.f;
}

// 1 / x to within two roundings, x in [1, 1e300]: the hardware's estimate and three Newton
// steps (from 2^-14, the least taken of the estimate, two would leave 2^-56 besides their
// roundings), without the full division's scaling.
__device__ __forceinline__ double reciprocal64(double x) {
  double r = __builtin_amdgcn_rcp(x);
  r = fma(fma(-x, r, 1.0), r, r);
  r = fma(fma(-x, r, 1.0), r, r);
  return fma(fma(-x, r, 1.0), r, r);
}

// Choice of one token by one wave by scores (mlora_route_scored). The scores decide
// which of two near experts is chosen, so their rounding is part of the result: they
// are computed in 64 bits and rounded to fp32, where the bias is added (one rounding)
// and a group's two best are (another). In 64 bits a score is off by what the difference
// of two logits, its exponential, the sum (22 roundings), the reciprocal and the product
// lose, up to about 2^-47 of it: one that lies as near to the middle of two fp32 values may
// become either. `key_lds`: E words of the wave's own. Lane g holds group g: at most 64
// groups.
//
// Bound by issue and latency: at 4096 tokens of 160 experts three 64-bit exponentials
// per lane are about a third of 9.1 us, the rounds of the choice most of the rest; 64 tokens of
// 256 experts take 6.2 us as 16 workgroups of 4 waves, and took 26 of 29.6 as one
// workgroup that also groups them (a CU's 64-bit rate).
template <typename E_, int NV>
__device__ __forceinline__ void choose_scored(const RouteArgs& a, int t, int lane, uint32_t* key_lds, int* id, float* w) {
  const E_* __restrict__ row = (const E_*)a.logits + (long long)t * a.E;
  float l[NV], s[NV], b[NV];
  uint32_t key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) l[i] = elem_f32<E_>(row, min(lane + kWave * i, a.E - 1));
#pragma unroll
  for (int i = 0; i < NV; ++i) b[i] = a.bias ? a.bias[min(lane + kWave * i, a.E - 1)] : 0.f;   // (requested with the logits)
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (lane + kWave * i >= a.E || !(l[i] > -INFINITY)) l[i] = -INFINITY;   // (NaN: as -inf)
  if (a.sigmoid) {   // uniform
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] = (float)reciprocal64(1.0 + exp(fmin(-(double)l[i], 200.0)));   // (0 in fp32 from 104 on)
  } else {
    uint32_t mk = logit_key(l[0]);
#pragma unroll
    for (int i = 1; i < NV; ++i) mk = max(mk, logit_key(l[i]));
    const float m = key_logit(wave_max(mk));             // (a row of no expert: NaN)
    double p[NV], sum = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      p[i] = !(l[i] > -INFINITY) ? 0.0 : l[i] == m ? 1.0 : exp((double)l[i] - (double)m);
      sum += p[i];
    }
    const double inv = 1.0 / wave_sum64(sum);
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] = (float)(p[i] * inv);   // (a row of no expert: NaN, chosen by none)
  }
  // (softmax scores alone are in the logits' order, which the logits show where scores
  // round to the same value or to 0)
  const bool by_logit = !a.sigmoid && !a.bias && a.groups <= 1;   // uniform
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const float c = by_logit ? l[i] : a.bias ? s[i] + b[i] : s[i];
    key[i] = l[i] > -INFINITY ? logit_key(c) : 0u;
  }
  if (a.groups > 1) {   // uniform
    const int per = a.E / a.groups;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + kWave * i < a.E) key_lds[lane + kWave * i] = key[i];
    // (the wave's own LDS writes are ordered before its reads)
    // lane g: the two best of group g, eight entries in flight
    uint32_t k1 = 0u, k2 = 0u;
    const int first = min(lane, a.groups - 1) * per;
    for (int j0 = 0; j0 < per; j0 += 8) {
      uint32_t k[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) k[u] = key_lds[first + min(j0 + u, per - 1)];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const uint32_t v = j0 + u < per ? k[u] : 0u;
        k2 = max(k2, min(k1, v));
        k1 = max(k1, v);
      }
    }
    // (a group with an expert is above none, whatever its sum)
    const uint32_t gk = lane >= a.groups || k1 == 0u ? 0u
                        : max(1u, logit_key(k2 == 0u ? key_logit(k1) : key_logit(k1) + key_logit(k2)));
    int above = 0;   // groups before this one in the order
    for (int g = 0; g < a.groups; ++g) {
      const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)gk, g);
      above += o > gk || (o == gk && g < lane);
    }
    const unsigned long long kept = __ballot(gk != 0u && above < a.top_groups);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (!((kept >> (min(lane + kWave * i, a.E - 1) / per)) & 1ull)) key[i] = 0u;
  }
  int my_id = -1;
  float mine = 0.f;
  for (int j = 0; j < a.k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) best = max(best, key[i]);
    const uint32_t m = wave_max(best);                 // uniform
    if (m == 0u) break;                                // nothing left to choose
    int win = -1;                                      // uniform
#pragma unroll
    for (int i = NV - 1; i >= 0; --i) {
      const unsigned long long h = __ballot(key[i] == m);
      if (h) win = kWave * i + (int)__builtin_ctzll(h);
    }
    float sw = s[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) sw = win / kWave == i ? s[i] : sw;
    sw = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(sw), win % kWave));
    if (lane == j) {
      my_id = win;
      mine = sw;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (win == lane + kWave * i) key[i] = 0u;
  }
  if (a.renorm) {   // uniform
    const float sum = wave_sum(mine);
    mine = sum > 0.f ? mine / sum : 0.f;
  }
  *id = my_id;
  *w = a.scale * mine;
}

// LDS of the grouping: counts per wave [kRtWaves][E], then per expert [E + 1],
// then, in the one-launch form, the choices [T k].
__host__ __device__ inline size_t route_lds_bytes(int E) { return ((size_t)(kRtWaves + 1) * E + 1) * 4; }

// Slots [s0, s1) of the flat choice list (`ids` holds them from s0 on) grouped
// by expert: base[e] is the sorted position of the block's next slot of expert e.
// Rounds of 1024 slots: a wave ranks its 64 slots among those of the same
// expert with one ballot per bit of the expert id, the waves' counts are added
// in wave order. The block's threads all take part (barriers).
__device__ __forceinline__ void group_slots(const RouteArgs& a, const int32_t* ids, int s0, int s1, int* cnt, int* base) {
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int bits = 32 - __clz(a.E);   // ids 0 .. E (E: not chosen)
  for (int r0 = s0; r0 < s1; r0 += kRtThreads) {
    const int s = r0 + tid;
    int e = s < s1 ? ids[s - s0] : -1;
    if (e < 0) e = a.E;
    for (int i = tid; i < kRtWaves * a.E; i += kRtThreads) cnt[i] = 0;
    __syncthreads();
    unsigned long long same = ~0ull;
    for (int b = 0; b < bits; ++b) {
      const unsigned long long m = __ballot((e >> b) & 1);
      same &= ((e >> b) & 1) ? m : ~m;
    }
    const int rank = (int)__popcll(same & ((1ull << lane) - 1ull));
    if (e < a.E && rank == 0) cnt[wave * a.E + e] = (int)__popcll(same);
    __syncthreads();
    // counts -> first positions, waves in order; base moves on
    for (int x = tid; x < a.E; x += kRtThreads) {
      int n[kRtWaves];
#pragma unroll
      for (int w = 0; w < kRtWaves; ++w) n[w] = cnt[w * a.E + x];
      int p = base[x];
#pragma unroll
      for (int w = 0; w < kRtWaves; ++w) {
        cnt[w * a.E + x] = p;
        p += n[w];
      }
      base[x] = p;
    }
    __syncthreads();
    if (s < s1) {
      const int p = e < a.E ? cnt[wave * a.E + e] + rank : -1;
      a.position[s] = p;
      if (p >= 0) a.token_index[p] = s / a.k;
    }
    if (r0 + kRtThreads < s1) __syncthreads();   // uniform
  }
}

// Exclusive scan of n[0 .. E) (one workgroup) into base, total returned to
// every thread.
__device__ __forceinline__ int scan_experts(int* n, int E) {
  __shared__ int wsum[kRtWaves];
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int v = tid < E ? n[tid] : 0;   // E <= kRtThreads
  int inc = v;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const int up = __shfl_up(inc, off, kWave);
    if (lane >= off) inc += up;
  }
  if (lane == kWave - 1) wsum[wave] = inc;
  __syncthreads();
  int before = 0, total = 0;
  for (int w = 0; w < kRtWaves; ++w) {
    if (w < wave) before += wsum[w];
    total += wsum[w];
  }
  if (tid < E) n[tid] = before + inc - v;
  __syncthreads();
  return total;
}

// The choice for a block of a.tpb tokens; the block's slots per expert are
// left in LDS (base), and its choices where `ids` is given.
// FORM: four tokens per wave (choose4), one (choose1), or one by scores
// (choose_scored, with `keys`: E words per wave).
constexpr int kRtOne = 0, kRtQuad = 1, kRtScored = 2;
template <typename E_, int NV, int FORM>
__device__ __forceinline__ void choose_block(const RouteArgs& a, int* base, int* ids, int* keys) {
  constexpr bool QUAD = FORM == kRtQuad;
  constexpr int TPW = QUAD ? 4 : 1;                      // tokens of a wave at a time
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, waves = blockDim.x / kWave;
  for (int i = tid; i < a.E; i += blockDim.x) base[i] = 0;
  __syncthreads();
  const int t0 = blockIdx.x * a.tpb, t1 = min(t0 + a.tpb, a.T);
  const int l = QUAD ? lane % 16 : lane;
  for (int tw = t0 + TPW * wave; tw < t1; tw += TPW * waves) {   // uniform
    const int t = QUAD ? tw + lane / 16 : tw;
    int id;
    float w;
    if constexpr (QUAD) choose4<E_, NV>(a, min(t, t1 - 1), t < t1, l, &id, &w);
    else if constexpr (FORM == kRtScored) choose_scored<E_, NV>(a, t, l, (uint32_t*)keys + wave * a.E, &id, &w);
    else choose1<E_, NV>(a, t, l, &id, &w);
    if (t < t1 && l < a.k) {
      a.expert[(long long)t * a.k + l] = id;
      a.weight[(long long)t * a.k + l] = w;
      if (ids) ids[(t - t0) * a.k + l] = id;
      if (id >= 0) atomicAdd(&base[id], 1);              // (LDS; a count does not depend on the order)
    }
  }
  __syncthreads();
}

// One workgroup holds the batch: choice and grouping in one launch.
template <typename E_, int NV, int FORM>
__global__ __launch_bounds__(kRtThreads) void k_route_one(RouteArgs a) {
  extern __shared__ int sm[];
  int* cnt = sm;
  int* base = sm + kRtWaves * a.E;
  int* ids = base + a.E + 1;
  choose_block<E_, NV, FORM>(a, base, ids, cnt);   // (the counts come later)
  const int total = scan_experts(base, a.E);
  const int tid = threadIdx.x, P = a.T * a.k;
  for (int e = tid; e <= a.E; e += kRtThreads) a.seg_start[e] = e < a.E ? base[e] : total;
  for (int p = total + tid; p < P; p += kRtThreads) a.token_index[p] = -1;
  __syncthreads();
  group_slots(a, ids, 0, P, cnt, base);
}

constexpr int kRcThreads = 512;

template <typename E_, int NV, int FORM>
__global__ __launch_bounds__(FORM == kRtScored ? kRtThreads : kRcThreads) void k_route_choose(RouteArgs a) {
  extern __shared__ int sm[];
  choose_block<E_, NV, FORM>(a, sm, nullptr, sm + a.E);
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.hist[(long long)blockIdx.x * a.E + e] = sm[e];
}

// Grouping by the blocks' counts: block b's first position of expert e is the
// number of slots of lower experts plus those of e in earlier blocks. Each
// block sums the counts [blocks][E] itself: G = 1024 / E threads per expert take
// every G-th block.
__global__ __launch_bounds__(kRtThreads) void k_route_group(RouteArgs a) {
  extern __shared__ int sm[];
  int* cnt = sm;
  int* base = sm + kRtWaves * a.E;
  __shared__ int before[kRtThreads];   // slots of the expert in earlier blocks
  const int tid = threadIdx.x, nb = gridDim.x, b = blockIdx.x;
  for (int e = tid; e < a.E; e += kRtThreads) {
    base[e] = 0;
    before[e] = 0;
  }
  __syncthreads();
  const int G = kRtThreads / a.E > 0 ? kRtThreads / a.E : 1;
  for (int e = tid; e < G * a.E; e += kRtThreads) {
    const int x = e % a.E, g = e / a.E;
    int all = 0, pre = 0;
    constexpr int U = 8;   // counts in flight
    for (int i0 = g; i0 < nb; i0 += U * G) {
      int n[U];
#pragma unroll
      for (int u = 0; u < U; ++u) n[u] = a.hist[(long long)min(i0 + u * G, nb - 1) * a.E + x];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * G;
        if (i < nb) all += n[u];
        if (i < b) pre += n[u];
      }
    }
    if (all) atomicAdd(&base[x], all);      // (LDS; sums of counts)
    if (pre) atomicAdd(&before[x], pre);
  }
  __syncthreads();
  const int total = scan_experts(base, a.E);
  if (b == 0)
    for (int e = tid; e <= a.E; e += kRtThreads) a.seg_start[e] = e < a.E ? base[e] : total;
  __syncthreads();
  for (int e = tid; e < a.E; e += kRtThreads) base[e] += before[e];
  const int s0 = b * a.tpb * a.k, s1 = min(s0 + a.tpb * a.k, a.T * a.k);
  for (int p = max(s0, total) + tid; p < s1; p += kRtThreads) a.token_index[p] = -1;
  __syncthreads();
  group_slots(a, a.expert + s0, s0, s1, cnt, base);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
static int route_tokens_per_block(int T) {
  const int t = ((T > 0 ? T : 1) + kRtMaxBlocks - 1) / kRtMaxBlocks;
  return (t + kRtMinTokens - 1) / kRtMinTokens * kRtMinTokens;
}

// By scores a wave takes a token (its score alone is some 60 instructions in 64
// bits), so the choice spreads over more and smaller blocks.
constexpr int kRsMinTokens = 4;
static int scored_tokens_per_block(int T) {
  const int t = (T + kRtMaxBlocks - 1) / kRtMaxBlocks;
  return t > kRsMinTokens ? t : kRsMinTokens;
}

// Counts of the most blocks that a batch of up to T tokens is cut into: a larger
// batch never has a smaller workspace (8193 tokens are fewer blocks than 8192).
size_t route_workspace_bytes(int T, int E, bool scored) {
  const int per = scored ? kRsMinTokens : kRtMinTokens;
  const int blocks = (T + per - 1) / per;
  return ((size_t)(blocks < kRtMaxBlocks ? blocks : kRtMaxBlocks) * E * 4 + 255) / 256 * 256;
}

// Batches of up to this many tokens take the one-launch form (64 tokens, 128
// experts, top 8: 8.2 us; two launches take 4.6 + 5.5 us and the gap between
// them at 4096 tokens, hardly less at a few).
constexpr int kRtOneTokens = 128;

template <typename E_, int NV, int FORM>
static void launch_route_nv(RouteArgs a, hipStream_t st) {
  const size_t lds = route_lds_bytes(a.E);
  if constexpr (FORM == kRtScored) {
    if (a.T > kRtWaves) {
      a.tpb = scored_tokens_per_block(a.T);
      const dim3 grid((a.T + a.tpb - 1) / a.tpb);
      const int waves = a.tpb < kRtWaves ? a.tpb : kRtWaves;
      hipLaunchKernelGGL((k_route_choose<E_, NV, FORM>), grid, dim3(waves * kWave), (size_t)a.E * 4 * (1 + waves), st, a);
      hipLaunchKernelGGL(k_route_group, grid, dim3(kRtThreads), lds, st, a);
      return;
    }
  }
  if (a.T <= kRtOneTokens) {
    a.tpb = a.T;
    hipLaunchKernelGGL((k_route_one<E_, NV, FORM>), dim3(1), dim3(kRtThreads), lds + (size_t)a.T * a.k * 4, st, a);
    return;
  }
  a.tpb = route_tokens_per_block(a.T);
  const dim3 grid((a.T + a.tpb - 1) / a.tpb);
  hipLaunchKernelGGL((k_route_choose<E_, NV, FORM>), grid, dim3(kRcThreads), (size_t)a.E * 4, st, a);
  hipLaunchKernelGGL(k_route_group, grid, dim3(kRtThreads), lds, st, a);
}

template <typename E_>
static void launch_route_t(const RouteArgs& a, hipStream_t st) {
  if (a.scored) {
    if (a.E <= 64) launch_route_nv<E_, 1, kRtScored>(a, st);
    else if (a.E <= 128) launch_route_nv<E_, 2, kRtScored>(a, st);
    else if (a.E <= 192) launch_route_nv<E_, 3, kRtScored>(a, st);
    else if (a.E <= 256) launch_route_nv<E_, 4, kRtScored>(a, st);
    else if (a.E <= 512) launch_route_nv<E_, 8, kRtScored>(a, st);
    else launch_route_nv<E_, MLORA_MAX_EXPERTS / kWave, kRtScored>(a, st);
  } else if (a.E > 256 || a.k > 16) launch_route_nv<E_, MLORA_MAX_EXPERTS / kWave, kRtOne>(a, st);
  else if (a.E <= 64) launch_route_nv<E_, 4, kRtQuad>(a, st);
  else if (a.E <= 128) launch_route_nv<E_, 8, kRtQuad>(a, st);
  else launch_route_nv<E_, 16, kRtQuad>(a, st);
}

void launch_route(const RouteArgs& a, bool bf16, hipStream_t st) {
  if (bf16) launch_route_t<uint16_t>(a, st);
  else launch_route_t<float>(a, st);
}

}  // namespace mlora
