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
// and no order that depends on timing: the result is unique.
#include "../../include/mlora.h"
#include "experts.h"

namespace mlora {

constexpr int kRtThreads = 1024, kRtWaves = kRtThreads / kWave;
constexpr int kRtMaxBlocks = 256;   // blocks of the grouping (each reads all their counts)
constexpr int kRtMinTokens = 16;    // tokens per block at least: one per wave

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

// Choice of one token by one wave: NV experts per lane (expert lane + 64 i).
// k rounds of a wave-wide maximum over (logit, lowest index); lane j keeps
// choice j.
template <typename E_, int NV>
__device__ __forceinline__ void choose(const RouteArgs& a, int t, int lane, int* id, float* w) {
  const E_* __restrict__ row = (const E_*)a.logits + (long long)t * a.E;
  uint32_t key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + kWave * i;
    key[i] = e < a.E ? logit_key(elem_f32<E_>(row, e)) : 0u;
  }
  uint32_t lv[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) lv[i] = key[i];
  int my_id = -1;
  uint32_t my_key = 0, top = 0;
  for (int j = 0; j < a.k; ++j) {
    // the lane's best (its lowest index wins ties), then the wave's
    uint32_t bk = key[0];
    int bi = lane;
#pragma unroll
    for (int i = 1; i < NV; ++i)
      if (key[i] > bk) {
        bk = key[i];
        bi = lane + kWave * i;
      }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      const uint32_t ok = __shfl_xor(bk, off, kWave);
      const int oi = __shfl_xor(bi, off, kWave);
      if (ok > bk || (ok == bk && oi < bi)) {
        bk = ok;
        bi = oi;
      }
    }
    if (bk == 0u) break;   // uniform: nothing left to choose
    if (j == 0) top = bk;
    if (lane == j) {
      my_id = bi;
      my_key = bk;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (bi == lane + kWave * i) key[i] = 0u;
  }
  const float m = key_logit(top);
  float mine = my_id >= 0 ? exp_from(key_logit(my_key), m) : 0.f;
  float sum = 0.f;
  if (a.renorm) {
    sum = mine;
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lv[i] != 0u) sum += exp_from(key_logit(lv[i]), m);
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, kWave);
  *id = my_id;
  *w = my_id >= 0 ? mine / sum : 0.f;
}

// LDS of a block: counts per wave [kRtWaves][E], then per expert [E + 1] and
// the tokens' choices (int16) of one round.
__host__ __device__ inline size_t route_lds_bytes(int E) { return ((size_t)(kRtWaves + 1) * E + 1) * 4; }

// Slots [s0, s1) of the flat choice list `ids` grouped by expert: base[e] is
// the sorted position of the block's next slot of expert e. Rounds of 1024
// slots: a wave ranks its 64 slots among those of the same expert with one
// ballot per bit of the expert id, the waves' counts are added in wave order.
// The block's threads all take part (barriers).
__device__ __forceinline__ void group_slots(const RouteArgs& a, const int32_t* ids, int s0, int s1, int* cnt, int* base) {
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int bits = 32 - __clz(a.E);   // ids 0 .. E (E: not chosen)
  for (int r0 = s0; r0 < s1; r0 += kRtThreads) {
    for (int i = tid; i < kRtWaves * a.E; i += kRtThreads) cnt[i] = 0;
    __syncthreads();
    const int s = r0 + tid;
    int e = s < s1 ? ids[s] : -1;
    if (e < 0) e = a.E;
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
      int p = base[x];
      for (int w = 0; w < kRtWaves; ++w) {
        const int n = cnt[w * a.E + x];
        cnt[w * a.E + x] = p;
        p += n;
      }
      base[x] = p;
    }
    __syncthreads();
    if (s < s1) {
      const int p = e < a.E ? cnt[wave * a.E + e] + rank : -1;
      a.position[s] = p;
      if (p >= 0) a.token_index[p] = s / a.k;
    }
    __syncthreads();
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
// left in LDS (base) and, with several blocks, in a.hist.
template <typename E_, int NV>
__device__ __forceinline__ void choose_block(const RouteArgs& a, int* base) {
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  for (int i = tid; i < a.E; i += kRtThreads) base[i] = 0;
  __syncthreads();
  const int t0 = blockIdx.x * a.tpb, t1 = min(t0 + a.tpb, a.T);
  for (int t = t0 + wave; t < t1; t += kRtWaves) {
    int id;
    float w;
    choose<E_, NV>(a, t, lane, &id, &w);
    if (lane < a.k) {
      a.expert[(long long)t * a.k + lane] = id;
      a.weight[(long long)t * a.k + lane] = w;
      if (id >= 0) atomicAdd(&base[id], 1);   // (LDS; a count does not depend on the order)
    }
  }
  __syncthreads();
}

// One workgroup holds the batch: choice and grouping in one launch.
template <typename E_, int NV>
__global__ __launch_bounds__(kRtThreads) void k_route_one(RouteArgs a) {
  extern __shared__ int sm[];
  int* cnt = sm;
  int* base = sm + kRtWaves * a.E;
  choose_block<E_, NV>(a, base);
  const int total = scan_experts(base, a.E);
  const int tid = threadIdx.x, P = a.T * a.k;
  for (int e = tid; e <= a.E; e += kRtThreads) a.seg_start[e] = e < a.E ? base[e] : total;
  for (int p = total + tid; p < P; p += kRtThreads) a.token_index[p] = -1;
  __syncthreads();
  group_slots(a, a.expert, 0, P, cnt, base);
}

template <typename E_, int NV>
__global__ __launch_bounds__(kRtThreads) void k_route_choose(RouteArgs a) {
  extern __shared__ int sm[];
  choose_block<E_, NV>(a, sm);
  for (int e = threadIdx.x; e < a.E; e += kRtThreads) a.hist[(long long)blockIdx.x * a.E + e] = sm[e];
}

// Grouping by the blocks' counts: block b's first position of expert e is the
// number of slots of lower experts plus those of e in earlier blocks. Each
// block sums the counts [blocks][E] itself: G threads per expert take every
// G-th block, G the largest power of two with G E <= 1024.
__global__ __launch_bounds__(kRtThreads) void k_route_group(RouteArgs a) {
  extern __shared__ int sm[];
  int* cnt = sm;                       // (first: partial sums)
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
    for (int i = g; i < nb; i += G) {
      const int n = a.hist[(long long)i * a.E + x];
      all += n;
      if (i < b) pre += n;
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
  group_slots(a, a.expert, s0, s1, cnt, base);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
static int route_tokens_per_block(int T) {
  const int t = ((T > 0 ? T : 1) + kRtMaxBlocks - 1) / kRtMaxBlocks;
  return (t + kRtMinTokens - 1) / kRtMinTokens * kRtMinTokens;
}

size_t route_workspace_bytes(int T, int E) {
  const int tpb = route_tokens_per_block(T);
  return ((size_t)((T + tpb - 1) / tpb) * E * 4 + 255) / 256 * 256;
}

// Batches of up to this many tokens take the one-launch form.
constexpr int kRtOneTokens = 64;

template <typename E_, int NV>
static void launch_route_nv(RouteArgs a, hipStream_t st) {
  const size_t lds = route_lds_bytes(a.E);
  if (a.T <= kRtOneTokens) {
    a.tpb = a.T;
    hipLaunchKernelGGL((k_route_one<E_, NV>), dim3(1), dim3(kRtThreads), lds, st, a);
    return;
  }
  a.tpb = route_tokens_per_block(a.T);
  const dim3 grid((a.T + a.tpb - 1) / a.tpb);
  hipLaunchKernelGGL((k_route_choose<E_, NV>), grid, dim3(kRtThreads), (size_t)a.E * 4, st, a);
  hipLaunchKernelGGL(k_route_group, grid, dim3(kRtThreads), lds, st, a);
}

template <typename E_>
static void launch_route_t(const RouteArgs& a, hipStream_t st) {
  if (a.E <= 64) launch_route_nv<E_, 1>(a, st);
  else if (a.E <= 128) launch_route_nv<E_, 2>(a, st);
  else if (a.E <= 256) launch_route_nv<E_, 4>(a, st);
  else launch_route_nv<E_, MLORA_MAX_EXPERTS / kWave>(a, st);
}

void launch_route(const RouteArgs& a, bool bf16, hipStream_t st) {
  if (bf16) launch_route_t<uint16_t>(a, st);
  else launch_route_t<float>(a, st);
}

}  // namespace mlora
