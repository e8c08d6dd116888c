// experts.h -- host-side launchers and device-side helpers of the routing and
// expert kernels (internal to the library).
#pragma once
#include "common.h"
#include "epilogue.h"

namespace mlora {

// ---- routing (kernels_route.hip) ----------------------------------------------
struct RouteArgs {
  const void* logits;     // [T, E] bf16 or fp32
  int T, E, k;
  int renorm;
  int32_t* expert;        // [T, k]
  float* weight;          // [T, k]
  int32_t* token_index;   // [T k]
  int32_t* seg_start;     // [E + 1]
  int32_t* position;      // [T, k]
  int32_t* hist;          // workspace: slots per expert of every block's tokens [blocks][E]
  int tpb;                // tokens per block
  // choice by scores (mlora_route_scored); scored = 0: by logits
  int scored, sigmoid;
  const float* bias;      // [E] or null
  int groups, top_groups;
  float scale;
};
size_t route_workspace_bytes(int T, int E, bool scored);
void launch_route(const RouteArgs& a, bool bf16, hipStream_t st);

// ---- products per expert (experts_kernels.h, kernels_experts*.hip) ----------------------------------
struct ExpertsArgs {
  const void* x;                // [n_rows, d_in]
  const void* W;                // [E, d_out, d_in]
  const float* w_scale;         // [E, d_out]: W holds e4m3 codes; null: W in x's type
  const uint8_t* w_mx;          // [E, planes, d_out, 4]: W holds MXFP4 codes, these are their scales
  const uint8_t* x_mx;          // [planes, n_rows, 4]: x holds MXFP4 codes too (with w_mx only)
  void* y;                      // [n_pos, d_y]; where f32_out fp32 [n_pos, f32_pitch(d_out)]
  const int32_t* seg_start;     // [E + 1]
  const int32_t* token_index;   // [n_pos] or null
  int n_rows, E, d_in, d_out, n_pos;
  int gated, f32_out;
  EpiView epi;                  // bias [E, d_out]; no residual
};
void launch_experts(const ExpertsArgs& a, bool bf16, hipStream_t st);
void launch_experts_mx(const ExpertsArgs& a, hipStream_t st);   // (w_mx given)

// Row pitch of the products on the way back: whole vectors of 4, also for odd d_out
// (columns past it hold anything).
__host__ __device__ __forceinline__ int f32_pitch(int d_out) { return (d_out + 3) & ~3; }

struct CombineArgs {
  const float* part;            // [n_pos, f32_pitch(d_out)]
  const int32_t* position;      // [T, k]
  const float* weight;          // [T, k]
  const void* residual;         // [T, d_out] or null
  void* out;                    // [T, d_out]
  int T, k, d_out, n_pos;
};
void launch_combine(const CombineArgs& a, bool bf16, hipStream_t st);

// A batch cut into runs of at most BT positions per expert. Every wave finds a
// run by itself, 64 experts per step (one load pair, a wave scan of the run
// counts, a ballot), so no barrier precedes the weight loads. Starts are clamped
// into [0, n_pos]: a lying seg_start drops or repeats positions but never leaves
// the arrays.
struct RunScan {   // of 64 experts, one per lane
  int s0, s1;      // positions
  int n, inc;      // runs, and their inclusive sum over the lanes
};
__device__ __forceinline__ RunScan scan_runs(const int32_t* __restrict__ seg_start, int E, int n_pos, int BT, int e0) {
  const int lane = threadIdx.x % kWave, e = min(e0 + lane, E - 1);
  RunScan r;
  r.s0 = min(max(seg_start[e], 0), n_pos);
  r.s1 = min(max(seg_start[e + 1], 0), n_pos);
  r.n = e0 + lane < E ? (max(r.s1 - r.s0, 0) + BT - 1) / BT : 0;
  r.inc = r.n;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const int up = __shfl_up(r.inc, off, kWave);
    if (lane >= off) r.inc += up;
  }
  return r;
}

// Runs in all; `first` is the scan from expert 0.
__device__ __forceinline__ int count_runs(const RunScan& first, const int32_t* __restrict__ seg_start, int E, int n_pos, int BT) {
  int n = __builtin_amdgcn_readlane(first.inc, kWave - 1);
  for (int e0 = kWave; e0 < E; e0 += kWave)
    n += __builtin_amdgcn_readlane(scan_runs(seg_start, E, n_pos, BT, e0).inc, kWave - 1);
  return n;
}

// Run `item`: its expert (or -1 past the last run), the expert's positions
// [*s0, *s1), its number of runs and the runs before it.
__device__ __forceinline__ int find_run(const RunScan& first, const int32_t* __restrict__ seg_start, int E, int n_pos, int BT,
                                        int item, int* s0, int* s1, int* runs, int* before) {
  int done = 0;
  for (int e0 = 0; e0 < E; e0 += kWave) {
    const RunScan r = e0 == 0 ? first : scan_runs(seg_start, E, n_pos, BT, e0);
    const unsigned long long m = __ballot(r.inc > item - done);
    if (m) {   // uniform
      const int l = (int)__builtin_ctzll(m);
      *s0 = __builtin_amdgcn_readlane(r.s0, l);
      *s1 = __builtin_amdgcn_readlane(r.s1, l);
      *runs = __builtin_amdgcn_readlane(r.n, l);
      *before = done + __builtin_amdgcn_readlane(r.inc, l) - *runs;
      return e0 + l;
    }
    done += __builtin_amdgcn_readlane(r.inc, kWave - 1);
  }
  return -1;
}

// The same, with the run's positions [*p0, *p1).
__device__ __forceinline__ int find_expert(const RunScan& first, const int32_t* __restrict__ seg_start, int E, int n_pos, int BT,
                                           int item, int* p0, int* p1) {
  int s0, s1, runs, before;
  const int e = find_run(first, seg_start, E, n_pos, BT, item, &s0, &s1, &runs, &before);
  if (e < 0) return -1;
  *p0 = s0 + BT * (item - before);
  *p1 = min(*p0 + BT, s1);
  return e;
}

}  // namespace mlora
