// api_experts.hip -- the exported C ABI of routing and expert products
// (include/mlora.h): host-side validation and dispatch.
#include <hip/hip_runtime.h>

#include "../../include/mlora.h"
#include "experts.h"

using namespace mlora;

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

int launched() { return hipGetLastError() == hipSuccess ? MLORA_OK : MLORA_ERR_HIP; }

bool batch_ok(int n_tokens, int n_experts, int top_k) {
  return n_tokens >= 0 && n_tokens <= MLORA_MAX_TOKENS && n_experts >= 1 && n_experts <= MLORA_MAX_EXPERTS &&
         top_k >= 1 && top_k <= MLORA_MAX_TOP_K && top_k <= n_experts &&
         (long long)n_tokens * top_k <= MLORA_MAX_POSITIONS;
}

// Checks shared by the two expert products. Returns a status. (The limit on
// n_pos d_out keeps a launch of the tiled forms, 512 threads per 128 x 128 tile
// and less than one part tile per expert and run, under 2^32 threads.)
int check_product(int dtype, const float* w_scale, int n_experts, int d_in, int d_out, long long n_pos) {
  if (dtype != MLORA_F32 && dtype != MLORA_BF16) return MLORA_ERR_DTYPE;
  if (w_scale && dtype != MLORA_BF16) return MLORA_ERR_DTYPE;
  if (n_experts < 1 || n_experts > MLORA_MAX_EXPERTS) return MLORA_ERR_SHAPE;
  if (d_in < 1 || d_in > MLORA_MAX_DIM || d_out < 1 || d_out > MLORA_MAX_DIM) return MLORA_ERR_SHAPE;
  if (d_in % (w_scale ? 16 : dtype == MLORA_F32 ? 4 : 8) != 0) return MLORA_ERR_SHAPE;
  if (n_pos < 0 || n_pos > MLORA_MAX_POSITIONS || n_pos * d_out > MLORA_MAX_PRODUCT) return MLORA_ERR_SHAPE;
  return MLORA_OK;
}

}  // namespace

extern "C" {

size_t mlora_route_workspace_bytes(int n_tokens, int n_experts, int top_k) {
  if (!batch_ok(n_tokens, n_experts, top_k)) return 0;
  const size_t b = route_workspace_bytes(n_tokens, n_experts);
  return b < 256 ? 256 : b;
}

int mlora_route(const void* logits, int dtype, int n_tokens, int n_experts, int top_k, int renormalize,
                int32_t* expert, float* weight, int32_t* token_index, int32_t* seg_start, int32_t* position,
                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (dtype != MLORA_F32 && dtype != MLORA_BF16) return MLORA_ERR_DTYPE;
  if (renormalize != 0 && renormalize != 1) return MLORA_ERR_INVALID_ARG;
  if (!batch_ok(n_tokens, n_experts, top_k)) return MLORA_ERR_SHAPE;
  if (!seg_start || !aligned16(seg_start)) return MLORA_ERR_INVALID_ARG;
  if (n_tokens > 0) {
    if (!logits || !expert || !weight || !token_index || !position || !workspace) return MLORA_ERR_INVALID_ARG;
    if (!aligned16(logits) || !aligned16(expert) || !aligned16(weight) || !aligned16(token_index) ||
        !aligned16(position) || !aligned16(workspace))
      return MLORA_ERR_INVALID_ARG;
    if (workspace_bytes < mlora_route_workspace_bytes(n_tokens, n_experts, top_k)) return MLORA_ERR_WORKSPACE;
  }
  RouteArgs a{};
  a.logits = logits;
  a.T = n_tokens;
  a.E = n_experts;
  a.k = top_k;
  a.renorm = renormalize;
  a.expert = expert;
  a.weight = weight;
  a.token_index = token_index;
  a.seg_start = seg_start;
  a.position = position;
  a.hist = (int32_t*)workspace;
  launch_route(a, dtype == MLORA_BF16, stream);
  return launched();
}

int mlora_experts_linear(const void* x, const void* W, const float* w_scale, int dtype, int n_rows,
                         int n_experts, int d_in, int d_out, const int32_t* seg_start,
                         const int32_t* token_index, int n_pos, const mlora_epilogue_t* epilogue, void* y,
                         hipStream_t stream) {
  if (const int st = check_product(dtype, w_scale, n_experts, d_in, d_out, n_pos)) return st;
  if (n_rows < 0 || n_rows > MLORA_MAX_POSITIONS) return MLORA_ERR_SHAPE;
  const int act = epilogue ? epilogue->act & ~MLORA_ACT_GATED : MLORA_ACT_NONE;
  const bool gated = epilogue && (epilogue->act & MLORA_ACT_GATED);
  if (act < MLORA_ACT_NONE || act > MLORA_ACT_GELU_TANH) return MLORA_ERR_INVALID_ARG;
  if (epilogue && (epilogue->residual || !aligned16(epilogue->bias))) return MLORA_ERR_INVALID_ARG;
  if (gated && d_out % 2 != 0) return MLORA_ERR_SHAPE;
  if (n_pos == 0) return MLORA_OK;
  if (n_rows < 1 || (!token_index && n_rows < n_pos)) return MLORA_ERR_SHAPE;
  if (!x || !W || !seg_start || !y) return MLORA_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(W) || !aligned16(y)) return MLORA_ERR_INVALID_ARG;
  ExpertsArgs a{};
  a.x = x;
  a.W = W;
  a.w_scale = w_scale;
  a.y = y;
  a.seg_start = seg_start;
  a.token_index = token_index;
  a.n_rows = n_rows;
  a.E = n_experts;
  a.d_in = d_in;
  a.d_out = d_out;
  a.n_pos = n_pos;
  a.gated = gated;
  a.epi.bias = epilogue ? epilogue->bias : nullptr;
  a.epi.act = act;
  launch_experts(a, dtype == MLORA_BF16, stream);
  return launched();
}

size_t mlora_experts_workspace_bytes(int n_tokens, int top_k, int n_experts, int d_out, int dtype) {
  if (!batch_ok(n_tokens, n_experts, top_k) || d_out < 1 || d_out > MLORA_MAX_DIM) return 0;
  if (dtype != MLORA_F32 && dtype != MLORA_BF16) return 0;
  if ((long long)n_tokens * top_k * d_out > MLORA_MAX_PRODUCT) return 0;
  const size_t b = ((size_t)n_tokens * top_k * f32_pitch(d_out) * 4 + 255) / 256 * 256;
  return b < 256 ? 256 : b;
}

int mlora_experts_combine(const void* h, const void* W, const float* w_scale, int dtype, int n_tokens,
                          int top_k, int n_experts, int d_in, int d_out, const int32_t* seg_start,
                          const int32_t* position, const float* weight, const void* bias,
                          const void* residual, void* out, void* workspace, size_t workspace_bytes,
                          hipStream_t stream) {
  if (!batch_ok(n_tokens, n_experts, top_k)) return MLORA_ERR_SHAPE;
  const int n_pos = n_tokens * top_k;
  if (const int st = check_product(dtype, w_scale, n_experts, d_in, d_out, n_pos)) return st;
  if (n_tokens == 0) return MLORA_OK;
  if (!h || !W || !seg_start || !position || !weight || !out || !workspace) return MLORA_ERR_INVALID_ARG;
  if (!aligned16(h) || !aligned16(W) || !aligned16(bias) || !aligned16(residual) || !aligned16(out) ||
      !aligned16(workspace))
    return MLORA_ERR_INVALID_ARG;
  if (workspace_bytes < mlora_experts_workspace_bytes(n_tokens, top_k, n_experts, d_out, dtype))
    return MLORA_ERR_WORKSPACE;
  ExpertsArgs a{};
  a.x = h;
  a.W = W;
  a.w_scale = w_scale;
  a.y = workspace;
  a.seg_start = seg_start;
  a.n_rows = n_pos;
  a.E = n_experts;
  a.d_in = d_in;
  a.d_out = d_out;
  a.n_pos = n_pos;
  a.f32_out = 1;
  a.epi.bias = bias;
  a.epi.act = MLORA_ACT_NONE;
  launch_experts(a, dtype == MLORA_BF16, stream);
  if (const int st = launched()) return st;
  CombineArgs c{};
  c.part = (const float*)workspace;
  c.position = position;
  c.weight = weight;
  c.residual = residual;
  c.out = out;
  c.T = n_tokens;
  c.k = top_k;
  c.d_out = d_out;
  c.n_pos = n_pos;
  launch_combine(c, dtype == MLORA_BF16, stream);
  return launched();
}

}  // extern "C"
