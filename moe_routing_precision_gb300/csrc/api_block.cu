// api_block.cu -- the extern "C" boundary of the operators around the routed
// experts (include/moe_route.h): host-side argument checks, then the launch.
// A rejected call launches nothing.
#include <cmath>

#include "block/block_ops.cuh"

namespace moe {
namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool dtype_ok(int32_t t) { return t == MOE_DT_BF16 || t == MOE_DT_F32; }
size_t dtype_size(int32_t t) { return t == MOE_DT_F32 ? 4 : 2; }
bool experts_ok(int32_t E, int32_t k) {
  return E >= 1 && E <= MOE_MAX_EXPERTS && k >= 1 && k <= MOE_MAX_TOPK && k <= E;
}
// Zero-fill of the outputs of an empty problem.
cudaError_t zero(void* p, size_t bytes, void* stream) {
  if (p == nullptr || bytes == 0) return cudaSuccess;
  return cudaMemsetAsync(p, 0, bytes, static_cast<cudaStream_t>(stream));
}

// What the two norm calls share.
bool norm_ok(int32_t stream_dtype, int32_t block_dtype, int64_t T, int32_t H, const void* y,
             const float* post_w, const void* gate, int32_t gate_kind, int32_t gate_act,
             float scale, const float* pre_w) {
  if (!dtype_ok(stream_dtype) || !dtype_ok(block_dtype)) return false;
  if (T < 0 || H < 1) return false;
  if (gate_kind < MOE_GATE_NONE || gate_kind > MOE_GATE_ELEMENT) return false;
  if (gate_act != MOE_GATE_ACT_NONE && gate_act != MOE_GATE_ACT_SIGMOID) return false;
  if (!std::isfinite(scale)) return false;
  if (y == nullptr && T > 0 && (post_w || gate_kind != MOE_GATE_NONE || !pre_w)) return false;
  const size_t ge = gate_kind == MOE_GATE_ELEMENT ? dtype_size(block_dtype) : 4;
  return aligned(post_w, 4) && aligned(pre_w, 4) && aligned(gate, ge) &&
         aligned(y, dtype_size(block_dtype));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_block_norm(const void* residual, int32_t stream_dtype, const void* y,
                            int32_t block_dtype, int64_t num_tokens, int32_t hidden,
                            const float* post_weight, const void* gate, int32_t gate_kind,
                            int32_t gate_act, float scale, const float* pre_weight, float eps,
                            void* h, void* n, float* rstd_post, float* rstd_pre, void* stream) {
  if (!norm_ok(stream_dtype, block_dtype, num_tokens, hidden, y, post_weight, gate, gate_kind,
               gate_act, scale, pre_weight))
    return MOE_ERR_INVALID_ARG;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return MOE_ERR_INVALID_ARG;
  if (hidden > MOE_NORM_MAX_HIDDEN || num_tokens >= ((int64_t)1 << 40) / hidden)
    return MOE_ERR_UNSUPPORTED;
  if (num_tokens == 0) return MOE_OK;
  const size_t es = dtype_size(stream_dtype), eb = dtype_size(block_dtype);
  if (!residual || !aligned(residual, es) || !aligned(h, es) || !aligned(n, eb) ||
      !aligned(rstd_post, 4) || !aligned(rstd_pre, 4))
    return MOE_ERR_INVALID_ARG;
  if ((y && !h) || (pre_weight != nullptr) != (n != nullptr) ||
      (gate != nullptr) != (gate_kind != MOE_GATE_NONE))
    return MOE_ERR_INVALID_ARG;
  LaunchCtx c;
  moe_status_t s = context(stream, &c);
  if (s != MOE_OK) return s;
  NormArgs a;
  a.residual = residual;
  a.y = y;
  a.gate = gate;
  a.post_w = post_weight;
  a.pre_w = pre_weight;
  a.T = num_tokens;
  a.H = hidden;
  a.gate_kind = gate_kind;
  a.gate_act = gate_act;
  a.scale = scale;
  a.eps = eps;
  a.h = y ? h : nullptr;
  a.n = n;
  a.rstd_post = rstd_post;
  a.rstd_pre = rstd_pre;
  cudaError_t e =
      launch_block_norm(c, a, stream_dtype == MOE_DT_F32, block_dtype == MOE_DT_F32);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

size_t moe_block_norm_backward_workspace_bytes(int64_t num_tokens, int32_t hidden) {
  if (num_tokens <= 0 || hidden < 1 || hidden > MOE_NORM_MAX_HIDDEN) return 0;
  const int64_t blocks = norm_partial_blocks(num_tokens, hidden);
  return ((size_t)blocks * 2 * (size_t)hidden * 4 + 255) / 256 * 256;
}

moe_status_t moe_block_norm_backward(
    const void* grad_h, const void* grad_n, const void* h, int32_t stream_dtype, const void* y,
    int32_t block_dtype, int64_t num_tokens, int32_t hidden, const float* post_weight,
    const void* gate, int32_t gate_kind, int32_t gate_act, float scale, const float* pre_weight,
    const float* rstd_post, const float* rstd_pre, void* grad_residual, void* grad_y,
    float* grad_post_weight, void* grad_gate, float* grad_pre_weight, void* workspace,
    size_t workspace_bytes, void* stream) {
  if (!norm_ok(stream_dtype, block_dtype, num_tokens, hidden, y, post_weight, gate, gate_kind,
               gate_act, scale, pre_weight))
    return MOE_ERR_INVALID_ARG;
  if (hidden > MOE_NORM_MAX_HIDDEN || num_tokens >= ((int64_t)1 << 40) / hidden)
    return MOE_ERR_UNSUPPORTED;
  if ((post_weight != nullptr) != (grad_post_weight != nullptr) ||
      (pre_weight != nullptr) != (grad_pre_weight != nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(grad_post_weight, 4) || !aligned(grad_pre_weight, 4)) return MOE_ERR_INVALID_ARG;
  const bool channel = gate_kind == MOE_GATE_CHANNEL;
  if (channel && (!grad_gate || !aligned(grad_gate, 4))) return MOE_ERR_INVALID_ARG;
  if (num_tokens == 0) {
    // no token: the gradients summed over the tokens are zero
    const size_t bytes = (size_t)hidden * 4;
    cudaError_t e = zero(grad_post_weight, bytes, stream);
    if (e == cudaSuccess) e = zero(grad_pre_weight, bytes, stream);
    if (e == cudaSuccess && channel) e = zero(grad_gate, bytes, stream);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e);
  }
  const size_t es = dtype_size(stream_dtype), eb = dtype_size(block_dtype);
  const size_t ge = gate_kind == MOE_GATE_ELEMENT ? eb : 4;
  if (!grad_residual || (y != nullptr) != (grad_y != nullptr) ||
      (gate != nullptr) != (gate_kind != MOE_GATE_NONE) ||
      (grad_gate != nullptr) != (gate_kind != MOE_GATE_NONE))
    return MOE_ERR_INVALID_ARG;
  if (pre_weight && (!grad_n || !h || !rstd_pre)) return MOE_ERR_INVALID_ARG;
  if (post_weight && !rstd_post) return MOE_ERR_INVALID_ARG;
  if (!aligned(grad_h, es) || !aligned(grad_n, eb) || !aligned(h, es) ||
      !aligned(grad_residual, es) || !aligned(grad_y, eb) || !aligned(grad_gate, ge) ||
      !aligned(rstd_post, 4) || !aligned(rstd_pre, 4))
    return MOE_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 16) ||
      workspace_bytes < moe_block_norm_backward_workspace_bytes(num_tokens, hidden))
    return MOE_ERR_INVALID_ARG;
  LaunchCtx c;
  moe_status_t s = context(stream, &c);
  if (s != MOE_OK) return s;
  NormArgs a;
  a.grad_h = grad_h;
  a.grad_n = grad_n;
  a.h = const_cast<void*>(h);
  a.y = y;
  a.gate = gate;
  a.post_w = post_weight;
  a.pre_w = pre_weight;
  a.T = num_tokens;
  a.H = hidden;
  a.gate_kind = gate_kind;
  a.gate_act = gate_act;
  a.scale = scale;
  a.rstd_post = const_cast<float*>(rstd_post);
  a.rstd_pre = const_cast<float*>(rstd_pre);
  a.grad_residual = grad_residual;
  a.grad_y = grad_y;
  a.grad_gate = grad_gate;
  a.grad_post_w = grad_post_weight;
  a.grad_pre_w = grad_pre_weight;
  a.partials = static_cast<float*>(workspace);
  cudaError_t e =
      launch_block_norm_backward(c, a, stream_dtype == MOE_DT_F32, block_dtype == MOE_DT_F32);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

size_t moe_balance_loss_workspace_bytes(int64_t num_tokens, int32_t num_experts,
                                        int32_t num_seqs) {
  if (num_tokens <= 0 || num_tokens >= ((int64_t)1 << 31) || num_experts < 1 ||
      num_experts > MOE_MAX_EXPERTS || num_seqs < 1 || num_seqs > 65535)
    return 0;
  // whatever the scores' alignment will be
  const size_t a = balance_workspace_bytes(num_tokens, num_experts, num_seqs, true);
  const size_t b = balance_workspace_bytes(num_tokens, num_experts, num_seqs, false);
  return a > b ? a : b;
}

moe_status_t moe_balance_loss(const float* scores, const int32_t* topk_idx, int64_t num_tokens,
                              int32_t num_experts, int32_t num_topk, int32_t score_func,
                              const int32_t* seq_offsets, int32_t num_seqs,
                              const uint8_t* token_mask, float* balance, float* z,
                              int32_t* counts, float* probs, int32_t* tokens, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (num_tokens < 0 || num_tokens >= ((int64_t)1 << 31) || !experts_ok(num_experts, num_topk))
    return MOE_ERR_INVALID_ARG;
  if (score_func != MOE_SCORE_SOFTMAX && score_func != MOE_SCORE_SIGMOID)
    return MOE_ERR_INVALID_ARG;
  if (num_seqs < 1 || num_seqs > 65535 || (!seq_offsets && num_seqs != 1))
    return MOE_ERR_INVALID_ARG;
  if (!balance || !z || !counts || !probs || !tokens) return MOE_ERR_INVALID_ARG;
  if (!aligned(balance, 4) || !aligned(z, 4) || !aligned(counts, 4) || !aligned(probs, 4) ||
      !aligned(tokens, 4) || !aligned(seq_offsets, 4))
    return MOE_ERR_INVALID_ARG;
  if (num_tokens == 0) {
    const size_t S = (size_t)num_seqs, SE = S * (size_t)num_experts;
    cudaError_t e = zero(balance, S * 4, stream);
    if (e == cudaSuccess) e = zero(z, S * 4, stream);
    if (e == cudaSuccess) e = zero(tokens, S * 4, stream);
    if (e == cudaSuccess) e = zero(counts, SE * 4, stream);
    if (e == cudaSuccess) e = zero(probs, SE * 4, stream);
    return e == cudaSuccess ? MOE_OK : cuda_fail(e);
  }
  if (!scores || !topk_idx || !aligned(scores, 4) || !aligned(topk_idx, 4))
    return MOE_ERR_INVALID_ARG;
  const size_t need =
      balance_workspace_bytes(num_tokens, num_experts, num_seqs, aligned(scores, 16));
  if (need > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < need))
    return MOE_ERR_INVALID_ARG;
  LaunchCtx c;
  moe_status_t s = context(stream, &c);
  if (s != MOE_OK) return s;
  BalanceArgs a;
  a.scores = scores;
  a.idx = topk_idx;
  a.T = num_tokens;
  a.E = num_experts;
  a.k = num_topk;
  a.func = score_func;
  a.S = num_seqs;
  a.seq = seq_offsets;
  a.mask = token_mask;
  a.balance = balance;
  a.z = z;
  a.counts = counts;
  a.probs = probs;
  a.tokens = tokens;
  a.ws = workspace;
  cudaError_t e = launch_balance_loss(c, a);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

moe_status_t moe_balance_loss_backward(const float* scores, int64_t num_tokens,
                                       int32_t num_experts, int32_t num_topk, int32_t score_func,
                                       const int32_t* seq_offsets, int32_t num_seqs,
                                       const uint8_t* token_mask, const int32_t* counts,
                                       const int32_t* tokens, const float* grad_balance,
                                       const float* grad_z, const int32_t* topk_idx,
                                       const float* topk_weights, const float* grad_topk_weights,
                                       float* grad_scores, void* stream) {
  if (num_tokens < 0 || num_tokens >= ((int64_t)1 << 31) || !experts_ok(num_experts, num_topk))
    return MOE_ERR_INVALID_ARG;
  if (score_func != MOE_SCORE_SOFTMAX && score_func != MOE_SCORE_SIGMOID)
    return MOE_ERR_INVALID_ARG;
  if (num_seqs < 1 || num_seqs > 65535 || (!seq_offsets && num_seqs != 1))
    return MOE_ERR_INVALID_ARG;
  if (num_tokens == 0) return MOE_OK;
  if (!scores || !counts || !tokens || !grad_scores) return MOE_ERR_INVALID_ARG;
  if (grad_topk_weights && (!topk_idx || !topk_weights)) return MOE_ERR_INVALID_ARG;
  if (!aligned(scores, 4) || !aligned(counts, 4) || !aligned(tokens, 4) ||
      !aligned(grad_balance, 4) || !aligned(grad_z, 4) || !aligned(topk_idx, 4) ||
      !aligned(topk_weights, 4) || !aligned(grad_topk_weights, 4) || !aligned(grad_scores, 4) ||
      !aligned(seq_offsets, 4))
    return MOE_ERR_INVALID_ARG;
  LaunchCtx c;
  moe_status_t s = context(stream, &c);
  if (s != MOE_OK) return s;
  BalanceArgs a;
  a.scores = scores;
  a.idx = topk_idx;
  a.T = num_tokens;
  a.E = num_experts;
  a.k = num_topk;
  a.func = score_func;
  a.S = num_seqs;
  a.seq = seq_offsets;
  a.mask = token_mask;
  a.counts = const_cast<int32_t*>(counts);
  a.tokens = const_cast<int32_t*>(tokens);
  a.grad_balance = grad_balance;
  a.grad_z = grad_z;
  a.w = topk_weights;
  a.grad_w = grad_topk_weights;
  a.grad_scores = grad_scores;
  cudaError_t e = launch_balance_loss_backward(c, a);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

moe_status_t moe_combine_backward(const void* grad_out, int32_t grad_dtype, const void* y,
                                  const float* topk_weights, const int32_t* pos,
                                  const int32_t* sorted_src, int64_t num_tokens, int32_t hidden,
                                  int32_t num_topk, int64_t num_rows, void* grad_y,
                                  float* grad_topk_weights, void* stream) {
  if (!dtype_ok(grad_dtype) || num_tokens < 0 || num_rows < 0 || hidden < 8 || hidden % 8 != 0 ||
      num_topk < 1 || num_topk > MOE_MAX_TOPK || num_rows >= ((int64_t)1 << 31))
    return MOE_ERR_INVALID_ARG;
  if (num_tokens * (hidden / 8) >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
  if (num_tokens == 0 && (num_rows == 0 || !sorted_src)) return MOE_OK;
  if (num_tokens > 0 && (!grad_out || !topk_weights || !pos || !grad_topk_weights))
    return MOE_ERR_INVALID_ARG;
  if (num_rows > 0 && ((num_tokens > 0 && !y) || !grad_y)) return MOE_ERR_INVALID_ARG;
  if (!aligned(grad_out, 16) || !aligned(y, 16) || !aligned(grad_y, 16) ||
      !aligned(topk_weights, 4) || !aligned(pos, 4) || !aligned(sorted_src, 4) ||
      !aligned(grad_topk_weights, 4))
    return MOE_ERR_INVALID_ARG;
  LaunchCtx c;
  moe_status_t s = context(stream, &c);
  if (s != MOE_OK) return s;
  cudaError_t e = launch_combine_backward(c, grad_out, grad_dtype == MOE_DT_F32, y, topk_weights,
                                          pos, num_rows > 0 ? sorted_src : nullptr, num_tokens,
                                          hidden, num_topk, num_rows, grad_y, grad_topk_weights);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

moe_status_t moe_expert_matvec_fp4(const void* x, int64_t num_x, const uint8_t* w,
                                   const void* w_sf, int32_t sf_type, int32_t group,
                                   const int32_t* offsets, const int32_t* sorted_src,
                                   int32_t num_experts, int32_t num_topk, int64_t num_rows,
                                   int32_t k_dim, int32_t n_dim, int32_t swiglu, void* out,
                                   int32_t out_dtype, void* stream) {
  if (group != 16 && group != 32 && group != 64 && group != 128) return MOE_ERR_UNSUPPORTED;
  if (sf_type != MOE_WSF_F32 && sf_type != MOE_WSF_UE8M0) return MOE_ERR_INVALID_ARG;
  if (out_dtype != MOE_OUT_BF16 && out_dtype != MOE_OUT_F32) return MOE_ERR_INVALID_ARG;
  if (num_experts < 1 || num_experts > MOE_MAX_EXPERTS || num_topk < 1 ||
      num_topk > MOE_MAX_TOPK || num_rows < 0 || num_x < 0 || n_dim < 1 || k_dim < 32 ||
      k_dim % 32 != 0 || k_dim % group != 0)
    return MOE_ERR_INVALID_ARG;
  if (!offsets && num_experts != 1) return MOE_ERR_INVALID_ARG;
  if (!sorted_src && num_x < num_rows) return MOE_ERR_INVALID_ARG;
  if (k_dim > 16384 || num_rows > MOE_MATVEC_MAX_ROWS ||
      (int64_t)k_dim * n_dim * (swiglu ? 2 : 1) >= ((int64_t)1 << 32) ||
      (int64_t)num_experts * n_dim * (swiglu ? 2 : 1) >= ((int64_t)1 << 31))
    return MOE_ERR_UNSUPPORTED;
  if (num_rows == 0) return MOE_OK;
  if ((num_x > 0 && !x) || !w || !w_sf || !out) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(offsets, 4) || !aligned(sorted_src, 4) ||
      !aligned(w_sf, 4) ||
      !aligned(out, out_dtype == MOE_OUT_F32 ? 4 : 2))
    return MOE_ERR_INVALID_ARG;
  LaunchCtx c;
  moe_status_t s = context(stream, &c);
  if (s != MOE_OK) return s;
  MatvecArgs a;
  a.x = x;
  a.num_x = num_x;
  a.w = w;
  a.sf = w_sf;
  a.sf_type = sf_type;
  a.group = group;
  a.offsets = offsets;
  a.src = sorted_src;
  a.E = num_experts;
  a.k = num_topk;
  a.R = num_rows;
  a.K = k_dim;
  a.N = n_dim;
  a.swiglu = swiglu ? 1 : 0;
  a.out = out;
  a.out_f32 = out_dtype == MOE_OUT_F32;
  cudaError_t e = launch_expert_matvec_fp4(c, a);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

moe_status_t moe_router_gate(const float* scores, int64_t num_tokens, int32_t num_experts,
                             int32_t num_topk, int32_t score_func, const float* bias,
                             int32_t num_groups, int32_t topk_groups, int32_t group_score,
                             int32_t renormalize, float scale, int32_t* topk_idx,
                             float* topk_weights, void* stream) {
  if (num_tokens < 0 || num_tokens >= ((int64_t)1 << 31) || !experts_ok(num_experts, num_topk))
    return MOE_ERR_INVALID_ARG;
  if (score_func != MOE_SCORE_SOFTMAX && score_func != MOE_SCORE_SIGMOID)
    return MOE_ERR_INVALID_ARG;
  if (num_groups < 1 || num_groups > MOE_MAX_GROUPS || num_experts % num_groups != 0 ||
      topk_groups < 1 || topk_groups > num_groups ||
      num_topk > num_experts / num_groups * topk_groups)
    return MOE_ERR_INVALID_ARG;
  if (group_score != MOE_GROUP_MAX && group_score != MOE_GROUP_TOP2) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return MOE_ERR_INVALID_ARG;
  if (num_tokens == 0) return MOE_OK;
  if (!scores || !topk_idx || !topk_weights || !aligned(scores, 4) || !aligned(bias, 4) ||
      !aligned(topk_idx, 4) || !aligned(topk_weights, 4))
    return MOE_ERR_INVALID_ARG;
  LaunchCtx c;
  moe_status_t s = context(stream, &c);
  if (s != MOE_OK) return s;
  RouterArgs a;
  a.scores = scores;
  a.T = num_tokens;
  a.E = num_experts;
  a.k = num_topk;
  a.func = score_func;
  a.bias = bias;
  a.G = num_groups;
  a.g = topk_groups;
  a.group_score = group_score;
  a.renorm = renormalize != 0;
  a.scale = scale;
  a.idx = topk_idx;
  a.w = topk_weights;
  cudaError_t e = launch_router_gate(c, a);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

moe_status_t moe_router_gate_backward(const float* scores, int64_t num_tokens,
                                      int32_t num_experts, int32_t num_topk, int32_t score_func,
                                      int32_t renormalize, float scale, const int32_t* topk_idx,
                                      const float* grad_topk_weights, const float* add,
                                      float* grad_scores, void* stream) {
  if (num_tokens < 0 || num_tokens >= ((int64_t)1 << 31) || !experts_ok(num_experts, num_topk))
    return MOE_ERR_INVALID_ARG;
  if (score_func != MOE_SCORE_SOFTMAX && score_func != MOE_SCORE_SIGMOID)
    return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return MOE_ERR_INVALID_ARG;
  if (num_tokens == 0) return MOE_OK;
  if (!scores || !topk_idx || !grad_topk_weights || !grad_scores || !aligned(scores, 4) ||
      !aligned(topk_idx, 4) || !aligned(grad_topk_weights, 4) || !aligned(add, 4) ||
      !aligned(grad_scores, 4))
    return MOE_ERR_INVALID_ARG;
  LaunchCtx c;
  moe_status_t s = context(stream, &c);
  if (s != MOE_OK) return s;
  RouterArgs a;
  a.scores = scores;
  a.T = num_tokens;
  a.E = num_experts;
  a.k = num_topk;
  a.func = score_func;
  a.renorm = renormalize != 0;
  a.scale = scale;
  a.idx = const_cast<int32_t*>(topk_idx);
  a.grad_w = grad_topk_weights;
  a.add = add;
  a.grad_scores = grad_scores;
  cudaError_t e = launch_router_gate_backward(c, a);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

moe_status_t moe_cast_int8(const void* x, int32_t dtype, int64_t num_rows, int32_t hidden,
                           int8_t* out, float* out_sf, void* stream) {
  if (!dtype_ok(dtype) || num_rows < 0 || hidden < 1) return MOE_ERR_INVALID_ARG;
  if (num_rows >= ((int64_t)1 << 31) || hidden > 1 << 30 ||
      num_rows >= ((int64_t)1 << 40) / hidden)
    return MOE_ERR_UNSUPPORTED;
  if (num_rows == 0) return MOE_OK;
  if (!x || !out || !out_sf || !aligned(x, dtype_size(dtype)) || !aligned(out_sf, 4))
    return MOE_ERR_INVALID_ARG;
  LaunchCtx c;
  moe_status_t s = context(stream, &c);
  if (s != MOE_OK) return s;
  cudaError_t e = launch_cast_int8(c, x, dtype == MOE_DT_F32, num_rows, hidden, out, out_sf);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

moe_status_t moe_expert_matmul_int8(const int8_t* x, const float* x_sf, int64_t num_x,
                                    const int8_t* w, const float* w_sf, const int32_t* offsets,
                                    const int32_t* sorted_src, int32_t num_experts,
                                    int32_t num_topk, int64_t num_rows, int32_t k_dim,
                                    int32_t n_dim, int32_t swiglu, void* out, int32_t out_dtype,
                                    void* stream) {
  if (out_dtype != MOE_OUT_BF16 && out_dtype != MOE_OUT_F32) return MOE_ERR_INVALID_ARG;
  if (num_experts < 1 || num_experts > MOE_MAX_EXPERTS || num_topk < 1 ||
      num_topk > MOE_MAX_TOPK || num_rows < 0 || num_x < 0 || n_dim < 1 || k_dim < 16 ||
      k_dim % 16 != 0)
    return MOE_ERR_INVALID_ARG;
  if (!offsets && num_experts != 1) return MOE_ERR_INVALID_ARG;
  if (!sorted_src && num_x < num_rows) return MOE_ERR_INVALID_ARG;
  if (k_dim > 65536 || num_rows >= ((int64_t)1 << 31) ||
      (int64_t)num_experts * n_dim * (swiglu ? 2 : 1) >= ((int64_t)1 << 31) - 512)
    return MOE_ERR_UNSUPPORTED;
  if (num_rows == 0) return MOE_OK;
  if ((num_x > 0 && (!x || !x_sf)) || !w || !w_sf || !out) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(x_sf, 4) || !aligned(w_sf, 4) ||
      !aligned(offsets, 4) || !aligned(sorted_src, 4) ||
      !aligned(out, out_dtype == MOE_OUT_F32 ? 4 : 2))
    return MOE_ERR_INVALID_ARG;
  LaunchCtx c;
  moe_status_t s = context(stream, &c);
  if (s != MOE_OK) return s;
  MatmulInt8Args a;
  a.x = x;
  a.x_sf = x_sf;
  a.num_x = num_x;
  a.w = w;
  a.w_sf = w_sf;
  a.offsets = offsets;
  a.src = sorted_src;
  a.E = num_experts;
  a.k = num_topk;
  a.R = num_rows;
  a.K = k_dim;
  a.N = n_dim;
  a.swiglu = swiglu ? 1 : 0;
  a.out = out;
  a.out_f32 = out_dtype == MOE_OUT_F32;
  a.wait_ns = (uint64_t)g_decode_timeout_ns.load();
  a.stages = g_matmul_int8_stages.load();
  cudaError_t e = launch_expert_matmul_int8(c, a);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

moe_status_t moe_debug_matmul_int8_form(int32_t num_experts, int64_t num_rows, int32_t k_dim,
                                        int32_t n_dim, int32_t swiglu, int32_t* form) {
  if (num_experts < 1 || num_experts > MOE_MAX_EXPERTS || num_rows < 1 ||
      num_rows >= ((int64_t)1 << 31) || k_dim < 16 || k_dim > 65536 || n_dim < 1 || !form)
    return MOE_ERR_INVALID_ARG;
  LaunchCtx c;
  moe_status_t s = context(nullptr, &c);
  if (s != MOE_OK) return s;
  MatmulInt8Args a;
  static const int32_t given = 0;
  a.offsets = &given;  // not read: the form goes by the sizes
  a.E = num_experts;
  a.R = num_rows;
  a.K = k_dim;
  a.N = n_dim;
  a.swiglu = swiglu ? 1 : 0;
  int f = 0, ctas = 0;
  cudaError_t e = expert_matmul_int8_form(c, a, &f, &ctas);
  *form = f;
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

}  // extern "C"
