// operators_api.cu -- the entry points of include/moe.h beside the layer's
// forward pass: tokens sorted by expert and back with their gradients, the
// router's gradient, and the experts' products in 8-bit integers.
#include "api_common.cuh"

using moe::aligned16;
using moe::at;
using moe::cuda_status;
using moe::current_device;
using moe::NvtxRange;
using moe::validate_config;

namespace {

// The operators' workspace: the header (device status word, and the 8-bit
// products' mark beside it), then one double per block of the router gradient.
constexpr size_t kHeaderBytes = 256;
constexpr size_t kOperatorWorkspace = kHeaderBytes + moe::kGradMaxBlocks * sizeof(double);

moe_status_t check_operator_workspace(const void* ws, size_t bytes) {
  if (ws == nullptr || !aligned16(ws)) return MOE_ERR_INVALID_ARGUMENT;
  return bytes < kOperatorWorkspace ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_OK;
}

// What the four row operators check alike.
moe_status_t check_rows(const moe_config_t* cfg, moe_dtype_t dtype, const int32_t* inverse) {
  const moe_status_t st = validate_config(cfg);
  if (st != MOE_OK) return st;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARGUMENT;
  if (cfg->num_tokens > 0 && inverse == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

// Whether p is memory of the current device, without touching it.
bool device_memory(const void* p) {
  int dev = 0;
  cudaPointerAttributes attr;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaPointerGetAttributes(&attr, p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return (attr.type == cudaMemoryTypeDevice && attr.device == dev) || attr.type == cudaMemoryTypeManaged;
}

bool given(const void* p) { return p != nullptr && aligned16(p); }
bool given_or_null(const void* p) { return aligned16(p); }

moe::RowsArgs rows_args(const moe_config_t* c, moe_dtype_t dtype, const int32_t* inverse, const float* weights,
                        int num_sms) {
  moe::RowsArgs a = {};
  a.inverse = inverse;
  a.weights = weights;
  a.T = c->num_tokens;
  a.k = c->top_k;
  a.R = c->num_tokens * c->top_k;
  a.vec = c->hidden_dim / (dtype == MOE_DTYPE_F32 ? 4 : 8);  // hidden_dim is a multiple of 8
  a.num_sms = num_sms;
  return a;
}

// K and N of one of the two contractions.
struct Shape {
  int K;
  int64_t N;
};
Shape shape_of(const moe_config_t* c, moe_contraction_t which) {
  if (which == MOE_GATE_UP) return {c->hidden_dim, 2 * static_cast<int64_t>(c->moe_dim)};
  return {c->moe_dim, c->hidden_dim};
}

moe_status_t check_int8(const moe_config_t* cfg, moe_contraction_t which) {
  const moe_status_t st = validate_config(cfg);
  if (st != MOE_OK) return st;
  if (which != MOE_GATE_UP && which != MOE_DOWN) return MOE_ERR_INVALID_ARGUMENT;
  const Shape s = shape_of(cfg, which);
  // 127 * 127 * K stays below 2^31, and column numbers are 32-bit
  if (s.K > MOE_INT8_MAX_K || s.N > (int64_t(1) << 30)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status_t moe_operator_workspace_size(const moe_config_t* cfg, size_t* bytes) {
  const moe_status_t st = validate_config(cfg);
  if (st != MOE_OK) return st;
  if (bytes == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  *bytes = kOperatorWorkspace;
  return MOE_OK;
}

moe_status_t moe_dispatch(const moe_config_t* cfg, moe_dtype_t dtype, const void* x, const int32_t* inverse,
                          const float* expert_weights, void* rows, moe_stream_t stream) {
  moe::refresh_switches();
  const NvtxRange api_range("moe_dispatch");
  moe_status_t st = check_rows(cfg, dtype, inverse);
  if (st != MOE_OK) return st;
  if (cfg->num_tokens == 0) return MOE_OK;
  if (!given(x) || !given(rows) || x == rows) return MOE_ERR_INVALID_ARGUMENT;
  int num_sms = 0;
  if ((st = current_device(&num_sms)) != MOE_OK) return st;
  moe::RowsArgs a = rows_args(cfg, dtype, inverse, expert_weights, num_sms);
  a.tok_in = x;
  a.rows_out = rows;
  return cuda_status(moe::launch_rows_spread(a, dtype == MOE_DTYPE_F32, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_dispatch_backward(const moe_config_t* cfg, moe_dtype_t dtype, const void* d_rows, const void* x,
                                   const int32_t* inverse, const float* expert_weights, void* d_x,
                                   float* d_expert_weights, moe_stream_t stream) {
  moe::refresh_switches();
  const NvtxRange api_range("moe_dispatch_backward");
  moe_status_t st = check_rows(cfg, dtype, inverse);
  if (st != MOE_OK) return st;
  if (cfg->num_tokens == 0) return MOE_OK;
  if (!given(d_rows) || !given(d_x) || !given_or_null(x)) return MOE_ERR_INVALID_ARGUMENT;
  if (d_expert_weights != nullptr && x == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  if (d_x == x || d_x == d_rows) return MOE_ERR_INVALID_ARGUMENT;  // not in place
  int num_sms = 0;
  if ((st = current_device(&num_sms)) != MOE_OK) return st;
  moe::RowsArgs a = rows_args(cfg, dtype, inverse, expert_weights, num_sms);
  a.rows_in = d_rows;
  a.tok_in = x;
  a.tok_out = d_x;
  a.d_weights = d_expert_weights;
  return cuda_status(moe::launch_rows_gather(a, dtype == MOE_DTYPE_F32, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_combine(const moe_config_t* cfg, moe_dtype_t dtype, const void* rows, const int32_t* inverse,
                         const float* expert_weights, void* out, moe_stream_t stream) {
  moe::refresh_switches();
  const NvtxRange api_range("moe_combine");
  moe_status_t st = check_rows(cfg, dtype, inverse);
  if (st != MOE_OK) return st;
  if (cfg->num_tokens == 0) return MOE_OK;
  if (!given(rows) || !given(out) || rows == out) return MOE_ERR_INVALID_ARGUMENT;
  int num_sms = 0;
  if ((st = current_device(&num_sms)) != MOE_OK) return st;
  moe::RowsArgs a = rows_args(cfg, dtype, inverse, expert_weights, num_sms);
  a.rows_in = rows;
  a.tok_out = out;
  return cuda_status(moe::launch_rows_gather(a, dtype == MOE_DTYPE_F32, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_combine_backward(const moe_config_t* cfg, moe_dtype_t dtype, const void* d_out, const void* rows,
                                  const int32_t* inverse, const float* expert_weights, void* d_rows,
                                  float* d_expert_weights, moe_stream_t stream) {
  moe::refresh_switches();
  const NvtxRange api_range("moe_combine_backward");
  moe_status_t st = check_rows(cfg, dtype, inverse);
  if (st != MOE_OK) return st;
  if (cfg->num_tokens == 0) return MOE_OK;
  if (!given(d_out) || !given(d_rows) || !given_or_null(rows)) return MOE_ERR_INVALID_ARGUMENT;
  if (d_expert_weights != nullptr && rows == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  if (d_rows == rows || d_rows == d_out) return MOE_ERR_INVALID_ARGUMENT;  // not in place
  int num_sms = 0;
  if ((st = current_device(&num_sms)) != MOE_OK) return st;
  moe::RowsArgs a = rows_args(cfg, dtype, inverse, expert_weights, num_sms);
  a.tok_in = d_out;
  a.rows_in = rows;
  a.rows_out = d_rows;
  a.d_weights = d_expert_weights;
  return cuda_status(moe::launch_rows_spread(a, dtype == MOE_DTYPE_F32, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_route_backward(const moe_config_t* cfg, const void* logits, const float* global_scale,
                                const int32_t* expert_indices, const float* d_expert_weights,
                                const float* d_sink_weights, void* d_logits, float* d_global_scale, void* workspace,
                                size_t workspace_bytes, moe_stream_t stream) {
  moe::refresh_switches();
  const NvtxRange api_range("moe_route_backward");
  moe_status_t st = validate_config(cfg);
  if (st != MOE_OK) return st;
  const bool sink = cfg->router == MOE_ROUTER_SIGMOID_SINK;
  // the softmax router has no global scale
  if (!sink && (global_scale != nullptr || d_global_scale != nullptr)) return MOE_ERR_INVALID_ARGUMENT;
  if (cfg->num_sink == 0 && d_sink_weights != nullptr) return MOE_ERR_INVALID_ARGUMENT;
  if (d_global_scale != nullptr) {
    if ((st = check_operator_workspace(workspace, workspace_bytes)) != MOE_OK) return st;
  }
  if (cfg->num_tokens > 0 && (logits == nullptr || expert_indices == nullptr || d_expert_weights == nullptr ||
                              d_logits == nullptr || d_logits == logits))
    return MOE_ERR_INVALID_ARGUMENT;
  if (cfg->num_tokens == 0 && d_global_scale == nullptr) return MOE_OK;
  int num_sms = 0;
  if ((st = current_device(&num_sms)) != MOE_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // no token: the gradient of the global scale is an empty sum
  if (cfg->num_tokens == 0) return cuda_status(cudaMemsetAsync(d_global_scale, 0, sizeof(float), s));
  moe::RouterGradArgs a = {};
  a.logits = logits;
  a.stride = cfg->logits_row_stride;
  a.T = cfg->num_tokens;
  a.E = cfg->num_experts;
  a.k = cfg->top_k;
  a.S = cfg->num_sink;
  a.route_scale = cfg->route_scale;
  a.global_scale = global_scale;
  a.idx = expert_indices;
  a.d_weights = d_expert_weights;
  a.d_sink = d_sink_weights;
  a.d_logits = d_logits;
  a.partial = d_global_scale != nullptr ? at<double>(workspace, kHeaderBytes) : nullptr;
  a.d_global_scale = d_global_scale;
  return cuda_status(moe::launch_route_grad(a, sink, cfg->logits_dtype == MOE_DTYPE_BF16, s));
}

moe_status_t moe_dispatch_int8(const moe_config_t* cfg, const void* x, const int32_t* inverse, int8_t* rows_q,
                               float* row_scales, moe_stream_t stream) {
  moe::refresh_switches();
  const NvtxRange api_range("moe_dispatch_int8");
  moe_status_t st = check_int8(cfg, MOE_GATE_UP);
  if (st != MOE_OK) return st;
  if (cfg->num_tokens == 0) return MOE_OK;
  if (!given(x) || inverse == nullptr || !given(rows_q) || row_scales == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  int num_sms = 0;
  if ((st = current_device(&num_sms)) != MOE_OK) return st;
  return cuda_status(moe::launch_quantize_rows(static_cast<const __nv_bfloat16*>(x), cfg->num_tokens, cfg->hidden_dim,
                                               inverse, cfg->top_k, cfg->num_tokens * cfg->top_k, nullptr, rows_q,
                                               row_scales, num_sms, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_quantize_rows(const moe_config_t* cfg, const void* h, const int32_t* expert_offsets, int8_t* rows_q,
                               float* row_scales, moe_stream_t stream) {
  moe::refresh_switches();
  const NvtxRange api_range("moe_quantize_rows");
  moe_status_t st = check_int8(cfg, MOE_DOWN);
  if (st != MOE_OK) return st;
  if (cfg->num_tokens == 0) return MOE_OK;
  if (!given(h) || !given(rows_q) || row_scales == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  int num_sms = 0;
  if ((st = current_device(&num_sms)) != MOE_OK) return st;
  const int R = cfg->num_tokens * cfg->top_k;
  return cuda_status(moe::launch_quantize_rows(
      static_cast<const __nv_bfloat16*>(h), R, cfg->moe_dim, nullptr, 1, R,
      expert_offsets != nullptr ? expert_offsets + cfg->num_experts : nullptr, rows_q, row_scales, num_sms,
      reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_quantize_weights(const moe_config_t* cfg, moe_contraction_t which, const void* w, int8_t* w_q,
                                  float* w_scales, moe_stream_t stream) {
  moe::refresh_switches();
  const NvtxRange api_range("moe_quantize_weights");
  moe_status_t st = check_int8(cfg, which);
  if (st != MOE_OK) return st;
  if (!given(w) || !given(w_q) || w_scales == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  int num_sms = 0;
  if ((st = current_device(&num_sms)) != MOE_OK) return st;
  const Shape s = shape_of(cfg, which);
  return cuda_status(moe::launch_quantize_weights(static_cast<const __nv_bfloat16*>(w), cfg->num_experts, s.K,
                                                  static_cast<int>(s.N), w_q, w_scales,
                                                  reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_grouped_linear_int8(const moe_config_t* cfg, moe_contraction_t which, const int8_t* rows_q,
                                     const float* row_scales, const int8_t* w_q, const float* w_scales,
                                     const void* bias, const int32_t* expert_offsets, void* out, void* workspace,
                                     size_t workspace_bytes, moe_stream_t stream) {
  moe::refresh_switches();
  const NvtxRange api_range("moe_grouped_linear_int8");
  moe_status_t st = check_int8(cfg, which);
  if (st != MOE_OK) return st;
  if (cfg->num_tokens == 0) {
    // nothing but the status, where there is a word for it: such a call may
    // come without pointers, as the other entry points take it
    if (check_operator_workspace(workspace, workspace_bytes) != MOE_OK || !device_memory(workspace)) return MOE_OK;
    moe::Int8GemmArgs a = {};
    a.down = which == MOE_DOWN ? 1 : 0;
    a.status = at<int>(workspace, 0);
    return cuda_status(moe::launch_int8_gemm(a, reinterpret_cast<cudaStream_t>(stream)));
  }
  if (!given(rows_q) || row_scales == nullptr || !given(w_q) || !given(w_scales) || expert_offsets == nullptr ||
      !given(out))
    return MOE_ERR_INVALID_ARGUMENT;
  if (cfg->has_bias ? !given(bias) : bias != nullptr) return MOE_ERR_INVALID_ARGUMENT;
  if ((st = check_operator_workspace(workspace, workspace_bytes)) != MOE_OK) return st;
  int num_sms = 0;
  if ((st = current_device(&num_sms)) != MOE_OK) return st;
  moe::Int8GemmArgs a = {};
  a.offsets = expert_offsets;
  a.E = cfg->num_experts;
  a.R = cfg->num_tokens * cfg->top_k;
  a.H = cfg->hidden_dim;
  a.D = cfg->moe_dim;
  a.down = which == MOE_DOWN ? 1 : 0;
  a.gate_up_format = cfg->gate_up_format;
  a.activation = cfg->activation;
  a.alpha = cfg->alpha;
  a.limit = cfg->limit;
  a.A = rows_q;
  a.a_scales = row_scales;
  a.W = w_q;
  a.w_scales = w_scales;
  a.bias = static_cast<const __nv_bfloat16*>(bias);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.status = at<int>(workspace, 0);
  a.num_sms = num_sms;
  return cuda_status(moe::launch_int8_gemm(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
