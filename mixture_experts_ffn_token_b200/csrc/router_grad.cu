// router_grad.cu -- the gradient of stage 1 (moe_route), one warp per token.
//
// Over the n = k (+ S sink) normalised entries, p = softmax(z) for the softmax
// router or softmax(log sigmoid(z)) for the sigmoid router with sink lanes,
// and w = c p with c = 1 or route_scale * global_scale:
//   dz_i = c p_i sum_j p_j (dw_i - dw_j)   [ * sigmoid(-z_i) for the sigmoid router ]
//   d global_scale = route_scale * sum over tokens and entries of p_i dw_i .
// The differences are taken before they are weighted, so a weight close to
// one costs its entry no digits.  The selection has no gradient, nor has the
// selection bias.  p is computed again from the logits: k + S reads a token,
// against k + S more outputs of the forward pass to keep.
//
// Bound by the store of the dense [T, E + S] gradient: a warp builds its row
// in shared memory (zeros, then the n entries) and stores it in order.
#include <algorithm>

#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kGradWarps = 4;

__device__ __forceinline__ float log_sigmoid_f(float z) { return fminf(z, 0.f) - log1pf(expf(-fabsf(z))); }

template <bool SINK, bool BF16>
__global__ void __launch_bounds__(32 * kGradWarps) route_grad_kernel(const RouterGradArgs a) {
  griddep_wait();  // the previous kernel's results are complete and visible
  griddep_launch_dependents();
  extern __shared__ float s_rows[];  // [kGradWarps][E + S]
  __shared__ double s_sum[kGradWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cols = a.E + a.S;
  float* row = s_rows + warp * cols;
  const int n = a.k + a.S;  // <= 32
  float c = 1.f;
  if constexpr (SINK) c = a.route_scale * (a.global_scale != nullptr ? *a.global_scale : 1.f);
  double total = 0.0;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kGradWarps + warp; t < a.T;
       t += static_cast<int64_t>(gridDim.x) * kGradWarps) {
    for (int i = lane; i < cols; i += 32) row[i] = 0.f;
    // lane i < k: the i-th selected expert; lanes k .. n-1: the sink lanes
    int col = -1;
    float dw = 0.f, z = 0.f;
    if (lane < a.k) {
      col = a.idx[t * a.k + lane];
      if (col < 0 || col >= a.E) col = -1;  // no expert: the entry takes no part
      dw = a.d_weights[t * a.k + lane];
    } else if (lane < n) {
      col = a.E + lane - a.k;
      dw = a.d_sink != nullptr ? a.d_sink[t * a.S + lane - a.k] : 0.f;
    }
    const bool on = col >= 0;
    if (!on) dw = 0.f;
    if (on) {
      if constexpr (BF16) z = __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[t * a.stride + col]);
      else z = static_cast<const float*>(a.logits)[t * a.stride + col];
    }
    const float l = !on ? -INFINITY : SINK ? log_sigmoid_f(z) : z;
    float m = l;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float ex = on ? expf(l - m) : 0.f;
    float sum = ex;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    const float p = on ? ex / sum : 0.f;
    float g = 0.f;
    for (int j = 0; j < n; ++j) {
      const float pj = __shfl_sync(0xffffffffu, p, j), dj = __shfl_sync(0xffffffffu, dw, j);
      const bool oj = __shfl_sync(0xffffffffu, static_cast<int>(on), j) != 0;
      if (oj && j != lane) g += pj * (dw - dj);
    }
    g *= c * p;
    if constexpr (SINK) {
      g *= 1.f / (1.f + expf(z));
      if (a.partial != nullptr) {
        double s = on ? static_cast<double>(p) * dw : 0.0;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        total += s;
      }
    }
    // an expert named twice gets the sum of its entries, in entry order
    const uint32_t peers = __match_any_sync(0xffffffffu, on ? col : -1 - lane);
    const bool twice = __any_sync(0xffffffffu, (peers & (peers - 1)) != 0);
    float v = g;
    if (twice) {
      v = 0.f;
      for (int j = 0; j < n; ++j) {
        const float gj = __shfl_sync(0xffffffffu, g, j);
        if ((peers >> j) & 1u) v += gj;
      }
    }
    __syncwarp();
    if (on && (peers & ((1u << lane) - 1u)) == 0) row[col] = v;
    __syncwarp();
    for (int i = lane; i < cols; i += 32) {
      if constexpr (BF16) static_cast<__nv_bfloat16*>(a.d_logits)[t * a.stride + i] = __float2bfloat16_rn(row[i]);
      else static_cast<float*>(a.d_logits)[t * a.stride + i] = row[i];
    }
    __syncwarp();
  }
  if (SINK && a.partial != nullptr) {
    if (lane == 0) s_sum[warp] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
      double s = 0.0;
      for (int w = 0; w < kGradWarps; ++w) s += s_sum[w];
      a.partial[blockIdx.x] = s;
    }
  }
}

// d_global_scale = route_scale * the sum of the blocks' parts, in a fixed order.
__global__ void __launch_bounds__(32) scale_grad_kernel(const double* partial, int n, float route_scale, float* out) {
  griddep_wait();  // the previous kernel's results are complete and visible
  griddep_launch_dependents();
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += 32) s += partial[i];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if (threadIdx.x == 0) *out = static_cast<float>(s * static_cast<double>(route_scale));
}

}  // namespace

cudaError_t launch_route_grad(const RouterGradArgs& a, bool sink, bool bf16, float* d_global_scale,
                              cudaStream_t stream) {
  const int64_t blocks = std::min<int64_t>((static_cast<int64_t>(a.T) + kGradWarps - 1) / kGradWarps, kGradMaxBlocks);
  const dim3 grid(static_cast<unsigned>(blocks)), block(32 * kGradWarps);
  const size_t smem = static_cast<size_t>(kGradWarps) * (a.E + a.S) * sizeof(float);  // at most 16.5 KB
  cudaError_t err;
  if (sink)
    err = bf16 ? launch_pdl(route_grad_kernel<true, true>, grid, block, smem, stream, a)
               : launch_pdl(route_grad_kernel<true, false>, grid, block, smem, stream, a);
  else
    err = bf16 ? launch_pdl(route_grad_kernel<false, true>, grid, block, smem, stream, a)
               : launch_pdl(route_grad_kernel<false, false>, grid, block, smem, stream, a);
  if (err != cudaSuccess || a.partial == nullptr) return err;
  return launch_pdl(scale_grad_kernel, dim3(1), dim3(32), 0, stream, a.partial, static_cast<int>(blocks),
                    a.route_scale, d_global_scale);
}

}  // namespace moe
