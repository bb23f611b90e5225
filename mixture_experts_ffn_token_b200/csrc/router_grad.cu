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
// Bound by the store of the dense [T, E + S] gradient and by instruction
// issue: W lanes (the smallest power of two that holds the n entries) work on
// a token, so a warp works on 32 / W, and its rows are zeroed in 16-byte
// stores while the entries' loads are in flight; the entries follow.  8192
// tokens of 128 + 2 lanes take 3.6 us, 4.8 with the global scale's gradient (a
// second launch that sums the blocks' parts in order; tokens of one block need
// none, 16 of them 4.8 -> 3.0 us a call); a warp per token that built its row in
// shared memory took 8.0 and 9.4.
#include <algorithm>

#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kGradWarps = 8;

__device__ __forceinline__ float log_sigmoid_f(float z) { return fminf(z, 0.f) - log1pf(expf(-fabsf(z))); }

// Zeroes `bytes` bytes at `dst` (whole elements of EL bytes) by one warp.
template <int EL>
__device__ __forceinline__ void zero_span(uint8_t* dst, int64_t bytes, int lane) {
  int64_t head = (16 - (reinterpret_cast<uintptr_t>(dst) & 15u)) & 15u;
  if (head > bytes) head = bytes;
  const int64_t body = (bytes - head) / 16, tail = head + 16 * body;
  for (int64_t i = lane; i < body; i += 32) *reinterpret_cast<uint4*>(dst + head + 16 * i) = make_uint4(0, 0, 0, 0);
  // at most 16 / EL - 1 elements on either side
  const int64_t at = lane < 16 ? static_cast<int64_t>(lane) * EL : tail + static_cast<int64_t>(lane - 16) * EL;
  if (at < (lane < 16 ? head : bytes)) {
    if constexpr (EL == 4) *reinterpret_cast<uint32_t*>(dst + at) = 0;
    else *reinterpret_cast<uint16_t*>(dst + at) = 0;
  }
}

template <bool SINK, bool BF16, int W>
__global__ void __launch_bounds__(32 * kGradWarps) route_grad_kernel(const RouterGradArgs a) {
  griddep_wait();  // the previous kernel's results are complete and visible
  griddep_launch_dependents();
  constexpr int kTokens = 32 / W;  // tokens of a warp
  constexpr int EL = BF16 ? 2 : 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = lane & (W - 1);  // this lane's entry
  const int cols = a.E + a.S;
  const int n = a.k + a.S;  // <= W
  float c = 1.f;
  if constexpr (SINK) c = a.route_scale * (a.global_scale != nullptr ? *a.global_scale : 1.f);
  double total = 0.0;
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kGradWarps + warp) * kTokens; t0 < a.T;
       t0 += static_cast<int64_t>(gridDim.x) * kGradWarps * kTokens) {
    const int64_t t = t0 + lane / W;
    const bool live = t < a.T;
    // entry i < k: the i-th selected expert; k .. n-1: the sink lanes
    int col = -1;
    float dw = 0.f, z = 0.f;
    if (live && i < a.k) {
      col = a.idx[t * a.k + i];
      if (col < 0 || col >= a.E) col = -1;  // no expert: the entry takes no part
      dw = a.d_weights[t * a.k + i];
    } else if (live && i < n) {
      col = a.E + i - a.k;
      dw = a.d_sink != nullptr ? a.d_sink[t * a.S + i - a.k] : 0.f;
    }
    // the rows' zeros, while those loads are in flight
    uint8_t* rows = static_cast<uint8_t*>(a.d_logits) + t0 * a.stride * EL;
    const int count = static_cast<int>(min(static_cast<int64_t>(kTokens), a.T - t0));
    if (a.stride == cols) {
      zero_span<EL>(rows, static_cast<int64_t>(count) * cols * EL, lane);
    } else {
      for (int r = 0; r < count; ++r) zero_span<EL>(rows + r * a.stride * EL, static_cast<int64_t>(cols) * EL, lane);
    }
    const bool on = col >= 0;
    if (on) {
      if constexpr (BF16) z = __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[t * a.stride + col]);
      else z = static_cast<const float*>(a.logits)[t * a.stride + col];
    } else {
      dw = 0.f;
    }
    const float l = !on ? -INFINITY : SINK ? log_sigmoid_f(z) : z;
    float m = l;
#pragma unroll
    for (int off = W / 2; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float ex = on ? expf(l - m) : 0.f;
    float sum = ex;
#pragma unroll
    for (int off = W / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    const float p = on ? ex / sum : 0.f;
    // the token's entries that take part, this one left out
    const uint32_t others = __ballot_sync(0xffffffffu, on) & ~(1u << lane);
    float g = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const float pj = __shfl_sync(0xffffffffu, p, j, W), dj = __shfl_sync(0xffffffffu, dw, j, W);
      if ((others >> (lane - i + j)) & 1u) g += pj * (dw - dj);
    }
    g *= c * p;
    if constexpr (SINK) {
      g *= 1.f / (1.f + expf(z));
      if (on) total += static_cast<double>(p) * static_cast<double>(dw);
    }
    // an expert named twice gets the sum of its entries, in entry order
    const int key = on ? (lane / W) * (kMaxExperts + 32) + col : -1 - lane;
    const uint32_t peers = __match_any_sync(0xffffffffu, key);
    float v = g;
    if (__any_sync(0xffffffffu, (peers & (peers - 1)) != 0)) {
      v = 0.f;
      for (int j = 0; j < 32; ++j) {
        const float gj = __shfl_sync(0xffffffffu, g, j);
        if ((peers >> j) & 1u) v += gj;
      }
    }
    __syncwarp();  // the zeros come before the entries
    if (on && (peers & ((1u << lane) - 1u)) == 0) {
      if constexpr (BF16) static_cast<__nv_bfloat16*>(a.d_logits)[t * a.stride + col] = __float2bfloat16_rn(v);
      else static_cast<float*>(a.d_logits)[t * a.stride + col] = v;
    }
  }
  if (SINK && a.partial != nullptr) {
    __shared__ double s_sum[kGradWarps];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    if (lane == 0) s_sum[warp] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
      double s = 0.0;
      for (int w = 0; w < kGradWarps; ++w) s += s_sum[w];
      // (one block's part is the sum: no second launch)
      if (gridDim.x == 1) *a.d_global_scale = static_cast<float>(s * static_cast<double>(a.route_scale));
      else a.partial[blockIdx.x] = s;
    }
  }
}

// d_global_scale = route_scale * the sum of the blocks' parts, in a fixed order.
constexpr int kSumThreads = 256;
__global__ void __launch_bounds__(kSumThreads) scale_grad_kernel(const double* partial, int n, float route_scale,
                                                                 float* out) {
  griddep_wait();  // the previous kernel's results are complete and visible
  griddep_launch_dependents();
  __shared__ double s_sum[kSumThreads / 32];
  double v[kGradMaxBlocks / kSumThreads], s = 0.0;
#pragma unroll
  for (int i = 0; i < kGradMaxBlocks / kSumThreads; ++i) {
    const int b = static_cast<int>(threadIdx.x) + i * kSumThreads;
    v[i] = b < n ? partial[b] : 0.0;
  }
#pragma unroll
  for (int i = 0; i < kGradMaxBlocks / kSumThreads; ++i) s += v[i];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0;
    for (int w = 0; w < kSumThreads / 32; ++w) s += s_sum[w];
    *out = static_cast<float>(s * static_cast<double>(route_scale));
  }
}

template <bool SINK, bool BF16>
cudaError_t launch_grad(const RouterGradArgs& a, int* blocks, cudaStream_t stream) {
  const int n = a.k + a.S, w = n <= 4 ? 4 : n <= 8 ? 8 : n <= 16 ? 16 : 32;
  const int64_t per_block = kGradWarps * (32 / w);
  *blocks = static_cast<int>(std::min<int64_t>((a.T + per_block - 1) / per_block, kGradMaxBlocks));
  const dim3 grid(static_cast<unsigned>(*blocks)), block(32 * kGradWarps);
  if (w == 4) return launch_pdl(route_grad_kernel<SINK, BF16, 4>, grid, block, 0, stream, a);
  if (w == 8) return launch_pdl(route_grad_kernel<SINK, BF16, 8>, grid, block, 0, stream, a);
  if (w == 16) return launch_pdl(route_grad_kernel<SINK, BF16, 16>, grid, block, 0, stream, a);
  return launch_pdl(route_grad_kernel<SINK, BF16, 32>, grid, block, 0, stream, a);
}

}  // namespace

cudaError_t launch_route_grad(const RouterGradArgs& a, bool sink, bool bf16, cudaStream_t stream) {
  int blocks = 0;
  const cudaError_t err = sink ? (bf16 ? launch_grad<true, true>(a, &blocks, stream) : launch_grad<true, false>(a, &blocks, stream))
                               : (bf16 ? launch_grad<false, true>(a, &blocks, stream) : launch_grad<false, false>(a, &blocks, stream));
  if (err != cudaSuccess || a.partial == nullptr || blocks == 1) return err;
  return launch_pdl(scale_grad_kernel, dim3(1), dim3(kSumThreads), 0, stream, a.partial, blocks, a.route_scale,
                    a.d_global_scale);
}

}  // namespace moe
