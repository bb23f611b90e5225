// rows.cu -- tokens sorted by expert and back, and the gradients of both.
//
// With p = inverse[t*k + j] the position of token t's j-th slot among the
// rows sorted by expert (a p outside [0, R): the slot went to no expert):
//   spread   rows[p] = w_tj * tok[t]                  (dispatch; combine's gradient)
//   gather   out[t]  = sum_j w_tj * rows[p]           (combine; dispatch's gradient)
//   and, for the gradient of the weights,  dw_tj = <tok[t], rows_in[p]>.
// Every kernel walks tokens, not positions: a token's row is read once for
// its k copies (or written once for its k terms), each position belongs to
// one slot, so nothing is accumulated across threads but the inner products,
// in a fixed order: results are the same bits on every run.
//
// All of them are bound by HBM: per token one row on the token side and k
// rows on the sorted side, each moved once.
#include <algorithm>

#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kRowThreads = 256;

// 16 bytes of a row: 8 bf16 or 4 fp32 values.
template <bool F32>
struct Vec {
  static constexpr int N = F32 ? 4 : 8;
  float v[N];
  __device__ __forceinline__ void unpack(const uint4& u) {
    if constexpr (F32) {
      v[0] = __uint_as_float(u.x);
      v[1] = __uint_as_float(u.y);
      v[2] = __uint_as_float(u.z);
      v[3] = __uint_as_float(u.w);
    } else {
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
      }
    }
  }
  // rounded to the row type once, here
  __device__ __forceinline__ uint4 pack() const {
    if constexpr (F32)
      return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    else
      return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                        pack_bf16x2(v[6], v[7]));
  }
};

// A block covers 2^cw_log columns (16-byte vectors) of 256 / 2^cw_log tokens.
struct Tiling {
  int cw_log, chunks;
};

Tiling tiling(int vec) {
  Tiling t;
  t.cw_log = 0;
  while ((1 << t.cw_log) < vec && t.cw_log < 7) ++t.cw_log;
  t.chunks = (vec + (1 << t.cw_log) - 1) >> t.cw_log;
  return t;
}

// The positions (-1: no slot) and weights of KB of a token's slots, all loaded
// before the first is used.
template <int KB>
__device__ __forceinline__ void load_slots(const RowsArgs& a, int64_t t, int j0, int (&p)[KB], float (&w)[KB]) {
#pragma unroll
  for (int q = 0; q < KB; ++q) {
    const bool in = j0 + q < a.k;
    p[q] = in ? __ldg(a.inverse + t * a.k + j0 + q) : -1;
    w[q] = in && a.weights != nullptr ? __ldg(a.weights + t * a.k + j0 + q) : 1.f;
  }
#pragma unroll
  for (int q = 0; q < KB; ++q)
    if (p[q] >= a.R) p[q] = -1;
}

// rows[p] = w * tok[t] for each of the token's slots.
template <bool F32, int KB>
__global__ void __launch_bounds__(kRowThreads) spread_kernel(const RowsArgs a, int cw_log, int chunks) {
  griddep_wait();  // the previous kernel's results are complete and visible
  griddep_launch_dependents();
  const uint32_t tile = blockIdx.x / static_cast<uint32_t>(chunks);
  const int c = static_cast<int>(((blockIdx.x - tile * chunks) << cw_log) + (threadIdx.x & ((1u << cw_log) - 1u)));
  const int64_t t = (static_cast<int64_t>(tile) << (8 - cw_log)) + (threadIdx.x >> cw_log);
  if (t >= a.T || c >= a.vec) return;
  const uint4 u = __ldg(static_cast<const uint4*>(a.tok_in) + t * a.vec + c);
  uint4* rows = static_cast<uint4*>(a.rows_out) + c;
  Vec<F32> x;
  x.unpack(u);
  for (int j0 = 0; j0 < a.k; j0 += KB) {
    int p[KB];
    float w[KB];
    load_slots<KB>(a, t, j0, p, w);
#pragma unroll
    for (int q = 0; q < KB; ++q) {
      uint4 o = u;
      if (a.weights != nullptr) {
        Vec<F32> y;
#pragma unroll
        for (int i = 0; i < Vec<F32>::N; ++i) y.v[i] = w[q] * x.v[i];
        o = y.pack();
      }
      if (p[q] >= 0) rows[static_cast<int64_t>(p[q]) * a.vec] = o;
    }
  }
}

// out[t] = sum_j w * rows[p], j ascending in fp32.
template <bool F32, int KB>
__global__ void __launch_bounds__(kRowThreads) gather_kernel(const RowsArgs a, int cw_log, int chunks) {
  griddep_wait();  // the previous kernel's results are complete and visible
  griddep_launch_dependents();
  const uint32_t tile = blockIdx.x / static_cast<uint32_t>(chunks);
  const int c = static_cast<int>(((blockIdx.x - tile * chunks) << cw_log) + (threadIdx.x & ((1u << cw_log) - 1u)));
  const int64_t t = (static_cast<int64_t>(tile) << (8 - cw_log)) + (threadIdx.x >> cw_log);
  if (t >= a.T || c >= a.vec) return;
  const uint4* rows = static_cast<const uint4*>(a.rows_in) + c;
  Vec<F32> acc;
#pragma unroll
  for (int i = 0; i < Vec<F32>::N; ++i) acc.v[i] = 0.f;
  for (int j0 = 0; j0 < a.k; j0 += KB) {
    int p[KB];
    float w[KB];
    uint4 u[KB];
    load_slots<KB>(a, t, j0, p, w);
#pragma unroll
    for (int q = 0; q < KB; ++q)
      if (p[q] >= 0) u[q] = __ldg(rows + static_cast<int64_t>(p[q]) * a.vec);
#pragma unroll
    for (int q = 0; q < KB; ++q) {
      if (p[q] >= 0) {
        Vec<F32> y;
        y.unpack(u[q]);
#pragma unroll
        for (int i = 0; i < Vec<F32>::N; ++i) acc.v[i] += w[q] * y.v[i];
      }
    }
  }
  static_cast<uint4*>(a.tok_out)[t * a.vec + c] = acc.pack();
}

// The same with the weights' gradient: one block per token, its k inner
// products reduced over the block in a fixed order.  SPREAD: rows[p] =
// w * tok[t] is written; else out[t] = sum_j w * rows[p] (KB >= k terms, kept
// in registers so that every row is read once).  A thread loads U columns of
// up to 8 / U rows before it uses the first.
template <bool F32, bool SPREAD, int KB, int U>
__global__ void __launch_bounds__(kRowThreads) rows_dot_kernel(const RowsArgs a) {
  griddep_wait();  // the previous kernel's results are complete and visible
  griddep_launch_dependents();
  __shared__ float s_part[kRowThreads / 32][KB];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int p[KB];
  float w[KB];
  load_slots<KB>(a, t, 0, p, w);
  const uint4* tok = static_cast<const uint4*>(a.tok_in) + t * a.vec;
  const uint4* rows = static_cast<const uint4*>(a.rows_in);
  constexpr int N = Vec<F32>::N;
  constexpr int kBatch = KB < 8 ? KB : 8;
  float dot[KB];
#pragma unroll
  for (int j = 0; j < KB; ++j) dot[j] = 0.f;
  for (int c0 = tid; c0 < a.vec; c0 += U * blockDim.x) {
    uint4 ux[U];
    Vec<F32> x[U], acc[U];
#pragma unroll
    for (int v = 0; v < U; ++v) {
      const int c = c0 + v * blockDim.x;
      ux[v] = c < a.vec ? __ldg(tok + c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j0 = 0; j0 < KB; j0 += kBatch) {
      uint4 u[U][kBatch];
#pragma unroll
      for (int v = 0; v < U; ++v) {
        const int c = c0 + v * blockDim.x;
#pragma unroll
        for (int q = 0; q < kBatch; ++q)
          u[v][q] = p[j0 + q] >= 0 && c < a.vec ? __ldg(rows + static_cast<int64_t>(p[j0 + q]) * a.vec + c)
                                                : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int v = 0; v < U; ++v) {
        const int c = c0 + v * blockDim.x;
        if (j0 == 0) {
          x[v].unpack(ux[v]);
#pragma unroll
          for (int i = 0; i < N; ++i) acc[v].v[i] = 0.f;
        }
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          if (p[j0 + q] < 0) continue;
          Vec<F32> y, o;
          y.unpack(u[v][q]);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            dot[j0 + q] += x[v].v[i] * y.v[i];
            if constexpr (SPREAD) o.v[i] = w[j0 + q] * x[v].v[i];
            else acc[v].v[i] += w[j0 + q] * y.v[i];
          }
          if constexpr (SPREAD) {
            if (c < a.vec) static_cast<uint4*>(a.rows_out)[static_cast<int64_t>(p[j0 + q]) * a.vec + c] = o.pack();
          }
        }
      }
    }
    if constexpr (!SPREAD) {
#pragma unroll
      for (int v = 0; v < U; ++v) {
        const int c = c0 + v * blockDim.x;
        if (c < a.vec) static_cast<uint4*>(a.tok_out)[t * a.vec + c] = acc[v].pack();
      }
    }
  }
#pragma unroll
  for (int j = 0; j < KB; ++j) {
    float v = dot[j];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (lane == 0) s_part[warp][j] = v;
  }
  __syncthreads();
  const int warps = blockDim.x >> 5;
  for (int j = tid; j < a.k; j += blockDim.x) {
    const int pj = a.inverse[t * a.k + j];
    float v = 0.f;
    for (int i = 0; i < warps; ++i) v += s_part[i][j];
    a.d_weights[t * a.k + j] = pj >= 0 && pj < a.R ? v : 0.f;
  }
}

template <bool F32, bool SPREAD, int KB, int U>
cudaError_t launch_dot_k(const RowsArgs& a, cudaStream_t stream) {
  int threads = 32;
  while (threads < kRowThreads && threads * U < a.vec) threads <<= 1;
  return launch_pdl(rows_dot_kernel<F32, SPREAD, KB, U>, dim3(static_cast<unsigned>(a.T)),
                    dim3(static_cast<unsigned>(threads)), 0, stream, a);
}

template <bool F32, bool SPREAD>
cudaError_t launch_dot(const RowsArgs& a, cudaStream_t stream) {
  if (a.k <= 1) return launch_dot_k<F32, SPREAD, 1, 4>(a, stream);
  if (a.k <= 2) return launch_dot_k<F32, SPREAD, 2, 4>(a, stream);
  if (a.k <= 4) return launch_dot_k<F32, SPREAD, 4, 2>(a, stream);
  if (a.k <= 6) return launch_dot_k<F32, SPREAD, 6, 1>(a, stream);
  if (a.k <= 8) return launch_dot_k<F32, SPREAD, 8, 1>(a, stream);
  if (a.k <= 16) return launch_dot_k<F32, SPREAD, 16, 1>(a, stream);
  return launch_dot_k<F32, SPREAD, 32, 1>(a, stream);
}

template <bool F32, int KB>
cudaError_t launch_copy(const RowsArgs& a, bool spread, cudaStream_t stream) {
  const Tiling tl = tiling(a.vec);
  const int per_block = kRowThreads >> tl.cw_log;
  const int64_t blocks = (static_cast<int64_t>(a.T) + per_block - 1) / per_block * tl.chunks;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks)), block(kRowThreads);
  if (spread) return launch_pdl(spread_kernel<F32, KB>, grid, block, 0, stream, a, tl.cw_log, tl.chunks);
  return launch_pdl(gather_kernel<F32, KB>, grid, block, 0, stream, a, tl.cw_log, tl.chunks);
}

template <bool F32>
cudaError_t launch_rows(const RowsArgs& a, bool spread, cudaStream_t stream) {
  if (a.d_weights != nullptr)
    return spread ? launch_dot<F32, true>(a, stream) : launch_dot<F32, false>(a, stream);
  if (a.k <= 2) return launch_copy<F32, 2>(a, spread, stream);
  if (a.k <= 4) return launch_copy<F32, 4>(a, spread, stream);
  return launch_copy<F32, 8>(a, spread, stream);
}

}  // namespace

cudaError_t launch_rows_spread(const RowsArgs& a, bool f32, cudaStream_t stream) {
  return f32 ? launch_rows<true>(a, true, stream) : launch_rows<false>(a, true, stream);
}

cudaError_t launch_rows_gather(const RowsArgs& a, bool f32, cudaStream_t stream) {
  return f32 ? launch_rows<true>(a, false, stream) : launch_rows<false>(a, false, stream);
}

}  // namespace moe
