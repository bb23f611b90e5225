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
// rows on the sorted side, each moved once.  On one B200 (6.56 TB/s copy rate),
// bf16: dispatch 8192 x 2048, k 6 in 38.1 us (0.94 of that rate), its gradient
// with the weights' 45.5 us (0.90), combine 38.8 us (0.92), its gradient with
// the weights' 74.2 us (0.90).  A few megabytes take launch, first loads and last
// wave, 2 to 4 us (combine 2048 x 2880, k 4: 12.3 us, 9.0 at the copy rate).
#include <algorithm>

#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kRowThreads = 256;
constexpr int kGatherLog = 7;
constexpr int kGatherThreads = 1 << kGatherLog;  // (2 to 4% less time than 256: the last wave is finer)

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

// A block covers u * 2^cw_log columns (16-byte vectors) of blockDim / 2^cw_log tokens.
struct Tiling {
  int cw_log, chunks;
};

Tiling tiling(int vec, int u) {
  Tiling t;
  t.cw_log = 0;
  while ((u << t.cw_log) < vec && t.cw_log < 7) ++t.cw_log;
  t.chunks = (vec + (u << t.cw_log) - 1) / (u << t.cw_log);
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

// out[t] = sum_j w * rows[p], j ascending in fp32.  A thread loads U columns of
// up to KB rows before it adds the first.
template <bool F32, int KB, int U>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const RowsArgs a, int cw_log, int chunks) {
  griddep_wait();  // the previous kernel's results are complete and visible
  griddep_launch_dependents();
  const uint32_t tile = blockIdx.x / static_cast<uint32_t>(chunks);
  const int cw = 1 << cw_log;
  const int c0 = static_cast<int>((blockIdx.x - tile * chunks) * U) * cw + (threadIdx.x & (cw - 1));
  const int64_t t = (static_cast<int64_t>(tile) << (kGatherLog - cw_log)) + (threadIdx.x >> cw_log);
  if (t >= a.T || c0 >= a.vec) return;
  const uint4* rows = static_cast<const uint4*>(a.rows_in) + c0;
  Vec<F32> acc[U];
#pragma unroll
  for (int v = 0; v < U; ++v)
#pragma unroll
    for (int i = 0; i < Vec<F32>::N; ++i) acc[v].v[i] = 0.f;
  for (int j0 = 0; j0 < a.k; j0 += KB) {
    int p[KB];
    float w[KB];
    uint4 u[U][KB];
    load_slots<KB>(a, t, j0, p, w);
#pragma unroll
    for (int v = 0; v < U; ++v)
#pragma unroll
      for (int q = 0; q < KB; ++q)
        if (p[q] >= 0 && c0 + v * cw < a.vec) u[v][q] = __ldg(rows + static_cast<int64_t>(p[q]) * a.vec + v * cw);
#pragma unroll
    for (int v = 0; v < U; ++v) {
#pragma unroll
      for (int q = 0; q < KB; ++q) {
        if (p[q] >= 0 && c0 + v * cw < a.vec) {
          Vec<F32> y;
          y.unpack(u[v][q]);
#pragma unroll
          for (int i = 0; i < Vec<F32>::N; ++i) acc[v].v[i] += w[q] * y.v[i];
        }
      }
    }
  }
#pragma unroll
  for (int v = 0; v < U; ++v)
    if (c0 + v * cw < a.vec) static_cast<uint4*>(a.tok_out)[t * a.vec + c0 + v * cw] = acc[v].pack();
}

// The same with the weights' gradient: one block per token, its k inner
// products reduced over the block in a fixed order.  SPREAD: rows[p] =
// w * tok[t] is written, with BATCHES `step` <= KB slots at a time, each time
// reading the token's row again (from L1); else out[t] = sum_j w * rows[p] (KB >= k terms, kept in
// registers so that every row is read once).  A thread loads U columns of up
// to 8 / U rows before it uses the first.  A row of at most 32 U vectors is
// a warp's (blockDim.y tokens a block, no sum across warps).
template <bool F32, bool SPREAD, int KB, int U, bool BATCHES>
__global__ void __launch_bounds__(kRowThreads) rows_dot_kernel(const RowsArgs a, int step) {
  static_assert(!BATCHES || SPREAD, "only spreading may take the slots in batches");
  griddep_wait();  // the previous kernel's results are complete and visible
  griddep_launch_dependents();
  __shared__ float s_part[kRowThreads / 32][KB];
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (t >= a.T) return;  // (whole warps, and then nothing is synchronised)
  const uint4* tok = static_cast<const uint4*>(a.tok_in) + t * a.vec;
  const uint4* rows = static_cast<const uint4*>(a.rows_in);
  constexpr int N = Vec<F32>::N;
  constexpr int kBatch = KB < 8 ? KB : 8;
  for (int b0 = 0; b0 < (BATCHES ? a.k : 1); b0 += BATCHES ? step : 1) {
    int p[KB];
    float w[KB];
    load_slots<KB>(a, t, b0, p, w);
    const int count = BATCHES ? min(step, a.k - b0) : a.k;
    if constexpr (BATCHES) {
#pragma unroll
      for (int j = 0; j < KB; ++j)
        if (j >= count) p[j] = -1;  // the next batch's
    }
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
      if (lane == 0) s_part[threadIdx.y + warp][j] = v;
    }
    if (blockDim.y > 1) __syncwarp();
    else __syncthreads();
    const int warps = blockDim.x >> 5;
    for (int j = tid; j < count; j += blockDim.x) {
      const int pj = a.inverse[t * a.k + b0 + j];
      float v = 0.f;
      for (int i = 0; i < warps; ++i) v += s_part[threadIdx.y + i][j];
      a.d_weights[t * a.k + b0 + j] = pj >= 0 && pj < a.R ? v : 0.f;
    }
    if constexpr (BATCHES) {  // the parts are read before the next batch's
      if (blockDim.y > 1) __syncwarp();
      else __syncthreads();
    }
  }
}

// The same for short rows (at most G U vectors): G lanes per token, 32 / G
// tokens a warp, the slots in batches of 8 that are loaded together; a batch's
// inner products are summed over the G lanes, and lane q stores slot q's.
// (16384 tokens of 64 bf16, k 16: 12.6 and 16.9 us where a warp or block per token
// takes 42.3 (gather) and 102 us (spread).)
template <bool F32, bool SPREAD, int G, int U>
__global__ void __launch_bounds__(kRowThreads) rows_dot_short_kernel(const RowsArgs a) {
  griddep_wait();  // the previous kernel's results are complete and visible
  griddep_launch_dependents();
  static_assert(G >= 8, "lane q of a group stores slot q of a batch");
  constexpr int N = Vec<F32>::N;
  constexpr int KB = 8;
  const int64_t t = (static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x) / G;
  const int i = threadIdx.x & (G - 1);
  const bool live = t < a.T;  // (every lane takes part in the sums)
  const uint4* rows = static_cast<const uint4*>(a.rows_in);
  Vec<F32> x[U], acc[U];
#pragma unroll
  for (int v = 0; v < U; ++v) {
    const int c = i + v * G;
    x[v].unpack(live && c < a.vec ? __ldg(static_cast<const uint4*>(a.tok_in) + t * a.vec + c) : make_uint4(0, 0, 0, 0));
#pragma unroll
    for (int e = 0; e < N; ++e) acc[v].v[e] = 0.f;
  }
  for (int j0 = 0; j0 < a.k; j0 += KB) {
    int p[KB];
    float w[KB], dot[KB];
    if (live) {
      load_slots<KB>(a, t, j0, p, w);
    } else {
#pragma unroll
      for (int q = 0; q < KB; ++q) p[q] = -1;
    }
    uint4 u[U][KB];
#pragma unroll
    for (int v = 0; v < U; ++v)
#pragma unroll
      for (int q = 0; q < KB; ++q)
        u[v][q] = p[q] >= 0 && i + v * G < a.vec ? __ldg(rows + static_cast<int64_t>(p[q]) * a.vec + i + v * G)
                                                 : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int q = 0; q < KB; ++q) {
      dot[q] = 0.f;
      if (p[q] < 0) continue;
#pragma unroll
      for (int v = 0; v < U; ++v) {
        const int c = i + v * G;
        Vec<F32> y, o;
        y.unpack(u[v][q]);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          dot[q] += x[v].v[e] * y.v[e];
          if constexpr (SPREAD) o.v[e] = w[q] * x[v].v[e];
          else acc[v].v[e] += w[q] * y.v[e];
        }
        if constexpr (SPREAD) {
          if (c < a.vec) static_cast<uint4*>(a.rows_out)[static_cast<int64_t>(p[q]) * a.vec + c] = o.pack();
        }
      }
    }
    float mine = 0.f;
#pragma unroll
    for (int q = 0; q < KB; ++q) {
      if (j0 + q < a.k) {  // (the same for the whole grid)
#pragma unroll
        for (int off = G / 2; off > 0; off >>= 1) dot[q] += __shfl_xor_sync(0xffffffffu, dot[q], off);
        if (i == q) mine = dot[q];
      }
    }
    if (live && i < KB && j0 + i < a.k) a.d_weights[t * a.k + j0 + i] = mine;
  }
  if constexpr (!SPREAD) {
#pragma unroll
    for (int v = 0; v < U; ++v) {
      const int c = i + v * G;
      if (live && c < a.vec) static_cast<uint4*>(a.tok_out)[t * a.vec + c] = acc[v].pack();
    }
  }
}

// out[t] = sum_j w * rows[p] (and the weights' gradient, DOT) for many tokens,
// through a ring in shared memory.  A warp walks whole tokens (or, without
// DOT, segments of them), 32 columns a step; each thread copies the k (+ 1)
// vectors of its own column with cp.async, S - 1 steps ahead, and reads back
// only what it copied itself, so nothing is synchronised.  Registers then hold
// one step while the ring keeps about 100 KB a SM in flight, across the ends
// of tokens: the reads are scattered rows, and the block form above, whose
// loads wait for their positions and drain at each token, reached 4.7 TB/s
// on them.
constexpr int kRingThreads = 256;
constexpr int kRingBytes = 104 * 1024;  // of a block of 256 threads, two a SM

// Where three steps of 256 threads do not fit, half the threads and as many
// blocks as fit: a step of nine rows and more is long, and it is warps that
// hide it (16384 x 1024, k 8: 71.4 us with 2 blocks of 5 steps, 53.8 with 4 of
// 3; with fewer rows the deeper ring of two blocks is the better, 8192 x 2880,
// k 4: 38.7 and 40.9 us).
template <int KB, bool DOT>
struct Ring {
  static constexpr int ROWS = KB + (DOT ? 1 : 0);
  static constexpr bool WIDE = ROWS * kRingThreads * 16 * 3 <= kRingBytes;
  static constexpr int THREADS = WIDE ? kRingThreads : kRingThreads / 2;
  static constexpr int FIT = kRingBytes / (ROWS * THREADS * 16);
  static constexpr int S = !WIDE ? 3 : FIT < 8 ? FIT : 8;
  static constexpr int BYTES = S * ROWS * THREADS * 16;
  static constexpr int BLOCKS = WIDE ? 2 : 222 * 1024 / (BYTES + 1024);  // of a SM
  static_assert(S >= 3 && BLOCKS >= 2, "the ring fits a SM");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <bool F32, bool DOT, int KB>
__global__ void __launch_bounds__(kRingThreads) gather_ring_kernel(const RowsArgs a, int segs, int seg_cols,
                                                                   int64_t jobs, int64_t warps) {
  griddep_wait();  // the previous kernel's results are complete and visible
  griddep_launch_dependents();
  using G = Ring<KB, DOT>;
  constexpr int N = Vec<F32>::N;
  extern __shared__ uint4 ring[];  // [S][ROWS][THREADS]
  const int tid = threadIdx.x, lane = tid & 31;
  const uint32_t mine = smem_u32(ring + tid);
  // neighbouring warps of a block take jobs far apart, so that a short grid
  // spreads over the SMs
  const int64_t first = blockIdx.x + static_cast<int64_t>(gridDim.x) * (tid >> 5);
  if (first >= warps) return;
  const uint4* rows = static_cast<const uint4*>(a.rows_in);
  const uint4* tok = static_cast<const uint4*>(a.tok_in);

  // ------------------------------------------------- the copying side
  int64_t job = first;     // job = (token, segment)
  int64_t t_in = 0;        // its token
  int c_in = 0, end_in = 0;  // this lane's column, the segment's end
  int p[KB];
  auto open_in = [&]() {
    if (job >= jobs) {
      c_in = end_in = 0;
      return;
    }
    t_in = job / segs;
    const int seg = static_cast<int>(job - t_in * segs);
    c_in = seg * seg_cols + lane;
    end_in = min(a.vec, (seg + 1) * seg_cols);
#pragma unroll
    for (int q = 0; q < KB; ++q) {
      p[q] = q < a.k ? __ldg(a.inverse + t_in * a.k + q) : -1;
      if (p[q] >= a.R) p[q] = -1;
    }
  };
  int slot_in = 0;
  auto copy_step = [&]() {
    if (c_in < end_in) {
      const uint32_t dst = mine + static_cast<uint32_t>(slot_in) * (G::ROWS * G::THREADS * 16);
#pragma unroll
      for (int q = 0; q < KB; ++q)
        if (p[q] >= 0) cp_async16(dst + q * (G::THREADS * 16), rows + static_cast<int64_t>(p[q]) * a.vec + c_in);
      if constexpr (DOT) cp_async16(dst + KB * (G::THREADS * 16), tok + t_in * a.vec + c_in);
    }
    cp_async_commit();  // (possibly empty: one group a step)
    slot_in = slot_in + 1 == G::S ? 0 : slot_in + 1;
    c_in += 32;
    if (c_in - lane >= end_in && job < jobs) {
      job += warps;
      open_in();
    }
  };
  open_in();
#pragma unroll
  for (int i = 0; i < G::S - 1; ++i) copy_step();

  // --------------------------------------------------- the using side
  int slot = 0;
  for (int64_t out_job = first; out_job < jobs; out_job += warps) {
    const int64_t t = out_job / segs;
    const int seg = static_cast<int>(out_job - t * segs);
    const int c0 = seg * seg_cols, end = min(a.vec, c0 + seg_cols);
    float w[KB], dot[KB];
    uint32_t on = 0;
#pragma unroll
    for (int q = 0; q < KB; ++q) {
      const int pos = q < a.k ? __ldg(a.inverse + t * a.k + q) : -1;
      if (pos >= 0 && pos < a.R) on |= 1u << q;
      w[q] = q < a.k && a.weights != nullptr ? __ldg(a.weights + t * a.k + q) : 1.f;
      dot[q] = 0.f;
    }
    for (int c = c0 + lane; c - lane < end; c += 32) {
      copy_step();
      cp_async_wait<G::S - 1>();
      const uint4* in = ring + slot * (G::ROWS * G::THREADS) + tid;
      slot = slot + 1 == G::S ? 0 : slot + 1;
      if (c < end) {
        Vec<F32> x, acc;
        if constexpr (DOT) x.unpack(in[KB * G::THREADS]);
#pragma unroll
        for (int i = 0; i < N; ++i) acc.v[i] = 0.f;
#pragma unroll
        for (int q = 0; q < KB; ++q) {
          if (!((on >> q) & 1u)) continue;
          Vec<F32> y;
          y.unpack(in[q * G::THREADS]);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            acc.v[i] += w[q] * y.v[i];
            if constexpr (DOT) dot[q] += x.v[i] * y.v[i];
          }
        }
        static_cast<uint4*>(a.tok_out)[t * a.vec + c] = acc.pack();
      }
    }
    if constexpr (DOT) {
#pragma unroll
      for (int q = 0; q < KB; ++q) {
        float v = dot[q];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        if (lane == 0 && q < a.k) a.d_weights[t * a.k + q] = v;
      }
    }
  }
}

template <bool F32, bool SPREAD, int KB, int U, bool BATCHES = false>
cudaError_t launch_dot_k(const RowsArgs& a, int step, cudaStream_t stream) {
  // whole warps that cover the row in the fewest equal steps
  const int rounds = (a.vec + kRowThreads * U - 1) / (kRowThreads * U);
  const int threads = ((a.vec + rounds * U - 1) / (rounds * U) + 31) / 32 * 32;
  const int tokens = threads == 32 ? kRowThreads / 32 : 1;
  return launch_pdl(rows_dot_kernel<F32, SPREAD, KB, U, BATCHES>, dim3(static_cast<unsigned>((a.T + tokens - 1) / tokens)),
                    dim3(static_cast<unsigned>(threads), static_cast<unsigned>(tokens)), 0, stream, a, step);
}

template <bool F32, bool DOT, int KB>
cudaError_t launch_ring(const RowsArgs& a, cudaStream_t stream) {
  using G = Ring<KB, DOT>;
  constexpr int kWarps = G::THREADS / 32;
  const cudaError_t err =
      opt_in_dynamic_smem(reinterpret_cast<const void*>(gather_ring_kernel<F32, DOT, KB>), G::BYTES);
  if (err != cudaSuccess) return err;
  const int64_t most = static_cast<int64_t>(a.num_sms) * G::BLOCKS * kWarps;  // warps resident at once
  // without the weights' gradient a token may be cut into segments of whole
  // 32-column steps, so that every warp has several jobs
  int segs = 1;
  if (!DOT) segs = static_cast<int>(std::min<int64_t>((a.vec + 63) / 64, std::max<int64_t>(1, 6 * most / a.T)));
  const int seg_cols = ((a.vec + segs - 1) / segs + 31) / 32 * 32;
  segs = (a.vec + seg_cols - 1) / seg_cols;
  const int64_t jobs = static_cast<int64_t>(a.T) * segs;
  // equal numbers of jobs per warp
  const int64_t rounds = (jobs + most - 1) / most, warps = (jobs + rounds - 1) / rounds;
  return launch_pdl(gather_ring_kernel<F32, DOT, KB>, dim3(static_cast<unsigned>((warps + kWarps - 1) / kWarps)),
                    dim3(G::THREADS), G::BYTES, stream, a, segs, seg_cols, jobs, warps);
}

template <bool F32, bool DOT>
cudaError_t launch_ring_k(const RowsArgs& a, cudaStream_t stream) {
  if constexpr (!DOT) {
    if (a.k <= 2) return launch_ring<F32, DOT, 2>(a, stream);
  }
  if (a.k <= 4) return launch_ring<F32, DOT, 4>(a, stream);
  if (a.k <= 6) return launch_ring<F32, DOT, 6>(a, stream);
  if constexpr (DOT) {
    if (a.k > 8) return launch_ring<F32, DOT, 16>(a, stream);
  }
  return launch_ring<F32, DOT, 8>(a, stream);
}

// The ring pays once it has many tokens to run ahead over; below, its start
// costs more than the waits it saves.  On one B200, bf16:
//   combine            8192 x 2880, k 4 (188 MB): 43.0 us by threads, 38.7 by the ring; 4096 x 4096, k 8
//                      (268 MB): 54.0, 48.7; but 2048 x 2880, k 4 (47 MB): 12.6, 15.6; k 16 (134 MB): 26.0, 28.9
//   dispatch backward  8192 x 2048, k 6 (201 MB): 57.5 by blocks, 45.6 by the ring; 1500 x 2048, k 6 (37 MB):
//                      12.7, 11.4; but 1024 x 1024, k 8 (17 MB): 7.1, 7.6; 512 x 4096, k 8: 11.3, 15.9; and with
//                      one or two rows a token the block form already runs at 0.94 of the copy rate.
bool use_ring(const RowsArgs& a) {
  const int64_t bytes = static_cast<int64_t>(a.R) * a.vec * 16;
  if (a.d_weights == nullptr) return a.k <= 8 && bytes >= (int64_t(128) << 20);
  return a.k >= 3 && a.k <= 16 && a.T >= 1024 && bytes >= (int64_t(24) << 20);
}

template <bool F32, bool SPREAD>
cudaError_t launch_dot(const RowsArgs& a, cudaStream_t stream) {
  if (a.k <= 1) return launch_dot_k<F32, SPREAD, 1, 4>(a, a.k, stream);
  if (a.k <= 2) return launch_dot_k<F32, SPREAD, 2, 4>(a, a.k, stream);
  if (a.k <= 4) return launch_dot_k<F32, SPREAD, 4, 2>(a, a.k, stream);
  if (a.k <= 6) return launch_dot_k<F32, SPREAD, 6, 1>(a, a.k, stream);
  if (a.k <= 8) return launch_dot_k<F32, SPREAD, 8, 1>(a, a.k, stream);
  if constexpr (SPREAD) {
    // equal batches of at most 8
    const int batches = (a.k + 7) / 8, step = (a.k + batches - 1) / batches;
    if (step <= 6) return launch_dot_k<F32, true, 6, 1, true>(a, step, stream);
    return launch_dot_k<F32, true, 8, 1, true>(a, step, stream);
  } else {
    if (a.k <= 16) return launch_dot_k<F32, false, 16, 1>(a, a.k, stream);
    return launch_dot_k<F32, false, 32, 1>(a, a.k, stream);
  }
}

template <bool F32, bool SPREAD, int G, int U>
cudaError_t launch_short(const RowsArgs& a, cudaStream_t stream) {
  const int64_t blocks = (static_cast<int64_t>(a.T) * G + kRowThreads - 1) / kRowThreads;
  return launch_pdl(rows_dot_short_kernel<F32, SPREAD, G, U>, dim3(static_cast<unsigned>(blocks)), dim3(kRowThreads), 0,
                    stream, a);
}

template <bool F32, bool SPREAD>
cudaError_t launch_grad(const RowsArgs& a, cudaStream_t stream) {
  if (a.vec <= 8) return launch_short<F32, SPREAD, 8, 1>(a, stream);
  if (a.vec <= 16) return launch_short<F32, SPREAD, 16, 1>(a, stream);
  if (a.vec <= 32) return launch_short<F32, SPREAD, 32, 1>(a, stream);
  if constexpr (!SPREAD) {
    if (a.vec <= 64) return launch_short<F32, SPREAD, 32, 2>(a, stream);
    if (use_ring(a)) return launch_ring_k<F32, true>(a, stream);
  }
  return launch_dot<F32, SPREAD>(a, stream);
}

template <bool F32, int KB, int U>
cudaError_t launch_copy(const RowsArgs& a, bool spread, cudaStream_t stream) {
  const Tiling tl = tiling(a.vec, spread ? 1 : U);
  const int threads = spread ? kRowThreads : kGatherThreads;
  const int per_block = threads >> tl.cw_log;
  const int64_t blocks = (static_cast<int64_t>(a.T) + per_block - 1) / per_block * tl.chunks;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks)), block(static_cast<unsigned>(threads));
  if (spread) return launch_pdl(spread_kernel<F32, KB>, grid, block, 0, stream, a, tl.cw_log, tl.chunks);
  return launch_pdl(gather_kernel<F32, KB, U>, grid, block, 0, stream, a, tl.cw_log, tl.chunks);
}

template <bool F32>
cudaError_t launch_rows(const RowsArgs& a, bool spread, cudaStream_t stream) {
  if (a.d_weights != nullptr)
    return spread ? launch_grad<F32, true>(a, stream) : launch_grad<F32, false>(a, stream);
  if (!spread && use_ring(a)) return launch_ring_k<F32, false>(a, stream);
  // two columns a thread pay for one or two rows (4096 x 4096, k 2: 21.4 -> 19.9 us), more do not, and for more
  // rows a column is enough (2048 x 2880, k 4: 12.6 us with one, 17.7 with two); loads that k does not fill cost too
  // (8192 x 2048, k 6: 47.4 us with eight, 39.9 with six)
  if (a.k <= 2) return launch_copy<F32, 2, 2>(a, spread, stream);
  if (a.k <= 4) return launch_copy<F32, 4, 1>(a, spread, stream);
  if (a.k <= 6) return launch_copy<F32, 6, 1>(a, spread, stream);
  return launch_copy<F32, 8, 1>(a, spread, stream);
}

}  // namespace

cudaError_t launch_rows_spread(const RowsArgs& a, bool f32, cudaStream_t stream) {
  return f32 ? launch_rows<true>(a, true, stream) : launch_rows<false>(a, true, stream);
}

cudaError_t launch_rows_gather(const RowsArgs& a, bool f32, cudaStream_t stream) {
  return f32 ? launch_rows<true>(a, false, stream) : launch_rows<false>(a, false, stream);
}

}  // namespace moe
