// int8_common.cuh -- what the two 8-bit grouped products share: the integer MMA,
// their parameters, the CSR check, the scaling and the gated activation.
#pragma once

#include <cmath>

#include "grouped_tiles.cuh"
#include "kernels.cuh"

namespace moe {

// Instruction descriptor for kind::i8, signed A and B, both K-major, 32-bit
// integer D: D format bits 4..5 = 2 (s32), A format 7..9 = 1 (s8), B format
// 10..12 = 1 (s8), N >> 3 at 17..22, M >> 4 at 24..28.
__host__ __device__ constexpr uint32_t idesc_s8_s32(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void mma_i8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The matrix descriptor of K-major rows of 128 B (8-row swizzle atoms 1024 B
// apart) as its two halves: the high one is constant, and the low one moves with
// the address in 16-byte units, so a step of K or a stage is one addition.  The
// issuing thread is what bounds short MMAs: building both descriptors anew took it
// some 85 cycles an MMA, against 128 of the tensor cores for the largest here.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return (1u << 16) | (saddr >> 4); }
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) {
  return (static_cast<uint64_t>(kDescHi) << 32) | lo;
}

// One stage: four K steps of 32 (32 B along the rows).  `fresh`: the first
// step starts the sum.
__device__ __forceinline__ void mma_i8_stage(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool fresh) {
  mma_i8_ss(d_tmem, desc_of(a_lo), desc_of(b_lo), idesc, fresh ? 0u : 1u);
  mma_i8_ss(d_tmem, desc_of(a_lo + 2), desc_of(b_lo + 2), idesc, 1u);
  mma_i8_ss(d_tmem, desc_of(a_lo + 4), desc_of(b_lo + 4), idesc, 1u);
  mma_i8_ss(d_tmem, desc_of(a_lo + 6), desc_of(b_lo + 6), idesc, 1u);
}

constexpr int MODE_CONCAT = 0;       // gate_up, [gate | up] columns
constexpr int MODE_INTERLEAVED = 1;  // gate_up, gate on even columns
constexpr int MODE_DOWN = 2;

struct Int8Params {
  const int32_t* offsets;
  const float* a_scales;
  const float* w_scales;
  const __nv_bfloat16* bias;
  __nv_bfloat16* out;
  int* status;
  int E, R;
  int N;        // weight columns of an expert (2D or H)
  int out_cols; // D or H
  int n_tiles, num_kb;
  float alpha, limit;  // limit: infinity for none
  int err_bit;
};

// The workspace's first two words: the device status, and a mark that gate_up
// leaves and down takes away.  A layer runs both on one workspace and reads the
// status once, after both: so gate_up starts the word anew, and down keeps what
// the gate_up before it recorded, which only the mark tells from what the memory
// held (a lone down starts the word anew; what gate_up cannot have recorded is
// not its).  `bad_csr` is what this call found so far; a wait that times out is
// recorded seconds later.  One thread of the last epilogue warp has read the
// words (csr_pieces) and writes them once its first loads are on their way: by
// thread 0 ahead of the barrier it cost one token 0.2 to 0.5 us.
constexpr int kGateUpMark = 0x6d6f6547;
__device__ __forceinline__ bool keeps_status() { return blockIdx.x == 0 && threadIdx.x == blockDim.x - 1; }
__device__ __forceinline__ void start_status(int* status, const int2& before, bool down, bool bad_csr) {
  constexpr int kOfGateUp = MOE_DEVICE_ERR_CSR | MOE_DEVICE_ERR_TIMEOUT_GEMM1;
  const bool keep = down && before.y == kGateUpMark && (before.x & ~kOfGateUp) == 0;
  status[0] = (keep ? before.x : 0) | (bad_csr ? MOE_DEVICE_ERR_CSR : 0);
  status[1] = down ? 0 : kGateUpMark;
}

// The gated activation with sigmoids throughout (0.5 (1 + tanh a) is
// sigmoid(2a)).  The exponential's error grows with its argument, 2 + 1.17 |x|
// steps of 2^-23: 2^-22 near zero, 2^-18 at -20, 2^-16 at -87, where the
// sigmoid ends, and so it stays below the bf16 rounding of h, 2^-8.  The
// quotient's is 2 steps.  For large negative gates the exponential overflows and
// the quotient is 0, as the limit is.  ACT is a template argument: a branch per
// element would keep the elements from overlapping.
template <int ACT>
__device__ __forceinline__ float gated(float g, float u, float alpha, float limit) {
  if constexpr (ACT != MOE_ACT_GELU_TANH) {
    // (comparisons, so that a NaN stays one; no limit is an infinite one)
    g = g > limit ? limit : g;
    u = u > limit ? limit : u < -limit ? -limit : u;
  }
  if constexpr (ACT == MOE_ACT_SILU) return __fdividef(g, 1.f + __expf(-g)) * u;
  if constexpr (ACT == MOE_ACT_SWIGLUOAI) return __fdividef(g, 1.f + __expf(-alpha * g)) * (u + 1.f);
  return __fdividef(g, 1.f + __expf(-1.5957691216057308f * (g + 0.044715f * g * g * g))) * u;
}

// What does not depend on the tile shape (n_tiles and num_kb are the kernel's).
inline Int8Params int8_params(const Int8GemmArgs& a) {
  Int8Params p = {};
  p.offsets = a.offsets;
  p.a_scales = a.a_scales;
  p.w_scales = a.w_scales;
  p.bias = a.bias;
  p.out = a.out;
  p.status = a.status;
  p.E = a.E;
  p.R = a.R;
  p.N = a.down ? a.H : 2 * a.D;
  p.out_cols = a.down ? a.H : a.D;
  p.alpha = a.alpha;
  p.limit = a.limit > 0.f ? a.limit : INFINITY;
  p.err_bit = a.down ? MOE_DEVICE_ERR_TIMEOUT_GEMM2 : MOE_DEVICE_ERR_TIMEOUT_GEMM1;
  return p;
}

// (acc * row scale) * column scale + bias: the same operations, and so the same
// bits, in both kernels.
__device__ __forceinline__ float int8_scaled(uint32_t acc, float row, float col, float bias) {
  return fmaf(static_cast<float>(static_cast<int>(acc)) * row, col, bias);
}

// Warp 0: validates the CSR in s_off and builds the per-expert prefix s_mt of
// pieces of `piece` rows; *bad_flag is set for offsets that are no CSR of at
// most R rows.
__device__ __forceinline__ void build_pieces(const int* s_off, int* s_mt, int* bad_flag, int E, int R, int piece,
                                             int lane) {
  const int per = (E + 31) / 32;
  const int e0 = min(lane * per, E), e1 = min(e0 + per, E);
  int local = 0;
  bool bad = false;
  for (int e = e0; e < e1; ++e) {
    const int lo = s_off[e], hi = s_off[e + 1];
    if (lo < 0 || hi < lo || hi > R) bad = true;
    else local += (hi - lo + piece - 1) / piece;
  }
  int incl = local;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  int run = incl - local;
  for (int e = e0; e < e1; ++e) {
    s_mt[e] = run;
    const int lo = s_off[e], hi = s_off[e + 1];
    if (lo >= 0 && hi > lo && hi <= R) run += (hi - lo + piece - 1) / piece;
  }
  if (lane == 31) s_mt[E] = incl;
  if (lane == 0 && s_off[0] != 0) bad = true;
  if (__any_sync(0xffffffffu, bad) && lane == 0) *bad_flag = 1;
}

// Tile t as decode_tile gives it, by a whole warp (all lanes, the same t): the
// expert is looked for from `from` on (at most t's), 32 experts at a time, which
// takes one step where decode_tile's halving takes log2(E) dependent ones.
__device__ __forceinline__ TileCoord warp_tile(int t, int from, int n_tiles, int E, const int* s_mt, const int* s_off,
                                               int piece) {
  const int lane = threadIdx.x & 31;
  int e = from;
  for (;;) {
    const int i = e + 1 + lane;
    const int ahead = __popc(__ballot_sync(0xffffffffu, i < E && s_mt[i < E ? i : E] * n_tiles <= t));
    e += ahead;
    if (ahead < 32) break;
  }
  TileCoord c;
  c.e = e;
  const int local = t - s_mt[e] * n_tiles, mt = s_mt[e + 1] - s_mt[e];
  c.n = mt == 1 ? local : local / mt;
  const int m = local - c.n * mt;
  c.row0 = s_off[e] + m * piece;
  c.rows = min(piece, s_off[e + 1] - c.row0);
  c.piece = s_mt[e] + m;
  return c;
}

// Reads and checks the offsets and builds s_mt; returns the number of pieces, 0
// for offsets that are no CSR (*bad_flag).  While the kernels before
// (as a rule the rows' quantiser) still run, `prefetch` is called by warp 0 to
// fetch the first tile's weights to L2, where their copies then find them: a
// hint, which cannot make a value stale.  The offsets that it goes by may still
// be changing, so it gets any CSR, and they are read again afterwards.  On return
// the kernels before are complete and visible, and `before` holds the status
// words for the thread that keeps them.
template <typename Prefetch>
__device__ __forceinline__ int csr_pieces(const Int8Params& g, int* s_off, int* s_mt, int* bad_flag, int piece,
                                          int2& before, Prefetch prefetch) {
  const int lane = threadIdx.x & 31;
  auto read = [&]() {
    for (int i = threadIdx.x; i <= g.E; i += blockDim.x) s_off[i] = __ldcg(g.offsets + i);
  };
  if (threadIdx.x == 0) *bad_flag = 0;
  read();
  __syncthreads();
  if (threadIdx.x < 32) {
    build_pieces(s_off, s_mt, bad_flag, g.E, g.R, piece, lane);
    __syncwarp();
    if (*bad_flag == 0) prefetch();
  }
  griddep_wait();
  before = keeps_status() ? __ldcg(reinterpret_cast<const int2*>(g.status)) : make_int2(0, 0);
  bool same = true;
  for (int i = threadIdx.x; i <= g.E; i += blockDim.x) same = same && s_off[i] == __ldcg(g.offsets + i);
  if (!__syncthreads_and(same)) {
    if (threadIdx.x == 0) *bad_flag = 0;
    read();
    __syncthreads();
    if (threadIdx.x < 32) build_pieces(s_off, s_mt, bad_flag, g.E, g.R, piece, lane);
    __syncthreads();
  }
  return *bad_flag != 0 ? 0 : s_mt[g.E];
}

}  // namespace moe
