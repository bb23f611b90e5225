// int8_gemm.cu -- the experts' products in 8-bit integers over rows sorted by
// expert:  y[p, n] = (sum_k A[p, k] W[e, n, k]) * a_scale[p] * w_scale[e, n] + b[e, n]
// for p in expert e's segment; the gate_up product also applies the gated
// activation and stores h [R, D], the down product stores [R, H].
//
// The integer sums are exact (32-bit accumulators in TMEM, K <= 131072), the
// scales, bias and activation are fp32, and the only rounding is the store to
// bf16.  Both operands are K-major (the weights are turned once, when they are
// quantised), so a 128-byte swizzle row holds 128 values of K: a stage of
// 48 KB carries twice the K of the bf16 kernel's, and streaming the weights
// costs half the bytes.
//
// One persistent CTA per SM, as in the bf16 kernel:
//   warp 0      TMA producer: per 128-wide K block one 128 x 128 B box of A
//               (64 or 16 rows for a tile of at most so many) and one 256 x
//               128 B tile of W into a 4-stage ring;
//   warp 1      MMA issuer: four tcgen05.mma kind::i8 128x256x32 a stage
//               (M = 64 for a tile of at most 64 rows), two 256-column
//               accumulators alternate between tiles;
//   warps 2..9  epilogue: 32 TMEM lanes and half of the columns each.
// Tiles walk the column blocks of an expert, row pieces innermost, so that
// CTAs running together share a weight block through L2.
//
// What bounds it, on one B200 (6.56 TB/s copy rate):
//   few rows per expert   the weights' stream: E 128, 2880 x 5760, 8192 rows in
//               341 us (6.4 TB/s); E 64, 1536 x 4096, 256 rows in 56 us, of
//               which 5 us pass before the first copy has landed and 1.4 us are
//               the seventh wave of 6.8; one token to 8 experts 13.8 us;
//   many rows   the 1000 W power limit: E 8, 4096 x 28672, 8192 rows in 0.84 ms
//               (2.3 POP/s) at 1.38 GHz in a loop, 0.71 ms (2.7) for a few
//               passes; 0.65 ms with all-zero weights at 1.965 GHz.  Pairs of CTAs
//               (256 x 256 tiles) drew the same power for the same time.
#include <cudaTypedefs.h>

#include <algorithm>

#include "grouped_tiles.cuh"
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int BM = 128;                    // rows per tile (TMEM lanes)
constexpr int BN = 256;                    // accumulator columns per tile
constexpr int BK = 128;                    // K per stage: one 128-byte swizzle row
constexpr int UMMA_K = 32;                 // K per tcgen05.mma (kind::i8)
constexpr int A_BYTES = BM * BK;           // 16 KB
constexpr int B_BYTES = BN * BK;           // 32 KB
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int STAGES = 4;
constexpr int HALF_ROWS = 64;              // tiles of at most 64 rows: M = 64
constexpr int FEW_ROWS = 16;               // tiles that copy only 16 rows of A
constexpr int NUM_EPI_WARPS = 8;
constexpr int NUM_THREADS = 64 + 32 * NUM_EPI_WARPS;
constexpr int CTRL_BYTES = 256;
constexpr uint32_t TMEM_COLS = 2 * BN;     // two accumulators

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
  int activation;
  float alpha, limit;
  int err_bit;
};

// The gated activation with sigmoids throughout (0.5 (1 + tanh a) is
// sigmoid(2a)): exp2 and reciprocal approximations of about 2^-22, below the
// bf16 rounding of h.  For large negative gates the exponential overflows and
// the quotient is 0, as the limit is.
__device__ __forceinline__ float gated(int act, float g, float u, float alpha, float limit) {
  if (act != 2 && limit > 0.f) {
    // (comparisons, so that a NaN stays one)
    g = g > limit ? limit : g;
    u = u > limit ? limit : u < -limit ? -limit : u;
  }
  if (act == 0) return __fdividef(g, 1.f + __expf(-g)) * u;
  if (act == 1) return __fdividef(g, 1.f + __expf(-alpha * g)) * (u + 1.f);
  return __fdividef(g, 1.f + __expf(-1.5957691216057308f * (g + 0.044715f * g * g * g))) * u;
}

// What one epilogue warp does of a tile: Cols::n output columns from column
// `col` on, whose accumulators start at TMEM column `tcol` (concatenated: the up
// columns BN / 2 further on), of the rows from row0 on that its lanes hold.  The
// M = 64 accumulator holds row r in lane 32*(r/16) + r%16.
struct Part {
  int col, tcol;
  int row0, lanes;  // rows row0 .. row0 + lanes - 1 of the tile
};
template <int MODE>
struct Cols {
  static constexpr int OUT = MODE == MODE_DOWN ? BN : BN / 2;  // output columns of a tile
  static constexpr int PER = BN / OUT;                         // accumulator columns per output column
  static constexpr int n = OUT / 2;                            // output columns of a warp
};

template <int MODE>
__device__ __forceinline__ Part warp_part(int tile_n, int quad, int part, bool half) {
  using C = Cols<MODE>;
  return {tile_n * C::OUT + part * C::n, MODE == MODE_CONCAT ? part * C::n : part * C::n * C::PER,
          half ? quad * 16 : quad * 32, half ? 16 : 32};
}

// A warp's weight columns, in groups of four: group i's scales lie in the 16
// bytes that row i of its staging block leaves free, its biases behind the
// block.  The loads are issued while the tile's product is still running,
// since the scales come from HBM.  Concatenated: the gate columns' groups,
// then the up columns'.
constexpr int kWarpStage = kStageWarpBytes + 256;

template <int MODE>
__device__ __forceinline__ void stage_columns(const Int8Params& p, const Part& w, int e, int lane, uint8_t* stage) {
  int c = -1;  // the group's first weight column, or -1 past the end
  if constexpr (MODE == MODE_CONCAT) {
    const int h = w.col + 4 * (lane & 15);
    if (h < p.out_cols) c = (lane < 16 ? 0 : p.out_cols) + h;
  } else {
    const int first = w.col * Cols<MODE>::PER + 4 * lane;
    if (first < p.N) c = first;
  }
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  uint2 b = make_uint2(0u, 0u);
  if (c >= 0) {
    const int64_t at = static_cast<int64_t>(e) * p.N + c;
    s = __ldg(reinterpret_cast<const float4*>(p.w_scales + at));
    if (p.bias != nullptr) b = __ldg(reinterpret_cast<const uint2*>(p.bias + at));
  }
  __syncwarp();  // every lane is done with the tile before
  *reinterpret_cast<float4*>(stage + lane * kStageRowBytes + 64) = s;
  *reinterpret_cast<uint2*>(stage + kStageWarpBytes + 8 * lane) = b;
  __syncwarp();
}

struct Col4 {
  float s[4], b[4];
};
__device__ __forceinline__ Col4 columns(const uint8_t* stage, int i) {
  const float4 s = *reinterpret_cast<const float4*>(stage + i * kStageRowBytes + 64);
  const uint2 b = *reinterpret_cast<const uint2*>(stage + kStageWarpBytes + 8 * i);
  return {{s.x, s.y, s.z, s.w}, {bf16_lo(b.x), bf16_hi(b.x), bf16_lo(b.y), bf16_hi(b.y)}};
}

__device__ __forceinline__ float scaled(uint32_t acc, float row, const Col4& c, int i) {
  return fmaf(static_cast<float>(static_cast<int>(acc)) * row, c.s[i], c.b[i]);
}

// 32 output columns of this thread's row, from column `rel` of the warp's
// columns, packed to bf16.
template <int MODE>
__device__ __forceinline__ void out_chunk(const Int8Params& p, const Part& w, uint32_t tacc, int rel, float row,
                                          const uint8_t* stage, uint32_t (&packed)[16]) {
  const int i0 = rel >> 2;
  if constexpr (MODE == MODE_DOWN) {
    uint32_t a[32];
    tmem_ld32(tacc + w.tcol + rel, a);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const Col4 c = columns(stage, i0 + (j >> 2));
      packed[j / 2] = pack_bf16x2(scaled(a[j], row, c, 0), scaled(a[j + 1], row, c, 1));
      packed[j / 2 + 1] = pack_bf16x2(scaled(a[j + 2], row, c, 2), scaled(a[j + 3], row, c, 3));
    }
  } else if constexpr (MODE == MODE_CONCAT) {
    uint32_t g[32], u[32];
    tmem_ld32(tacc + w.tcol + rel, g);
    tmem_ld32(tacc + w.tcol + BN / 2 + rel, u);
    tmem_ld_wait();
    const int i1 = i0 + 16;
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const Col4 cg = columns(stage, i0 + (j >> 2)), cu = columns(stage, i1 + (j >> 2));
      float h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        h[i] = gated(p.activation, scaled(g[j + i], row, cg, i), scaled(u[j + i], row, cu, i), p.alpha, p.limit);
      packed[j / 2] = pack_bf16x2(h[0], h[1]);
      packed[j / 2 + 1] = pack_bf16x2(h[2], h[3]);
    }
  } else {
    uint32_t a[64];
    tmem_ld32(tacc + w.tcol + 2 * rel, a);
    tmem_ld32(tacc + w.tcol + 2 * rel + 32, a + 32);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 64; j += 4) {
      const Col4 c = columns(stage, 2 * i0 + (j >> 2));
      const float h0 = gated(p.activation, scaled(a[j], row, c, 0), scaled(a[j + 1], row, c, 1), p.alpha, p.limit);
      const float h1 = gated(p.activation, scaled(a[j + 2], row, c, 2), scaled(a[j + 3], row, c, 3), p.alpha, p.limit);
      packed[j / 4] = pack_bf16x2(h0, h1);
    }
  }
}

// One tile's epilogue for one warp, rs its thread's row scale; row0 the tile's
// first row and rows how many there are.  Each 32 x 32 block is turned through the staging block so that a store instruction writes 8 rows
// x 64 contiguous bytes.
template <int MODE>
__device__ __forceinline__ void epilogue(const Int8Params& p, const Part& w, uint32_t tacc, int row0, int rows, int lane,
                                         float rs, uint8_t* stage) {
  const int q = lane & 3;
  uint8_t* my_row = stage + lane * kStageRowBytes;
#pragma unroll 1
  for (int rel = 0; rel < Cols<MODE>::n; rel += kOutChunk) {
    if (w.col + rel >= p.out_cols) break;
    uint32_t packed[16];
    out_chunk<MODE>(p, w, tacc, rel, rs, stage, packed);
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<uint4*>(my_row + 16 * c) =
          make_uint4(packed[4 * c], packed[4 * c + 1], packed[4 * c + 2], packed[4 * c + 3]);
    __syncwarp();
    const int col = w.col + rel + 8 * q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int l = 8 * i + (lane >> 2);  // the lane whose row this is
      const int r = w.row0 + l;
      if (l < w.lanes && r < rows && col < p.out_cols)
        *reinterpret_cast<uint4*>(p.out + (static_cast<int64_t>(row0) + r) * p.out_cols + col) =
            *reinterpret_cast<const uint4*>(stage + l * kStageRowBytes + 16 * q);
    }
  }
}

template <int MODE>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapAh,
                     const __grid_constant__ CUtensorMap mapAf, const __grid_constant__ CUtensorMap mapB,
                     const Int8Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint8_t* ctrl = smem + STAGES * STAGE_BYTES;
  const uint32_t full0 = smem_u32(ctrl);        // STAGES mbarriers
  const uint32_t empty0 = full0 + 8 * STAGES;   // STAGES mbarriers
  const uint32_t tfull0 = empty0 + 8 * STAGES;  // 2 mbarriers
  const uint32_t tempty0 = tfull0 + 16;         // 2 mbarriers
  const uint32_t drain_bar = tempty0 + 16;      // 1 mbarrier
  static_assert((2 * STAGES + 5) * 8 <= 128, "mbarriers overflow their part of the control block");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 128);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctrl + 132);
  int* bad_flag = reinterpret_cast<int*>(ctrl + 136);
  int* s_off = reinterpret_cast<int*>(ctrl + CTRL_BYTES);
  int* s_mt = s_off + (p.E + 1);
  uint8_t* s_stage =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_mt + p.E + 1) + 15) & ~uintptr_t(15));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull0 + 8 * a, 1);
      mbar_init(tempty0 + 8 * a, 32 * NUM_EPI_WARPS);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    *bad_flag = 0;
    fence_mbar_init();
    tma_prefetch_map(&mapA);
    tma_prefetch_map(&mapB);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  griddep_wait();  // the offsets and operands of the kernels before are complete and visible
  // the status word of this call starts at zero: only this CTA records a bad
  // CSR, and a timed-out wait of another comes seconds later
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;
  for (int i = threadIdx.x; i <= p.E; i += NUM_THREADS) s_off[i] = p.offsets[i];
  __syncthreads();
  if (warp == 0) {
    // Validate the CSR and build the per-expert prefix of tile pieces.
    const int per = (p.E + 31) / 32;
    const int e0 = min(lane * per, p.E), e1 = min(e0 + per, p.E);
    int local = 0;
    bool bad = false;
    for (int e = e0; e < e1; ++e) {
      const int cnt = s_off[e + 1] - s_off[e];
      if (cnt < 0 || s_off[e] < 0 || s_off[e + 1] > p.R) bad = true;
      else local += (cnt + BM - 1) / BM;
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
      const int cnt = s_off[e + 1] - s_off[e];
      if (cnt > 0) run += (cnt + BM - 1) / BM;
    }
    if (lane == 31) s_mt[p.E] = incl;
    if (lane == 0 && s_off[0] != 0) bad = true;
    if (__any_sync(0xffffffffu, bad) && lane == 0) *bad_flag = 1;
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  const bool bad = *bad_flag != 0;
  if (bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.status, MOE_DEVICE_ERR_CSR);
  const int total = bad ? 0 : s_mt[p.E] * p.n_tiles;

  if (warp == 0) {
    if (lane == 0) {
      // -------------------------------------------------- TMA producer
      int it = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
        const TileCoord tc = decode_tile(t, p.n_tiles, p.E, s_mt, s_off, BM);
        // rows of A to copy: all 128, or 64 of a tile of at most 64, or 16 of one
        // of at most 16; the rest of the stage holds old rows, whose sums are
        // not stored
        const bool half = tc.rows <= HALF_ROWS, few = tc.rows <= FEW_ROWS;
        const int a_rows = few ? FEW_ROWS : half ? HALF_ROWS : BM;
        const CUtensorMap* ma = few ? &mapAf : half ? &mapAh : &mapA;
        const uint32_t bytes = static_cast<uint32_t>(a_rows * BK + B_BYTES);
        for (int kb = 0; kb < p.num_kb; ++kb, ++it) {
          const int s = it % STAGES;
          const uint32_t ph = static_cast<uint32_t>(it / STAGES) & 1u;
          if (!mbar_wait(empty0 + 8 * s, ph ^ 1u, abort_flag, kTimeoutNs)) {
            ok = false;
            break;
          }
          const uint32_t sa = sbase + s * STAGE_BYTES, sb = sa + A_BYTES;
          const uint32_t fb = full0 + 8 * s;
          mbar_arrive_expect_tx(fb, bytes);
          tma_load_2d(sa, ma, fb, kb * BK, tc.row0);
          if constexpr (MODE == MODE_CONCAT) tma_load_4d(sb, &mapB, fb, kb * BK, tc.n * (BN / 2), 0, tc.e);
          else tma_load_3d(sb, &mapB, fb, kb * BK, tc.n * BN, tc.e);
        }
      }
      if (ok) {
        // wait until the MMAs have released every stage, so that no commit
        // arrival lands after this CTA exits
        for (int i = 0; i < STAGES; ++i, ++it) {
          const int s = it % STAGES;
          const uint32_t ph = static_cast<uint32_t>(it / STAGES) & 1u;
          if (!mbar_wait(empty0 + 8 * s, ph ^ 1u, abort_flag, kTimeoutNs)) break;
        }
      } else {
        // aborted: let the copies already issued land before shared memory is
        // released (time-bounded, independent of the abort flag)
        for (int s = 0; s < STAGES; ++s) {
          if (it > s) {
            const int last = s + ((it - 1 - s) / STAGES) * STAGES;
            wait_time_only(full0 + 8 * s, static_cast<uint32_t>(last / STAGES) & 1u);
          }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------------------------------------------- MMA issuer
      int it = 0, ti = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < total; t += gridDim.x, ++ti) {
        const int acc = ti & 1;
        if (!mbar_wait(tempty0 + 8 * acc, (static_cast<uint32_t>(ti >> 1) & 1u) ^ 1u, abort_flag, kTimeoutNs)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
        const TileCoord tc = decode_tile(t, p.n_tiles, p.E, s_mt, s_off, BM);
        const uint32_t idesc = tc.rows <= HALF_ROWS ? idesc_s8_s32(HALF_ROWS, BN) : idesc_s8_s32(BM, BN);
        for (int kb = 0; kb < p.num_kb; ++kb, ++it) {
          const int s = it % STAGES;
          if (!mbar_wait(full0 + 8 * s, static_cast<uint32_t>(it / STAGES) & 1u, abort_flag, kTimeoutNs)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t sa = sbase + s * STAGE_BYTES, sb = sa + A_BYTES;
#pragma unroll
          for (int kk = 0; kk < BK / UMMA_K; ++kk) {
            // K-major rows of 128 B, 8-row swizzle atoms 1024 B apart; a
            // 32-wide K step is 32 B along the row
            mma_i8_ss(d_tmem, smem_desc_sw128(sa + kk * UMMA_K, 16, 1024),
                      smem_desc_sw128(sb + kk * UMMA_K, 16, 1024), idesc, (kb | kk) != 0 ? 1u : 0u);
          }
          mma_commit(empty0 + 8 * s);
        }
        if (!ok) break;
        mma_commit(tfull0 + 8 * acc);
      }
      if (!ok) {
        // aborted: every MMA issued so far must finish before TMEM is freed
        mma_commit(drain_bar);
        wait_time_only(drain_bar, 0);
      }
    }
  } else {
    // -------------------------------------------------------- epilogue
    const int quad = warp & 3;         // this warp may access TMEM lanes 32*quad..+31
    const int part = (warp - 2) >> 2;  // which half of the tile's columns
    uint8_t* stage = s_stage + (warp - 2) * kWarpStage;
    int ti = 0;
    for (int t = blockIdx.x; t < total; t += gridDim.x, ++ti) {
      const TileCoord tc = decode_tile(t, p.n_tiles, p.E, s_mt, s_off, BM);
      const int acc = ti & 1;
      const Part w = warp_part<MODE>(tc.n, quad, part, tc.rows <= HALF_ROWS);
      const float rs = lane < w.lanes && w.row0 + lane < tc.rows ? __ldg(p.a_scales + tc.row0 + w.row0 + lane) : 0.f;
      stage_columns<MODE>(p, w, tc.e, lane, stage);
      const bool got = mbar_wait(tfull0 + 8 * acc, static_cast<uint32_t>(ti >> 1) & 1u, abort_flag, kTimeoutNs);
      if (!__all_sync(0xffffffffu, got)) break;
      tc_fence_after_sync();
      const uint32_t tacc = tmem_base + static_cast<uint32_t>(acc * BN) + (static_cast<uint32_t>(quad * 32) << 16);
      epilogue<MODE>(p, w, tacc, tc.row0, tc.rows, lane, rs, stage);
      tc_fence_before_sync();
      mbar_arrive(tempty0 + 8 * acc);
    }
  }

  __syncthreads();
  griddep_launch_dependents();  // this CTA has no tiles left: the next kernel may begin launching
  if (threadIdx.x == 0 && *abort_flag) atomicOr(p.status, p.err_bit);
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

constexpr size_t smem_bytes(int E) {
  return 1024 + STAGES * STAGE_BYTES + CTRL_BYTES + 2 * static_cast<size_t>(E + 1) * 4 + 16 + NUM_EPI_WARPS * kWarpStage;
}

template <int MODE>
cudaError_t launch_mode(const Int8GemmArgs& a, cudaStream_t stream) {
  const bool down = MODE == MODE_DOWN;
  const int K = down ? a.D : a.H;
  const cuuint64_t pitch = static_cast<cuuint64_t>(int8_pitch(K));
  const cuuint64_t N = down ? a.H : 2 * static_cast<cuuint64_t>(a.D), E = a.E;
  constexpr CUtensorMapDataType kU8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  CUtensorMap mapA, mapAh, mapAf, mapB;
  {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(a.R)};
    const cuuint64_t strides[1] = {pitch};
    const cuuint32_t box[2] = {BK, BM}, half_box[2] = {BK, HALF_ROWS}, few_box[2] = {BK, FEW_ROWS};
    if (!encode_tiled_map(&mapA, kU8, a.A, 2, dims, strides, box) ||
        !encode_tiled_map(&mapAh, kU8, a.A, 2, dims, strides, half_box) ||
        !encode_tiled_map(&mapAf, kU8, a.A, 2, dims, strides, few_box))
      return cudaErrorInvalidValue;
  }
  if (MODE == MODE_CONCAT) {
    // {K, D, 2 (gate/up), E}: a CTA's gate rows, then the matching up rows
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(a.D), 2, E};
    const cuuint64_t strides[3] = {pitch, a.D * pitch, N * pitch};
    const cuuint32_t box[4] = {BK, BN / 2, 2, 1};
    if (!encode_tiled_map(&mapB, kU8, a.W, 4, dims, strides, box)) return cudaErrorInvalidValue;
  } else {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(K), N, E};
    const cuuint64_t strides[2] = {pitch, N * pitch};
    const cuuint32_t box[3] = {BK, BN, 1};
    if (!encode_tiled_map(&mapB, kU8, a.W, 3, dims, strides, box)) return cudaErrorInvalidValue;
  }
  Int8Params p;
  p.offsets = a.offsets;
  p.a_scales = a.a_scales;
  p.w_scales = a.w_scales;
  p.bias = a.bias;
  p.out = a.out;
  p.status = a.status;
  p.E = a.E;
  p.R = a.R;
  p.N = static_cast<int>(N);
  p.out_cols = down ? a.H : a.D;
  p.n_tiles = (p.out_cols + (down ? BN : BN / 2) - 1) / (down ? BN : BN / 2);
  p.num_kb = (K + BK - 1) / BK;
  p.activation = a.activation;
  p.alpha = a.alpha;
  p.limit = a.limit;
  p.err_bit = down ? MOE_DEVICE_ERR_TIMEOUT_GEMM2 : MOE_DEVICE_ERR_TIMEOUT_GEMM1;
  const void* kernel = reinterpret_cast<const void*>(int8_gemm_kernel<MODE>);
  const cudaError_t err = opt_in_dynamic_smem(kernel, static_cast<int>(smem_bytes(kMaxExperts)));
  if (err != cudaSuccess) return err;
  const int64_t max_tiles = (static_cast<int64_t>(a.R) / BM + std::min(a.E, a.R)) * p.n_tiles;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(max_tiles, a.num_sms)));
  return launch_pdl(int8_gemm_kernel<MODE>, grid, dim3(NUM_THREADS), smem_bytes(a.E), stream, mapA, mapAh, mapAf, mapB,
                    p);
}

}  // namespace

cudaError_t launch_int8_gemm(const Int8GemmArgs& a, cudaStream_t stream) {
  if (a.R == 0) return cudaSuccess;
  if (a.down) return launch_mode<MODE_DOWN>(a, stream);
  return a.gate_up_format == 0 ? launch_mode<MODE_CONCAT>(a, stream) : launch_mode<MODE_INTERLEAVED>(a, stream);
}

}  // namespace moe
