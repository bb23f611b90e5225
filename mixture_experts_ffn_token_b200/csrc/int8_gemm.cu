// int8_gemm.cu -- the experts' products in 8-bit integers over rows sorted by
// expert:  y[p, n] = (sum_k A[p, k] W[e, n, k]) * a_scale[p] * w_scale[e, n] + b[e, n]
// for p in expert e's segment; the gate_up product also applies the gated
// activation and stores h [R, D], the down product stores [R, H].
//
// The integer sums are exact (32-bit accumulators in TMEM, K <= 131072).  The
// sum's conversion to fp32, the two scales and the bias round to 2^-24 each, the
// activation as int8_common.cuh says, and the store to bf16 to 2^-8.  Both operands are K-major (the weights are turned once, when they are
// quantised), so a 128-byte swizzle row holds 128 values of K: a stage of
// 48 KB carries twice the K of the bf16 kernel's, and streaming the weights
// costs half the bytes.
//
// One persistent CTA per SM, as in the bf16 kernel:
//   warp 0      TMA producer: per 128-wide K block one 128 x 128 B box of A
//               (64 rows for a tile of at most 64) and one 256 x 128 B tile of
//               W into a 4-stage ring;
//   warp 1      MMA issuer: four tcgen05.mma kind::i8 128x256x32 a stage
//               (M = 64 for a tile of at most 64 rows), two 256-column
//               accumulators alternate between tiles;
//   warps 2..9  epilogue: 32 TMEM lanes and half of the columns each.
// Tiles walk the column blocks of an expert, row pieces innermost, so that
// CTAs running together share a weight block through L2.
//
// What bounds it, on one B200: with a long K the 1000 W power limit (E 8, 4096 x
// 28672, 8192 rows in 0.80 to 0.85 ms, 2.3 POP/s, at 1.38 GHz in a loop, 0.65 ms with all-zero weights at 1.965 GHz; pairs of CTAs with 256 x
// 256 tiles drew the same power for the same time), with a short one the
// epilogue, whose shared-memory traffic fills 60% of its cycles (E 50, 240 x 2328,
// 32200 rows in 72 us with the quantiser, 30 at the copy rate).
#include <cudaTypedefs.h>

#include <algorithm>

#include "int8_common.cuh"

namespace moe {
namespace {

constexpr int BM = 128;                    // rows per tile (TMEM lanes)
constexpr int BN = 256;                    // accumulator columns per tile
constexpr int BK = 128;                    // K per stage: one 128-byte swizzle row
constexpr int A_BYTES = BM * BK;           // 16 KB
constexpr int B_BYTES = BN * BK;           // 32 KB
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int STAGES = 4;
constexpr int HALF_ROWS = 64;              // tiles of at most 64 rows: M = 64
constexpr int HALF_A_BYTES = HALF_ROWS * BK;
constexpr int NUM_EPI_WARPS = 8;
constexpr int NUM_THREADS = 64 + 32 * NUM_EPI_WARPS;
constexpr int CTRL_BYTES = 256;
constexpr uint32_t TMEM_COLS = 2 * BN;     // two accumulators

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

// An epilogue warp's shared memory: a block of 32 rows x 64 B that turns 32 x 32
// outputs, its 128 weight columns' scales, and their biases.  16-byte piece c
// of the block's row r lies at piece c ^ (r / 2 % 4), so that neither a piece of
// eight rows nor four pieces of two rows meet in a bank.
constexpr int kScalesAt = 32 * 64, kBiasAt = kScalesAt + 128 * 4;
constexpr int kWarpStage = kBiasAt + 128 * 2;
__device__ __forceinline__ uint8_t* turned(uint8_t* stage, int r, int c) {
  return stage + r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// What a tile's epilogue needs from memory, fetched a tile ahead, since it comes
// from HBM: the scales and biases in groups of four columns, one a lane
// (concatenated: the gate columns' groups, then the up columns').

struct Ahead {
  TileCoord tc;
  Part w;
  float rs;   // the scale of this lane's row
  float4 s;   // this lane's group
  uint2 b;
};
template <int MODE>
__device__ __forceinline__ Ahead fetch(const Int8Params& p, int t, int from, const int* s_mt, const int* s_off, int quad, int part,
                                       int lane) {
  Ahead f;
  f.tc = warp_tile(t, from, p.n_tiles, p.E, s_mt, s_off, BM);
  f.w = warp_part<MODE>(f.tc.n, quad, part, f.tc.rows <= HALF_ROWS);
  f.rs = lane < f.w.lanes && f.w.row0 + lane < f.tc.rows ? __ldg(p.a_scales + f.tc.row0 + f.w.row0 + lane) : 0.f;
  int c = -1;  // the group's first weight column, or -1 past the end
  if constexpr (MODE == MODE_CONCAT) {
    const int h = f.w.col + 4 * (lane & 15);
    if (h < p.out_cols) c = (lane < 16 ? 0 : p.out_cols) + h;
  } else {
    const int first = f.w.col * Cols<MODE>::PER + 4 * lane;
    if (first < p.N) c = first;
  }
  f.s = make_float4(0.f, 0.f, 0.f, 0.f);
  f.b = make_uint2(0u, 0u);
  if (c >= 0) {
    const int64_t at = static_cast<int64_t>(f.tc.e) * p.N + c;
    f.s = __ldg(reinterpret_cast<const float4*>(p.w_scales + at));
    if (p.bias != nullptr) f.b = __ldg(reinterpret_cast<const uint2*>(p.bias + at));
  }
  return f;
}

struct Col4 {
  float s[4], b[4];
};
__device__ __forceinline__ Col4 columns(const uint8_t* stage, int i) {
  const float4 s = *reinterpret_cast<const float4*>(stage + kScalesAt + 16 * i);
  const uint2 b = *reinterpret_cast<const uint2*>(stage + kBiasAt + 8 * i);
  return {{s.x, s.y, s.z, s.w}, {bf16_lo(b.x), bf16_hi(b.x), bf16_lo(b.y), bf16_hi(b.y)}};
}

__device__ __forceinline__ float scaled(uint32_t acc, float row, const Col4& c, int i) {
  return int8_scaled(acc, row, c.s[i], c.b[i]);
}

// 16 outputs of this thread's row, from column `rel` of the warp's columns.
template <int MODE, int ACT>
__device__ __forceinline__ void outputs(const Int8Params& p, const Part& w, uint32_t tacc, int rel, float row,
                                        const uint8_t* stage, float (&h)[16]) {
  if constexpr (MODE == MODE_DOWN) {
    uint32_t a[16];
    tmem_ld16(tacc + w.tcol + rel, a);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      const Col4 c = columns(stage, (rel + j) >> 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[j + i] = scaled(a[j + i], row, c, i);
    }
  } else if constexpr (MODE == MODE_CONCAT) {
    uint32_t g[16], u[16];
    tmem_ld16(tacc + w.tcol + rel, g);
    tmem_ld16(tacc + w.tcol + BN / 2 + rel, u);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      const Col4 cg = columns(stage, (rel + j) >> 2), cu = columns(stage, 16 + ((rel + j) >> 2));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        h[j + i] = gated<ACT>(scaled(g[j + i], row, cg, i), scaled(u[j + i], row, cu, i), p.alpha, p.limit);
    }
  } else {
    uint32_t a[32];
    tmem_ld32(tacc + w.tcol + 2 * rel, a);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const Col4 c = columns(stage, (2 * rel + j) >> 2);
      h[j / 2] = gated<ACT>(scaled(a[j], row, c, 0), scaled(a[j + 1], row, c, 1), p.alpha, p.limit);
      h[j / 2 + 1] = gated<ACT>(scaled(a[j + 2], row, c, 2), scaled(a[j + 3], row, c, 3), p.alpha, p.limit);
    }
  }
}

// One tile's epilogue for one warp, rs its thread's row scale; row0 the tile's
// first row and rows how many there are.  Each 32 x 32 block is turned through
// the staging block so that a store instruction writes 8 rows x 64 contiguous
// bytes.  The loops stay rolled at 16 outputs: unrolled further the code
// outgrows the instruction cache that ten warps share.
template <int MODE, int ACT>
__device__ __forceinline__ void epilogue(const Int8Params& p, const Part& w, uint32_t tacc, int row0, int rows, int lane,
                                         float rs, uint8_t* stage) {
  const int q = lane & 3;
#pragma unroll 1
  for (int rel = 0; rel < Cols<MODE>::n; rel += 16) {
    if (w.col + (rel & ~(kOutChunk - 1)) >= p.out_cols) break;
    float h[16];
    outputs<MODE, ACT>(p, w, tacc, rel, rs, stage, h);
    const int c0 = (rel & 16) >> 3;  // first of the two pieces of the row
    if (c0 == 0) __syncwarp();       // the block before is stored
#pragma unroll
    for (int c = 0; c < 2; ++c)
      *reinterpret_cast<uint4*>(turned(stage, lane, c0 + c)) =
          make_uint4(pack_bf16x2(h[8 * c], h[8 * c + 1]), pack_bf16x2(h[8 * c + 2], h[8 * c + 3]),
                     pack_bf16x2(h[8 * c + 4], h[8 * c + 5]), pack_bf16x2(h[8 * c + 6], h[8 * c + 7]));
    if (c0 == 0) continue;
    __syncwarp();
    const int col = w.col + rel - 16 + 8 * q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int l = 8 * i + (lane >> 2);  // the lane whose row this is
      const int r = w.row0 + l;
      if (l < w.lanes && r < rows && col < p.out_cols)
        *reinterpret_cast<uint4*>(p.out + (static_cast<int64_t>(row0) + r) * p.out_cols + col) =
            *reinterpret_cast<const uint4*>(turned(stage, l, q));
    }
  }
}

template <int MODE, int ACT>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapAh,
                     const __grid_constant__ CUtensorMap mapB, const Int8Params p) {
  extern __shared__ uint8_t smem_raw[];
  // (by an offset, so that the compiler still knows it for shared memory)
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
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
  uint8_t* s_stage = ctrl + CTRL_BYTES;  // NUM_EPI_WARPS of kWarpStage
  int* s_off = reinterpret_cast<int*>(s_stage + NUM_EPI_WARPS * kWarpStage);
  int* s_mt = s_off + (p.E + 1);
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
    fence_mbar_init();
    tma_prefetch_map(&mapA);
    tma_prefetch_map(&mapB);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  int2 before;
  const int pieces = csr_pieces(p, s_off, s_mt, bad_flag, BM, before, [&]() {
    const int t = blockIdx.x;
    if (t >= s_mt[p.E] * p.n_tiles) return;
    const TileCoord tc = decode_tile(t, p.n_tiles, p.E, s_mt, s_off, BM);
    if (lane < min(p.num_kb, STAGES)) {
      if constexpr (MODE == MODE_CONCAT) tma_prefetch_4d(&mapB, lane * BK, tc.n * (BN / 2), 0, tc.e);
      else tma_prefetch_3d(&mapB, lane * BK, tc.n * BN, tc.e);
    }
  });
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  const int total = pieces * p.n_tiles;

  if (warp == 0) {
    if (lane == 0) {
      // -------------------------------------------------- TMA producer
      int it = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
        const TileCoord tc = decode_tile(t, p.n_tiles, p.E, s_mt, s_off, BM);
        const bool half = tc.rows <= HALF_ROWS;
        const CUtensorMap* ma = half ? &mapAh : &mapA;
        const uint32_t bytes = half ? HALF_A_BYTES + B_BYTES : STAGE_BYTES;
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
    // ------------------------------------------------------ MMA issuer
    // (a whole warp of which one lane issues: then the loop's values are uniform,
    // and an MMA costs the thread no 40 cycles: E 8, 4096 x 28672, 8192 rows 827 ->
    // 800 us; the copying warp likewise makes a short K slower, 75.6 -> 77.6)
    int s = 0, ti = 0, e = 0;
    uint32_t ph = 0;
    bool ok = true;
    const bool leader = elect_one();
    for (int t = blockIdx.x; ok && t < total; t += gridDim.x, ++ti) {
      const int acc = ti & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(tempty0 + 8 * acc, (static_cast<uint32_t>(ti >> 1) & 1u) ^ 1u, abort_flag,
                                             kTimeoutNs))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
      const TileCoord tc = warp_tile(t, e, p.n_tiles, p.E, s_mt, s_off, BM);
      e = tc.e;
      const uint32_t idesc = tc.rows <= HALF_ROWS ? idesc_s8_s32(HALF_ROWS, BN) : idesc_s8_s32(BM, BN);
      for (int kb = 0; kb < p.num_kb; ++kb) {
        if (!__all_sync(0xffffffffu, mbar_wait(full0 + 8 * s, ph, abort_flag, kTimeoutNs))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        if (leader) {
          const uint32_t a_lo = desc_lo(sbase + s * STAGE_BYTES);
          mma_i8_stage(d_tmem, a_lo, a_lo + A_BYTES / 16, idesc, kb == 0);
          mma_commit(empty0 + 8 * s);
        }
        __syncwarp();
        if (++s == STAGES) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (!ok) break;
      if (leader) mma_commit(tfull0 + 8 * acc);
      __syncwarp();
    }
    if (!ok && leader) {
      // aborted: every MMA issued so far must finish before TMEM is freed
      mma_commit(drain_bar);
      wait_time_only(drain_bar, 0);
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------- epilogue
    const int quad = warp & 3;         // this warp may access TMEM lanes 32*quad..+31
    const int part = (warp - 2) >> 2;  // which half of the tile's columns
    uint8_t* stage = s_stage + (warp - 2) * kWarpStage;
    Ahead next = {};
    if (static_cast<int>(blockIdx.x) < total) next = fetch<MODE>(p, blockIdx.x, 0, s_mt, s_off, quad, part, lane);
    if (keeps_status()) start_status(p.status, before, MODE == MODE_DOWN, *bad_flag != 0);
    int ti = 0;
    for (int t = blockIdx.x; t < total; t += gridDim.x, ++ti) {
      const int acc = ti & 1;
      const TileCoord tc = next.tc;
      const Part w = next.w;
      const float rs = next.rs;
      __syncwarp();  // every lane is done with the tile before
      *reinterpret_cast<float4*>(stage + kScalesAt + 16 * lane) = next.s;
      *reinterpret_cast<uint2*>(stage + kBiasAt + 8 * lane) = next.b;
      __syncwarp();
      if (t + static_cast<int>(gridDim.x) < total)
        next = fetch<MODE>(p, t + gridDim.x, tc.e, s_mt, s_off, quad, part, lane);
      const bool got = mbar_wait(tfull0 + 8 * acc, static_cast<uint32_t>(ti >> 1) & 1u, abort_flag, kTimeoutNs);
      if (!__all_sync(0xffffffffu, got)) break;
      tc_fence_after_sync();
      const uint32_t tacc = tmem_base + static_cast<uint32_t>(acc * BN) + (static_cast<uint32_t>(quad * 32) << 16);
      epilogue<MODE, ACT>(p, w, tacc, tc.row0, tc.rows, lane, rs, stage);
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
  return 1024 + STAGES * STAGE_BYTES + CTRL_BYTES + NUM_EPI_WARPS * kWarpStage +
         2 * static_cast<size_t>(E + 1) * 4;
}

template <int MODE, int ACT>
cudaError_t launch_mode(const Int8GemmArgs& a, cudaStream_t stream) {
  const bool down = MODE == MODE_DOWN;
  const int K = down ? a.D : a.H;
  const cuuint64_t pitch = static_cast<cuuint64_t>(int8_pitch(K));
  const cuuint64_t N = down ? a.H : 2 * static_cast<cuuint64_t>(a.D), E = a.E;
  constexpr CUtensorMapDataType kU8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  CUtensorMap mapA, mapAh, mapB;
  {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(a.R)};
    const cuuint64_t strides[1] = {pitch};
    const cuuint32_t box[2] = {BK, BM}, half_box[2] = {BK, HALF_ROWS};
    if (!encode_tiled_map(&mapA, kU8, a.A, 2, dims, strides, box) ||
        !encode_tiled_map(&mapAh, kU8, a.A, 2, dims, strides, half_box))
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
  Int8Params p = int8_params(a);
  p.n_tiles = (p.out_cols + (down ? BN : BN / 2) - 1) / (down ? BN : BN / 2);
  p.num_kb = (K + BK - 1) / BK;
  const cudaError_t err = opt_in_dynamic_smem(reinterpret_cast<const void*>(int8_gemm_kernel<MODE, ACT>),
                                              static_cast<int>(smem_bytes(kMaxExperts)));
  if (err != cudaSuccess) return err;
  const int64_t max_tiles = (static_cast<int64_t>(a.R) / BM + std::min(a.E, a.R)) * p.n_tiles;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(max_tiles, a.num_sms)));
  return launch_pdl(int8_gemm_kernel<MODE, ACT>, grid, dim3(NUM_THREADS), smem_bytes(a.E), stream, mapA, mapAh, mapB, p);
}

// A call of no tokens: only the status words are written.
__global__ void int8_status_kernel(int* status, int down) {
  griddep_wait();  // the previous kernel's results are complete and visible
  griddep_launch_dependents();
  start_status(status, *reinterpret_cast<const int2*>(status), down != 0, false);
}

template <int MODE>
cudaError_t launch_gate_up(const Int8GemmArgs& a, cudaStream_t stream) {
  if (a.activation == MOE_ACT_SILU) return launch_mode<MODE, MOE_ACT_SILU>(a, stream);
  if (a.activation == MOE_ACT_SWIGLUOAI) return launch_mode<MODE, MOE_ACT_SWIGLUOAI>(a, stream);
  return launch_mode<MODE, MOE_ACT_GELU_TANH>(a, stream);
}

}  // namespace

cudaError_t launch_int8_gemm(const Int8GemmArgs& a, cudaStream_t stream) {
  if (a.R == 0) return launch_pdl(int8_status_kernel, dim3(1), dim3(1), 0, stream, a.status, a.down);
  // Few rows per expert go to the kernel with the operands exchanged
  // (int8_few.cu): on one B200, 2 rows per expert (E 135, K 64, 8848 columns) 104 us
  // here, 28 there; 24 rows (E 49, K 72) 18.8, 12.6; 64 rows (E 123, K 208) 107, 97;
  // 80 rows (E 32, K 1024) 32.3, 32.4; 96 rows (E 128, K 2048) 70, 71; 128 rows (E 18,
  // K 344) 21, 26.  So does what this one's 256-column tiles would leave half of the
  // SMs idle with, in 128-column tiles (4 experts, 93 rows, K 6984: 39 us here, 22 there).
  const int64_t experts = std::min(a.E, a.R), columns = a.down ? a.H : 2 * static_cast<int64_t>(a.D);
  const int64_t tiles = (a.R / BM + experts) * ((columns + BN - 1) / BN);
  if (2 * tiles <= a.num_sms) return launch_int8_few(a, 128, stream);
  if (a.R <= 80 * experts) return launch_int8_few(a, 256, stream);
  if (a.down) return launch_mode<MODE_DOWN, MOE_ACT_SILU>(a, stream);  // (no activation)
  return a.gate_up_format == 0 ? launch_gate_up<MODE_CONCAT>(a, stream) : launch_gate_up<MODE_INTERLEAVED>(a, stream);
}

}  // namespace moe
