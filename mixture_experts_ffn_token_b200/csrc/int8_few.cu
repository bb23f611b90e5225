// int8_few.cu -- the experts' products in 8-bit integers when an expert has few
// rows (int8_gemm.cu has the many): the same products, bit for bit, with the
// operands exchanged.  The weights' columns lie along the MMA's M side (TMEM
// lanes) and the rows along N, rounded up to 16, so that neither the tensor
// cores nor the epilogue work on rows that are not there: with the rows on the M
// side a tile of 2 rows costs the epilogue as much as one of 64.
//
// Tiles are `wc` weight columns (256, or 128 where that leaves SMs without a
// tile) by up to 128 rows.  Roles are those of int8_gemm.cu; a stage holds wc x
// 128 B of W and the rows that a tile can have (16 to 128, from R) by 128 B, of
// which the smallest box that holds the tile's is copied.  Where even 128-column
// tiles leave SMs idle, the CTAs of a cluster share a tile's K.
//
// What bounds it, on one B200 (6.56 TB/s copy rate), the rows' quantiser included:
// the weights' stream (E 64, K 4096, 2 x 1536 columns, 256 rows in 124 us, 6.5
// TB/s; K 1536, 4096 columns in 53.3 us, of which about 3 are start-up and 1.4 the
// seventh wave of 6.8; one token to 8 of those experts 12.5 us, 7.7 at the copy
// rate); with few tiles the chain of stages in one SM, 0.15 us for each 128 of K
// (one row of K 7168: 17.3 us by one SM, 9.6 by clusters of eight); with a short K
// the epilogue's latency (E 135, K 64, 8848 columns, 2 rows per expert: 27.7 us,
// 0.9 a tile and SM).
//
// For gate_up a gate and its up column have to meet in one warp: interleaved
// columns are neighbours, and concatenated ones are copied in groups of 8 gate
// and 8 up columns (a {K, 8, 2, D/8, E} view of W), so they are 8 lanes apart.
// Two rows at a time, the gate lane finishes the first and the up lane the
// second.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>

#include "int8_common.cuh"

namespace moe {
namespace {

constexpr int BK = 128;       // K per stage: one 128-byte swizzle row
constexpr int NUM_EPI_WARPS = 8;
constexpr int NUM_THREADS = 64 + 32 * NUM_EPI_WARPS;
constexpr int CTRL_BYTES = 512;
constexpr int RING_BYTES = 192 * 1024;
constexpr int MAX_STAGES = 10;
constexpr int AHEAD_BYTES = 128 * 1024;
constexpr int BR = 128;                     // rows of a tile
constexpr int MMA_COLS = 128;               // weight columns of an MMA (its M)
constexpr uint32_t TMEM_COLS = 2 * 2 * BR;  // two accumulators of at most two MMAs

struct FewParams {
  Int8Params g;
  int wc;       // weight columns of a tile
  int blocks;   // MMAs across them
  int cap;      // rows of a stage: 16, 32, 64 or 128, whatever holds a tile's
  int stages;
  int split;    // CTAs of a cluster that share a tile's K
  int ahead;    // weight boxes fetched to L2 before the kernels before are done
};

// Stores v[0..N) -- this lane's column at N rows, the rows of two lanes `d`
// apart being the same -- as pairs of columns: of two rows the even lane of a
// pair stores the first and the odd lane the second, four bytes each.  `odd`:
// this lane holds the second column.  row(i) is the tile row of v[i], or -1.
template <int N, typename Row>
__device__ __forceinline__ void store_pairs(const float (&v)[N], bool odd, int d, __nv_bfloat16* out, int64_t stride,
                                            int col, bool in, Row row) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float other = __shfl_xor_sync(0xffffffffu, odd ? v[i] : v[i + 1], d);
    const int r = row(odd ? i + 1 : i);
    const uint32_t word = odd ? pack_bf16x2(other, v[i + 1]) : pack_bf16x2(v[i], other);
    if (in && r >= 0) *reinterpret_cast<uint32_t*>(out + r * stride + (odd ? col - 1 : col)) = word;
  }
}

// The first NR rows of `a`, from their integer sums: `scales` holds the rows' and
// `ws` this lane's column's, `out` is the first row's, `left` how many rows there are.
template <int MODE, int ACT, int NR>
__device__ __forceinline__ void finish_some(const Int8Params& g, const uint32_t (&a)[16], const float* scales, float ws,
                                            float bias, int lane, __nv_bfloat16* out, int col, int left) {
  constexpr int kMate = MODE == MODE_CONCAT ? 8 : 1;  // lanes between a gate and its up column
  const bool is_up = MODE != MODE_DOWN && (lane & kMate) != 0;
  const bool in = col < g.out_cols;
  const int64_t stride = g.out_cols;
  float v[NR];
#pragma unroll
  for (int i = 0; i < NR; i += 4) {
    const float4 rs = *reinterpret_cast<const float4*>(scales + i);
    v[i] = int8_scaled(a[i], rs.x, ws, bias);
    v[i + 1] = int8_scaled(a[i + 1], rs.y, ws, bias);
    v[i + 2] = int8_scaled(a[i + 2], rs.z, ws, bias);
    v[i + 3] = int8_scaled(a[i + 3], rs.w, ws, bias);
  }
  if constexpr (MODE == MODE_DOWN) {
    store_pairs(v, (lane & 1) != 0, 1, out, stride, col, in, [&](int i) { return i < left ? i : -1; });
  } else {
    float h[NR / 2];  // of rows 2i (gate lane) or 2i + 1 (up lane)
#pragma unroll
    for (int i = 0; i < NR / 2; ++i) {
      const float other = __shfl_xor_sync(0xffffffffu, is_up ? v[2 * i] : v[2 * i + 1], kMate);
      h[i] = is_up ? gated<ACT>(other, v[2 * i + 1], g.alpha, g.limit) : gated<ACT>(v[2 * i], other, g.alpha, g.limit);
    }
    constexpr int kNext = MODE == MODE_CONCAT ? 1 : 2;  // lanes between neighbouring h columns
    store_pairs(h, (lane & kNext) != 0, kNext, out, stride, col, in, [&](int i) {
      const int r = 2 * i + (is_up ? 1 : 0);
      return r < left ? r : -1;
    });
  }
}

// 16 rows of a tile, or the first four of a tile that has no more (E 135, K 64, 2
// rows per expert: 39.2 -> 37.0 us; the last few rows of longer tiles stay with
// the others, since taking both ways in turn costs more than it saves).
template <int MODE, int ACT>
__device__ __forceinline__ void finish_rows(const Int8Params& g, const uint32_t (&a)[16], const float* scales, float ws,
                                            float bias, int lane, __nv_bfloat16* out, int col, int left, bool few) {
  if (few) finish_some<MODE, ACT, 4>(g, a, scales, ws, bias, lane, out, col, left);
  else finish_some<MODE, ACT, 16>(g, a, scales, ws, bias, lane, out, col, left);
}

// SPLIT: a cluster of `split` CTAs shares each tile's K, one tile a cluster (128
// columns).  Each leaves its integer sums in shared memory, in the ring that is
// then done with, and CTA q finishes every split-th 16 rows from q on with the
// sums of all: they are whole numbers, so the results are the same bits.
template <int MODE, int ACT, bool SPLIT>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    int8_few_kernel(const __grid_constant__ CUtensorMap mapA16, const __grid_constant__ CUtensorMap mapA32,
                    const __grid_constant__ CUtensorMap mapA64, const __grid_constant__ CUtensorMap mapA128,
                    const __grid_constant__ CUtensorMap mapB, const FewParams p) {
  extern __shared__ uint8_t smem_raw[];
  // (by an offset, so that the compiler still knows it for shared memory)
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  uint8_t* ctrl = smem + RING_BYTES;
  const uint32_t full0 = smem_u32(ctrl);            // MAX_STAGES mbarriers
  const uint32_t empty0 = full0 + 8 * MAX_STAGES;   // MAX_STAGES mbarriers
  const uint32_t tfull0 = empty0 + 8 * MAX_STAGES;  // 2 mbarriers
  const uint32_t tempty0 = tfull0 + 16;             // 2 mbarriers
  const uint32_t drain_bar = tempty0 + 16;          // 1 mbarrier
  static_assert((2 * MAX_STAGES + 5) * 8 <= 256, "mbarriers overflow their part of the control block");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 256);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctrl + 260);
  int* bad_flag = reinterpret_cast<int*>(ctrl + 264);
  float* s_scales = reinterpret_cast<float*>(ctrl + CTRL_BYTES);  // [NUM_EPI_WARPS][BR]
  int* s_off = reinterpret_cast<int*>(s_scales + NUM_EPI_WARPS * BR);
  int* s_mt = s_off + (p.g.E + 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // this CTA's tiles and its part of their K
  const int rank = SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
  const int first = SPLIT ? static_cast<int>(blockIdx.x) / p.split : static_cast<int>(blockIdx.x);
  const int step = SPLIT ? static_cast<int>(gridDim.x) / p.split : static_cast<int>(gridDim.x);
  const int kb0 = SPLIT ? p.g.num_kb * rank / p.split : 0;
  const int kb1 = SPLIT ? p.g.num_kb * (rank + 1) / p.split : p.g.num_kb;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
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
    tma_prefetch_map(&mapB);
    tma_prefetch_map(&mapA16);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  int2 before;
  const int pieces = csr_pieces(p.g, s_off, s_mt, bad_flag, BR, before, [&]() {
    if (first >= s_mt[p.g.E] * p.g.n_tiles) return;
    const TileCoord tc = warp_tile(first, 0, p.g.n_tiles, p.g.E, s_mt, s_off, BR);
    for (int kb = kb0 + lane; kb < min(kb1, kb0 + p.ahead); kb += 32) {
      if constexpr (MODE == MODE_CONCAT) tma_prefetch_5d(&mapB, kb * BK, 0, 0, tc.n * (p.wc / 16), tc.e);
      else tma_prefetch_3d(&mapB, kb * BK, tc.n * p.wc, tc.e);
    }
  });
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  const int total = pieces * p.g.n_tiles;
  const int w_bytes = p.wc * BK, stage_bytes = w_bytes + p.cap * BK;

  // Both single-thread roles run as whole warps of which one lane issues: then
  // the loops' values are uniform.
  if (warp == 0) {
    // ---------------------------------------------------- TMA producer
    int it = 0, s = 0, e = 0;
    uint32_t ph = 0;
    bool ok = true;
    const bool leader = elect_one();
    for (int t = first; ok && t < total; t += step) {
      const TileCoord tc = warp_tile(t, e, p.g.n_tiles, p.g.E, s_mt, s_off, BR);
      e = tc.e;
      // the smallest box that holds the rows
      const int rows = tc.rows <= 16 ? 16 : tc.rows <= 32 ? 32 : tc.rows <= 64 ? 64 : 128;
      const CUtensorMap* ma = rows == 16 ? &mapA16 : rows == 32 ? &mapA32 : rows == 64 ? &mapA64 : &mapA128;
      const uint32_t bytes = static_cast<uint32_t>(w_bytes + rows * BK);
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        if (!__all_sync(0xffffffffu, mbar_wait(empty0 + 8 * s, ph ^ 1u, abort_flag, kTimeoutNs))) {
          ok = false;
          break;
        }
        if (leader) {
          const uint32_t sw = sbase + s * stage_bytes, fb = full0 + 8 * s;
          mbar_arrive_expect_tx(fb, bytes);
          if constexpr (MODE == MODE_CONCAT) tma_load_5d(sw, &mapB, fb, kb * BK, 0, 0, tc.n * (p.wc / 16), tc.e);
          else tma_load_3d(sw, &mapB, fb, kb * BK, tc.n * p.wc, tc.e);
          tma_load_2d(sw + w_bytes, ma, fb, kb * BK, tc.row0);
        }
        __syncwarp();
        if (++s == p.stages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    if (ok) {
      // wait until the MMAs have released every stage, so that no commit
      // arrival lands after this CTA exits
      for (int i = 0; i < p.stages; ++i) {
        if (!mbar_wait(empty0 + 8 * s, ph ^ 1u, abort_flag, kTimeoutNs)) break;
        if (++s == p.stages) {
          s = 0;
          ph ^= 1u;
        }
      }
    } else {
      // aborted: let the copies already issued land before shared memory is
      // released (time-bounded, independent of the abort flag)
      for (int i = 0; i < p.stages; ++i) {
        if (it > i) {
          const int last = i + ((it - 1 - i) / p.stages) * p.stages;
          wait_time_only(full0 + 8 * i, static_cast<uint32_t>(last / p.stages) & 1u);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA issuer
    int s = 0, ti = 0, e = 0;
    uint32_t ph = 0;
    bool ok = true;
    const bool leader = elect_one();
    for (int t = first; ok && t < total; t += step, ++ti) {
      const int acc = ti & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(tempty0 + 8 * acc, (static_cast<uint32_t>(ti >> 1) & 1u) ^ 1u, abort_flag,
                                             kTimeoutNs))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * 2 * BR);
      const TileCoord tc = warp_tile(t, e, p.g.n_tiles, p.g.E, s_mt, s_off, BR);
      e = tc.e;
      const uint32_t idesc = idesc_s8_s32(MMA_COLS, (tc.rows + 15) & ~15);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!__all_sync(0xffffffffu, mbar_wait(full0 + 8 * s, ph, abort_flag, kTimeoutNs))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        if (leader) {
          const uint32_t w_lo = desc_lo(sbase + s * stage_bytes), r_lo = w_lo + (w_bytes >> 4);
          mma_i8_stage(d_tmem, w_lo, r_lo, idesc, kb == kb0);
          if (p.blocks == 2) mma_i8_stage(d_tmem + BR, w_lo + MMA_COLS * BK / 16, r_lo, idesc, kb == kb0);
          mma_commit(empty0 + 8 * s);
        }
        __syncwarp();
        if (++s == p.stages) {
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
  }

  // ---------------------------------------------------------- epilogue
  if (warp >= 2) {
    const int quad = warp & 3;         // this warp may access TMEM lanes 32*quad..+31
    const int part = (warp - 2) >> 2;  // two blocks: the block; one: every other 16 rows
    float* scales = s_scales + (warp - 2) * BR;
    const int block = p.blocks == 2 ? part : 0;
    const int wrow = block * MMA_COLS + quad * 32 + lane;  // this lane's weight column within the tile
    constexpr int kMate = MODE == MODE_CONCAT ? 8 : 1;  // lanes between a gate and its up column
    const bool is_up = MODE != MODE_DOWN && (lane & kMate) != 0;
    // What a tile's epilogue needs from memory: fetched a tile ahead, since the
    // scales come from HBM and a tile of few rows takes less than their latency.
    struct Ahead {
      TileCoord tc;
      int col;               // this lane's output column
      float ws, bias;        // and its column of W's
      float rs[BR / 32];     // scales of rows lane, lane + 32, ...
    };
    auto fetch = [&](int t, int from) {
      Ahead f;
      f.tc = warp_tile(t, from, p.g.n_tiles, p.g.E, s_mt, s_off, BR);
      int wcol;
      if constexpr (MODE == MODE_CONCAT) {
        f.col = f.tc.n * (p.wc / 2) + (wrow >> 4) * 8 + (wrow & 7);
        wcol = (is_up ? p.g.out_cols : 0) + f.col;
      } else {
        wcol = f.tc.n * p.wc + wrow;
        f.col = MODE == MODE_INTERLEAVED ? wcol >> 1 : wcol;
      }
      f.ws = f.bias = 0.f;
      if (f.col < p.g.out_cols) {
        const int64_t at = static_cast<int64_t>(f.tc.e) * p.g.N + wcol;
        f.ws = __ldg(p.g.w_scales + at);
        if (p.g.bias != nullptr) f.bias = __bfloat162float(p.g.bias[at]);
      }
#pragma unroll
      for (int i = 0; i < BR / 32; ++i) {
        const int r = lane + 32 * i;
        f.rs[i] = r < f.tc.rows ? __ldg(p.g.a_scales + f.tc.row0 + r) : 0.f;
      }
      return f;
    };
    Ahead next = {};
    if (first < total) next = fetch(first, 0);
    if (keeps_status()) start_status(p.g.status, before, MODE == MODE_DOWN, *bad_flag != 0);
    if constexpr (SPLIT) {
      const TileCoord tc = next.tc;
#pragma unroll
      for (int i = 0; i < BR / 32; ++i) scales[lane + 32 * i] = next.rs[i];
      __syncwarp();
      const bool got = first < total && __all_sync(0xffffffffu, mbar_wait(tfull0, 0, abort_flag, kTimeoutNs));
      tc_fence_after_sync();
      const uint32_t tacc = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
      // rows r0 .. r0 + 15 of the CTAs' sums, four rows of a column together (the
      // copies and products that used this memory are complete: tfull)
      const uint32_t mine = sbase + static_cast<uint32_t>(quad * 32 + lane) * 16;
      constexpr uint32_t kFour = MMA_COLS * 16;
      if (got) {
        for (int r0 = 16 * part; r0 < tc.rows; r0 += 32) {
          if (((r0 >> 4) & (p.split - 1)) == rank) continue;
          uint32_t a[16];
          tmem_ld16(tacc + static_cast<uint32_t>(r0), a);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 4; ++i)
            st_shared_v4(mine + (r0 / 4 + i) * kFour, make_uint4(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]));
        }
      }
      __syncwarp();
      cluster_sync();
      if (got) {
        for (int r0 = 16 * part; r0 < tc.rows; r0 += 32) {
          if (((r0 >> 4) & (p.split - 1)) != rank) continue;
          uint32_t a[16];
          tmem_ld16(tacc + static_cast<uint32_t>(r0), a);
          tmem_ld_wait();
          for (int q0 = 1; q0 < p.split; q0 += 4) {  // four CTAs' loads in flight
            uint4 b[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t from = map_to_rank(mine, static_cast<uint32_t>((rank + q0 + j) & (p.split - 1)));
#pragma unroll
              for (int i = 0; i < 4; ++i)
                b[j][i] = q0 + j < p.split ? ld_cluster_v4(from + (r0 / 4 + i) * kFour) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                a[4 * i] += b[j][i].x;
                a[4 * i + 1] += b[j][i].y;
                a[4 * i + 2] += b[j][i].z;
                a[4 * i + 3] += b[j][i].w;
              }
          }
          finish_rows<MODE, ACT>(p.g, a, scales + r0, next.ws, next.bias, lane,
                                 p.g.out + (static_cast<int64_t>(tc.row0) + r0) * p.g.out_cols, next.col, tc.rows - r0,
                                 tc.rows <= 4);
        }
      }
      tc_fence_before_sync();
    }
    int ti = 0;
    for (int t = first; !SPLIT && t < total; t += step, ++ti) {
      const TileCoord tc = next.tc;
      const int acc = ti & 1, col = next.col;
      const float ws = next.ws, bias = next.bias;
      __syncwarp();  // every lane is done with the tile before
#pragma unroll
      for (int i = 0; i < BR / 32; ++i) scales[lane + 32 * i] = next.rs[i];
      __syncwarp();
      if (t + step < total) next = fetch(t + step, tc.e);
      const bool got = mbar_wait(tfull0 + 8 * acc, static_cast<uint32_t>(ti >> 1) & 1u, abort_flag, kTimeoutNs);
      if (!__all_sync(0xffffffffu, got)) break;
      tc_fence_after_sync();
      const uint32_t tacc = tmem_base + static_cast<uint32_t>((acc * 2 + block) * BR) +
                            (static_cast<uint32_t>(quad * 32) << 16);
      __nv_bfloat16* out = p.g.out + static_cast<int64_t>(tc.row0) * p.g.out_cols;
      const int r_step = p.blocks == 2 ? 16 : 32;
#pragma unroll 1
      for (int r0 = p.blocks == 2 ? 0 : 16 * part; r0 < tc.rows; r0 += r_step) {
        uint32_t a[16];
        tmem_ld16(tacc + static_cast<uint32_t>(r0), a);
        tmem_ld_wait();
        finish_rows<MODE, ACT>(p.g, a, scales + r0, ws, bias, lane, out + static_cast<int64_t>(r0) * p.g.out_cols, col,
                               tc.rows - r0, tc.rows <= 4);
      }
      tc_fence_before_sync();
      mbar_arrive(tempty0 + 8 * acc);
    }
  }

  __syncwarp();
  if constexpr (SPLIT) {
    if (warp < 2) cluster_sync();  // (the epilogue's, between leaving the sums and reading them)
    cluster_sync();                // the others have read this CTA's sums
  }
  __syncthreads();
  griddep_launch_dependents();  // this CTA has no tiles left: the next kernel may begin launching
  if (threadIdx.x == 0 && *abort_flag) atomicOr(p.g.status, p.g.err_bit);
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

constexpr size_t smem_bytes(int E) {
  return 1024 + RING_BYTES + CTRL_BYTES + NUM_EPI_WARPS * BR * 4 + 2 * static_cast<size_t>(E + 1) * 4;
}

// K is split where the tiles leave SMs idle: by the largest power of two up to 8
// that finds SMs for all (clusters of 4 and 8 fit within groups of SMs, so some
// stay out) and leaves four stages to each.
int k_split(int64_t tiles, int num_kb, int num_sms) {
  int split = 1;
  while (split < 8 && tiles * 2 * split <= (split == 1 ? num_sms : num_sms * 7 / 8) && num_kb >= 8 * split) split *= 2;
  return split;
}

template <int MODE, int ACT>
cudaError_t launch_mode(const Int8GemmArgs& a, int wc, cudaStream_t stream) {
  const bool down = MODE == MODE_DOWN;
  const int K = down ? a.D : a.H;
  const cuuint64_t pitch = static_cast<cuuint64_t>(int8_pitch(K));
  const cuuint64_t N = down ? a.H : 2 * static_cast<cuuint64_t>(a.D), E = a.E;
  constexpr CUtensorMapDataType kU8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  // a tile has at most R rows: one token's few rows leave room for more stages,
  // and need fewer maps
  const int cap = a.R <= 16 ? 16 : a.R <= 32 ? 32 : a.R <= 64 ? 64 : BR;
  CUtensorMap mapA[4], mapB;
  for (int i = 0; i < 4; ++i) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(a.R)};
    const cuuint64_t strides[1] = {pitch};
    const cuuint32_t box[2] = {BK, 16u << i};
    if ((16 << i) > cap) mapA[i] = mapA[i - 1];  // (no tile asks for it)
    else if (!encode_tiled_map(&mapA[i], kU8, a.A, 2, dims, strides, box)) return cudaErrorInvalidValue;
  }
  if (MODE == MODE_CONCAT) {
    const cuuint64_t D = a.D;
    const cuuint64_t dims[5] = {static_cast<cuuint64_t>(K), 8, 2, D / 8, E};
    const cuuint64_t strides[4] = {pitch, D * pitch, 8 * pitch, N * pitch};
    const cuuint32_t box[5] = {BK, 8, 2, static_cast<cuuint32_t>(wc / 16), 1};
    if (!encode_tiled_map(&mapB, kU8, a.W, 5, dims, strides, box)) return cudaErrorInvalidValue;
  } else {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(K), N, E};
    const cuuint64_t strides[2] = {pitch, N * pitch};
    const cuuint32_t box[3] = {BK, static_cast<cuuint32_t>(wc), 1};
    if (!encode_tiled_map(&mapB, kU8, a.W, 3, dims, strides, box)) return cudaErrorInvalidValue;
  }
  FewParams p;
  p.g = int8_params(a);
  const int tile_cols = down ? wc : wc / 2;
  p.g.n_tiles = (p.g.out_cols + tile_cols - 1) / tile_cols;
  p.g.num_kb = (K + BK - 1) / BK;
  p.wc = wc;
  p.blocks = wc / MMA_COLS;
  p.cap = cap;
  p.stages = std::min(MAX_STAGES, RING_BYTES / ((wc + p.cap) * BK));
  p.ahead = std::min(p.g.num_kb, AHEAD_BYTES / (wc * BK));
  const int64_t max_tiles = (static_cast<int64_t>(a.R) / BR + std::min(a.E, a.R)) * p.g.n_tiles;
  p.split = wc == MMA_COLS ? k_split(max_tiles, p.g.num_kb, a.num_sms) : 1;
  const auto kernel = p.split > 1 ? int8_few_kernel<MODE, ACT, true> : int8_few_kernel<MODE, ACT, false>;
  const cudaError_t err =
      opt_in_dynamic_smem(reinterpret_cast<const void*>(kernel), static_cast<int>(smem_bytes(kMaxExperts)));
  if (err != cudaSuccess) return err;
  // (a cluster has one tile at most)
  const int64_t ctas = p.split > 1 ? max_tiles * p.split : std::min<int64_t>(max_tiles, a.num_sms);
  return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(ctas)), dim3(NUM_THREADS), p.split, smem_bytes(a.E), stream,
                            mapA[0], mapA[1], mapA[2], mapA[3], mapB, p);
}

template <int MODE>
cudaError_t launch_gate_up(const Int8GemmArgs& a, int wc, cudaStream_t stream) {
  if (a.activation == MOE_ACT_SILU) return launch_mode<MODE, MOE_ACT_SILU>(a, wc, stream);
  if (a.activation == MOE_ACT_SWIGLUOAI) return launch_mode<MODE, MOE_ACT_SWIGLUOAI>(a, wc, stream);
  return launch_mode<MODE, MOE_ACT_GELU_TANH>(a, wc, stream);
}

}  // namespace

cudaError_t launch_int8_few(const Int8GemmArgs& a, int wc, cudaStream_t stream) {
  if (a.down) return launch_mode<MODE_DOWN, MOE_ACT_SILU>(a, wc, stream);  // (no activation)
  return a.gate_up_format == 0 ? launch_gate_up<MODE_CONCAT>(a, wc, stream)
                               : launch_gate_up<MODE_INTERLEAVED>(a, wc, stream);
}

}  // namespace moe
