// kernels.cuh -- launchers of the sm_100a kernels, called by the C ABI
// (moe_api.cu).  Every launcher only enqueues work on `stream` and returns
// the launch status.
#pragma once

#include "common.cuh"

namespace moe {

// Runtime switches (environment variables, all optional):
//   MOE_B200_PDL=0             no programmatic dependent launch
//   MOE_B200_PDL_COOP=0        none on the two cooperative launches (CSR build, FFN)
//   MOE_B200_CSR_FUSED=0       the CSR build as three launches
//   MOE_B200_SINGLE_LAUNCH=0   the two grouped GEMMs as two launches
//   MOE_B200_CTA_PAIR=2        CTA-pair GEMM tiles (single launch unless
//                              MOE_B200_SINGLE_LAUNCH=0)
//   MOE_B200_PAIR_COOP=0       the single-launch pair without the cooperative
//                              attribute (its grid still comes from the
//                              cluster occupancy query; if some cluster is not
//                              resident, the bounded dependency waits report
//                              a timeout instead of hanging)
//   MOE_B200_B_ONE_BOX=0       four copies per B stage tile
//   MOE_B200_TILE_SCHEDULE=static|dynamic   tile order of the single launch
//   MOE_B200_FUSED_GATHER=1    the gate_up GEMM gathers its rows of x itself
//   MOE_B200_TEST_STALL_DOWN_TILES_MS, MOE_B200_TEST_STALL_CSR_MS   test hooks
//                              that make a bounded wait run out (see the kernels)
// Every API call takes one snapshot of them (refresh_switches) for all of
// its launches; switches() returns the calling thread's snapshot.
struct Switches {
  bool pdl = true;
  bool csr_fused = true;
  long test_stall_csr_ms = 0;
  bool fused_gather = false;
  bool b_one_box = true;
  int cta_pair = 1;
  long test_stall_down_ms = 0;
  char tile_schedule = 0;  // 's', 'd', or 0 (chosen by rows per expert)
  bool single_launch = true;
  bool pdl_coop = true;
  bool pair_coop = true;
};
void refresh_switches();
const Switches& switches();

// Launches `kernel` on `stream`, allowing it to overlap the tail of the
// kernel before it (programmatic dependent launch) unless
// MOE_B200_PDL=0; every kernel of this library calls griddep_wait() before
// touching global memory, so the overlap never changes what it reads.
bool pdl_enabled();

// Raises the dynamic shared-memory limit of kernel `func` to `bytes` on the
// current device the first time it is asked for that (device, kernel); once
// that has succeeded, later calls return without calling the runtime.  Every
// caller passes the kernel's largest possible size, so one opt-in serves all
// launches.  Thread-safe.
cudaError_t opt_in_dynamic_smem(const void* func, int bytes);

// The same with clusters of `cluster` blocks (1: none).
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, int cluster, size_t smem,
                                      cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (pdl_enabled()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                              Args... args) {
  return launch_pdl_cluster(kernel, grid, block, 1, smem, stream, args...);
}

// ------------------------------------------------------------------ router
struct RouterArgs {
  const void* logits;
  int logits_bf16;
  int64_t stride;
  int T, E, k, S;
  int sink;                  // 0 softmax top-k, 1 sigmoid + sink lanes
  const float* expert_bias;  // [E] or null
  const float* global_scale; // device [1] or null
  float route_scale;
  int32_t* idx;              // [T,k]
  float* w;                  // [T,k]
  float* sink_w;             // [T,S] or null
  int* status_reset;         // status_reset[0] (status) and [1] (CSR grid barrier) zeroed by the first thread, or null
};
cudaError_t launch_router(const RouterArgs& a, cudaStream_t stream);

// Routing plus the whole CSR build (offsets, permutation) in one CTA, for
// problems with at most kSmallSlots routed slots and kSmallExperts experts.
constexpr int kSmallWarps = 32;
constexpr int kSmallSlots = 2048;
constexpr int kSmallExperts = 512;
cudaError_t launch_route_csr_small(const RouterArgs& a, int32_t* offsets, int32_t* perm, int* status,
                                   const uint8_t* mask, cudaStream_t stream);

// ---------------------------------------------------------------------- CSR
constexpr int kCsrChunk = 2048;      // slots per CTA
constexpr int kCsrThreads = 512;     // 16 warps x 128 slots
inline int csr_num_chunks(int64_t R) { return static_cast<int>((R + kCsrChunk - 1) / kCsrChunk); }
// mask (may be null): slots of tokens whose mask byte is 0 take no place.
cudaError_t launch_csr_count(const int32_t* idx, int R, int E, int32_t* chunk_counts, int* status,
                             const uint8_t* mask, int k, cudaStream_t stream);
cudaError_t launch_csr_scan(const int32_t* chunk_counts, int nchunks, int E, int32_t* chunk_base,
                            int32_t* offsets, cudaStream_t stream);
cudaError_t launch_csr_scatter(const int32_t* idx, int R, int E, const int32_t* chunk_base, int32_t* perm,
                               int32_t* inv, const uint8_t* mask, int k, cudaStream_t stream);
// The three CSR kernels as one cooperative launch (one CTA per chunk), used
// when the chunks fit on the GPU at once (csr_num_chunks(R) <= num_sms) unless
// MOE_B200_CSR_FUSED=0; *barrier must be zero at launch.
bool csr_fused_enabled(int R, int num_sms);
cudaError_t launch_csr_fused(const int32_t* idx, int R, int E, int32_t* chunk_counts, int32_t* offsets, int32_t* perm,
                             int32_t* inv, int* status, int* barrier, const uint8_t* mask, int k,
                             cudaStream_t stream);
// shared slots: offsets[i] = i*T, perm[i*T + t] = t*Ns + i; also clears
// zero[0 .. n_zero) (may be null / 0).
cudaError_t launch_shared_index(int T, int Ns, int32_t* offsets, int32_t* perm, int num_sms, cudaStream_t stream,
                                int* zero = nullptr, int n_zero = 0);

// ----------------------------------------------------- gather and combine
// scale (may be null): per-slot factor applied to the gathered row.
// zero[0 .. n_zero) (may be null / 0) is cleared by the same launch.
cudaError_t launch_gather(const __nv_bfloat16* x, const int32_t* perm, const int32_t* offsets, int E, int R,
                          int k, int H, const float* scale, __nv_bfloat16* Xp, int* status, int num_sms,
                          cudaStream_t stream, int* zero = nullptr, int n_zero = 0);
// Ys (may be null, Ns = 0): shared-expert rows added after the routed ones;
// mask (may be null): masked tokens get zero rows.
cudaError_t launch_combine(const __nv_bfloat16* Y, int T, int H, int k, const __nv_bfloat16* Ys, int Ns,
                           const uint8_t* mask, __nv_bfloat16* out, int num_sms, cudaStream_t stream);

// ------------------------------------------------------------ grouped GEMM
struct GroupedGemmArgs {
  // routing (device)
  const int32_t* offsets;   // [E+1]
  const int32_t* perm;      // [R]
  const float* weights;     // [R] routing weight per slot (down GEMM), or null for 1
  int E, R, T, k;
  // problem
  int H, D;
  int gate_up_format;       // 0 concatenated, 1 interleaved
  int activation;           // 0 silu, 1 swigluoai, 2 gelu_tanh
  float alpha, limit;
  // operands (device)
  const __nv_bfloat16* A;   // Xp [R,H] (gate_up) or h [R,D] (down)
  // gate_up only: A is x [T,H] itself and a slot's A row is its row within
  // its expert's segment (the shared experts' slots, token order per expert)
  int a_direct = 0;
  // gate_up only: A is x [T,H] and the kernel gathers each tile's rows by the
  // permutation itself (token = perm[p] / k); no Xp is read
  int gather = 0;
  const __nv_bfloat16* W;   // [E,H,2D] (gate_up) or [E,D,H] (down)
  const __nv_bfloat16* bias;// [E,2D] / [E,H] or null
  __nv_bfloat16* out;       // h [R,D] (gate_up) or Y [R,H] slot rows (down)
  int* status;
  int num_sms;
};
cudaError_t launch_gemm_gate_up(const GroupedGemmArgs& a, cudaStream_t stream);
cudaError_t launch_gemm_down(const GroupedGemmArgs& a, cudaStream_t stream);

// Both contractions in one persistent cooperative launch: `up` describes the
// gate_up GEMM (A = Xp, out = h) and `down` the down GEMM (A = h, out = Y,
// which must not alias Xp).  A down tile of a 128-row piece waits (bounded)
// until every gate_up tile of that piece has stored its h columns, counted
// in arrivals[piece]; the counters must be zero at launch (launch_gather
// clears them) and hold at least mega_ffn_counters(R, E) entries: one per
// possible 128-row piece, and last the tile scheduler's counter.
int mega_ffn_counters(int R, int E);
cudaError_t launch_mega_ffn(const GroupedGemmArgs& up, const GroupedGemmArgs& down, int* arrivals,
                            cudaStream_t stream);

// Encodes a 128-byte-swizzled tensor map of `rank` dimensions; strides in bytes, from the second dimension on.
bool encode_tiled_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int rank, const cuuint64_t* dims,
                      const cuuint64_t* strides_bytes, const cuuint32_t* box);

// Resolves cuTensorMapEncodeTiled through the runtime (no libcuda link).
bool tensor_map_encoder_available();

// Whether the gate_up GEMM gathers its rows of x itself in this process
// (MOE_B200_FUSED_GATHER=1 with single-CTA tiles; off by default).
bool fused_gather_enabled();

// ------------------------------------ tokens sorted by expert and back
// Rows are `vec` 16-byte vectors.  spread: rows_out[p] = w * tok_in[t]; gather:
// tok_out[t] = sum_j w * rows_in[p]; with d_weights (may be null) also
// d_weights[t*k+j] = <tok_in[t], rows_in[p]>.  p = inverse[t*k+j].
struct RowsArgs {
  const void* tok_in;
  void* tok_out;
  const void* rows_in;
  void* rows_out;
  const int32_t* inverse;  // [R]
  const float* weights;    // [R] or null for 1
  float* d_weights;        // [R] or null
  int T, k, R, vec;
  int num_sms;
};
cudaError_t launch_rows_spread(const RowsArgs& a, bool f32, cudaStream_t stream);
cudaError_t launch_rows_gather(const RowsArgs& a, bool f32, cudaStream_t stream);

// ------------------------------------------------------ router gradient
constexpr int kGradMaxBlocks = 1024;
struct RouterGradArgs {
  const void* logits;
  int64_t stride;            // of logits and d_logits
  int T, E, k, S;
  float route_scale;
  const float* global_scale; // device [1] or null
  const int32_t* idx;        // [T,k]
  const float* d_weights;    // [T,k]
  const float* d_sink;       // [T,S] or null for zero
  void* d_logits;            // [T,stride], columns 0 .. E+S-1 written
  double* partial;           // [kGradMaxBlocks] or null: no d_global_scale
  float* d_global_scale;     // [1], with partial
};
cudaError_t launch_route_grad(const RouterGradArgs& a, bool sink, bool bf16, cudaStream_t stream);

// ------------------------------------------------------------ 8-bit experts
// Bytes of a row of n 8-bit values: TMA row strides are multiples of 16.
inline int int8_pitch(int n) { return (n + 15) / 16 * 16; }
// q[p] = the row quantised by its largest magnitude, scales[p] = that / 127,
// for the k positions p of every row (inverse, may be null: p = the row).
// total (may be null): device int, rows from it on are left alone.
cudaError_t launch_quantize_rows(const __nv_bfloat16* in, int rows, int n, const int32_t* inverse, int k, int R,
                                 const int32_t* total, int8_t* q, float* scales, int num_sms, cudaStream_t stream);
// W [E,K,N] bf16 -> q [E,N,int8_pitch(K)], scales [E,N] (per column).
cudaError_t launch_quantize_weights(const __nv_bfloat16* w, int E, int K, int N, int8_t* q, float* scales,
                                    cudaStream_t stream);
struct Int8GemmArgs {
  const int32_t* offsets;    // [E+1]
  int E, R, H, D;
  int down;                  // 0: gate_up with the activation, 1: down
  int gate_up_format;
  int activation;
  float alpha, limit;
  const int8_t* A;           // [R, int8_pitch(K)]
  const float* a_scales;     // [R]
  const int8_t* W;           // [E, N, int8_pitch(K)]
  const float* w_scales;     // [E, N]
  const __nv_bfloat16* bias; // [E, N] or null
  __nv_bfloat16* out;        // [R, D] or [R, H], in sorted order
  int* status;
  int num_sms;
};
cudaError_t launch_int8_gemm(const Int8GemmArgs& a, cudaStream_t stream);
// The same for few rows per expert, in tiles of wc weight columns (256 or 128).
cudaError_t launch_int8_few(const Int8GemmArgs& a, int wc, cudaStream_t stream);

}  // namespace moe
