// int8_quant.cu -- bf16 to 8-bit integers with one scale per token row (or per
// weight column): with m the largest magnitude,  scale = m / 127  and
// q = rint(127 a / m), ties to even, so |q| <= 127 and q * scale is a to
// within half a step.
//
// The rounding is exact although it is one multiply by a rounded reciprocal:
// with 8-bit significands A and M, a / m = A / (M 2^s), a quotient 127 a / m that
// is no tie lies at least 1 / (2 M 2^s) from one, and the reciprocal's error
// moves it by less than 2^-23 of itself, 127 A 2^-23 / (M 2^s), which is under
// 1/128 of that.  The ties are a = m/2 (63.5, to 64) and those of an m whose
// reciprocal times 127 is a power of two (exact).  The reciprocal is rounded up,
// so 63.5 never falls below its tie.
// Bound by HBM: each value read once and each place written once.
// Rows of denormal size are scaled by 2^64 first.  A row that holds an
// infinity or a NaN gets a NaN scale, so that its products are NaN.
#include <algorithm>

#include "kernels.cuh"

namespace moe {
namespace {

// |bf16| pairs compared as integers: the order of their bits is the order of
// their magnitudes, with NaN above infinity above all else.
__device__ __forceinline__ uint32_t absmax2(uint32_t m, uint32_t v) { return __vmaxu2(m, v & 0x7fff7fffu); }
__device__ __forceinline__ uint32_t absmax8(uint32_t m, const uint4& u) {
  return absmax2(absmax2(absmax2(absmax2(m, u.x), u.y), u.z), u.w);
}

struct Quant {
  float pre, inv, scale;
};

// From the bits of the largest magnitude.
__device__ __forceinline__ Quant quant_of(uint32_t bits) {
  const float m = __uint_as_float(bits << 16);
  Quant q;
  q.pre = m < 0x1p-100f ? 0x1p64f : 1.f;
  q.inv = m > 0.f ? __fdiv_ru(127.f, m * q.pre) : 0.f;
  q.scale = bits >= 0x7f80u ? __uint_as_float(0x7fffffffu) : __fdiv_rn(m, 127.f);
  return q;
}

// rint(a * inv) in the low byte: adding 1.5 * 2^23 rounds to an integer.
__device__ __forceinline__ uint32_t q_bits(float a, const Quant& q) {
  return __float_as_uint(fmaf(a * q.pre, q.inv, 12582912.f));
}

__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// 8 bf16 values to 8 bytes.
__device__ __forceinline__ uint2 quant8(const uint4& u, const Quant& q) {
  return make_uint2(
      pack4(q_bits(bf16_lo(u.x), q), q_bits(bf16_hi(u.x), q), q_bits(bf16_lo(u.y), q), q_bits(bf16_hi(u.y), q)),
      pack4(q_bits(bf16_lo(u.z), q), q_bits(bf16_hi(u.z), q), q_bits(bf16_lo(u.w), q), q_bits(bf16_hi(u.w), q)));
}

// 2^g_log threads per row (a warp at least, 256 / 2^g_log rows a block), 16
// values a thread and step; the row stays in registers between the maximum
// and the rounding (up to HELD steps), so it is read once and its k copies
// are written once each.
constexpr int kQuantThreads = 512;

template <int HELD>
__global__ void __launch_bounds__(kQuantThreads) quantize_rows_kernel(const __nv_bfloat16* __restrict__ in, int rows,
                                                                      int n, int g_log,
                                                                      const int32_t* __restrict__ inverse, int k,
                                                                      int R, const int32_t* __restrict__ total,
                                                                      int8_t* __restrict__ q,
                                                                      float* __restrict__ scales) {
  griddep_wait();  // the previous kernel's results are complete and visible
  griddep_launch_dependents();
  const int steps = 1 << g_log, tid = threadIdx.x & (steps - 1), group = threadIdx.x >> g_log;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> g_log) + group;
  const bool live = row < rows && (total == nullptr || row < *total);
  const int chunks = (n + 15) / 16, vec = live ? n / 8 : 0;  // nothing is read of a row that is not live
  const uint4* src = reinterpret_cast<const uint4*>(in + row * n);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 a[HELD], b[HELD];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    const int c = tid + i * steps;
    a[i] = 2 * c < vec ? __ldg(src + 2 * c) : zero;
    b[i] = 2 * c + 1 < vec ? __ldg(src + 2 * c + 1) : zero;
  }
#pragma unroll
  for (int i = 0; i < HELD; ++i) m = absmax8(absmax8(m, a[i]), b[i]);
  for (int c = tid + HELD * steps; 2 * c < vec; c += steps) {
    m = absmax8(m, __ldg(src + 2 * c));
    if (2 * c + 1 < vec) m = absmax8(m, __ldg(src + 2 * c + 1));
  }
  m = max(m & 0xffffu, m >> 16);
  m = __reduce_max_sync(0xffffffffu, m);
  if (steps > 32) {
    __shared__ uint32_t s_max[kQuantThreads / 32];
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
    __syncthreads();
    for (int w = 0; w < (steps >> 5); ++w) m = max(m, s_max[group * (steps >> 5) + w]);
  }
  if (!live) return;
  const Quant qt = quant_of(m);
  const int64_t pitch = 16 * static_cast<int64_t>(chunks);
  auto store = [&](int c, const uint4& va, const uint4& vb) {
    const uint2 lo = quant8(va, qt), hi = quant8(vb, qt);
    uint4 o = make_uint4(lo.x, lo.y, hi.x, hi.y);
    if (2 * c + 1 >= vec) o.z = o.w = 0;  // the padding of the row
    for (int j = 0; j < k; ++j) {
      const int64_t p = inverse != nullptr ? __ldg(inverse + row * k + j) : row;
      if (p >= 0 && p < R) *reinterpret_cast<uint4*>(q + p * pitch + 16 * c) = o;
    }
  };
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    const int c = tid + i * steps;
    if (c < chunks) store(c, a[i], b[i]);
  }
  for (int c = tid + HELD * steps; c < chunks; c += steps)
    store(c, __ldg(src + 2 * c), 2 * c + 1 < vec ? __ldg(src + 2 * c + 1) : zero);
  for (int j = tid; j < k; j += steps) {
    const int64_t p = inverse != nullptr ? inverse[row * k + j] : row;
    if (p >= 0 && p < R) scales[p] = qt.scale;
  }
}

// Weights [E, K, N] bf16 to [E, N, pitch] 8-bit, one scale per column.  A
// block owns 64 columns of one expert: it reads its K x 64 strip for the
// maxima, and again (from L2, mostly) to round it, turning 128 x 64 blocks
// through shared memory so that both sides move whole sectors.  E 8, 4096 x
// 28672 in 737 us, 0.58 of the copy rate: the strips of all blocks together do
// not stay in L2 between the two readings.  One block of 1024 threads a SM,
// whose strips would (936 us), and a cluster that holds its strip in shared
// memory (1176 us) were slower, and this runs once per model.
constexpr int kWCols = 64, kWRows = 128, kWThreads = 256;
constexpr int kWPitch = kWRows + 4;  // bytes; a word stride of 33

__global__ void __launch_bounds__(kWThreads) quantize_weights_kernel(const __nv_bfloat16* __restrict__ w, int K, int N,
                                                                     int strips, int8_t* __restrict__ q,
                                                                     float* __restrict__ scales) {
  griddep_wait();  // the previous kernel's results are complete and visible
  griddep_launch_dependents();
  const int64_t e = blockIdx.x / static_cast<uint32_t>(strips);
  const int n0 = (blockIdx.x - static_cast<uint32_t>(e) * strips) * kWCols;
  const int tid = threadIdx.x;
  const int g = tid & 7, r = tid >> 3;  // this thread's 8 columns, its row of 32
  const int col = n0 + 8 * g;
  const bool in = col < N;  // N is a multiple of 8
  const __nv_bfloat16* src = w + (e * K) * N + col;
  uint32_t m[4] = {0, 0, 0, 0};
  if (in) {
#pragma unroll 4
    for (int k = r; k < K; k += 32) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(src + static_cast<int64_t>(k) * N));
      m[0] = absmax2(m[0], u.x);
      m[1] = absmax2(m[1], u.y);
      m[2] = absmax2(m[2], u.z);
      m[3] = absmax2(m[3], u.w);
    }
  }
  __shared__ uint32_t s_m[32][33];
  __shared__ Quant s_q[kWCols];
  __shared__ __align__(16) uint8_t s_t[kWCols * kWPitch];
#pragma unroll
  for (int i = 0; i < 4; ++i) s_m[r][4 * g + i] = m[i];
  __syncthreads();
  if (tid < 32) {
    uint32_t v = 0;
    for (int i = 0; i < 32; ++i) v = __vmaxu2(v, s_m[i][tid]);
    s_q[2 * tid] = quant_of(v & 0xffffu);
    s_q[2 * tid + 1] = quant_of(v >> 16);
  }
  __syncthreads();
  if (tid < kWCols && n0 + tid < N) scales[e * N + n0 + tid] = s_q[tid].scale;
  const int pitch = (K + 15) / 16 * 16;
  for (int k0 = 0; k0 < K; k0 += kWRows) {
    // four consecutive rows of 8 columns -> one word of each of 8 columns
    uint4 u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = k0 + 4 * r + i;
      u[i] = in && k < K ? __ldg(reinterpret_cast<const uint4*>(src + static_cast<int64_t>(k) * N))
                         : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const Quant qt = s_q[8 * g + c];
      uint32_t b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t word = c < 2 ? u[i].x : c < 4 ? u[i].y : c < 6 ? u[i].z : u[i].w;
        b[i] = q_bits((c & 1) ? bf16_hi(word) : bf16_lo(word), qt);
      }
      *reinterpret_cast<uint32_t*>(s_t + (8 * g + c) * kWPitch + 4 * r) = pack4(b[0], b[1], b[2], b[3]);
    }
    __syncthreads();
    // 64 columns x 8 pieces of 16 bytes along K
#pragma unroll
    for (int i = 0; i < kWCols * 8 / kWThreads; ++i) {
      const int piece = tid + i * kWThreads;
      const int cc = piece >> 3, kk = (piece & 7) * 16;
      if (n0 + cc < N && k0 + kk < pitch) {
        const uint32_t* s = reinterpret_cast<const uint32_t*>(s_t + cc * kWPitch + kk);
        uint4 o = make_uint4(s[0], s[1], s[2], s[3]);
        if (k0 + kk + 8 >= K) o.z = o.w = 0;  // the padding (K is a multiple of 8)
        *reinterpret_cast<uint4*>(q + (e * N + n0 + cc) * pitch + k0 + kk) = o;
      }
    }
    __syncthreads();
  }
}

template <int HELD>
cudaError_t launch_rows(const __nv_bfloat16* in, int rows, int n, const int32_t* inverse, int k, int R,
                        const int32_t* total, int8_t* q, float* scales, cudaStream_t stream) {
  // as many threads as hold the row in registers
  const int chunks = (n + 15) / 16;
  int g_log = 5;
  while ((HELD << g_log) < chunks && (1 << g_log) < kQuantThreads) ++g_log;
  const int threads = std::max(256, 1 << g_log), per_block = threads >> g_log;
  return launch_pdl(quantize_rows_kernel<HELD>, dim3(static_cast<unsigned>((rows + per_block - 1) / per_block)),
                    dim3(static_cast<unsigned>(threads)), 0, stream, in, rows, n, g_log, inverse, k, R, total, q,
                    scales);
}

}  // namespace

cudaError_t launch_quantize_rows(const __nv_bfloat16* in, int rows, int n, const int32_t* inverse, int k, int R,
                                 const int32_t* total, int8_t* q, float* scales, int num_sms, cudaStream_t stream) {
  if (rows == 0) return cudaSuccess;
  // Four steps a thread keep most in flight (8192 rows of 14336: 70.3 us with two, 56.7 with four; of 2880: 17.6,
  // 15.4), two where a warp then holds a short row (49152 of 768: 24.6 us, 29.8 with four), and with few rows one,
  // for the shortest way through (32 rows of 4096 to 8 places: 2.4 us, 3.4 with two, 4.6 with four).
  if (rows <= 2 * num_sms) return launch_rows<1>(in, rows, n, inverse, k, R, total, q, scales, stream);
  if (n <= 1024) return launch_rows<2>(in, rows, n, inverse, k, R, total, q, scales, stream);
  return launch_rows<4>(in, rows, n, inverse, k, R, total, q, scales, stream);
}

cudaError_t launch_quantize_weights(const __nv_bfloat16* w, int E, int K, int N, int8_t* q, float* scales,
                                    cudaStream_t stream) {
  const int strips = (N + kWCols - 1) / kWCols;
  const int64_t blocks = static_cast<int64_t>(E) * strips;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl(quantize_weights_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kWThreads), 0, stream, w, K, N,
                    strips, q, scales);
}

}  // namespace moe
