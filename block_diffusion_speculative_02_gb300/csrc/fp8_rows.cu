// Rows and weights rounded to 8 bits (e4m3) with a scale for each block of 128.
//
// For a block with the largest magnitude a (at least 2^-117):
//   scale = a / 448,  code = e4m3(h * (448 / a)),  a value is scale * code.
// Everything before the codes is fp32.  All three calls are bound by memory: each element is
// read once and written once, 16 of them (32 bytes in, 16 out) to a thread, so that 8
// neighbouring lanes hold a block and find its maximum in three shuffles.
#include <cmath>

#include "fp8.cuh"

namespace dflash {
namespace fp8 {
namespace {

// --------------------------------------------------------------------------------------------
// rows: h = RMSNorm(x + residual) * norm_w
// --------------------------------------------------------------------------------------------
struct NormParams {
  const uint16_t* x;
  const uint16_t* residual;
  const uint16_t* norm_w;
  uint16_t* sum;
  uint8_t* q;
  float* scale;
  long long x_pitch, residual_pitch, sum_pitch;
  int rows, cols;
  float eps;
};

constexpr int kWarpRows = 8;    // rows of a CTA where a warp takes one
constexpr int kMostLanes = 512; // threads of a CTA that takes one

// Below this mean of squares some of them may have left the range of fp32 (2^-126), and with eps
// so small they count.
__device__ __forceinline__ float least_mean() { return __uint_as_float((127 - 100) << 23); }

// The sum over a row of what each of its threads has, the same bits in all of them.
template <bool kWarp>
__device__ __forceinline__ float row_sum(float x, int t, int step) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (!kWarp) {
    __shared__ float part[32];           // (between two sums the row's threads meet in row_max)
    if ((t & 31) == 0) part[t >> 5] = x;
    __syncthreads();
    x = (t & 31) < (step >> 5) ? part[t & 31] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  }
  return x;
}

// The largest magnitude (as bits) of a row, likewise.
template <bool kWarp>
__device__ __forceinline__ uint32_t row_max(uint32_t m, int t, int step) {
  m = warp_max_u32(m);
  if (!kWarp) {
    __shared__ uint32_t part[32];
    if ((t & 31) == 0) part[t >> 5] = m;
    __syncthreads();
    m = warp_max_u32((t & 31) < (step >> 5) ? part[t & 31] : 0u);
  }
  return m;
}

// The mean of squares of a row where some leave the range of fp32 (elements past 2^64, or a row of
// tiny ones over next to no eps), and what it is the mean for: the row times 2^k, which brings its
// largest element, or sqrt(eps) if that is larger, next to 1.  h stays what it was,
//   (2^k s) / sqrt(mean (2^k s)^2 + 2^2k eps).
// A row with an infinity or NaN, or of zeros over nothing, stays as it is.  (A call, which takes a
// copy of the row: as part of the kernel it cost every row of 5120 and 8192 columns 1 to 2 %.)
template <int kN, bool kWarp>
__device__ __noinline__ float2 wide_mean(const float (&v)[kN], float mean, int cols, float eps,
                                         int t, int step) {
  uint32_t m = 0;
#pragma unroll 1
  for (int i = 0; i < kN; ++i) m = max(m, abs_bits(v[i]));
  m = max(row_max<kWarp>(m, t, step), __float_as_uint(sqrtf(eps)));
  if (m == 0 || m >= 0x7F800000u) return make_float2(mean, 1.f);
  const int k = max(254 - static_cast<int>(m >> 23), 1);              // biased
  const float up = __uint_as_float(static_cast<uint32_t>(k) << 23);
  float ss = 0.f;
#pragma unroll 1
  for (int i = 0; i < kN; ++i) ss = fmaf(v[i] * up, v[i] * up, ss);
  return make_float2(row_sum<kWarp>(ss, t, step) / cols + eps * up * up, up);
}

// A row to a CTA (or, up to 512 columns, to a warp): kChunks pieces of 16 columns stay
// in the thread's registers from the sum of squares to the codes, so the row is read once.
template <int kChunks, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 32 * kWarpRows : kMostLanes)
norm_rows_kernel(const NormParams p) {
  const int t = threadIdx.x, step = blockDim.x;
  const int row = kWarp ? blockIdx.x * kWarpRows + threadIdx.y : blockIdx.x;
  const int pieces = p.cols / 16;
  griddep_wait();
  griddep_launch_dependents();           // (they wait for the end of this grid before they read)
  if (row >= p.rows) return;                                  // whole warps
  float v[kChunks][16];
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int i = t + c * step;
    uint4 x[2] = {}, r[2] = {};
    if (i < pieces) {
      load16(p.x + row * p.x_pitch + 16 * i, x);
      if (p.residual) load16(p.residual + row * p.residual_pitch + 16 * i, r);
    }
    widen16(x, v[c]);
    if (p.residual) {
      float w[16];
      widen16(r, w);
#pragma unroll
      for (int j = 0; j < 16; ++j) v[c][j] += w[j];
    }
    if (p.norm_w) {
#pragma unroll
      for (int j = 0; j < 16; ++j) ss = fmaf(v[c][j], v[c][j], ss);
    }
  }
  if (p.sum) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int i = t + c * step;
      if (i >= pieces) continue;
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        o[j] = static_cast<uint32_t>(float_to_bf16_bits(v[c][2 * j])) |
               static_cast<uint32_t>(float_to_bf16_bits(v[c][2 * j + 1])) << 16;
      uint4* dst = reinterpret_cast<uint4*>(p.sum + row * p.sum_pitch + 16 * i);
      dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
      dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
  if (p.norm_w) {
    float mean = row_sum<kWarp>(ss, t, step) / p.cols + p.eps;
    if (!(mean >= least_mean() && mean < __uint_as_float(0x7F800000u))) {
      float copy[kChunks * 16];
#pragma unroll
      for (int i = 0; i < kChunks * 16; ++i) copy[i] = v[i >> 4][i & 15];
      const float2 wide = wide_mean<kChunks * 16, kWarp>(copy, mean, p.cols, p.eps, t, step);
      mean = wide.x;
#pragma unroll
      for (int i = 0; i < kChunks * 16; ++i) v[i >> 4][i & 15] *= wide.y;
    }
    const float inv = rsqrtf(mean);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int i = t + c * step;
      if (i >= pieces) continue;
      uint4 w[2];
      float g[16];
      load16(p.norm_w + 16 * i, w);
      widen16(w, g);
#pragma unroll
      for (int j = 0; j < 16; ++j) v[c][j] = v[c][j] * inv * g[j];
    }
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int i = t + c * step;
    const uint32_t m = max8(i < pieces ? max16(v[c]) : 0u);
    if (i >= pieces) continue;
    float s, r;
    scale_of(m, &s, &r);
    *reinterpret_cast<uint4*>(p.q + static_cast<size_t>(row) * p.cols + 16 * i) =
        codes16(v[c], r);
    if ((i & 7) == 0) p.scale[static_cast<size_t>(i >> 3) * p.rows + row] = s;
  }
}

// --------------------------------------------------------------------------------------------
// rows: h = silu(gate) * up
// --------------------------------------------------------------------------------------------
struct SiluParams {
  const uint16_t* x;
  uint8_t* q;
  float* scale;
  long long x_pitch;
  int rows, cols, blocks;
};

constexpr int kSiluThreads = 256;

// g / (1 + exp(-g)) as (g / 8) / (1 / 8 + exp(-g) / 8): a divisor past 2^126 has no reciprocal
// but zero, and exp(-g) reaches 2^128.  Relative to it the result is off by at most 6 + |g| units of
// 2^-23: the exponent |g| + 1 (the constant and the fma, 2^-24 of |g| log2 e each), the exponential
// 2, the reciprocal 1, the sum and the product half a unit each.
__device__ __forceinline__ float silu(float g) {
  constexpr float kLog2e = 1.44269504f;
  const float t = g * 0.125f;
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fmaf(t, -8.f * kLog2e, -3.f)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(0.125f + e));
  return t * r;
}

// 8 lanes to a block of 128 columns.
__global__ void __launch_bounds__(kSiluThreads) silu_rows_kernel(const SiluParams p) {
  const long long unit = (static_cast<long long>(blockIdx.x) * kSiluThreads + threadIdx.x) >> 3;
  const long long row = unit / p.blocks;
  const int b = static_cast<int>(unit - row * p.blocks);
  const int col = b * kBlockK + (threadIdx.x & 7) * 16;
  griddep_wait();
  griddep_launch_dependents();           // (they wait for the end of this grid before they read)
  const bool live = row < p.rows && col < p.cols;
  uint4 g4[2] = {}, u4[2] = {};
  if (live) {
    const uint16_t* src = p.x + row * p.x_pitch + col;
    load16(src, g4);
    load16(src + p.cols, u4);
  }
  float g[16], u[16];
  widen16(g4, g);
  widen16(u4, u);
#pragma unroll
  for (int j = 0; j < 16; ++j) u[j] *= silu(g[j]);
  const uint32_t m = max8(max16(u));
  if (!live) return;
  float s, r;
  scale_of(m, &s, &r);
  *reinterpret_cast<uint4*>(p.q + row * p.cols + col) = codes16(u, r);
  if ((threadIdx.x & 7) == 0) p.scale[static_cast<size_t>(b) * p.rows + row] = s;
}

// --------------------------------------------------------------------------------------------
// weights
// --------------------------------------------------------------------------------------------
struct WeightParams {
  const uint16_t* w;
  uint8_t* q;
  float* scale;
  int n, k, n_blocks, k_blocks;
};

constexpr int kWeightThreads = 256;

// A CTA to a block of 128 x 128, 64 elements to a thread.
__global__ void __launch_bounds__(kWeightThreads) weight_kernel(const WeightParams p) {
  __shared__ uint32_t part[kWeightThreads / 32];
  const int t = threadIdx.x;
  const int kb = blockIdx.x % p.k_blocks, rest = blockIdx.x / p.k_blocks;
  const int nb = rest % p.n_blocks, g = rest / p.n_blocks;
  const int col = kb * kBlockK + (t & 7) * 16;
  const size_t base = static_cast<size_t>(g) * p.n * p.k + col;
  griddep_wait();
  griddep_launch_dependents();           // (they wait for the end of this grid before they read)
  uint4 x[4][2];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = nb * kBlockK + (t >> 3) + 32 * i;
    x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
    if (row < p.n && col < p.k) load16(p.w + base + static_cast<size_t>(row) * p.k, x[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[16];
    widen16(x[i], v);
    m = max(m, max16(v));
  }
  m = warp_max_u32(m);
  if ((t & 31) == 0) part[t >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWeightThreads / 32; ++i) m = max(m, part[i]);
  float s, r;
  scale_of(m, &s, &r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = nb * kBlockK + (t >> 3) + 32 * i;
    if (row >= p.n || col >= p.k) continue;
    float v[16];
    widen16(x[i], v);
    *reinterpret_cast<uint4*>(p.q + base + static_cast<size_t>(row) * p.k) = codes16(v, r);
  }
  if (t == 0) p.scale[blockIdx.x] = s;
}

constexpr int kMaxCols = 16 * 4 * kMostLanes;   // of dflash_fp8_norm_rows

template <int kChunks>
int launch_norm(const NormParams& p, cudaStream_t st) {
  const int lanes = (p.cols / 16 + kChunks - 1) / kChunks;
  return launch(norm_rows_kernel<kChunks, false>, dim3(p.rows), dim3((lanes + 31) / 32 * 32), 0,
                st, p);
}

bool bad_pitch(long long pitch, long long least) { return pitch < least; }

}  // namespace
}  // namespace fp8
}  // namespace dflash

using namespace dflash;
using namespace dflash::fp8;

extern "C" int dflash_fp8_norm_rows(int32_t rows, int32_t cols, const void* x, int64_t x_pitch,
                                    const void* residual, int64_t residual_pitch,
                                    const void* norm_w, float rms_eps, void* sum_out,
                                    int64_t sum_pitch, void* q, float* scale,
                                    dflash_stream_t stream) {
  DFLASH_ENTRY("dflash_fp8_norm_rows");
  if (rows < 0 || cols < 1 || !(rms_eps >= 0.f) || std::isinf(rms_eps)) return DFLASH_E_ARG;
  if (cols % 16 || cols > kMaxCols) return DFLASH_E_UNSUPPORTED;
  if (rows == 0) return DFLASH_OK;
  if (!x || !q || !scale) return DFLASH_E_ARG;
  if (bad_pitch(x_pitch, cols) || (residual && bad_pitch(residual_pitch, cols)) ||
      (sum_out && bad_pitch(sum_pitch, cols)))
    return DFLASH_E_ARG;
  // in place: each row where it was
  if (sum_out && ((sum_out == x && sum_pitch != x_pitch) ||
                  (sum_out == residual && sum_pitch != residual_pitch)))
    return DFLASH_E_ARG;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(norm_w) || !aligned16(sum_out) ||
      !aligned16(q) || x_pitch % 8 || (residual && residual_pitch % 8) ||
      (sum_out && sum_pitch % 8) || reinterpret_cast<uintptr_t>(scale) % 4)
    return DFLASH_E_ALIGN;
  NormParams p = {};
  p.x = static_cast<const uint16_t*>(x);
  p.residual = static_cast<const uint16_t*>(residual);
  p.norm_w = static_cast<const uint16_t*>(norm_w);
  p.sum = static_cast<uint16_t*>(sum_out);
  p.q = static_cast<uint8_t*>(q);
  p.scale = scale;
  p.x_pitch = x_pitch;
  p.residual_pitch = residual_pitch;
  p.sum_pitch = sum_pitch;
  p.rows = rows;
  p.cols = cols;
  p.eps = rms_eps;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (cols <= 16 * 32)
    return launch(norm_rows_kernel<1, true>,
                  dim3((static_cast<unsigned>(rows) + kWarpRows - 1) / kWarpRows),
                  dim3(32, kWarpRows), 0, st, p);
  if (cols <= 16 * kMostLanes) return launch_norm<1>(p, st);
  if (cols <= 16 * 2 * kMostLanes) return launch_norm<2>(p, st);
  return launch_norm<4>(p, st);
}

extern "C" int dflash_fp8_silu_mul(int32_t rows, int32_t cols, const void* gate_up,
                                   int64_t pitch, void* q, float* scale, dflash_stream_t stream) {
  DFLASH_ENTRY("dflash_fp8_silu_mul");
  if (rows < 0 || cols < 1) return DFLASH_E_ARG;
  if (cols % 16) return DFLASH_E_UNSUPPORTED;
  if (rows == 0) return DFLASH_OK;
  if (!gate_up || !q || !scale || bad_pitch(pitch, 2ll * cols)) return DFLASH_E_ARG;
  if (!aligned16(gate_up) || !aligned16(q) || pitch % 8 || reinterpret_cast<uintptr_t>(scale) % 4)
    return DFLASH_E_ALIGN;
  SiluParams p = {};
  p.x = static_cast<const uint16_t*>(gate_up);
  p.q = static_cast<uint8_t*>(q);
  p.scale = scale;
  p.x_pitch = pitch;
  p.rows = rows;
  p.cols = cols;
  p.blocks = static_cast<int>(blocks(cols));
  const long long threads = 8ll * rows * p.blocks;
  const long long grid = (threads + kSiluThreads - 1) / kSiluThreads;
  if (grid > 0x7FFFFFFFll) return DFLASH_E_UNSUPPORTED;
  return launch(silu_rows_kernel, dim3(static_cast<unsigned>(grid)), dim3(kSiluThreads), 0,
                reinterpret_cast<cudaStream_t>(stream), p);
}

extern "C" int dflash_fp8_weight(int32_t n_groups, int32_t n_out, int32_t n_in, const void* w,
                                 void* q, float* scale, dflash_stream_t stream) {
  DFLASH_ENTRY("dflash_fp8_weight");
  if (n_groups < 1 || n_out < 1 || n_in < 1 || !w || !q || !scale) return DFLASH_E_ARG;
  if (n_in % 16) return DFLASH_E_UNSUPPORTED;
  if (!aligned16(w) || !aligned16(q) || reinterpret_cast<uintptr_t>(scale) % 4)
    return DFLASH_E_ALIGN;
  WeightParams p = {};
  p.w = static_cast<const uint16_t*>(w);
  p.q = static_cast<uint8_t*>(q);
  p.scale = scale;
  p.n = n_out;
  p.k = n_in;
  p.n_blocks = static_cast<int>(blocks(n_out));
  p.k_blocks = static_cast<int>(blocks(n_in));
  // (in double: three factors of 31 bits pass 64)
  if (static_cast<double>(n_groups) * p.n_blocks * p.k_blocks > 2147483647.0)
    return DFLASH_E_UNSUPPORTED;
  const long long grid = static_cast<long long>(n_groups) * p.n_blocks * p.k_blocks;
  return launch(weight_kernel, dim3(static_cast<unsigned>(grid)), dim3(kWeightThreads), 0,
                reinterpret_cast<cudaStream_t>(stream), p);
}
