// Per-head RMSNorm of queries and keys with the position rotation in the same
// pass.
//
// "DFlash双实现对比" (hotelren.com) §1: the drafter and its target are Qwen3
// models, which norm every query and key head before rotating it.
//
//   y = x / sqrt(mean(x^2) + eps) * w;   out_d = y_d cos a_d - y_{d+D/2} sin a_d,
//   out_{d+D/2} = y_{d+D/2} cos a_d + y_d sin a_d,   a_d = pos * theta^(-2d/D)
//
// The angle in turns, pos * f_d with f_d = theta^(-2d/D) / 2 pi, is formed modulo
// one in 64-bit integers: f_d (at most 1 / 2 pi, so below 2^62 units of 2^-64
// turns) is rounded once, to the 53 bits of a double, and the wrapped product is
// exact: the error is below pos 2^-55 turns, 2^-24 at the farthest position.
#include <cmath>

#include "kv4.cuh"

namespace dflash {
namespace {

struct TurnTable {
  unsigned long long f[64];   // theta^(-2d/D) / (2 pi) in units of 2^-64 turns
};

struct NormRopeParams {
  const uint16_t* x[2];       // q, k
  uint16_t* y[2];
  long long x_pitch[2], y_pitch[2];
  const uint16_t* w[2];
  const int32_t* pos;
  int n_tokens, heads[2];
  float eps;
  TurnTable turns;
};

constexpr int kThreads = 128;

// One CTA per row: 16 threads a head, each with D/32 dims of either half.
template <int D>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const NormRopeParams p) {
  constexpr int kHalf = D / 2, kE = kHalf / 16;
  __shared__ float2 sc[kHalf];
  griddep_wait();
  griddep_launch_dependents();
  const int n = blockIdx.x;
  const int pos = p.pos[n];
  if (pos < 0) return;
  for (int d = threadIdx.x; d < kHalf; d += kThreads) {
    const unsigned long long turns = p.turns.f[d] * static_cast<unsigned long long>(pos);
    // the fraction in half turns, -1 <= a < 1
    const float a = static_cast<float>(static_cast<long long>(turns)) * 0x1p-63f;
    float sn, cs;
    sincospif(a, &sn, &cs);
    sc[d] = make_float2(cs, sn);
  }
  __syncthreads();
  const int l = threadIdx.x & 15, d0 = l * kE;
  const int total = p.heads[0] + p.heads[1];
  // (whole warps run the same number of times: a warp holds two heads)
  for (int hh = threadIdx.x >> 4; hh < ((total + 1) & ~1); hh += kThreads / 16) {
    const bool live = hh < total;
    const int which = live && hh >= p.heads[0], h = live ? hh - (which ? p.heads[0] : 0) : 0;
    const uint16_t* x = p.x[which] + n * p.x_pitch[which] + static_cast<long long>(h) * D;
    float a[kE], b[kE];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      a[i] = bf16_bits_to_float(x[d0 + i]);
      b[i] = bf16_bits_to_float(x[kHalf + d0 + i]);
      ss += a[i] * a[i] + b[i] * b[i];
    }
#pragma unroll
    for (int o = 8; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const uint16_t* w = p.w[which];
    const float r = w ? rsqrtf(ss * (1.f / D) + p.eps) : 1.f;
    uint16_t* y = p.y[which] + n * p.y_pitch[which] + static_cast<long long>(h) * D;
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      float u = a[i], v = b[i];
      if (w) {
        u *= r * bf16_bits_to_float(w[d0 + i]);
        v *= r * bf16_bits_to_float(w[kHalf + d0 + i]);
      }
      const float2 cs = sc[d0 + i];
      if (live) {
        y[d0 + i] = float_to_bf16_bits(u * cs.x - v * cs.y);
        y[kHalf + d0 + i] = float_to_bf16_bits(v * cs.x + u * cs.y);
      }
    }
  }
}

}  // namespace
}  // namespace dflash

using namespace dflash;

extern "C" int dflash_qk_norm_rope(const dflash_kv4_dims* dims, const void* q, int64_t q_pitch,
                                   const void* k, int64_t k_pitch, const void* q_norm_w,
                                   const void* k_norm_w, const int32_t* pos, float rope_theta,
                                   float rms_eps, void* q_out, int64_t q_out_pitch, void* k_out,
                                   int64_t k_out_pitch, dflash_stream_t stream) {
  DFLASH_ENTRY("dflash_qk_norm_rope");
  const int rc = check_kv4_dims(dims);
  if (rc) return rc;
  if (!q || !k || !pos || !q_out || !k_out) return DFLASH_E_ARG;
  if (!(rope_theta >= 1.0f) || !(rms_eps >= 0.0f) || std::isinf(rope_theta) ||
      std::isinf(rms_eps))
    return DFLASH_E_ARG;
  const int D = dims->head_dim;
  const int64_t qw = static_cast<int64_t>(dims->n_q_heads) * D;
  const int64_t kw = static_cast<int64_t>(dims->n_kv_heads) * D;
  if (q_pitch < qw || q_out_pitch < qw || k_pitch < kw || k_out_pitch < kw) return DFLASH_E_ARG;
  if (((q_pitch | q_out_pitch | k_pitch | k_out_pitch) & 7) || !aligned16(q) || !aligned16(k) ||
      !aligned16(q_out) || !aligned16(k_out) || !aligned16(q_norm_w) || !aligned16(k_norm_w))
    return DFLASH_E_ALIGN;
  NormRopeParams p = {};
  p.x[0] = static_cast<const uint16_t*>(q);
  p.x[1] = static_cast<const uint16_t*>(k);
  p.y[0] = static_cast<uint16_t*>(q_out);
  p.y[1] = static_cast<uint16_t*>(k_out);
  p.x_pitch[0] = q_pitch;
  p.x_pitch[1] = k_pitch;
  p.y_pitch[0] = q_out_pitch;
  p.y_pitch[1] = k_out_pitch;
  p.w[0] = static_cast<const uint16_t*>(q_norm_w);
  p.w[1] = static_cast<const uint16_t*>(k_norm_w);
  p.pos = pos;
  p.n_tokens = dims->n_tokens;
  p.heads[0] = dims->n_q_heads;
  p.heads[1] = dims->n_kv_heads;
  p.eps = rms_eps;
  for (int d = 0; d < D / 2; ++d)
    p.turns.f[d] = static_cast<unsigned long long>(std::llround(std::ldexp(
        std::pow(static_cast<double>(rope_theta), -2.0 * d / D) / 6.283185307179586476925, 64)));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid(dims->n_tokens), block(kThreads);
  return D == 128 ? launch(qk_norm_rope_kernel<128>, grid, block, 0, st, p)
                  : launch(qk_norm_rope_kernel<64>, grid, block, 0, st, p);
}
