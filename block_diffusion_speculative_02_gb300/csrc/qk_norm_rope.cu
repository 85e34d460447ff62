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

constexpr int kThreads = 256;

// One CTA per row: 16 threads a head, each with D/32 dims of either half (8 or 4 bytes at
// a time, both halves of a rotated pair in one thread), kBatch heads in flight.  Bound
// by the 4 bytes an element moves.
template <int D>
__global__ void __launch_bounds__(kThreads, 5) qk_norm_rope_kernel(const NormRopeParams p) {
  constexpr int kHalf = D / 2, kE = kHalf / 16, kW = kE / 2, kBatch = 3;
  __shared__ float2 sc[kHalf];
  griddep_wait();
  griddep_launch_dependents();
  const long long n = blockIdx.x;
  const int pos = p.pos[n];
  const int l = threadIdx.x & 15, d0 = l * kE;
  const int total = p.heads[0] + p.heads[1];
  uint32_t x[kBatch][2][kW];             // of a head: both halves, two dims to a word
  auto place = [&](int hh, int* which) {
    *which = hh >= p.heads[0];
    return static_cast<long long>(hh - (*which ? p.heads[0] : 0)) * D + d0;
  };
  auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int hh = h0 + u * (kThreads / 16);
      if (hh >= total) continue;
      int which;
      const long long at = place(hh, &which);
      const uint16_t* src = p.x[which] + n * p.x_pitch[which] + at;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (kW == 2)
          *reinterpret_cast<uint2*>(x[u][half]) =
              *reinterpret_cast<const uint2*>(src + half * kHalf);
        else
          x[u][half][0] = *reinterpret_cast<const uint32_t*>(src + half * kHalf);
      }
    }
  };
  const int h_first = threadIdx.x >> 4;
  load(h_first);                         // (before the position is known to be one)
  if (pos < 0) return;
  for (int d = threadIdx.x; d < kHalf; d += kThreads) {
    const unsigned long long turns = p.turns.f[d] * static_cast<unsigned long long>(pos);
    // the fraction in half turns, -1 <= a < 1
    const float a = static_cast<float>(static_cast<long long>(turns)) * 0x1p-63f;
    float sn, cs;
    sincospif(a, &sn, &cs);
    sc[d] = make_float2(cs, sn);
  }
  float2 cs[kE];
  uint32_t w[2][2][kW];                  // gains: q or k, half, two dims to a word
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint16_t* src = p.w[i] + half * kHalf + d0;
#pragma unroll
      for (int e = 0; e < kW; ++e) w[i][half][e] = 0x3F803F80u;          // 1, 1
      if (!p.w[i]) continue;
      if (kW == 2)
        *reinterpret_cast<uint2*>(w[i][half]) = *reinterpret_cast<const uint2*>(src);
      else
        w[i][half][0] = *reinterpret_cast<const uint32_t*>(src);
    }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < kE; ++e) cs[e] = sc[d0 + e];
  for (int h0 = h_first; h0 < ((total + 1) & ~1); h0 += kBatch * (kThreads / 16)) {
    if (h0 != h_first) load(h0);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      // (whole warps go on together: a warp holds two heads)
      const int hh = h0 + u * (kThreads / 16);
      if (hh >= ((total + 1) & ~1)) break;
      const bool live = hh < total;
      int which;
      const long long at = place(live ? hh : 0, &which);
      float a[kE], b[kE], ss = 0.f;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const uint32_t lo = x[u][0][e / 2], hi = x[u][1][e / 2];
        a[e] = __uint_as_float(e & 1 ? lo & 0xFFFF0000u : lo << 16);
        b[e] = __uint_as_float(e & 1 ? hi & 0xFFFF0000u : hi << 16);
        if (!live) a[e] = b[e] = 0.f;
        ss += a[e] * a[e] + b[e] * b[e];
      }
#pragma unroll
      for (int o = 8; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float r = p.w[which] ? rsqrtf(ss * (1.f / D) + p.eps) : 1.f;
      uint32_t y[2][kW];
#pragma unroll
      for (int e = 0; e < kE; e += 2) {
        float o0[2], o1[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t w0 = which ? w[1][0][e / 2] : w[0][0][e / 2];
          const uint32_t w1 = which ? w[1][1][e / 2] : w[0][1][e / 2];
          const float g = a[e + i] * (r * __uint_as_float(i ? w0 & 0xFFFF0000u : w0 << 16));
          const float v = b[e + i] * (r * __uint_as_float(i ? w1 & 0xFFFF0000u : w1 << 16));
          o0[i] = g * cs[e + i].x - v * cs[e + i].y;
          o1[i] = v * cs[e + i].x + g * cs[e + i].y;
        }
        y[0][e / 2] = pack_bf16(o0[0], o0[1]);
        y[1][e / 2] = pack_bf16(o1[0], o1[1]);
      }
      if (live) {
        uint16_t* dst = p.y[which] + n * p.y_pitch[which] + at;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (kW == 2)
            *reinterpret_cast<uint2*>(dst + half * kHalf) = make_uint2(y[half][0], y[half][kW - 1]);
          else
            *reinterpret_cast<uint32_t*>(dst + half * kHalf) = y[half][0];
        }
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
