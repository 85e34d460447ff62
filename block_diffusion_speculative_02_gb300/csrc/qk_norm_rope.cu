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

// The table of (theta, D), kept for the thread's next call: 64 powers take as long as the launch.
const TurnTable& turn_table(float theta, int D) {
  struct Kept {
    float theta = 0.f;
    int D = 0;
    TurnTable table;
  };
  static thread_local Kept kept;
  if (kept.theta != theta || kept.D != D) {
    for (int d = 0; d < D / 2; ++d)
      kept.table.f[d] = static_cast<unsigned long long>(std::llround(std::ldexp(
          std::pow(static_cast<double>(theta), -2.0 * d / D) / 6.283185307179586476925, 64)));
    kept.theta = theta;
    kept.D = D;
  }
  return kept.table;
}

constexpr int kThreads = 256, kGroups = kThreads / 16;

// 16 threads take a head, each D / 32 dims of either half (8 or 4 bytes at a time, both halves
// of a rotated pair in one thread).  What a pair is multiplied by, gains and angle, is the same for
// every head of q (and of k): w cos and w sin are formed once a row, and 1 / rms goes on at the
// end.
template <int D>
struct Heads {
  static constexpr int kHalf = D / 2, kE = kHalf / 16, kW = kE / 2;

  template <int kBatch>
  static __device__ __forceinline__ void load(const uint16_t* row, int heads, int h0, int d0,
                                              uint32_t (&x)[kBatch][2][kW]) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int h = h0 + u * kGroups;
      if (h >= heads) continue;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint16_t* src = row + static_cast<long long>(h) * D + half * kHalf + d0;
        if (kW == 2)
          *reinterpret_cast<uint2*>(x[u][half]) = *reinterpret_cast<const uint2*>(src);
        else
          x[u][half][0] = *reinterpret_cast<const uint32_t*>(src);
      }
    }
  }

  // All heads of a row; the first kBatch of this thread are in x.
  template <int kBatch>
  static __device__ __forceinline__ void run(const uint16_t* row, uint16_t* out, int heads,
                                             const uint16_t* w, float eps, const float2* angle,
                                             uint32_t (&x)[kBatch][2][kW]) {
    const int d0 = (threadIdx.x & 15) * kE, h_first = threadIdx.x >> 4;
    float2 lo_c[kE], hi_c[kE];           // what a, b give of out_d, and of out_{d + D/2}
    {
      uint32_t g[2][kW];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int e = 0; e < kW; ++e) g[half][e] = 0x3F803F80u;               // 1, 1
        if (!w) continue;
        const uint16_t* src = w + half * kHalf + d0;
        if (kW == 2)
          *reinterpret_cast<uint2*>(g[half]) = *reinterpret_cast<const uint2*>(src);
        else
          g[half][0] = *reinterpret_cast<const uint32_t*>(src);
      }
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const float2 cs = angle[d0 + e];
        const float g0 = __uint_as_float(e & 1 ? g[0][e / 2] & 0xFFFF0000u : g[0][e / 2] << 16);
        const float g1 = __uint_as_float(e & 1 ? g[1][e / 2] & 0xFFFF0000u : g[1][e / 2] << 16);
        lo_c[e] = make_float2(g0 * cs.x, -g1 * cs.y);
        hi_c[e] = make_float2(g0 * cs.y, g1 * cs.x);
      }
    }
    // (whole warps go on together: a warp holds two heads)
    const int warp_first = h_first & ~1;
#pragma unroll 1
    for (int i = 0; warp_first + i < heads; i += kBatch * kGroups) {
      if (i) load<kBatch>(row, heads, h_first + i, d0, x);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (warp_first + i + u * kGroups >= heads) break;
        const int h = h_first + i + u * kGroups;
        const bool live = h < heads;
        float a[kE], b[kE], ss = 0.f;
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          const uint32_t lo = live ? x[u][0][e / 2] : 0u, hi = live ? x[u][1][e / 2] : 0u;
          a[e] = __uint_as_float(e & 1 ? lo & 0xFFFF0000u : lo << 16);
          b[e] = __uint_as_float(e & 1 ? hi & 0xFFFF0000u : hi << 16);
          ss += a[e] * a[e] + b[e] * b[e];
        }
        float r = 1.f;
        if (w) {
#pragma unroll
          for (int o = 8; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          r = rsqrtf(ss * (1.f / D) + eps);
        }
        uint32_t y[2][kW];
#pragma unroll
        for (int e = 0; e < kE; e += 2) {
          float o0[2], o1[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            o0[k] = r * (a[e + k] * lo_c[e + k].x + b[e + k] * lo_c[e + k].y);
            o1[k] = r * (a[e + k] * hi_c[e + k].x + b[e + k] * hi_c[e + k].y);
          }
          y[0][e / 2] = pack_bf16(o0[0], o0[1]);
          y[1][e / 2] = pack_bf16(o1[0], o1[1]);
        }
        if (live) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint16_t* dst = out + static_cast<long long>(h) * D + half * kHalf + d0;
            if (kW == 2)
              *reinterpret_cast<uint2*>(dst) = make_uint2(y[half][0], y[half][kW - 1]);
            else
              *reinterpret_cast<uint32_t*>(dst) = y[half][0];
          }
        }
      }
    }
  }
};

// One CTA per row, five of them to an SM.  Floor: the 4 bytes an element moves.  8191 rows of
// 64 + 8 heads of 128 dims take 56.5 us, 5.35 TB/s; before the products above were formed
// once a row the instruction slots were the bound (69% of them, 60 us).  Two heads of a
// thread in flight in place of four 59 us, six CTAs to an SM 58 us.  (Five CTAs leave 48
// registers a thread: 56 bytes of it go to local memory at 128 dims.)
template <int D>
__global__ void __launch_bounds__(kThreads, 5) qk_norm_rope_kernel(const NormRopeParams p) {
  using H = Heads<D>;
  __shared__ float2 angle[H::kHalf];
  griddep_wait();
  griddep_launch_dependents();
  const long long n = blockIdx.x;
  const int pos = p.pos[n];
  const int d0 = (threadIdx.x & 15) * H::kE, h_first = threadIdx.x >> 4;
  const uint16_t* q = p.x[0] + n * p.x_pitch[0];
  const uint16_t* k = p.x[1] + n * p.x_pitch[1];
  uint32_t xq[4][2][H::kW], xk[1][2][H::kW];
  H::template load<4>(q, p.heads[0], h_first, d0, xq);   // (before the position is known to be one)
  H::template load<1>(k, p.heads[1], h_first, d0, xk);
  if (pos < 0) return;
  for (int d = threadIdx.x; d < H::kHalf; d += kThreads) {
    const unsigned long long turns = p.turns.f[d] * static_cast<unsigned long long>(pos);
    // the fraction in half turns, -1 <= a < 1
    const float a = static_cast<float>(static_cast<long long>(turns)) * 0x1p-63f;
    float sn, cs;
    sincospif(a, &sn, &cs);
    angle[d] = make_float2(cs, sn);
  }
  __syncthreads();
  H::template run<4>(q, p.y[0] + n * p.y_pitch[0], p.heads[0], p.w[0], p.eps, angle, xq);
  H::template run<1>(k, p.y[1] + n * p.y_pitch[1], p.heads[1], p.w[1], p.eps, angle, xk);
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
  p.turns = turn_table(rope_theta, D);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid(dims->n_tokens), block(kThreads);
  return D == 128 ? launch(qk_norm_rope_kernel<128>, grid, block, 0, st, p)
                  : launch(qk_norm_rope_kernel<64>, grid, block, 0, st, p);
}
