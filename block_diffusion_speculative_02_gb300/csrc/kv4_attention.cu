// Attention of a ragged batch's rows over a KV cache held in 4 bits.
//
// "DFlash双实现对比" (hotelren.com) §2 and "dflash-mlx" (dpshk.com) 单次前向验证 ⑤:
// the drafter's block attends to its context and itself, the target's verify
// forward to the cache and, causally, to the block.  Here the new rows are in the
// cache already, so both are one product over its rows:
//   out[t, h] = softmax(q[t, h] K^T scale) V over the rows below
//   m = L - T + t + 1 (causal) or L.
//
// One CTA per (sequence, KV head, 16 query rows); keys come in tiles of 32, are
// expanded to fp32 in shared memory, and the running maximum and sum of the softmax
// are kept in fp32.
#include <cmath>

#include "kv4.cuh"

namespace dflash {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 16;
constexpr int kTile = 32;

struct Kv4AttnParams {
  Kv4Store s;
  int batch, n_tokens, max_tokens, n_q_heads, group, causal;
  int paged, page_size, max_pages, limit;
  const int32_t* seq_len;
  const int32_t* start;
  const int32_t* page_table;
  const uint16_t* q;
  uint16_t* out;
  float scale;
  uint32_t* status;
};

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_attention_kernel(const Kv4AttnParams p) {
  __shared__ float ks[kTile][D + 1], vs[kTile][D], qs[kRows][D], ps[kRows][kTile];
  __shared__ float row_m[kRows], row_l[kRows], row_f[kRows];
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
  const int lo = p.start[b], hi = p.start[b + 1], len = p.seq_len[b];
  const int T = hi - lo;
  if (lo < 0 || hi < lo || hi > p.n_tokens || T > p.max_tokens || len < 0 || len > p.limit) {
    if (blockIdx.x == 0 && h == 0 && tid == 0) set_status(p.status, DFLASH_ST_CAPACITY);
    return;
  }
  const int G = p.group, r0 = blockIdx.x * kRows, rows = min(kRows, T * G - r0);
  if (rows <= 0) return;
  auto seen = [&](int r) {
    return max(0, p.causal ? min(len, len - T + (r0 + r) / G + 1) : len);
  };
  auto at = [&](int r) {
    return (static_cast<size_t>(lo + (r0 + r) / G) * p.n_q_heads + h * G + (r0 + r) % G) * D;
  };
  for (int i = tid; i < kRows * D; i += kThreads)
    qs[i / D][i % D] = i / D < rows ? bf16_bits_to_float(p.q[at(i / D) + i % D]) : 0.f;
  if (tid < kRows) {
    row_m[tid] = -INFINITY;
    row_l[tid] = 0.f;
  }
  constexpr int kPer = kRows * D / kThreads;
  const int d = tid % D, or0 = tid / D * kPer;
  float o[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) o[i] = 0.f;
  const float qk = p.scale * 1.4426950408889634f * pow2(gain_exp(p.s.k_exp, h));
  const int end = seen(rows - 1);
  for (int key0 = 0; key0 < end; key0 += kTile) {
    __syncthreads();
    for (int i = tid; i < kTile * (D / 16); i += kThreads) {
      const int j = i / (D / 16), g = i % (D / 16), key = key0 + j;
      int slab = b, row = key;
      bool ok = key < len;
      if (ok && p.paged) {
        slab = p.page_table[static_cast<size_t>(b) * p.max_pages + key / p.page_size];
        row = key % p.page_size;
        if (slab < 0 || slab >= p.s.n_slabs) {
          ok = false;
          set_status(p.status, DFLASH_ST_PAGE_MISSING);
        }
      }
      float fk = 0.f, fv = 0.f;
      uint2 kc = make_uint2(0, 0);
      uint32_t vc[2] = {0, 0};
      if (ok) {
        const uint8_t* cell = p.s.cells + cell_index(p.s, slab, h, row) * Cell<D>::kBytes;
        const int r = row % kCellRows;
        kc = *reinterpret_cast<const uint2*>(cell + Cell<D>::k_codes(r, g));
        for (int e = 0; e < 8; ++e)
          vc[e / 4] |= static_cast<uint32_t>(cell[Cell<D>::v_codes(r, 8 * g + e)]) << (8 * (e & 3));
        const uint32_t sc = cell[Cell<D>::k_scale(r, g)] | cell[Cell<D>::v_scale(r, g)] << 8;
        const float2 f = f16x2_to_float2(e4m3x2_to_f16x2(sc));
        fk = f.x;
        fv = f.y;
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t kx[4], vx[4];
        e2m1x8_to_f16x2(half ? kc.y : kc.x, kx);
        e2m1x8_to_f16x2(vc[half], vx);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 a = f16x2_to_float2(kx[e]), c = f16x2_to_float2(vx[e]);
          ks[j][16 * g + 8 * half + 2 * e] = a.x * fk;
          ks[j][16 * g + 8 * half + 2 * e + 1] = a.y * fk;
          vs[j][16 * g + 8 * half + 2 * e] = c.x * fv;
          vs[j][16 * g + 8 * half + 2 * e + 1] = c.y * fv;
        }
      }
    }
    __syncthreads();
    // a warp takes two rows, a lane one key
    const int lane = tid & 31;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = (tid >> 5) * 2 + i;
      float s = 0.f;
      for (int e = 0; e < D; ++e) s = fmaf(qs[r][e], ks[lane][e], s);
      s = r < rows && key0 + lane < seen(r) ? s * qk : -INFINITY;
      float m = s;
#pragma unroll
      for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
      const float old = row_m[r], now = fmaxf(old, m);
      const float base = now == -INFINITY ? 0.f : now;
      const float e = exp2f(s - base);
      float sum = e;
#pragma unroll
      for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      ps[r][lane] = e;
      __syncwarp();
      if (lane == 0) {
        const float f = exp2f(old - base);
        row_f[r] = f;
        row_l[r] = row_l[r] * f + sum;
        row_m[r] = now;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      float a = o[i] * row_f[or0 + i];
      for (int j = 0; j < kTile; ++j) a = fmaf(ps[or0 + i][j], vs[j][d], a);
      o[i] = a;
    }
  }
  __syncthreads();
  const float gv = pow2(gain_exp(p.s.v_exp, h));
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (or0 + i < rows) {
      const float l = row_l[or0 + i];
      // a row that sees nothing is zero (l is NaN, not 0, for a row with NaN)
      p.out[at(or0 + i) + d] = float_to_bf16_bits(l == 0.f ? 0.f : o[i] / l * gv);
    }
}

}  // namespace

size_t kv4_attention_bytes(const dflash_kv4_dims&) { return 256; }

}  // namespace dflash

using namespace dflash;

extern "C" int dflash_kv4_attention(const dflash_kv4_dims* dims, const void* q,
                                    const int32_t* start, const dflash_kv4_view* cache,
                                    float scale, int causal, void* out, void* ws,
                                    size_t ws_bytes, dflash_stream_t stream) {
  DFLASH_ENTRY("dflash_kv4_attention");
  int rc = check_kv4_dims(dims);
  if (rc) return rc;
  if (!q || !start || !out || !cache || !cache->kv.seq_len || !std::isfinite(scale))
    return DFLASH_E_ARG;
  Kv4AttnParams p = {};
  if ((rc = kv4_store(*dims, cache, &p.s))) return rc;
  if (!aligned16(q) || !aligned16(out)) return DFLASH_E_ALIGN;
  Kv4Plan plan;
  if ((rc = make_kv4_plan(*dims, &plan))) return rc;
  if (!ws || ws_bytes < plan.total) return DFLASH_E_WORKSPACE;
  p.batch = dims->batch;
  p.n_tokens = dims->n_tokens;
  p.max_tokens = dims->max_tokens;
  p.n_q_heads = dims->n_q_heads;
  p.group = dims->n_q_heads / dims->n_kv_heads;
  p.causal = causal != 0;
  p.paged = cache->kv.page_table != nullptr;
  p.page_size = cache->kv.page_size;
  p.max_pages = cache->kv.max_pages;
  p.limit = p.paged ? p.max_pages * p.page_size : cache->kv.capacity;
  p.seq_len = cache->kv.seq_len;
  p.start = start;
  p.page_table = cache->kv.page_table;
  p.q = static_cast<const uint16_t*>(q);
  p.out = static_cast<uint16_t*>(out);
  p.scale = scale;
  p.status = ws_at<uint32_t>(ws, plan.off_status);
  const long long rows = static_cast<long long>(p.max_tokens) * p.group;
  const long long tiles = (rows + kRows - 1) / kRows;
  if (tiles > INT32_MAX) return DFLASH_E_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(tiles), dims->n_kv_heads, p.batch);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return dims->head_dim == 128
             ? launch(kv4_attention_kernel<128>, grid, dim3(kThreads), 0, st, p)
             : launch(kv4_attention_kernel<64>, grid, dim3(kThreads), 0, st, p);
}
