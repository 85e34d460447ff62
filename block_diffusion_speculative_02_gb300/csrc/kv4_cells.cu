// K/V rows into the 4-bit cells of a cache, and back.
//
// For 16 consecutive dims x of one head, times the power of two 2^-exp[head]:
//   scale = e4m3(max |x| / 6),  code = e2m1(x / scale),  x ~ 2^exp scale code.
// Both quotients are divided with one rounding (IEEE), so a quotient that lies
// halfway between two codes stays there and rounds to even: x has 8 significant
// bits, 6 times an e4m3 midpoint 7 and an e2m1 midpoint times a scale 7, so a
// quotient is either a midpoint or at least 2^-8 of its size away from it.
#include "kv4.cuh"

namespace dflash {
namespace {

constexpr int kThreads = 128;

// Row of the pool -> slab and row in it; false for rows outside it.
__device__ __forceinline__ bool find_slot(const Kv4Store& s, int slot, int* slab, int* row,
                                          uint32_t* status) {
  if (slot < 0) return false;
  *slab = slot / s.slab_rows;
  *row = slot - *slab * s.slab_rows;
  if (*slab >= s.n_slabs) {
    set_status(status, DFLASH_ST_CAPACITY);
    return false;
  }
  return true;
}

// 16 bf16 (two 16-byte loads) to 16 codes (8 bytes) and their scale.
__device__ __forceinline__ uint2 quantise16(const uint16_t* x, float gain, uint32_t* scale,
                                            bool* bad) {
  const uint4 a = reinterpret_cast<const uint4*>(x)[0], b = reinterpret_cast<const uint4*>(x)[1];
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float v[16], m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i] = __uint_as_float(i & 1 ? (w[i / 2] & 0xFFFF0000u) : (w[i / 2] << 16)) * gain;
    if (!(fabsf(v[i]) <= 3.4028234e38f)) *bad = true;
    if (isnan(v[i])) v[i] = 0.f;
    m = fmaxf(m, fabsf(v[i]));
  }
  *scale = to_e4m3(__fdiv_rn(m, 6.f));
  if (*scale == 0) return make_uint2(0, 0);
  const float s = f16x2_to_float2(e4m3x2_to_f16x2(*scale)).x;
  uint32_t o[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 16; i += 2)
    o[i / 8] |= to_e2m1x2(__fdiv_rn(v[i], s), __fdiv_rn(v[i + 1], s)) << (i % 8 * 4);
  return make_uint2(o[0], o[1]);
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(
    const Kv4Store s, const uint16_t* __restrict__ k, long long k_pitch,
    const uint16_t* __restrict__ v, long long v_pitch, const int32_t* __restrict__ slot,
    long long units, uint32_t* status) {
  constexpr int kG = D / 16;
  griddep_wait();
  griddep_launch_dependents();
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= units) return;
  const int g = static_cast<int>(i % kG);
  const int h = static_cast<int>(i / kG % s.n_kv_heads);
  const long long n = i / kG / s.n_kv_heads;
  int slab, row;
  if (!find_slot(s, slot[n], &slab, &row, status)) return;
  uint8_t* cell = s.cells + cell_index(s, slab, h, row) * Cell<D>::kBytes;
  const int r = row % kCellRows;
  bool bad = false;
  uint32_t ks, vs;
  const uint2 kc = quantise16(k + n * k_pitch + h * D + 16 * g, pow2(-gain_exp(s.k_exp, h)), &ks,
                              &bad);
  const uint2 vc = quantise16(v + n * v_pitch + h * D + 16 * g, pow2(-gain_exp(s.v_exp, h)), &vs,
                              &bad);
  *reinterpret_cast<uint2*>(cell + Cell<D>::k_codes(r, g)) = kc;
  cell[Cell<D>::k_scale(r, g)] = static_cast<uint8_t>(ks);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    cell[Cell<D>::v_codes(r, 8 * g + j)] =
        static_cast<uint8_t>((j < 4 ? vc.x : vc.y) >> (8 * (j & 3)));
  cell[Cell<D>::v_scale(r, g)] = static_cast<uint8_t>(vs);
  if (bad) set_status(status, DFLASH_ST_BAD_VALUE);
}

// Eight codes with their scale and gain as eight bf16 (exact).
__device__ __forceinline__ uint4 values8(uint32_t codes, float f) {
  uint32_t h[4], o[4];
  e2m1x8_to_f16x2(codes, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = f16x2_to_float2(h[i]);
    o[i] = static_cast<uint32_t>(float_to_bf16_bits(x.x * f)) |
           static_cast<uint32_t>(float_to_bf16_bits(x.y * f)) << 16;
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_gather_kernel(
    const Kv4Store s, const int32_t* __restrict__ slot, uint16_t* __restrict__ k,
    uint16_t* __restrict__ v, long long units, uint32_t* status) {
  constexpr int kG = D / 16;
  griddep_wait();
  griddep_launch_dependents();
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= units) return;
  const int g = static_cast<int>(i % kG);
  const int h = static_cast<int>(i / kG % s.n_kv_heads);
  const long long n = i / kG / s.n_kv_heads;
  int slab, row;
  if (!find_slot(s, slot[n], &slab, &row, status)) return;
  const uint8_t* cell = s.cells + cell_index(s, slab, h, row) * Cell<D>::kBytes;
  const int r = row % kCellRows;
  const uint2 kc = *reinterpret_cast<const uint2*>(cell + Cell<D>::k_codes(r, g));
  uint32_t vc[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    vc[j / 4] |= static_cast<uint32_t>(cell[Cell<D>::v_codes(r, 8 * g + j)]) << (8 * (j & 3));
  const uint32_t sc = cell[Cell<D>::k_scale(r, g)] | cell[Cell<D>::v_scale(r, g)] << 8;
  const float2 f = f16x2_to_float2(e4m3x2_to_f16x2(sc));
  const float fk = f.x * pow2(gain_exp(s.k_exp, h)), fv = f.y * pow2(gain_exp(s.v_exp, h));
  uint4* ko = reinterpret_cast<uint4*>(k + (n * s.n_kv_heads + h) * D + 16 * g);
  uint4* vo = reinterpret_cast<uint4*>(v + (n * s.n_kv_heads + h) * D + 16 * g);
  ko[0] = values8(kc.x, fk);
  ko[1] = values8(kc.y, fk);
  vo[0] = values8(vc[0], fv);
  vo[1] = values8(vc[1], fv);
}

}  // namespace

int kv4_store(const dflash_kv4_dims& d, const dflash_kv4_view* v, Kv4Store* s) {
  if (!v || !v->kv.k) return DFLASH_E_ARG;
  const dflash_kv_view& c = v->kv;
  long long rows;
  if (c.page_table) {
    if (c.page_size < 1 || c.max_pages < 1 || c.n_pages < 1) return DFLASH_E_ARG;
    if (c.page_size % kCellRows) return DFLASH_E_UNSUPPORTED;
    if (static_cast<long long>(c.max_pages) * c.page_size > INT32_MAX) return DFLASH_E_UNSUPPORTED;
    s->slab_rows = c.page_size;
    s->n_slabs = c.n_pages;
  } else {
    if (c.capacity < 1) return DFLASH_E_ARG;
    if (c.capacity % kCellRows) return DFLASH_E_UNSUPPORTED;
    s->slab_rows = c.capacity;
    s->n_slabs = d.batch;
  }
  rows = static_cast<long long>(s->slab_rows) * s->n_slabs;
  if (rows > INT32_MAX) return DFLASH_E_UNSUPPORTED;   // slots are int32
  if (!aligned16(c.k)) return DFLASH_E_ALIGN;
  s->cells = static_cast<uint8_t*>(c.k);
  s->k_exp = v->k_exp;
  s->v_exp = v->v_exp;
  s->n_kv_heads = d.n_kv_heads;
  return DFLASH_OK;
}

}  // namespace dflash

using namespace dflash;

extern "C" int dflash_kv4_append(const dflash_kv4_dims* dims, const void* k, int64_t k_pitch,
                                 const void* v, int64_t v_pitch, const int32_t* slot,
                                 const dflash_kv4_view* cache, void* ws, size_t ws_bytes,
                                 dflash_stream_t stream) {
  DFLASH_ENTRY("dflash_kv4_append");
  int rc = check_kv4_dims(dims);
  if (rc) return rc;
  if (!k || !v || !slot) return DFLASH_E_ARG;
  Kv4Store s;
  if ((rc = kv4_store(*dims, cache, &s))) return rc;
  const int64_t width = static_cast<int64_t>(dims->n_kv_heads) * dims->head_dim;
  if (k_pitch < width || v_pitch < width) return DFLASH_E_ARG;
  if (((k_pitch | v_pitch) & 7) || !aligned16(k) || !aligned16(v)) return DFLASH_E_ALIGN;
  if (!ws || ws_bytes < 64) return DFLASH_E_WORKSPACE;
  const long long units =
      static_cast<long long>(dims->n_tokens) * dims->n_kv_heads * (dims->head_dim / 16);
  const long long ctas = (units + kThreads - 1) / kThreads;
  if (ctas > INT32_MAX) return DFLASH_E_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(ctas)), block(kThreads);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto* kernel = dims->head_dim == 128 ? kv4_append_kernel<128> : kv4_append_kernel<64>;
  return launch(kernel, grid, block, 0, st, s, static_cast<const uint16_t*>(k),
                static_cast<long long>(k_pitch), static_cast<const uint16_t*>(v),
                static_cast<long long>(v_pitch), slot, units, ws_at<uint32_t>(ws, 0));
}

extern "C" int dflash_kv4_gather(const dflash_kv4_dims* dims, const int32_t* slot,
                                 const dflash_kv4_view* cache, void* k_out, void* v_out, void* ws,
                                 size_t ws_bytes, dflash_stream_t stream) {
  DFLASH_ENTRY("dflash_kv4_gather");
  int rc = check_kv4_dims(dims);
  if (rc) return rc;
  if (!k_out || !v_out || !slot) return DFLASH_E_ARG;
  Kv4Store s;
  if ((rc = kv4_store(*dims, cache, &s))) return rc;
  if (!aligned16(k_out) || !aligned16(v_out)) return DFLASH_E_ALIGN;
  if (!ws || ws_bytes < 64) return DFLASH_E_WORKSPACE;
  const long long units =
      static_cast<long long>(dims->n_tokens) * dims->n_kv_heads * (dims->head_dim / 16);
  const long long ctas = (units + kThreads - 1) / kThreads;
  if (ctas > INT32_MAX) return DFLASH_E_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(ctas)), block(kThreads);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto* kernel = dims->head_dim == 128 ? kv4_gather_kernel<128> : kv4_gather_kernel<64>;
  return launch(kernel, grid, block, 0, st, s, slot, static_cast<uint16_t*>(k_out),
                static_cast<uint16_t*>(v_out), units, ws_at<uint32_t>(ws, 0));
}
