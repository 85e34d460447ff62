// K/V rows into the 4-bit cells of a cache, and back.
//
// For 16 consecutive dims x of one head, times the power of two 2^-exp[head]:
//   scale = e4m3(max |x| / 6),  code = e2m1(x / scale),  x ~ 2^exp scale code.
// A quotient that lies halfway between two codes has to stay there, to round to even: x has
// 8 significant bits, 6 times an e4m3 midpoint 7 and an e2m1 midpoint times a scale 7, so
// a quotient is either a midpoint or at least 2^-8 of its size away from it.  Products with
// the reciprocals, within 2^-22 of the quotients, are therefore rounded once more, to fewer
// bits than would lose a midpoint: max / 6 to 12 significant ones (a midpoint has 5, and the
// others stay on their side), x / scale to a multiple of 2^-14 (midpoints, 0.25 and up,
// are such multiples, every other quotient up to 6 is 2^-10 or more away from them).  (IEEE
// divisions took most of the kernel's time.)
#include "kv4.cuh"

namespace dflash {
namespace {

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

// 16 bf16 to 16 codes (8 bytes) and their scale.
__device__ __forceinline__ uint2 quantise16(const uint4& a, const uint4& b, float gain,
                                            uint32_t* scale, bool* bad) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  // the largest magnitude among the bits (two halves at once): they order as the values do
  auto largest = [&w] {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; i += 2)
      m = __vimax3_u16x2(m, w[i] & 0x7FFF7FFFu, w[i + 1] & 0x7FFF7FFFu);
    return max(m & 0xFFFFu, m >> 16);
  };
  float m = __uint_as_float(largest() << 16) * gain;
  if (!(m <= 3.4028234e38f)) {           // infinite (also times the gain) or NaN
    *bad = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if ((w[i] & 0x7FFFu) > 0x7F80u) w[i] &= 0xFFFF0000u;
      if ((w[i] >> 16 & 0x7FFFu) > 0x7F80u) w[i] &= 0xFFFFu;
    }
    m = __uint_as_float(largest() << 16) * gain;
  }
  // (4097 q less what it is past q: q in 12 bits; past 448 the scale saturates)
  const float q = fminf(m * (1.f / 6.f), 1024.f), t = __fmul_rn(q, 4097.f);
  *scale = to_e4m3(__fsub_rn(t, __fsub_rn(t, q)));
  if (*scale == 0) return make_uint2(0, 0);
  // (the gain is a power of two: its product with the reciprocal rounds nothing)
  float inv = f16x2_to_float2(e4m3x2_to_f16x2(*scale)).x;
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(inv));             // within 2^-23
  inv *= gain;
  // (an ulp between 512 and 1024 is 2^-14; quotients past 6 saturate, rounded or not)
  auto snap = [inv](uint32_t x) {
    return __fadd_rn(__fadd_rn(__fmul_rn(__uint_as_float(x), inv), 768.f), -768.f);
  };
  uint32_t o[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    o[i / 4] |= to_e2m1x2(snap(w[i] << 16), snap(w[i] & 0xFFFF0000u)) << (i % 4 * 8);
  return make_uint2(o[0], o[1]);
}

// Sixteen rows of the batch and one head to a CTA: a thread holds 16 dims of one row of K
// and V.  Their codes meet in shared memory in the cell's own layout, so that the rows'
// bytes, which lie 16 apart in a cell of V, leave 16 rows side by side; sixteen rows that
// are one whole cell leave as it is, 16 bytes a store.
// Floor: 2 bytes an element in, 0.5625 out (or back).  Prompts of 17,600 rows in all, 8 heads of
// 128 dims, take 21 us in and 33 back (48 one after the other: the way back then finds cells in
// L2), 4.3 and 2.8 TB/s: what bounds them is the passage through shared memory (its barriers and
// byte accesses) and the conversions, not the copies.  A few rows
// per sequence (blocks at batch 32) are launch and two dependent loads.
template <int D>
struct CellIo {
  static constexpr int kG = D / 16;
  static constexpr int kThreads = kCellRows * kG;
  static constexpr int kBytes = Cell<D>::kBytes;
};

// Eight bytes turned: byte j of the result is byte (j + n) % 8, 0 <= n <= 8.  The bytes of V of
// the threads of one row lie 128 apart, in one bank: each starts with another one.
__device__ __forceinline__ uint2 turn_right(uint2 x, int n) {
  if (n & 4) x = make_uint2(x.y, x.x);
  const uint32_t s = 8 * (n & 3);
  return make_uint2(__funnelshift_r(x.x, x.y, s), __funnelshift_r(x.y, x.x, s));
}

// The rows' places; true if they are rows 0 .. 15 of one cell.
template <int D>
__device__ __forceinline__ bool find_rows(const Kv4Store& s, const int32_t* slot, long long n0,
                                          long long n_tokens, int h, uint8_t** cells, int* rows,
                                          uint32_t* status) {
  if (threadIdx.x < kCellRows) {
    uint8_t* c = nullptr;
    int slab, row = 0;
    const long long n = n0 + threadIdx.x;
    if (n < n_tokens && find_slot(s, slot[n], &slab, &row, status))
      c = s.cells + cell_index(s, slab, h, row) * Cell<D>::kBytes;
    cells[threadIdx.x] = c;
    rows[threadIdx.x] = row % kCellRows;
  }
  __syncthreads();
  const int i = threadIdx.x % kCellRows;
  return __syncthreads_and(cells[0] != nullptr && cells[i] == cells[0] && rows[i] == i);
}

template <int D>
__global__ void __launch_bounds__(CellIo<D>::kThreads) kv4_append_kernel(
    const Kv4Store s, const uint16_t* __restrict__ k, long long k_pitch,
    const uint16_t* __restrict__ v, long long v_pitch, const int32_t* __restrict__ slot,
    long long n_tokens, uint32_t* status) {
  using C = CellIo<D>;
  __shared__ __align__(16) uint8_t image[C::kBytes];     // row i of the CTA in row i
  __shared__ uint8_t* cells[kCellRows];
  __shared__ int rows[kCellRows];
  griddep_wait();
  griddep_launch_dependents();
  // (heads vary fastest: neighbours read and write next to each other)
  const int h = blockIdx.x % s.n_kv_heads, r = threadIdx.x / C::kG, g = threadIdx.x % C::kG;
  const long long n0 = static_cast<long long>(blockIdx.x / s.n_kv_heads) * kCellRows, n = n0 + r;
  // (the rows are on their way before their places are known: two latencies side by side)
  uint4 kx[2] = {}, vx[2] = {};
  if (n < n_tokens) {
    const uint4* ks = reinterpret_cast<const uint4*>(k + n * k_pitch + h * D + 16 * g);
    const uint4* vs = reinterpret_cast<const uint4*>(v + n * v_pitch + h * D + 16 * g);
    kx[0] = ks[0];
    kx[1] = ks[1];
    vx[0] = vs[0];
    vx[1] = vs[1];
  }
  const float k_gain = pow2(-gain_exp(s.k_exp, h)), v_gain = pow2(-gain_exp(s.v_exp, h));
  const bool whole = find_rows<D>(s, slot, n0, n_tokens, h, cells, rows, status);
  if (cells[r]) {
    bool bad = false;
    uint32_t ks, vs;
    const uint2 kc = quantise16(kx[0], kx[1], k_gain, &ks, &bad);
    const uint2 vc = quantise16(vx[0], vx[1], v_gain, &vs, &bad);
    *reinterpret_cast<uint2*>(image + Cell<D>::k_codes(r, g)) = kc;
    image[Cell<D>::k_scale(r, g)] = static_cast<uint8_t>(ks);
    const uint2 turned = turn_right(vc, g);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      image[Cell<D>::v_codes(r, 8 * g + (j + g) % 8)] =
          static_cast<uint8_t>((j < 4 ? turned.x : turned.y) >> (8 * (j & 3)));
    image[Cell<D>::v_scale(r, g)] = static_cast<uint8_t>(vs);
    if (bad) set_status(status, DFLASH_ST_BAD_VALUE);
  }
  __syncthreads();
  if (whole) {
    for (int i = threadIdx.x; i < C::kBytes / 16; i += C::kThreads)
      reinterpret_cast<uint4*>(cells[0])[i] = reinterpret_cast<const uint4*>(image)[i];
    return;
  }
  // 16 lanes, 16 rows: K in pieces of 16 bytes, its scales in words, V byte by byte
  const int lr = threadIdx.x % kCellRows, lu = threadIdx.x / kCellRows;
  uint8_t* cell = cells[lr];
  if (!cell) return;
  const int to = rows[lr];
  for (int i = lu; i < D / 32; i += C::kG)
    *reinterpret_cast<uint4*>(cell + Cell<D>::k_codes(to, 2 * i)) =
        *reinterpret_cast<const uint4*>(image + Cell<D>::k_codes(lr, 2 * i));
  for (int i = lu; i < D / 64; i += C::kG)
    *reinterpret_cast<uint32_t*>(cell + Cell<D>::k_scale(to, 4 * i)) =
        *reinterpret_cast<const uint32_t*>(image + Cell<D>::k_scale(lr, 4 * i));
#pragma unroll
  for (int j = 0; j < 8; ++j)
    cell[Cell<D>::v_codes(to, lu + j * C::kG)] = image[Cell<D>::v_codes(lr, lu + j * C::kG)];
  cell[Cell<D>::v_scale(to, lu)] = image[Cell<D>::v_scale(lr, lu)];
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
__global__ void __launch_bounds__(CellIo<D>::kThreads) kv4_gather_kernel(
    const Kv4Store s, const int32_t* __restrict__ slot, uint16_t* __restrict__ k,
    uint16_t* __restrict__ v, long long n_tokens, uint32_t* status) {
  using C = CellIo<D>;
  __shared__ __align__(16) uint8_t image[C::kBytes];
  __shared__ uint8_t* cells[kCellRows];
  __shared__ int rows[kCellRows];
  griddep_wait();
  griddep_launch_dependents();
  const int h = blockIdx.x % s.n_kv_heads;
  const long long n0 = static_cast<long long>(blockIdx.x / s.n_kv_heads) * kCellRows;
  if (find_rows<D>(s, slot, n0, n_tokens, h, cells, rows, status)) {
    for (int i = threadIdx.x; i < C::kBytes / 16; i += C::kThreads)
      reinterpret_cast<uint4*>(image)[i] = reinterpret_cast<const uint4*>(cells[0])[i];
  } else {
    const int lr = threadIdx.x % kCellRows, lu = threadIdx.x / kCellRows;
    const uint8_t* cell = cells[lr];
    if (cell) {
      const int to = rows[lr];
      for (int i = lu; i < D / 32; i += C::kG)
        *reinterpret_cast<uint4*>(image + Cell<D>::k_codes(lr, 2 * i)) =
            *reinterpret_cast<const uint4*>(cell + Cell<D>::k_codes(to, 2 * i));
      for (int i = lu; i < D / 64; i += C::kG)
        *reinterpret_cast<uint32_t*>(image + Cell<D>::k_scale(lr, 4 * i)) =
            *reinterpret_cast<const uint32_t*>(cell + Cell<D>::k_scale(to, 4 * i));
#pragma unroll
      for (int j = 0; j < 8; ++j)
        image[Cell<D>::v_codes(lr, lu + j * C::kG)] = cell[Cell<D>::v_codes(to, lu + j * C::kG)];
      image[Cell<D>::v_scale(lr, lu)] = cell[Cell<D>::v_scale(to, lu)];
    }
  }
  __syncthreads();
  const int r = threadIdx.x / C::kG, g = threadIdx.x % C::kG;
  if (!cells[r]) return;
  const uint2 kc = *reinterpret_cast<const uint2*>(image + Cell<D>::k_codes(r, g));
  uint32_t turned[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    turned[j / 4] |= static_cast<uint32_t>(image[Cell<D>::v_codes(r, 8 * g + (j + g) % 8)])
                     << (8 * (j & 3));
  const uint2 vc = turn_right(make_uint2(turned[0], turned[1]), 8 - g % 8);
  const uint32_t sc = image[Cell<D>::k_scale(r, g)] | image[Cell<D>::v_scale(r, g)] << 8;
  const float2 f = f16x2_to_float2(e4m3x2_to_f16x2(sc));
  const float fk = f.x * pow2(gain_exp(s.k_exp, h)), fv = f.y * pow2(gain_exp(s.v_exp, h));
  const size_t at = (static_cast<size_t>(n0 + r) * s.n_kv_heads + h) * D + 16 * g;
  uint4* ko = reinterpret_cast<uint4*>(k + at);
  uint4* vo = reinterpret_cast<uint4*>(v + at);
  ko[0] = values8(kc.x, fk);
  ko[1] = values8(kc.y, fk);
  vo[0] = values8(vc.x, fv);
  vo[1] = values8(vc.y, fv);
}

}  // namespace

int kv4_store(const dflash_kv4_dims& d, const dflash_kv4_view* v, Kv4Store* s) {
  if (!v || !v->kv.k) return DFLASH_E_ARG;
  const dflash_kv_view& c = v->kv;
  if (c.page_table) {
    if (c.page_size < 1 || c.max_pages < 1 || c.n_pages < 1) return DFLASH_E_ARG;
    if (c.page_size % kCellRows) return DFLASH_E_UNSUPPORTED;
    s->slab_rows = c.page_size;
    s->n_slabs = c.n_pages;
  } else {
    if (c.capacity < 1) return DFLASH_E_ARG;
    if (c.capacity % kCellRows) return DFLASH_E_UNSUPPORTED;
    s->slab_rows = c.capacity;
    s->n_slabs = d.batch;
  }
  const long long rows = static_cast<long long>(s->slab_rows) * s->n_slabs;
  // slots and cell numbers are int32, and the tiles of a longest sequence end below 2^31
  const long long limit =
      c.page_table ? static_cast<long long>(c.max_pages) * c.page_size : c.capacity;
  if (rows > INT32_MAX || rows / kCellRows * d.n_kv_heads > INT32_MAX || limit > INT32_MAX - 512)
    return DFLASH_E_UNSUPPORTED;
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
  const long long ctas =
      static_cast<long long>((dims->n_tokens - 1) / kCellRows + 1) * dims->n_kv_heads;
  if (ctas > INT32_MAX) return DFLASH_E_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(ctas));
  const dim3 block(kCellRows * (dims->head_dim / 16));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto* kernel = dims->head_dim == 128 ? kv4_append_kernel<128> : kv4_append_kernel<64>;
  return launch(kernel, grid, block, 0, st, s, static_cast<const uint16_t*>(k),
                static_cast<long long>(k_pitch), static_cast<const uint16_t*>(v),
                static_cast<long long>(v_pitch), slot,
                static_cast<long long>(dims->n_tokens), ws_at<uint32_t>(ws, 0));
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
  const long long ctas =
      static_cast<long long>((dims->n_tokens - 1) / kCellRows + 1) * dims->n_kv_heads;
  if (ctas > INT32_MAX) return DFLASH_E_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(ctas));
  const dim3 block(kCellRows * (dims->head_dim / 16));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto* kernel = dims->head_dim == 128 ? kv4_gather_kernel<128> : kv4_gather_kernel<64>;
  return launch(kernel, grid, block, 0, st, s, slot, static_cast<uint16_t*>(k_out),
                static_cast<uint16_t*>(v_out), static_cast<long long>(dims->n_tokens),
                ws_at<uint32_t>(ws, 0));
}
