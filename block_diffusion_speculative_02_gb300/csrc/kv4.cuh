// The 4-bit KV cache as its kernels see it: cell layout, number formats and
// the argument checks its calls share.
#pragma once

#include "common.cuh"
#include "host.h"

namespace dflash {

constexpr int kCellRows = 16;
constexpr int kMaxKv4Batch = 4096;
constexpr int kMaxKv4Group = 64;
constexpr int kMaxGainExp = 64;

// Byte offsets inside the cell (16 rows of one KV head) of head dim D.
template <int D>
struct Cell {
  static constexpr int kBytes = 18 * D;
  static constexpr int kV = 8 * D;
  static constexpr int kKScale = 16 * D;
  static constexpr int kVScale = 17 * D;
  // the 8 bytes with dims 16 g .. 16 g + 15 of row r of K
  __host__ __device__ static constexpr int k_codes(int r, int g) {
    return (g >> 1) * 256 + r * 16 + (g & 1) * 8;
  }
  // the byte with dims 2 p, 2 p + 1 of row r of V
  __host__ __device__ static constexpr int v_codes(int r, int p) { return kV + p * 16 + r; }
  __host__ __device__ static constexpr int k_scale(int r, int g) {
    return kKScale + r * (D / 16) + g;
  }
  __host__ __device__ static constexpr int v_scale(int r, int g) { return kVScale + g * 16 + r; }
};

// Where the rows of a cache lie: slabs (pages, or sequences of a contiguous
// cache) of slab_rows rows, every slab [Hkv][slab_rows / 16] cells.
struct Kv4Store {
  uint8_t* cells;
  const int32_t* k_exp;
  const int32_t* v_exp;
  int n_kv_heads, slab_rows, n_slabs;
};

// Index of the cell that holds row `row` of slab `slab` for head h.
__device__ __forceinline__ size_t cell_index(const Kv4Store& s, int slab, int h, int row) {
  return (static_cast<size_t>(slab) * s.n_kv_heads + h) * (s.slab_rows / kCellRows) +
         row / kCellRows;
}

__device__ __forceinline__ int gain_exp(const int32_t* e, int h) {
  return e ? max(-kMaxGainExp, min(kMaxGainExp, e[h])) : 0;
}

__device__ __forceinline__ float pow2(int e) {  // -126 <= e <= 127
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Two bf16, to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// e4m3 code of x, to nearest even, saturating at 448.
__device__ __forceinline__ uint32_t to_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xFFu;
}

// Two e4m3 codes as f16x2 (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("{.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;}"
      : "=r"(r)
      : "r"(codes));
  return r;
}

// Two e2m1 codes (low nibble first) of one byte, to nearest even, saturating at 6.
__device__ __forceinline__ uint32_t to_e2m1x2(float lo, float hi) {
  uint16_t r;
  asm("{.reg .b8 t;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\t"
      "mov.b16 %0, {t, 0};}"
      : "=h"(r)
      : "f"(hi), "f"(lo));
  return r;
}

// The two e2m1 codes of byte B of a word as f16x2 (exact).
template <int B>
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b%2;}"
      : "=r"(r)
      : "r"(w), "n"(B));
  return r;
}

// The eight e2m1 codes of a word as four f16x2 (exact).
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&o)[4]) {
  o[0] = e2m1x2_to_f16x2<0>(w);
  o[1] = e2m1x2_to_f16x2<1>(w);
  o[2] = e2m1x2_to_f16x2<2>(w);
  o[3] = e2m1x2_to_f16x2<3>(w);
}

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t h) {
  float2 r;
  asm("{.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.f32.f16 %0, lo;\n\t"
      "cvt.f32.f16 %1, hi;}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h));
  return r;
}

// ----------------------------------------------------------------------------
// host side
// ----------------------------------------------------------------------------
int check_kv4_dims(const dflash_kv4_dims* d);

// Workspace: the status word, the page needs of dflash_kv_reserve, and the
// attention's plan and partial results.
struct Kv4Plan {
  size_t off_status, off_need, off_att, total;
};
int make_kv4_plan(const dflash_kv4_dims& d, Kv4Plan* p);
size_t kv4_attention_bytes(const dflash_kv4_dims& d);

// Checks the view and fills the store.
int kv4_store(const dflash_kv4_dims& d, const dflash_kv4_view* v, Kv4Store* s);

}  // namespace dflash
