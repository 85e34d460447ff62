// Products of rows and weights held in 8 bits (e4m3) with a scale for each block of 128, plain
// and grouped by expert: the entry points, and which kernel takes a call.
#include <algorithm>
#include <cmath>

#include "fp8_linear.cuh"

namespace dflash {
namespace fp8 {
namespace {

// Which kernel takes a call (of p: sizes, whether there are start and rows, and the SMs); `rows`: of
// an expert, on average.
//
// Up to 16 rows (32, if there is one expert) the weights are streamed with the smallest tile that
// holds the rows: 128 experts of 4 rows by index x 1536 x 2048 take 53, 51, 52 us with tiles of 16,
// 32, 64 rows; 8 experts of 8 rows x 4096 x 2048 9.7, 10.7, 13.8; 24 rows x 4096 x 4096 7.9, 6.6,
// 7.5.  More rows: whichever the estimates say is the fastest.  Of 264 sizes of products by expert
// (4 to 128 experts of 1 to 1000 rows, by index and in order) the choice is 1.7 % slower on average
// than the fastest kernel.  The estimates were fitted to bursts (one call again and again, weights in
// L2 as far as they fit).  They order the kernels; as times they are low where many experts go to
// pairs: 64 experts of 512 rows on average x 2048 x 1408 85 us, 104 measured (117 in continuous use);
// 128 of 512 x 1536 x 2048 170, 208 (239).
//
// Examples, in us, of bursts.  Few features leave SMs without a tile: 128 rows x 4096 x 12288 take 17 streamed
// in shares of K, 30 with tiles; x 2560 x 2560 8.1 and 8.4; 200 rows x 512 x 768 4.4 and 5.3.
// Among tiles the fewest waves win, each worth its time: 512 rows x 4096 x 4096 take 12.6 with
// 128 x 128 tiles, 14.6 with 128 x 256, 14.1 with pairs; 128 rows x 24576 27, 24, 33; 512 rows x
// 24576 59, 54, 45; 2000 rows x 12288 x 256 16.0, 13.4, 13.3.  By index the copies of the rows bound
// the tiles: 16 experts of 80 rows x 1536 x 2048 take 14.5 with 128 x 256 tiles, 16.9 streamed 32
// rows at a time, 20 64 rows; in order 11.9, 16.3, 16.7; 64 experts of 400 rows 104, in order 91
// (pairs 88).  (Pairs by index were slower at every size.)
Choice choose(const Linear& p) {
  const int rows = static_cast<int>((static_cast<long long>(p.m) + p.groups - 1) / p.groups);
  if (rows <= (p.start ? 8 : 16)) return {16, 128};
  if (rows <= (p.start ? 16 : 32)) return {32, 128};
  // us: the start, and the waves of a tile's blocks and its end
  const auto cost = [&](int tile_rows, int features, int at_once, double start, double block,
                        double end) {
    const double tiles = row_tiles(p, tile_rows) * ((p.n + features - 1) / features);
    return start + std::ceil(tiles / at_once) * (p.k_blocks * block + end);
  };
  const double wide = p.rows ? cost(128, 256, p.sms, 4.2, 0.6, 0.8)
                             : cost(128, 256, p.sms, 3.6, 0.45, 0.8),
               pair = p.rows ? wide : cost(256, 256, p.sms / 2, 4.2, 0.33, 0.87),
               small = p.rows ? wide : cost(128, 128, p.sms, 3.0, 0.28, 0.6);
  const double tiles = std::min(small, std::min(wide, pair));
  const double thin = stream_cost(p, 32), thick = stream_cost(p, 64);
  if ((!p.start && rows <= 64) || std::min(thin, thick) < tiles)
    return {thin < thick ? 32 : 64, 128};
  if (tiles == small && !p.rows) return {128, 128};
  if (tiles == wide) return {128, 256};
  return {256, 256};
}

int run(Linear& p, cudaStream_t st) {
  p.sms = current_num_sms();
  if (p.sms <= 0) return DFLASH_E_CUDA;
  const Choice c = choose(p);
  return c.rows < 128 ? run_stream(p, c.rows, st) : run_tiles(p, c, st);
}

// Sizes that the kernels do not take, of the product and of x (rows of the weights and tiles are
// counted in 31 bits).
bool too_large(int m, int n_src, int groups, int n, int k) {
  return k % 16 || groups > kMaxGroups || static_cast<long long>(groups) * n > 0x7FFFFFFFll - 256 ||
         m > 0x7FFFFFFF - 256 || n > 0x7FFFFFFF - 256 || n_src > 0x7FFFFFFF - 256;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// What both calls check, and the fields they share.
int check(int m, int n_src, int groups, int n, int k, const void* x, const float* xs,
          const void* w, const float* ws, void* out, int64_t out_pitch, void* wsp,
          size_t ws_bytes, Linear* p) {
  if (m < 0 || n_src < 0 || groups < 1 || n < 1 || k < 1) return DFLASH_E_ARG;
  if (too_large(m, n_src, groups, n, k)) return DFLASH_E_UNSUPPORTED;
  if (m == 0) return DFLASH_OK;
  if (!x || !xs || !w || !ws || !out || out_pitch < n || n_src < 1) return DFLASH_E_ARG;
  if (!aligned16(x) || !aligned16(w) || !aligned4(xs) || !aligned4(ws) ||
      (reinterpret_cast<uintptr_t>(out) & 1u))
    return DFLASH_E_ALIGN;
  if (!wsp || ws_bytes < 64) return DFLASH_E_WORKSPACE;
  if (!aligned4(wsp)) return DFLASH_E_ALIGN;
  *p = Linear{};
  p->x = static_cast<const uint8_t*>(x);
  p->w = static_cast<const uint8_t*>(w);
  p->xs = xs;
  p->ws = ws;
  p->out = static_cast<uint16_t*>(out);
  p->out_pitch = out_pitch;
  p->status = static_cast<uint32_t*>(wsp);
  p->m = m;
  p->n = n;
  p->k = k;
  p->n_src = n_src;
  p->groups = groups;
  p->k_blocks = static_cast<int>(blocks(k));
  p->n_blocks = static_cast<int>(blocks(n));
  p->vector = aligned16(out) && out_pitch % 8 == 0;
  return DFLASH_OK;
}

}  // namespace
}  // namespace fp8
}  // namespace dflash

using namespace dflash;
using namespace dflash::fp8;

extern "C" int dflash_fp8_linear(int32_t rows, int32_t n_out, int32_t n_in, const void* x,
                                 const float* x_scale, const void* w, const float* w_scale,
                                 void* out, int64_t out_pitch, void* ws, size_t ws_bytes,
                                 dflash_stream_t stream) {
  DFLASH_ENTRY("dflash_fp8_linear");
  Linear p;
  const int rc = check(rows, rows, 1, n_out, n_in, x, x_scale, w, w_scale, out, out_pitch, ws,
                       ws_bytes, &p);
  if (rc || rows == 0) return rc;
  return run(p, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int dflash_fp8_grouped(int32_t n_rows, int32_t n_src, int32_t n_groups, int32_t n_out,
                                  int32_t n_in, const void* x, const float* x_scale,
                                  const void* w, const float* w_scale, const int32_t* start,
                                  const int32_t* rows, void* out, int64_t out_pitch, void* ws,
                                  size_t ws_bytes, dflash_stream_t stream) {
  DFLASH_ENTRY("dflash_fp8_grouped");
  Linear p;
  const int rc = check(n_rows, n_src, n_groups, n_out, n_in, x, x_scale, w, w_scale, out,
                       out_pitch, ws, ws_bytes, &p);
  if (rc || n_rows == 0) return rc;
  if (!start || (!rows && n_src != n_rows)) return DFLASH_E_ARG;
  if (!aligned4(start) || !aligned4(rows)) return DFLASH_E_ALIGN;
  // (rows named by an index are found by 32-bit offsets in units of 16 bytes)
  if (rows && static_cast<long long>(n_src) * (n_in / 16) >= 0xFFFFFFFFll)
    return DFLASH_E_UNSUPPORTED;
  p.start = start;
  p.rows = rows;
  return run(p, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int dflash_fp8_plan(int32_t n_rows, int32_t n_groups, int32_t n_out, int32_t n_in,
                               int by_index, int32_t num_sms, int32_t* tile_rows,
                               int32_t* tile_features, int32_t* shares) {
  static const int32_t some = 0;
  const int groups = n_groups > 0 ? n_groups : 1;
  if (n_rows < 1 || n_groups < 0 || n_out < 1 || n_in < 1 || num_sms < 0 || !tile_rows ||
      !tile_features || !shares)
    return DFLASH_E_ARG;
  if (too_large(n_rows, 1, groups, n_out, n_in)) return DFLASH_E_UNSUPPORTED;
  Linear p = {};
  p.m = n_rows;
  p.n = n_out;
  p.k = n_in;
  p.groups = groups;
  p.k_blocks = static_cast<int>(blocks(n_in));
  p.n_blocks = static_cast<int>(blocks(n_out));
  p.start = n_groups > 0 ? &some : nullptr;
  p.rows = n_groups > 0 && by_index ? &some : nullptr;
  p.sms = num_sms > 0 ? num_sms : current_num_sms();
  if (p.sms <= 0) return DFLASH_E_CUDA;
  const Choice c = choose(p);
  *tile_rows = c.rows;
  *tile_features = c.features;
  *shares = c.rows < 128 ? stream_shares(p, c.rows) : 1;
  return DFLASH_OK;
}
