// Products of rows and weights held in 8 bits (e4m3) with a scale for each block of 128, plain
// and grouped by expert: the entry points, and which kernel takes a call.
#include "fp8_linear.cuh"

namespace dflash {
namespace fp8 {
namespace {

// Which kernel takes a call; `rows`: of an expert, on average.
//
// Up to 64 rows the weights are streamed, with the smallest tile that holds the rows: 16 rows x
// 4096 x 4096 take 6.1, 7.0, 11.1 us with tiles of 16, 32, 64 rows (128 x 128 tiles: 18), 64 rows
// 10.6, 8.7, 8.9 (11.5).
//
// By expert (rows of 128 experts x 1536 x 2048 by index, in us): 32 rows each take 81, 66, 64 with
// tiles of 16, 32, 64 rows, 109 with 128 x 256; 80 rows 89 and 98; 192 rows 162, 153 and 155 with
// pairs; 384 rows 292, 247, 231.  Rows in order reach the tiles sooner: 80 rows 80 and 80, 256 rows
// 150, 126, 131, 512 rows 206 with 128 x 256 and 201 with pairs.
//
// Up to 128 rows, where features are so few that four CTAs share a tile's K, the stream is still
// the better one: 128 rows x 4096 x 12288 take 18 us, 30 with 128 x 128 tiles.
//
// Among tiles the fewest waves win, each worth its time: at K = 4096 a wave of 128 x 128 tiles takes
// 10 us, of 128 x 256 18 (its weights and rows need most of what L2 gives), of pairs 13.7.
// 512 rows x 4096 x 4096 take 12.6, 14.6, 14.1 us; 128 rows x 24576 27, 24, 33; 512 rows x 24576 60,
// 54, 46.
int choose(Linear& p, cudaStream_t st) {
  p.sms = current_num_sms();
  if (p.sms <= 0) return DFLASH_E_CUDA;
  const int rows = (p.m + p.groups - 1) / p.groups;
  if (rows <= 16) return run_stream(p, 16, st);
  if (rows <= 32) return run_stream(p, 32, st);
  if (rows <= (p.rows ? 96 : 64)) return run_stream(p, 64, st);
  if (p.start)
    return run_tiles(p, rows <= 320 ? Tiles::k128x256 : Tiles::k256x256, st);
  if (rows <= 128 && most_tiles(p, 64, 128) <= p.sms / 2) return run_stream(p, 64, st);
  const auto cost = [&](int tile_rows, int features, int at_once, double wave) {
    const long long tiles = most_tiles(p, tile_rows, features);
    return static_cast<double>((tiles + at_once - 1) / at_once) * wave;
  };
  const double small = cost(128, 128, p.sms, 10), wide = cost(128, 256, p.sms, 18),
               pair = cost(256, 256, p.sms / 2, 13.7);
  if (small <= wide && small <= pair) return run_tiles(p, Tiles::k128x128, st);
  return run_tiles(p, wide < pair ? Tiles::k128x256 : Tiles::k256x256, st);
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// What both calls check, and the fields they share.
int check(int m, int n_src, int groups, int n, int k, const void* x, const float* xs,
          const void* w, const float* ws, void* out, int64_t out_pitch, void* wsp,
          size_t ws_bytes, Linear* p) {
  if (m < 0 || n_src < 0 || groups < 1 || n < 1 || k < 1) return DFLASH_E_ARG;
  if (k % 16 || groups > kMaxGroups) return DFLASH_E_UNSUPPORTED;
  // rows of the weights and tiles are counted in 31 bits
  if (static_cast<long long>(groups) * n > 0x7FFFFFFFll - 256 || m > 0x7FFFFFFF - 256 ||
      n > 0x7FFFFFFF - 256 || n_src > 0x7FFFFFFF - 256)
    return DFLASH_E_UNSUPPORTED;
  if (m == 0) return DFLASH_OK;
  if (!x || !xs || !w || !ws || !out || out_pitch < n || n_src < 1) return DFLASH_E_ARG;
  if (!aligned16(x) || !aligned16(w) || !aligned4(xs) || !aligned4(ws) ||
      (reinterpret_cast<uintptr_t>(out) & 1u))
    return DFLASH_E_ALIGN;
  if (!wsp || ws_bytes < 64) return DFLASH_E_WORKSPACE;
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
  return choose(p, reinterpret_cast<cudaStream_t>(stream));
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
  return choose(p, reinterpret_cast<cudaStream_t>(stream));
}
