// What the two kernels of the 8-bit products share (fp8_tiles.cu: many rows, fp8_stream.cu: few).
//
//   out[m, n] = sum_b sx[b, m] sw[n / 128, b] sum_{k in block b} x[m, k] w[n, k]
//
// The inner sum of a block of 128 columns is one step of the tensor cores (tcgen05, four
// products of K = 32 into a fresh TMEM accumulator); the outer one is kept in fp32 registers:
// the epilogue warps read each block's accumulator while the next blocks are multiplied, and
// add it times both scales.  One rounding, to bf16, at the end.
//
// Grouped by expert: rows start[e] .. start[e + 1] - 1 take the weights of expert e.  Every CTA
// turns start into a table of row tiles, so the number of rows of an expert never reaches the host.
// Tiles end with their expert: rows past it are multiplied (they are other rows of x, or zeros
// past its end), not stored.
//
// Rows of x that an index names are copied by one or two warps, 16 bytes a thread, into the order
// of the swizzle.  (Copies of four rows by the TMA took 50 to 150 ns each, 8 us a tile of 128 rows.)
#pragma once

#include "fp8.cuh"
#include "kv4_attention.cuh"   // elect_one, the register split, the shared-memory limit

namespace dflash {
namespace fp8 {

constexpr int kMaxGroups = 1024;
constexpr int kMaxStages = 8;
constexpr int kInfo = 4;            // tiles whose places are written down at a time

struct Linear {
  const uint8_t* x;      // [n_src][k]
  const uint8_t* w;      // [groups][n][k]
  const float* xs;       // [k / 128][n_src]
  const float* ws;       // [groups][n / 128][k / 128]
  const int32_t* start;  // [groups + 1], or null: one group, all rows
  const int32_t* rows;   // [m] or null
  uint16_t* out;
  long long out_pitch;
  uint32_t* status;
  int m, n, k, n_src, groups;
  int k_blocks, n_blocks;
  int n_tiles;
  int n_stages;
  int vector;            // out and its pitch are aligned to 16 bytes
  int sms;               // of the device
  int box_rows;          // rows of a copy of x: of a tile, or all there are if they are fewer (rows
                         // past the end of x, which the TMA fills with zeros, cost 2 ns each)
};

// What is the same all over the warp anyway, so that the compiler sees it and keeps what is
// made of it in uniform registers: where it does not, an instruction of the tensor cores or of
// the copies costs some 150 clocks to issue (measured), and a block of K takes ten.
__device__ __forceinline__ int same(int x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ bool all(bool x) { return __all_sync(0xffffffffu, x); }

using kv4::elect_one;
using kv4::wait_on;

// Both barriers' phases, tried together first: one after the other each try costs the warp
// that issues the products some 130 clocks.
__device__ __forceinline__ bool wait_both(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb,
                                          uint32_t* status) {
  uint32_t ok;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
      "and.pred p, p, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(a)), "r"(pa), "r"(smem_u32(b)), "r"(pb)
      : "memory");
  if (all(ok)) return true;
  // (lanes that saw the phase in the last try and lanes that gave up decide together, before the
  // second wait, which the warp enters as a whole or not at all)
  if (!all(wait_on(a, pa, status))) return false;
  return all(wait_on(b, pb, status));
}

// --------------------------------------------------------------------------------------------
// tensor cores and copies
// --------------------------------------------------------------------------------------------
// Instruction descriptor, kind::f8f6f4: A = B = e4m3 (0), D = fp32, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

template <bool kPair = false>
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
#define DFLASH_MMA(group)                                                              \
  asm volatile(                                                                        \
      "{\n\t.reg .pred p;\n\t"                                                     \
      "setp.ne.b32 p, %4, 0;\n\t"                                                    \
      "tcgen05.mma." group ".kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),    \
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)                                      \
      : "memory")
  if (kPair)
    DFLASH_MMA("cta_group::2");
  else
    DFLASH_MMA("cta_group::1");
#undef DFLASH_MMA
}

// Arrive on `bar`, of a pair in both CTAs, once the products issued so far are done.
template <bool kPair>
__device__ __forceinline__ void mma_done(uint64_t* bar) {
  if (kPair)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    umma_commit(bar);
}

// Likewise, in this CTA only.
template <bool kPair>
__device__ __forceinline__ void mma_done_here(uint64_t* bar) {
  if (kPair)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            smem_u32(bar))
        : "memory");
  else
    umma_commit(bar);
}

template <bool kPair>
__device__ __forceinline__ void tmem_take(uint32_t* slot, uint32_t cols) {
  if (kPair) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(slot)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(slot, cols);
    tmem_relinquish();
  }
}

template <bool kPair>
__device__ __forceinline__ void tmem_give(uint32_t taddr, uint32_t cols) {
  if (kPair)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols)
                 : "memory");
  else
    tmem_dealloc(taddr, cols);
}

// Copy four bytes (size 0: write a zero).
__device__ __forceinline__ void cp_async4(void* dst, const void* src, uint32_t size) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(size)
               : "memory");
}

// Arrive (one of the count) once this thread's copies so far are there.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// Arrive at a named barrier of n threads without waiting at it.
__device__ __forceinline__ void named_bar_arrive(uint32_t id, uint32_t n) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// A watcher's turn: waits at both mbarriers for the warps that meet it at named barrier `id` (n
// threads with its own), and returns whether to go on waiting.  While it does (ok), it only arrives
// there.  Once a wait gave up, the rest are skipped, and it syncs instead: arriving without a wait
// between would run ahead of the other warps, and the barrier's count no longer mean one turn.
__device__ __forceinline__ bool hand_over(bool ok, uint64_t* a, uint32_t pa, uint64_t* b,
                                          uint32_t pb, uint32_t id, uint32_t n, uint32_t* status) {
  ok = ok && wait_both(a, pa, b, pb, status);
  if (ok)
    named_bar_arrive(id, n);
  else
    named_bar_sync(id, n);
  return ok;
}

// The barrier of this name in the first CTA of a pair (a single CTA: its own).
template <bool kPair>
__device__ __forceinline__ uint32_t first_cta(uint64_t* bar) {
  uint32_t a = smem_u32(bar);
  if (kPair) asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(bar)));
  return a;
}

template <bool kPair>
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  if (kPair)
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
  else
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// 2-D tiled load whose bytes count at a barrier of either CTA of a pair.
template <bool kPair>
__device__ __forceinline__ void tma_box(void* dst, const CUtensorMap* map, uint32_t bar, int c0,
                                        int c1, uint64_t policy) {
#define DFLASH_LOAD(group)                                                                    \
  asm volatile(                                                                               \
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes" group \
      ".L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(dst)),                 \
      "l"(map), "r"(bar), "r"(c0), "r"(c1), "l"(policy)                                       \
      : "memory")
  if (kPair)
    DFLASH_LOAD(".cta_group::2");
  else
    DFLASH_LOAD("");
#undef DFLASH_LOAD
}

// 32 TMEM lanes x 16 columns of fp32; thread i gets lane (base + i), two columns to a word.
// The load, the wait for it and the pairs are one statement, so that the pairs are made where
// the load puts them (apart, the compiler moved every value twice).
__device__ __forceinline__ void tmem_pairs(uint32_t taddr, uint64_t (&d)[8]) {
  asm volatile(
      "{\n\t.reg .b32 r<16>;\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{r0, r1, r2, r3, r4, r5, r6, r7, r8, r9, r10, r11, r12, r13, r14, r15}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n\t"
      "mov.b64 %0, {r0, r1};\n\tmov.b64 %1, {r2, r3};\n\t"
      "mov.b64 %2, {r4, r5};\n\tmov.b64 %3, {r6, r7};\n\t"
      "mov.b64 %4, {r8, r9};\n\tmov.b64 %5, {r10, r11};\n\t"
      "mov.b64 %6, {r12, r13};\n\tmov.b64 %7, {r14, r15};\n\t}\n"
      : "=l"(d[0]), "=l"(d[1]), "=l"(d[2]), "=l"(d[3]), "=l"(d[4]), "=l"(d[5]), "=l"(d[6]),
        "=l"(d[7])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 halves(uint64_t d) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(d));
  return f;
}

// a += f * t, both halves.
__device__ __forceinline__ void fma_pair(uint64_t& a, uint64_t t, uint64_t f) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(t), "l"(f));
}

__device__ __forceinline__ uint32_t pack_bf16(uint64_t d) {
  const float2 f = halves(d);
  const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// --------------------------------------------------------------------------------------------
// row tiles of the groups
// --------------------------------------------------------------------------------------------
// In shared memory: first row and number of rows of each group, and how many row tiles the
// groups before it have.  A group whose rows do not lie in 0 .. m, or that starts before the end of
// one before it, counts none: no row has two owners, and there are no more tiles than most_tiles.
struct Groups {
  int* first;   // [groups]
  int* count;   // [groups]
  int* tiles;   // [groups + 1]
};

__host__ __device__ constexpr int groups_bytes(int groups) { return (3 * groups + 1) * 4; }

__device__ __forceinline__ Groups groups_at(uint8_t* smem, int groups) {
  int* p = reinterpret_cast<int*>(smem);
  return {p, p + groups, p + 2 * groups};
}

// By the whole block, of n threads.
__device__ __forceinline__ void fill_groups(const Linear& p, const Groups& g, int tile_rows,
                                            int n) {
  if (!p.start) {
    if (threadIdx.x == 0) {
      g.first[0] = 0;
      g.count[0] = p.m;
      g.tiles[0] = 0;
      g.tiles[1] = (p.m + tile_rows - 1) / tile_rows;
    }
    return;                              // (the caller's barrier follows)
  }
  int bad = 0;
  for (int e = threadIdx.x; e < p.groups; e += n) {
    int a = p.start[e], b = p.start[e + 1];
    if (a < 0 || b < a || b > p.m) {
      bad = 1;
      a = b = 0;
    }
    g.first[e] = a;
    g.count[e] = b - a;
  }
  if (__syncthreads_or(bad)) {           // (where none is, every group starts where one ended)
    if (threadIdx.x == 0) {
      set_status(p.status, DFLASH_ST_CAPACITY);
      int end = 0;
      for (int e = 0; e < p.groups; ++e) {
        if (g.count[e] == 0) continue;
        if (g.first[e] < end)
          g.count[e] = 0;
        else
          end = g.first[e] + g.count[e];
      }
    }
    __syncthreads();
  }
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int sum = 0;
    for (int e0 = 0; e0 < p.groups; e0 += 32) {
      const int e = e0 + lane;
      const int own = e < p.groups ? (g.count[e] + tile_rows - 1) / tile_rows : 0;
      int t = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) t += y;
      }
      if (e < p.groups) g.tiles[e] = sum + t - own;
      sum += __shfl_sync(0xffffffffu, t, 31);
    }
    if (lane == 0) g.tiles[p.groups] = sum;
  }
}

// The group that row tile i (< tiles[groups]) belongs to: the last one with tiles[e] <= i.
__device__ __forceinline__ int group_of(const Groups& g, int groups, int i) {
  int lo = 0, hi = groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (g.tiles[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

constexpr int kBand = 64;   // row tiles of a band
constexpr int kChunk = 4;   // feature tiles that neighbours take of the same rows

struct Tile {
  int e, n, row, count;     // group, feature tile, first row, its rows (1 ..)
};

// Tile t of the walk: groups one after the other, in a group bands of kBand row tiles, in a band
// chunks of kChunk feature tiles, in a chunk the features fastest.  A wave shares weights, which
// leave memory once a band; a band's rows stay in L2; neighbours ask for the same rows at the same
// time.  (8192 rows x 4096 x 12288 in continuous use: 313 us, 325 with the rows fastest; 128 experts
// of 512 rows by index x 1536 x 2048 257 and 254, of 200 rows 125 and 126; other sizes alike.)
template <int kRows>
__device__ __forceinline__ Tile tile_at(const Linear& p, const Groups& g, int t) {
  const int e = p.groups > 1 ? group_of(g, p.groups, t / p.n_tiles) : 0;
  int r = t - g.tiles[e] * p.n_tiles;
  const int band = r / (kBand * p.n_tiles);
  r -= band * kBand * p.n_tiles;
  const int height = min(kBand, g.tiles[e + 1] - g.tiles[e] - band * kBand);
  const int chunk = r / (kChunk * height);
  r -= chunk * kChunk * height;
  const int width = min(kChunk, p.n_tiles - chunk * kChunk);
  const int i = band * kBand + r / width, n = chunk * kChunk + r % width;
  return {e, n, g.first[e] + i * kRows, min(kRows, g.count[e] - i * kRows)};
}

// The row of x that row at of a tile is made of; none: -1.
__device__ __forceinline__ int source_row(const Linear& p, const Tile& tile, int at) {
  if (at >= tile.count) return -1;
  if (!p.rows) return tile.row + at;
  const int r = p.rows[tile.row + at];
  if (r >= 0 && r < p.n_src) return r;
  set_status(p.status, DFLASH_ST_CAPACITY);
  return -1;
}

// Where rows named by an index are, for the copies: row r of kRows at sources[place_of(r)], in
// units of 16 bytes from x on, or kNoRow (zeros).  The rows that eight lanes copy lie side by side.
constexpr uint32_t kNoRow = 0xFFFFFFFFu;

template <int kRows>
__device__ __forceinline__ int place_of(int r) {
  return (r & 3) * (kRows / 4) + (r >> 2);
}

// By one warp: block columns col .. col + 127 of kRows rows of x (from row `first` of kOf on), into
// the order of the 128-byte swizzle.  Few instructions a copy count here: the warp has few turns
// and registers.
template <int kRows, int kOf>
__device__ __forceinline__ void copy_rows(const Linear& p, uint8_t* dst, int col,
                                          const uint32_t* sources, int first, int lane) {
  const int c = lane & 7, at = col + c * 16;
  const uint32_t* from = sources + (lane >> 3) * (kOf / 4) + first / 4;
  const uint8_t* x = p.x + (at < p.k ? at : 0);
  const uint32_t to = smem_u32(dst) + (first + (lane >> 3)) * kBlockK;
#pragma unroll
  for (int i = 0; i < kRows / 4; i += 4) {
    const uint4 s = *reinterpret_cast<const uint4*>(from + i);
    const uint32_t v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = (i + j) * 4;                     // and lane >> 3; first is a multiple of 8
      const bool there = v[j] != kNoRow && at < p.k;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                       to + row * kBlockK + ((c ^ ((row + (lane >> 3)) & 7)) << 4)),
                   "l"(x + (there ? static_cast<size_t>(v[j]) * 16 : 0)), "r"(there ? 16 : 0)
                   : "memory");
    }
  }
}

// One warp's copies: each block into the next stage.  They arrive at the stage's barrier themselves
// (landed, 32 for a warp) when they are there; who hands them on to the tensor cores fences.
// (Announced by the warp itself two blocks later, 128 experts of 200 rows x 1536 x 2048 took 155
// us, 112 this way, in bursts.)
struct RowCopies {
  uint32_t stage = 0, phase = 0;   // of the next block to copy

  template <int kRows, int kOf>
  __device__ __forceinline__ bool tile(const Linear& p, uint8_t* base, int stage_bytes,
                                       uint64_t* empty, uint64_t* landed, int b_first, int b_last,
                                       const uint32_t* sources, int first, int lane) {
#pragma unroll 1
    for (int b = b_first; b < b_last; ++b) {
      if (!all(wait_on(&empty[stage], phase ^ 1, p.status))) return false;
      copy_rows<kRows, kOf>(p, base + stage * stage_bytes, b * kBlockK, sources, first, lane);
      cp_async_arrive(&landed[stage]);
      if (++stage == static_cast<uint32_t>(p.n_stages)) {
        stage = 0;
        phase ^= 1;
      }
    }
    return true;
  }
};

// --------------------------------------------------------------------------------------------
// host
// --------------------------------------------------------------------------------------------
// 2-D map over a row-major [rows, cols] matrix of bytes, box 128 columns x box_rows, 128-byte
// swizzle.
inline int make_map(CUtensorMap* map, const void* base, long long cols, long long rows,
                    int box_rows) {
  return make_tmap_2d_u8(map, base, static_cast<uint64_t>(cols), static_cast<uint64_t>(rows),
                         static_cast<uint64_t>(cols), kBlockK, static_cast<uint32_t>(box_rows));
}

// Tiles, at most: one row tile more for each group than the rows fill.
inline long long most_tiles(const Linear& p, int tile_rows, int tile_cols) {
  const long long n_tiles = (static_cast<long long>(p.n) + tile_cols - 1) / tile_cols;
  if (!p.start) return (static_cast<long long>(p.m) + tile_rows - 1) / tile_rows * n_tiles;
  return (p.m / tile_rows + static_cast<long long>(p.groups < p.m ? p.groups : p.m)) * n_tiles;
}

// Row tiles, about: the rows of an expert are not known here, so that on average 0.6 of a tile of
// each goes without rows.
inline double row_tiles(const Linear& p, int tile_rows) {
  if (!p.start) return (p.m + tile_rows - 1) / tile_rows;
  const double with_rows = p.groups < p.m ? p.groups : p.m, own = p.m / with_rows / tile_rows + 0.6;
  return with_rows * (own > 1 ? own : 1);
}

// Rows and features of a tile.
struct Choice {
  int rows, features;
};
// Tiles of 128 rows x 128 or 256 features, or, of a pair of CTAs, 256 x 256; of rows by index
// 128 x 256.
int run_tiles(const Linear& p, Choice tile, cudaStream_t st);
// At most `rows` (16, 32 or 64) rows at a time against weights streamed once.
int run_stream(const Linear& p, int rows, cudaStream_t st);
// CTAs that share a tile's K there, and about how many us that takes (32 or 64).
int stream_shares(const Linear& p, int rows);
double stream_cost(const Linear& p, int rows);

}  // namespace fp8
}  // namespace dflash
