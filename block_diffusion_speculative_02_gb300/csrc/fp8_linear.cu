// Products of rows and weights held in 8 bits (e4m3) with a scale for each block of 128, plain
// and grouped by expert:
//
//   out[m, n] = sum_b sx[b, m] sw[n / 128, b] sum_{k in block b} x[m, k] w[n, k]
//
// The inner sum of a block of 128 columns is one step of the tensor cores (tcgen05, four
// products of K = 32 into a fresh TMEM accumulator); the outer one is kept in fp32 registers:
// the epilogue warps read each block's accumulator while the next block is multiplied, and
// add it times both scales.  One rounding, to bf16, at the end.
//
// Grouped: rows start[e] .. start[e + 1] - 1 take the weights of expert e.  Every CTA turns
// start into a table of row tiles, so the number of rows of an expert never reaches the host.
// Tiles end with their expert: rows past it are multiplied (they are other rows of x, or zeros
// past its end), not stored.
#include "fp8.cuh"
#include "kv4_attention.cuh"   // bounded waits that hold one register, register split

namespace dflash {
namespace fp8 {
namespace {

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
  if (__all_sync(0xffffffffu, ok)) return true;
  ok = wait_on(a, pa, status) && wait_on(b, pb, status);
  return __all_sync(0xffffffffu, ok);
}

constexpr int kMaxGroups = 1024;

struct Linear {
  const float* xs;       // [K / 128][n_src]
  const float* ws;       // [groups][N / 128][K / 128]
  const int32_t* start;  // [groups + 1], or null: one group, all rows
  const int32_t* rows;   // [m] or null
  uint16_t* out;
  long long out_pitch;
  uint32_t* status;
  int m, n, n_src, groups;
  int k_blocks, n_blocks;
  int n_tiles;
  int n_stages;
  int vector;            // 16-byte stores: out and its pitch are aligned
};

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
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
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

// Four rows of a map whose box is one row high, one below the other in shared memory.  A row
// past the map's end reads as zeros.
template <bool kPair>
__device__ __forceinline__ void tma_gather4(void* dst, const CUtensorMap* map, uint32_t bar,
                                            int c0, int r0, int r1, int r2, int r3,
                                            uint64_t policy) {
#define DFLASH_LOAD(group)                                                                     \
  asm volatile(                                                                                \
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes" \
      group ".L2::cache_hint [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(smem_u32(dst)), \
      "l"(map), "r"(bar), "r"(c0), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "l"(policy)             \
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

// What is the same all over the warp anyway, so that the compiler sees it and keeps what is
// made of it in uniform registers: where it does not, an instruction of the tensor cores or of
// the copies costs some 150 clocks to issue (measured), and a block of K takes ten.
__device__ __forceinline__ int same(int x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ bool all(bool x) { return __all_sync(0xffffffffu, x); }

__device__ __forceinline__ uint32_t pack_bf16(uint64_t d) {
  const float2 f = halves(d);
  const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// --------------------------------------------------------------------------------------------
// row tiles of the groups
// --------------------------------------------------------------------------------------------
// In shared memory: first row and number of rows of each group, and how many row tiles the
// groups before it have.  A group whose rows do not lie in 0 .. m counts none.
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
  for (int e = threadIdx.x; e < p.groups; e += n) {
    int a = p.start[e], b = p.start[e + 1];
    if (a < 0 || b < a || b > p.m) {
      set_status(p.status, DFLASH_ST_CAPACITY);
      a = b = 0;
    }
    g.first[e] = a;
    g.count[e] = b - a;
  }
  __syncthreads();
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

struct Tile {
  int e, n, row, count;     // group, feature tile, first row, its rows (1 ..)
};

// Tile t of the walk: groups one after the other, in a group bands of kBand row tiles, in a band
// the row tile fastest: the CTAs of a wave share weights, and a band's rows stay in L2.
template <int kRows>
__device__ __forceinline__ Tile tile_at(const Linear& p, const Groups& g, int t) {
  const int e = p.groups > 1 ? group_of(g, p.groups, t / p.n_tiles) : 0;
  int r = t - g.tiles[e] * p.n_tiles;
  const int band = r / (kBand * p.n_tiles);
  r -= band * kBand * p.n_tiles;
  const int height = min(kBand, g.tiles[e + 1] - g.tiles[e] - band * kBand);
  const int n = r / height, i = band * kBand + r - n * height;
  return {e, n, g.first[e] + i * kRows, min(kRows, g.count[e] - i * kRows)};
}

// The rows of x that a tile's rows at .. at + 3 are made of, for a copy by row; none: past the
// end of x, which reads as zeros.
__device__ __forceinline__ void rows_of(const Linear& p, const Tile& tile, int at, int (&r)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = at + i < tile.count ? p.rows[tile.row + at + i] : p.n_src;
    if (r[i] < 0 || r[i] >= p.n_src) {
      if (at + i < tile.count) set_status(p.status, DFLASH_ST_CAPACITY);
      r[i] = p.n_src;
    }
  }
}

// --------------------------------------------------------------------------------------------
// tiles of 128 rows (or, of a pair of CTAs, 256) x kN features
// --------------------------------------------------------------------------------------------
// One thread issues the products, of a pair (kPair) for both SMs: each holds 128 rows of x and half
// of the features' weights, and gets the sums of its own rows.  Per block of K a pair of SMs moves
// and reads half as many bytes of weights as two single ones.
//
// A block's sums leave TMEM in the time of the next block's products (512 cycles at 256
// features): 16 warps take a quarter of the features of 32 rows each, so that four warps of
// a scheduler cover each other's waits.  (8 warps with twice the features each left the tensor
// cores idle 60 % of the time.)  They wait at named barriers, where a warp takes no turn: one more
// warp watches the accumulators' mbarriers for them.  (With all of them trying an mbarrier, a
// try took the warps that issue the products 400 clocks and more.)
constexpr int kTileRows = 128;
// Warps: 0 copies, 1 and 3 products, 2 scales, 4 and 5 watch, two idle, 16 of the epilogue.
constexpr int kTileWarps = 24;
constexpr int kEpiWarp = 8, kEpiWarps = 16;
// Registers a thread: 80 at the start; the epilogue's warps take from the others, within the
// block's 768 x 80.
constexpr int kRegsStart = 80, kRegsRest = 32, kRegsEpi = 104;
static_assert(kEpiWarp * kRegsRest + kEpiWarps * kRegsEpi <= kTileWarps * kRegsStart,
              "register split");
constexpr int kMaxStages = 8;
constexpr int kRing = 8;                        // blocks whose scales are in shared memory
constexpr int kScaleRow = kTileRows + 2;        // of the rows, then of the weights
constexpr int kSmemLimit = 227 * 1024;

template <bool kPair, int kN>
__host__ __device__ constexpr int tile_stage_bytes() {
  return (kTileRows + kN / (kPair ? 2 : 1)) * kBlockK;
}

// kW features of 32 rows, one row to a lane, go through shared memory (in the order that the copies
// swizzle to) and leave as one copy; where rows of another expert are among the 32, or out
// is not aligned, row by row.  The copy is on its way when this returns.
template <int kW>
__device__ __forceinline__ void store_rows(const Linear& p, const CUtensorMap* map,
                                           const uint64_t* acc, uint8_t* buf, int row,
                                           int rows_left, int col, int lane) {
  static_assert(kW == 64 || kW == 32, "swizzles");
  const auto at = [&](int r, int c) {
    return buf + r * kW * 2 + ((kW == 64 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
  };
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
#pragma unroll
  for (int c = 0; c < kW / 8; ++c)
    *reinterpret_cast<uint4*>(at(lane, c)) =
        make_uint4(pack_bf16(acc[4 * c]), pack_bf16(acc[4 * c + 1]), pack_bf16(acc[4 * c + 2]),
                   pack_bf16(acc[4 * c + 3]));
  // (The map ends with out: rows past its end are not written, nor are columns, of which a copy
  // takes eight or none.)
  if (p.vector && (rows_left >= 32 || !p.start) && (col + kW <= p.n || p.n % 8 == 0)) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && rows_left > 0 && col < p.n) {
      asm volatile(
          "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
          "r"(col), "r"(row), "r"(smem_u32(buf))
          : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
    return;
  }
  __syncwarp();
  const int most = min(32, rows_left);
  if (p.vector && col + kW <= p.n) {
    constexpr int kLanes = kW / 8;           // to a row
    const int c = lane % kLanes;
#pragma unroll
    for (int i = 0; i < kLanes; ++i) {
      const int r = i * (32 / kLanes) + lane / kLanes;
      const uint4 v = *reinterpret_cast<const uint4*>(at(r, c));
      if (r < most)
        *reinterpret_cast<uint4*>(p.out + static_cast<long long>(row + r) * p.out_pitch + col +
                                  8 * c) = v;
    }
  } else {
    for (int r = 0; r < most; ++r)
#pragma unroll
      for (int j = lane; j < kW; j += 32)
        if (col + j < p.n)
          p.out[static_cast<long long>(row + r) * p.out_pitch + col + j] =
              *reinterpret_cast<const uint16_t*>(at(r, j >> 3) + (j & 7) * 2);
  }
  __syncwarp();
}

template <bool kPair, int kN>
__global__ void __launch_bounds__(kTileWarps * 32, 1)
tile_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
            const __grid_constant__ CUtensorMap map_out, const Linear p) {
  constexpr int kCtas = kPair ? 2 : 1;
  constexpr int kRows = kTileRows * kCtas;
  constexpr int kStage = tile_stage_bytes<kPair, kN>();
  constexpr int kHalf = kN / 2;          // features of a product
  constexpr int kShare = kHalf / kCtas;  // of these, features whose weights this CTA holds
  constexpr int kOwn = kN / 4;           // features of an epilogue warp
  constexpr int kStore = 32 * kOwn * 2;  // its rows on their way out
  constexpr int kCols = 2 * kN;          // TMEM columns: two accumulators of each half
  constexpr int kBlocksN = kN / kBlockK;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  uint8_t* store = smem + p.n_stages * kStage;
  float* scales = reinterpret_cast<float*>(store + kEpiWarps * kStore);   // [kRing][128 rows, weights]
  int4* tiles = reinterpret_cast<int4*>(scales + kRing * kScaleRow);  // [2 halves][4] for the
                                                                      // epilogue
  uint64_t* full = reinterpret_cast<uint64_t*>(tiles + 8);
  uint64_t* empty = full + p.n_stages;
  uint64_t* tfull = empty + p.n_stages;  // [2 halves][2] accumulators are there
  uint64_t* tempty = tfull + 4;          // [2 halves][2] read (of a pair: in the first CTA)
  uint64_t* mdrain = tempty + 4;         // [2 halves]
  uint64_t* sfull = mdrain + 2;          // [kRing] scales are there
  uint64_t* sempty = sfull + kRing;      // [kRing] both halves' sums of that block are there
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sempty + kRing);
  const Groups groups = groups_at(reinterpret_cast<uint8_t*>(tmem_slot + 1), p.groups);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = kPair ? static_cast<int>(cluster_ctarank()) : 0;
  const int t_first = blockIdx.x / kCtas, t_step = gridDim.x / kCtas;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.n_stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 2);           // the products of both halves
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], kEpiWarps / 2 * kCtas);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&mdrain[i], 1);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sfull[i], 32);
      mbar_init(&sempty[i], 2);
    }
    fence_mbar_init();
  }
  if (warp == 1) tmem_take<kPair>(tmem_slot, kCols);
  if (warp == 2 && elect_one()) {
    tma_prefetch_desc(&map_x);
    tma_prefetch_desc(&map_w);
    if (p.vector) tma_prefetch_desc(&map_out);
  }
  griddep_wait();
  griddep_launch_dependents();           // (they wait for the end of this grid before they read)
  fill_groups(p, groups, kRows, kTileWarps * 32);
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();             // the other CTA's barriers are there
  tc_fence_after();
  const uint32_t tmem = same(*tmem_slot);
  const int total = groups.tiles[p.groups] * p.n_tiles;   // (below 2^31: the host)
  if (warp < kEpiWarp) kv4::regs_down<kRegsRest>();

  if (warp == 0) {
    const uint64_t pol = l2_policy_evict_normal();
    uint32_t stage = 0, phase = 0;
    int issued = 0;
    bool ok = true;
    for (int t = t_first; all(ok && t < total); t += t_step) {
      const Tile tile = tile_at<kRows>(p, groups, t);
      int r[4] = {};
      if (p.rows) rows_of(p, tile, rank * kTileRows + lane * 4, r);
      const int x_row = same(tile.row) + rank * kTileRows;
      const int w_row = same(tile.e * p.n + tile.n * kN) + rank * kShare;
#pragma unroll 1
      for (int b = 0; b < p.k_blocks; ++b) {
        ok = all(wait_on(&empty[stage], phase ^ 1, p.status));
        if (!ok) break;
        uint8_t* a = smem + stage * kStage;
        const uint32_t bar = first_cta<kPair>(&full[stage]);
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], kCtas * kStage);
          if (!p.rows) tma_box<kPair>(a, &map_x, bar, b * kBlockK, x_row, pol);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            tma_box<kPair>(a + (kTileRows + h * kShare) * kBlockK, &map_w, bar, b * kBlockK,
                           w_row + h * kHalf, pol);
        }
        if (p.rows) {
          __syncwarp();
          tma_gather4<kPair>(a + lane * 4 * kBlockK, &map_x, bar, b * kBlockK, r[0], r[1], r[2],
                             r[3], pol);
        }
        ++issued;
        if (++stage == static_cast<uint32_t>(p.n_stages)) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    // No copy may still be landing, and no product's arrival be on its way, when the CTA exits:
    // every stage has been read.  (Given up: what the first CTA's barriers counted has landed.)
    if (lane == 0)
      for (int st = 0; st < p.n_stages && st < issued; ++st) {
        const int last = st + ((issued - 1 - st) / p.n_stages) * p.n_stages;
        if (!ok && rank) break;
        if (!mbar_wait_drain(ok ? &empty[st] : &full[st],
                             static_cast<uint32_t>((last / p.n_stages) & 1), p.status))
          break;
      }
  } else if (warp == 1 || warp == 3) {
    if (rank == 0) {
      // a warp to each half of the features
      const int half = warp >> 1;
      constexpr uint32_t idesc = idesc_e4m3(kRows, kHalf);
      const uint64_t a_desc = umma_sdesc_sw128(smem_u32(smem));
      const uint64_t b_desc =
          umma_sdesc_sw128(smem_u32(smem) + (kTileRows + half * kShare) * kBlockK);
      const uint32_t acc = tmem + half * 2 * kHalf;
      uint64_t* done = tfull + 2 * half;
      uint64_t* read = tempty + 2 * half;
      uint32_t stage = 0, phase = 0, slot = 0, tphase = 0;
      bool ok = true;
      for (int t = t_first; all(ok && t < total); t += t_step) {
#pragma unroll 1
        for (int b = 0; b < p.k_blocks; ++b) {
          // (the wait for a phase before the first passes at once)
          ok = wait_both(&read[slot], tphase ^ 1, &full[stage], phase, p.status);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t ad = a_desc + stage * (kStage >> 4), bd = b_desc + stage * (kStage >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_e4m3<kPair>(acc + slot * kHalf, ad + 2 * kk, bd + 2 * kk, idesc, kk ? 1u : 0u);
            mma_done<kPair>(&done[slot]);
            mma_done<kPair>(&empty[stage]);
          }
          tphase ^= slot;
          slot ^= 1;
          if (++stage == static_cast<uint32_t>(p.n_stages)) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (elect_one()) mma_done_here<kPair>(&mdrain[half]);
      if (lane == 0) mbar_wait_drain(&mdrain[half], 0, p.status);
    }
  } else if (warp == 2) {
    // Copies the scales, kRing - 2 blocks ahead of the sums: that those of a block are there says
    // that those of two blocks before were read, their scales too.
    uint32_t it = 0;
    bool ok = true;
    for (int t = t_first; all(ok && t < total); t += t_step) {
      const Tile tile = tile_at<kRows>(p, groups, t);
      // the scales of four rows to a lane, and of the tile's blocks of features
      const float* xs[4];
      uint32_t x_size[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = rank * kTileRows + lane + 32 * i;
        int src = -1;
        if (at < tile.count) src = p.rows ? p.rows[tile.row + at] : tile.row + at;
        x_size[i] = src >= 0 && src < p.n_src ? 4 : 0;          // none: a zero
        xs[i] = p.xs + (x_size[i] ? src : 0);
      }
      const int nb = tile.n * kBlocksN + lane;
      const uint32_t w_size = lane < kBlocksN && nb < p.n_blocks ? 4 : 0;
      const float* ws =
          p.ws + (static_cast<long long>(tile.e) * p.n_blocks + (w_size ? nb : 0)) * p.k_blocks;
#pragma unroll 1
      for (int b = 0; b < p.k_blocks; ++b, ++it) {
        if (it >= kRing - 2) {
          const uint32_t seen = it - (kRing - 2);
          ok = all(wait_on(&sempty[seen % kRing], (seen / kRing) & 1, p.status));
        }
        if (!ok) break;
        float* to = scales + (it % kRing) * kScaleRow;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          cp_async4(to + lane + 32 * i, xs[i], x_size[i]);
          xs[i] += p.n_src;
        }
        if (lane < kBlocksN) cp_async4(to + kTileRows + lane, ws + b, w_size);
        cp_async_arrive(&sfull[it % kRing]);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == 4 || warp == 5) {
    // Watches the accumulators of half of the features, and the scales, for the epilogue.  Once a
    // wait gave up, the rest are skipped: the epilogue goes through its blocks all the same.
    // A tile's place is written down for the epilogue, which needs it at the tile's end, beside its
    // first block; of the ring, three are in use.
    const int half = warp & 1;
    bool ok = true;
    uint32_t it = 0, at = 4 * half;
    for (int t = t_first; all(t < total); t += t_step) {
      const auto note = [&] {
        const Tile tile = tile_at<kRows>(p, groups, t);
        if (lane == 0) tiles[at] = make_int4(tile.row, tile.count, tile.n, 0);
        at = 4 * half + ((at + 1) & 3);
      };
      if (p.k_blocks == 1) note();
#pragma unroll 1
      for (int b = 0; b < p.k_blocks; ++b, ++it) {
        const uint32_t slot = it & 1;
        ok = ok && wait_both(&tfull[2 * half + slot], (it >> 1) & 1, &sfull[it % kRing],
                             (it / kRing) & 1, p.status);
        named_bar_arrive(1 + 2 * half + slot, 32 * (kEpiWarps / 2 + 1));
        if (elect_one()) mbar_arrive(&sempty[it % kRing]);
        if (b == 0 && p.k_blocks > 1) note();
      }
    }
  } else if (warp >= kEpiWarp) {
    kv4::regs_up<kRegsEpi>();
    const int quad = warp & 3, part = (warp - kEpiWarp) >> 2;
    uint8_t* buf = store + (warp - kEpiWarp) * kStore;
    const int half = part >> 1;
    const uint32_t from = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * 2 * kHalf +
                          (part & 1) * kOwn;
    const float* x_scale = scales + quad * 32 + lane;
    const float* w_scale = scales + kTileRows + part * kOwn / kBlockK;
    const uint32_t read = first_cta<kPair>(tempty + 2 * half);
    uint32_t it = 0, at = 4 * half;
    for (int t = t_first; t < total; t += t_step) {
      uint64_t acc[kOwn / 2];
#pragma unroll
      for (int i = 0; i < kOwn / 2; ++i) acc[i] = 0;
#pragma unroll 1
      for (int b = 0; b < p.k_blocks; ++b, ++it) {
        const uint32_t slot = it & 1;
        named_bar_sync(1 + 2 * half + slot, 32 * (kEpiWarps / 2 + 1));
        tc_fence_after();
        const uint32_t in_ring = it % kRing * kScaleRow;
        const float f1 = x_scale[in_ring] * w_scale[in_ring];
        const uint64_t f = pair_of(f1, f1);
        const uint32_t ta = from + slot * kHalf;
#pragma unroll
        for (int c = 0; c < kOwn; c += 16) {
          uint64_t v[8];
          tmem_pairs(ta + c, v);
          if (c + 16 == kOwn) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_at<kPair>(read + slot * 8);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) fma_pair(acc[c / 2 + i], v[i], f);
        }
      }
      const int4 tile = tiles[at];                       // first row, rows, feature tile
      at = 4 * half + ((at + 1) & 3);
      const int in = rank * kTileRows + quad * 32;
      store_rows<kOwn>(p, &map_out, acc, buf, tile.x + in, tile.y - in, tile.z * kN + part * kOwn,
                       lane);
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();             // neither leaves while the other's products use it
  if (warp == 1) {
    tc_fence_after();
    tmem_give<kPair>(tmem, kCols);
  }
}

// --------------------------------------------------------------------------------------------
// few rows: the weights streamed once
// --------------------------------------------------------------------------------------------
// The operands change places: 128 features are the product's M, kT rows its N, so that a step
// moves 16 KB of weights for each 128 kT bytes of x and the tensor cores are not kept busy with
// rows that are not there.  Bound by the weights.  Two CTAs share an SM, so that one's start and
// end hide behind the other's stream.  Where there are fewer tiles than that, the CTAs of a
// cluster take a share of K each; they add their sums through distributed shared memory, in the
// order of the shares.
constexpr int kStreamThreads = 192;      // copies, products, 4 epilogue warps
constexpr int kStreamBufs = 4;           // accumulators in TMEM
constexpr int kStreamSmem = 112 * 1024;  // of a CTA: two on an SM

template <int kT>
__host__ __device__ constexpr int stream_stage_bytes() {
  return (128 + kT) * kBlockK;
}

__device__ __forceinline__ float ld_cluster(uint32_t addr, uint32_t rank) {
  uint32_t remote;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
  return v;
}

template <int kT>
__global__ void __launch_bounds__(kStreamThreads, 2)
stream_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
              const Linear p, const int split) {
  constexpr int kStage = stream_stage_bytes<kT>();
  constexpr int kCols = kStreamBufs * kT;
  constexpr int kScales = (kT + 31) / 32;          // scales of a step to a lane
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  float* factors = reinterpret_cast<float*>(smem + p.n_stages * kStage);   // [4 warps][2][kT]
  uint64_t* full = reinterpret_cast<uint64_t*>(factors + 8 * kT);
  uint64_t* empty = full + p.n_stages;
  uint64_t* tfull = empty + p.n_stages;            // [kStreamBufs]
  uint64_t* tempty = tfull + kStreamBufs;
  uint64_t* mdrain = tempty + kStreamBufs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mdrain + 1);
  const Groups groups = groups_at(reinterpret_cast<uint8_t*>(tmem_slot + 1), p.groups);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int b_first = static_cast<int>(static_cast<long long>(p.k_blocks) * rank / split);
  const int b_last = static_cast<int>(static_cast<long long>(p.k_blocks) * (rank + 1) / split);
  const int t_first = blockIdx.x / split, t_step = gridDim.x / split;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.n_stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kStreamBufs; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 4);
    }
    mbar_init(mdrain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kCols);
    tmem_relinquish();
  }
  if (warp == 2 && elect_one()) {
    tma_prefetch_desc(&map_x);
    tma_prefetch_desc(&map_w);
  }
  griddep_wait();
  griddep_launch_dependents();           // (they wait for the end of this grid before they read)
  fill_groups(p, groups, kT, kStreamThreads);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = same(*tmem_slot);
  const int total = groups.tiles[p.groups] * p.n_tiles;

  if (warp == 0) {
    const uint64_t pol = l2_policy_evict_normal();
    uint32_t stage = 0, phase = 0;
    int issued = 0;
    bool ok = true;
    for (int t = t_first; all(ok && t < total); t += t_step) {
      const Tile tile = tile_at<kT>(p, groups, t);
      int r[4] = {};
      if (p.rows && lane < kT / 4) rows_of(p, tile, lane * 4, r);
      const int x_row = same(tile.row), w_row = same(tile.e * p.n + tile.n * 128);
#pragma unroll 1
      for (int b = b_first; b < b_last; ++b) {
        ok = all(wait_on(&empty[stage], phase ^ 1, p.status));
        if (!ok) break;
        uint8_t* a = smem + stage * kStage;
        if (elect_one()) {
          mbar_arrive_expect_tx(&full[stage], kStage);
          tma_load_2d(a, &map_w, &full[stage], b * kBlockK, w_row, pol);
          if (!p.rows)
            tma_load_2d(a + 128 * kBlockK, &map_x, &full[stage], b * kBlockK, x_row, pol);
        }
        if (p.rows) {
          __syncwarp();
          if (lane < kT / 4)
            tma_gather4<false>(a + (128 + lane * 4) * kBlockK, &map_x, smem_u32(&full[stage]),
                               b * kBlockK, r[0], r[1], r[2], r[3], pol);
        }
        ++issued;
        if (++stage == static_cast<uint32_t>(p.n_stages)) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    // no copy may still be landing when the CTA exits
    if (lane == 0)
      for (int st = 0; st < p.n_stages && st < issued; ++st) {
        const int last = st + ((issued - 1 - st) / p.n_stages) * p.n_stages;
        mbar_wait_drain(&full[st], static_cast<uint32_t>((last / p.n_stages) & 1), p.status);
      }
  } else if (warp == 1) {
    constexpr uint32_t idesc = idesc_e4m3(128, kT);
    const uint64_t a_desc = umma_sdesc_sw128(smem_u32(smem));
    const uint64_t b_desc = umma_sdesc_sw128(smem_u32(smem) + 128 * kBlockK);
    uint32_t stage = 0, phase = 0, slot = 0, tphase = 0;
    bool ok = true;
    for (int t = t_first; all(ok && t < total); t += t_step) {
#pragma unroll 1
      for (int b = b_first; b < b_last; ++b) {
        // (the wait for a phase before the first passes at once)
        ok = wait_both(&tempty[slot], tphase ^ 1, &full[stage], phase, p.status);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t ad = a_desc + stage * (kStage >> 4), bd = b_desc + stage * (kStage >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_e4m3(tmem + slot * kT, ad + 2 * kk, bd + 2 * kk, idesc, kk ? 1u : 0u);
          umma_commit(&empty[stage]);
          umma_commit(&tfull[slot]);
        }
        __syncwarp();
        if (++slot == kStreamBufs) {
          slot = 0;
          tphase ^= 1;
        }
        if (++stage == static_cast<uint32_t>(p.n_stages)) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (elect_one()) umma_commit(mdrain);
    if (lane == 0) mbar_wait_drain(mdrain, 0, p.status);
  }

  // TMEM lane = feature, column = row of x
  const int et = (warp & 3) * 32 + lane;
  bool ok = true;
  uint64_t acc[kT / 2];
  Tile tile = {};
  if (warp >= 2) {
    const uint32_t from = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    float* mine = factors + (warp - 2) * 2 * kT;
    uint32_t it = 0;
    for (int t = t_first; ok && t < total; t += t_step) {
      tile = tile_at<kT>(p, groups, t);
      const float* ws =
          p.ws + (static_cast<long long>(tile.e) * p.n_blocks + tile.n) * p.k_blocks;
      int src[kScales];
      float x0[kScales], x1[kScales];
      auto scales = [&](int b, float (&to)[kScales]) {
#pragma unroll
        for (int i = 0; i < kScales; ++i)
          to[i] = src[i] >= 0 && b < b_last
                      ? p.xs[static_cast<long long>(b) * p.n_src + src[i]] * ws[b]
                      : 0.f;
      };
#pragma unroll
      for (int i = 0; i < kScales; ++i) {
        const int at = lane + 32 * i;
        src[i] = -1;
        if (at < tile.count) src[i] = p.rows ? p.rows[tile.row + at] : tile.row + at;
        if (src[i] >= p.n_src) src[i] = -1;
      }
      scales(b_first, x0);
      scales(b_first + 1, x1);
#pragma unroll
      for (int i = 0; i < kT / 2; ++i) acc[i] = 0;
#pragma unroll 1
      for (int b = b_first; b < b_last; ++b, ++it) {
        float* f = mine + (it & 1) * kT;
#pragma unroll
        for (int i = 0; i < kScales; ++i) {
          if (lane + 32 * i < kT) f[lane + 32 * i] = x0[i];
          x0[i] = x1[i];
        }
        scales(b + 2, x1);
        const uint32_t slot = it % kStreamBufs;
        ok = all(wait_on(&tfull[slot], (it / kStreamBufs) & 1, p.status));
        if (!ok) break;
        tc_fence_after();
        const uint32_t ta = from + slot * kT;
#pragma unroll
        for (int c = 0; c < kT; c += 16) {
          uint64_t v[8];
          tmem_pairs(ta + c, v);
          if (c + 16 == kT) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[slot]);
          }
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const ulonglong2 g = *reinterpret_cast<const ulonglong2*>(f + c + 2 * i);
            fma_pair(acc[c / 2 + i], v[i], g.x);
            fma_pair(acc[c / 2 + i + 1], v[i + 1], g.y);
          }
        }
      }
      if (!ok) break;
      const int n = tile.n * 128 + et;
      if (split == 1) {
        if (n < p.n) {
          uint16_t* dst = p.out + static_cast<long long>(tile.row) * p.out_pitch + n;
#pragma unroll
          for (int j = 0; j < kT; ++j) {
            if (j < tile.count) *dst = float_to_bf16_bits(j & 1 ? halves(acc[j / 2]).y : halves(acc[j / 2]).x);
            dst += p.out_pitch;
          }
        }
      } else {
        // (every copy and product of this CTA is done: the stages are free)
        float* part = reinterpret_cast<float*>(smem) + et;
#pragma unroll
        for (int j = 0; j < kT; ++j) part[j * 128] = j & 1 ? halves(acc[j / 2]).y : halves(acc[j / 2]).x;
      }
    }
  }
  if (split > 1) {
    __syncwarp();
    cluster_sync();
    if (warp >= 2 && ok && t_first < total) {
      const int n = tile.n * 128 + et;
      const uint32_t part = smem_u32(smem) + et * 4;
      for (int j = rank; j < tile.count; j += split) {
        float sum = ld_cluster(part + j * 512, 0);
        for (int r = 1; r < split; ++r) sum += ld_cluster(part + j * 512, r);
        if (n < p.n)
          p.out[static_cast<long long>(tile.row + j) * p.out_pitch + n] = float_to_bf16_bits(sum);
      }
    }
    __syncwarp();
    cluster_sync();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

// --------------------------------------------------------------------------------------------
// host
// --------------------------------------------------------------------------------------------
// 2-D map over a row-major [rows, cols] matrix of bytes, box 128 columns x box_rows, 128-byte
// swizzle.
int make_map(CUtensorMap* map, const void* base, long long cols, long long rows, int box_rows) {
  return make_tmap_2d_u8(map, base, static_cast<uint64_t>(cols), static_cast<uint64_t>(rows),
                         static_cast<uint64_t>(cols), kBlockK, static_cast<uint32_t>(box_rows));
}

// Tiles, at most: one row tile more for each group than the rows fill.
long long most_tiles(const Linear& p, int tile_rows, int tile_cols) {
  const long long n_tiles = (static_cast<long long>(p.n) + tile_cols - 1) / tile_cols;
  if (!p.start) return (static_cast<long long>(p.m) + tile_rows - 1) / tile_rows * n_tiles;
  return (p.m / tile_rows + static_cast<long long>(p.groups < p.m ? p.groups : p.m)) * n_tiles;
}

template <bool kPair, int kN>
int run_tiles(Linear p, const void* x, const void* w, int k, cudaStream_t st) {
  constexpr int kCtas = kPair ? 2 : 1;
  constexpr int kStage = tile_stage_bytes<kPair, kN>();
  p.n_tiles = (p.n + kN - 1) / kN;
  constexpr int kStoreBytes = kEpiWarps * 32 * (kN / 4) * 2;
  const int tail = kStoreBytes + kRing * kScaleRow * 4 + 8 * 16 + (10 + 2 * kRing) * 8 + 4 + groups_bytes(p.groups);
  p.n_stages = (kSmemLimit - 1024 - tail) / (kStage + 16);
  if (p.n_stages > kMaxStages) p.n_stages = kMaxStages;
  const int smem = 1024 + p.n_stages * (kStage + 16) + tail;
  CUtensorMap mx, mw, mo = {};
  int rc = make_map(&mx, x, k, p.n_src, p.rows ? 1 : kTileRows);
  if (!rc) rc = make_map(&mw, w, k, static_cast<long long>(p.groups) * p.n, kN / 2 / kCtas);
  if (!rc && p.vector) rc = make_tmap_2d_store_bf16(&mo, p.out, p.n, p.m, p.out_pitch * 2, kN / 4, 32);
  const auto kernel = tile_kernel<kPair, kN>;
  static std::atomic<uint64_t> ready{0};
  if (!rc)
    rc = kv4::smem_limit_once(&ready, reinterpret_cast<const void*>(kernel), kSmemLimit,
                              kRegsStart);
  if (rc) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kTileWarps * 32);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // clusters that fit at once (one CTA to an SM), once per process
  static const int most = [&] {
    const int nsm = current_num_sms();
    if (nsm <= 0) return 0;
    cudaLaunchConfig_t q = cfg;
    q.gridDim = dim3(nsm / kCtas * kCtas);
    q.dynamicSmemBytes = kSmemLimit;
    int n = 0;
    return cudaOccupancyMaxActiveClusters(&n, kernel, &q) == cudaSuccess ? n : 0;
  }();
  if (most < 1) return DFLASH_E_CUDA;
  const long long tiles = most_tiles(p, kTileRows * kCtas, kN);
  if (tiles > 0x7FFFFFFF - 256ll * kBand) return DFLASH_E_UNSUPPORTED;
  cfg.gridDim = dim3(static_cast<unsigned>(tiles < most ? tiles : most) * kCtas);
  cfg.numAttrs = 2;
  return cuda_err(cudaLaunchKernelEx(&cfg, kernel, mx, mw, mo, p));
}

// CTAs that share a tile's K: the fewest time units, where a wave (two CTAs to an SM) costs its
// blocks of K and kStreamStart for the start, the end and the joining.
constexpr int kStreamStart = 6;

int stream_split(const Linear& p, long long tiles, int nsm) {
  int best = 1;
  long long cost = 0;
  for (int s = 1; s <= 8 && s <= p.k_blocks; s *= 2) {
    const long long waves = (tiles * s + 2 * nsm - 1) / (2 * nsm);
    const long long c = waves * ((p.k_blocks + s - 1) / s + kStreamStart);
    if (s == 1 || c < cost) {
      best = s;
      cost = c;
    }
  }
  return best;
}

template <int kT>
int run_stream(Linear p, const void* x, const void* w, int k, cudaStream_t st) {
  p.n_tiles = (p.n + 127) / 128;
  const int tail = 8 * kT * 4 + (2 * kStreamBufs + 1) * 8 + 4 + groups_bytes(p.groups);
  p.n_stages = (kStreamSmem - 1024 - tail) / (stream_stage_bytes<kT>() + 16);
  if (p.n_stages > 8) p.n_stages = 8;
  const int smem = 1024 + p.n_stages * (stream_stage_bytes<kT>() + 16) + tail;
  CUtensorMap mx, mw;
  int rc = make_map(&mx, x, k, p.n_src, p.rows ? 1 : kT);
  if (!rc) rc = make_map(&mw, w, k, static_cast<long long>(p.groups) * p.n, 128);
  static std::atomic<uint64_t> ready{0};
  const void* kernel = reinterpret_cast<const void*>(stream_kernel<kT>);
  if (!rc) rc = kv4::smem_limit_once(&ready, kernel, kStreamSmem);
  if (rc) return rc;
  const int nsm = current_num_sms();
  if (nsm <= 0) return DFLASH_E_CUDA;
  const long long tiles = most_tiles(p, kT, 128);
  if (tiles > 0x7FFFFFFF / 16) return DFLASH_E_UNSUPPORTED;
  const int split = stream_split(p, tiles, nsm);
  // shares of K: one tile to a cluster; whole tiles: two CTAs to an SM walk them
  const long long ctas = split > 1 ? tiles * split : tiles < 2 * nsm ? tiles : 2 * nsm;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kStreamThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  return cuda_err(cudaLaunchKernelEx(&cfg, stream_kernel<kT>, mx, mw, p, split));
}

// Few rows (of an expert, on average) stream the weights, many fill the tiles.
int run(const Linear& p, const void* x, const void* w, int k, cudaStream_t st) {
  if (const char* v = getenv("VAR")) {
    if (v[0] == 'p' && v[1] == '2') return run_tiles<true, 256>(p, x, w, k, st);
    if (v[0] == 'p' && v[1] == '1') return run_tiles<true, 128>(p, x, w, k, st);
    if (v[0] == 's' && v[1] == '2') return run_tiles<false, 256>(p, x, w, k, st);
    if (v[0] == 's' && v[1] == '1') return run_tiles<false, 128>(p, x, w, k, st);
    if (v[0] == 't' && v[1] == '1') return run_stream<16>(p, x, w, k, st);
    if (v[0] == 't' && v[1] == '3') return run_stream<32>(p, x, w, k, st);
    if (v[0] == 't' && v[1] == '6') return run_stream<64>(p, x, w, k, st);
  }
  const int rows = (p.m + p.groups - 1) / p.groups;
  if (rows <= 16) return run_stream<16>(p, x, w, k, st);
  if (rows <= 32) return run_stream<32>(p, x, w, k, st);
  if (rows <= 64) return run_stream<64>(p, x, w, k, st);
  if (p.n > 128) return run_tiles<false, 256>(p, x, w, k, st);
  return run_tiles<false, 128>(p, x, w, k, st);
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
  p->xs = xs;
  p->ws = ws;
  p->out = static_cast<uint16_t*>(out);
  p->out_pitch = out_pitch;
  p->status = static_cast<uint32_t*>(wsp);
  p->m = m;
  p->n = n;
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
  return run(p, x, w, n_in, reinterpret_cast<cudaStream_t>(stream));
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
  p.start = start;
  p.rows = rows;
  return run(p, x, w, n_in, reinterpret_cast<cudaStream_t>(stream));
}
