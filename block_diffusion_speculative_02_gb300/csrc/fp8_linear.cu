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

using kv4::wait_on;

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

__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Four rows of a map whose box is one row high, one below the other in shared memory.  A row
// past the map's end reads as zeros.
__device__ __forceinline__ void tma_gather4(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int c0, int r0, int r1, int r2, int r3,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "l"(policy)
      : "memory");
}

// 32 TMEM lanes x 32 columns; thread i gets lane (base + i).  The registers hold the values
// after tmem_wait32 on them.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
      "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
  asm volatile(""
               : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]),
                 "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// acc += f * t, pairwise (one instruction for two).
__device__ __forceinline__ void add_scaled(float2* acc, const uint32_t (&t)[32], float f) {
  const float2 ff = make_float2(f, f);
#pragma unroll
  for (int i = 0; i < 16; ++i)
    acc[i] = __ffma2_rn(make_float2(__uint_as_float(t[2 * i]), __uint_as_float(t[2 * i + 1])), ff,
                        acc[i]);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return static_cast<uint32_t>(float_to_bf16_bits(lo)) |
         static_cast<uint32_t>(float_to_bf16_bits(hi)) << 16;
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

// By one warp.
__device__ __forceinline__ void fill_groups(const Linear& p, const Groups& g, int tile_rows,
                                            int lane) {
  int sum = 0;
  for (int e0 = 0; e0 < p.groups; e0 += 32) {
    const int e = e0 + lane;
    int a = 0, b = 0;
    if (e < p.groups) {
      a = p.start ? p.start[e] : 0;
      b = p.start ? p.start[e + 1] : p.m;
      if (a < 0 || b < a || b > p.m) {
        set_status(p.status, DFLASH_ST_CAPACITY);
        a = b = 0;
      }
    }
    const int own = (b - a + tile_rows - 1) / tile_rows;
    int t = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += y;
    }
    if (e < p.groups) {
      g.first[e] = a;
      g.count[e] = b - a;
      g.tiles[e] = sum + t - own;
    }
    sum += __shfl_sync(0xffffffffu, t, 31);
  }
  if (lane == 0) g.tiles[p.groups] = sum;
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
// tiles of 128 rows x kN features
// --------------------------------------------------------------------------------------------
constexpr int kTileRows = 128;
constexpr int kTileWarps = 12;        // copies, products, two idle, 8 epilogue warps
constexpr int kEpiWarp = 4;           // the first epilogue warp
// Registers a thread: 168 at the start; the accumulators' warps take from the others, within
// the block's 384 x 168.
constexpr int kRegsStart = 168, kRegsRest = 72, kRegsEpi = 216;
static_assert(kEpiWarp * kRegsRest + 8 * kRegsEpi <= kTileWarps * kRegsStart, "register split");
constexpr int kStoreBytes = 8 * 4096; // 32 rows x 64 features of each epilogue warp
constexpr int kSmemLimit = 227 * 1024;

template <int kN>
__host__ __device__ constexpr int tile_stage_bytes() {
  return (kTileRows + kN) * kBlockK;
}

// A lane of a warp's tile: 64 features of 32 rows go through shared memory, so that a row's
// features leave side by side.
__device__ __forceinline__ void store_rows(const Linear& p, const float2* acc, uint8_t* buf,
                                           int row, int rows_left, int col, int lane) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float2* a = acc + 4 * c;
    *reinterpret_cast<uint4*>(buf + lane * 128 + ((c ^ (lane & 7)) << 4)) =
        make_uint4(pack_bf16(a[0].x, a[0].y), pack_bf16(a[1].x, a[1].y),
                   pack_bf16(a[2].x, a[2].y), pack_bf16(a[3].x, a[3].y));
  }
  __syncwarp();
  const int most = min(32, rows_left);
  if (p.vector && col + 64 <= p.n) {
    const int c = lane & 7;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = i * 4 + (lane >> 3);
      const uint4 v = *reinterpret_cast<const uint4*>(buf + r * 128 + ((c ^ (r & 7)) << 4));
      if (r < most)
        *reinterpret_cast<uint4*>(p.out + static_cast<long long>(row + r) * p.out_pitch + col +
                                  8 * c) = v;
    }
  } else {
    for (int r = 0; r < most; ++r) {
      uint16_t* dst = p.out + static_cast<long long>(row + r) * p.out_pitch + col;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = lane + 32 * h;
        if (col + j < p.n)
          dst[j] = *reinterpret_cast<const uint16_t*>(buf + r * 128 +
                                                      (((j >> 3) ^ (r & 7)) << 4) + (j & 7) * 2);
      }
    }
  }
  __syncwarp();
}

template <int kN>
__global__ void __launch_bounds__(kTileWarps * 32, 1)
tile_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
            const Linear p) {
  constexpr int kStage = tile_stage_bytes<kN>();
  constexpr int kHalf = kN / 2;          // features of an epilogue warp
  constexpr int kCols = 2 * kN;          // TMEM columns: two accumulators
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  uint8_t* store = smem + p.n_stages * kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(store + kStoreBytes);
  uint64_t* empty = full + p.n_stages;
  uint64_t* tfull = empty + p.n_stages;  // [2]
  uint64_t* tempty = tfull + 2;          // [2]
  uint64_t* mdrain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mdrain + 1);
  const Groups groups = groups_at(reinterpret_cast<uint8_t*>(tmem_slot + 1), p.groups);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.n_stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 8);
    }
    mbar_init(mdrain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kCols);
    tmem_relinquish();
  }
  griddep_wait();
  if (warp == 2) fill_groups(p, groups, kTileRows, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int total = groups.tiles[p.groups] * p.n_tiles;   // (below 2^31: the host)
  if (warp < kEpiWarp) kv4::regs_down<kRegsRest>();

  if (warp == 0) {
    const uint64_t pol = l2_policy_evict_normal();
    uint32_t stage = 0, phase = 0;
    int issued = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
      const Tile tile = tile_at<kTileRows>(p, groups, t);
      int r[4] = {};
      if (p.rows) rows_of(p, tile, lane * 4, r);
      for (int b = 0; b < p.k_blocks; ++b) {
        ok = __all_sync(0xffffffffu, wait_on(&empty[stage], phase ^ 1, p.status));
        if (!ok) break;
        uint8_t* a = smem + stage * kStage;
        if (lane == 0) {
          mbar_arrive_expect_tx(&full[stage], kStage);
          if (!p.rows) tma_load_2d(a, &map_x, &full[stage], b * kBlockK, tile.row, pol);
          tma_load_2d(a + kTileRows * kBlockK, &map_w, &full[stage], b * kBlockK,
                      tile.e * p.n + tile.n * kN, pol);
        }
        if (p.rows) {
          __syncwarp();
          tma_gather4(a + lane * 4 * kBlockK, &map_x, &full[stage], b * kBlockK, r[0], r[1], r[2],
                      r[3], pol);
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
    const uint32_t base = smem_u32(smem);
    constexpr uint32_t idesc = idesc_e4m3(kTileRows, kN);
    uint32_t stage = 0, phase = 0, it = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
      for (int b = 0; b < p.k_blocks; ++b, ++it) {
        const uint32_t slot = it & 1;
        // (the wait for a phase before the first passes at once)
        ok = wait_on(&tempty[slot], ((it >> 1) & 1) ^ 1, p.status) &&
             wait_on(&full[stage], phase, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t at = base + stage * kStage;
          const uint64_t ad = umma_sdesc_sw128(at);
          const uint64_t bd = umma_sdesc_sw128(at + kTileRows * kBlockK);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_e4m3(tmem + slot * kN, ad + 2 * kk, bd + 2 * kk, idesc, kk ? 1u : 0u);
          umma_commit(&empty[stage]);
          umma_commit(&tfull[slot]);
        }
        __syncwarp();
        if (++stage == static_cast<uint32_t>(p.n_stages)) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (lane == 0) {
      umma_commit(mdrain);
      mbar_wait_drain(mdrain, 0, p.status);
    }
  } else if (warp >= kEpiWarp) {
    kv4::regs_up<kRegsEpi>();
    const int quad = warp & 3, half = (warp - kEpiWarp) >> 2;
    uint8_t* buf = store + (warp - kEpiWarp) * 4096;
    const uint32_t from = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * kHalf;
    uint32_t it = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
      const Tile tile = tile_at<kTileRows>(p, groups, t);
      const int at = quad * 32 + lane;                        // this thread's row of the tile
      const int col = tile.n * kN + half * kHalf;
      int src = -1;
      if (at < tile.count) src = p.rows ? p.rows[tile.row + at] : tile.row + at;
      if (src >= p.n_src) src = -1;
      const float* xs = p.xs + max(src, 0);
      const float* ws = p.ws + (static_cast<long long>(tile.e) * p.n_blocks +
                                min(col / kBlockK, p.n_blocks - 1)) * p.k_blocks;
      float2 acc[kHalf / 2];
#pragma unroll
      for (int i = 0; i < kHalf / 2; ++i) acc[i] = make_float2(0.f, 0.f);
      // the scales are read two blocks ahead
      float x0 = 0.f, x1 = 0.f, w0 = 0.f, w1 = 0.f;
      const bool there = src >= 0;
      if (there) {
        x0 = xs[0];
        w0 = ws[0];
        if (p.k_blocks > 1) {
          x1 = xs[p.n_src];
          w1 = ws[1];
        }
      }
#pragma unroll 1
      for (int b = 0; b < p.k_blocks; ++b, ++it) {
        const float f = x0 * w0;
        x0 = x1;
        w0 = w1;
        if (there && b + 2 < p.k_blocks) {
          x1 = xs[static_cast<long long>(b + 2) * p.n_src];
          w1 = ws[b + 2];
        }
        const uint32_t slot = it & 1;
        ok = __all_sync(0xffffffffu, wait_on(&tfull[slot], (it >> 1) & 1, p.status));
        if (!ok) break;
        tc_fence_after();
        const uint32_t ta = from + slot * kN;
        uint32_t v[2][32];
        tmem_ld32(ta, v[0]);
#pragma unroll
        for (int c = 0; c < kHalf / 32; ++c) {
          tmem_wait32(v[c & 1]);
          if (c + 1 < kHalf / 32) tmem_ld32(ta + 32 * (c + 1), v[(c + 1) & 1]);
          if (c + 1 == kHalf / 32) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[slot]);
          }
          add_scaled(acc + 16 * c, v[c & 1], f);
        }
      }
      if (!ok) break;
#pragma unroll
      for (int c = 0; c < kHalf; c += 64)
        store_rows(p, acc + c / 2, buf, tile.row + quad * 32, tile.count - quad * 32, col + c,
                   lane);
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
  griddep_launch_dependents();
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
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
  griddep_wait();
  if (warp == 2) fill_groups(p, groups, kT, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int total = groups.tiles[p.groups] * p.n_tiles;

  if (warp == 0) {
    const uint64_t pol = l2_policy_evict_normal();
    uint32_t stage = 0, phase = 0;
    int issued = 0;
    bool ok = true;
    for (int t = t_first; ok && t < total; t += t_step) {
      const Tile tile = tile_at<kT>(p, groups, t);
      int r[4] = {};
      if (p.rows && lane < kT / 4) rows_of(p, tile, lane * 4, r);
      for (int b = b_first; b < b_last; ++b) {
        ok = __all_sync(0xffffffffu, wait_on(&empty[stage], phase ^ 1, p.status));
        if (!ok) break;
        uint8_t* a = smem + stage * kStage;
        if (lane == 0) {
          mbar_arrive_expect_tx(&full[stage], kStage);
          tma_load_2d(a, &map_w, &full[stage], b * kBlockK, tile.e * p.n + tile.n * 128, pol);
          if (!p.rows)
            tma_load_2d(a + 128 * kBlockK, &map_x, &full[stage], b * kBlockK, tile.row, pol);
        }
        if (p.rows) {
          __syncwarp();
          if (lane < kT / 4)
            tma_gather4(a + (128 + lane * 4) * kBlockK, &map_x, &full[stage], b * kBlockK, r[0],
                        r[1], r[2], r[3], pol);
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
    const uint32_t base = smem_u32(smem);
    constexpr uint32_t idesc = idesc_e4m3(128, kT);
    uint32_t stage = 0, phase = 0, it = 0;
    bool ok = true;
    for (int t = t_first; ok && t < total; t += t_step) {
      for (int b = b_first; b < b_last; ++b, ++it) {
        const uint32_t slot = it % kStreamBufs;
        // (the wait for a phase before the first passes at once)
        ok = wait_on(&tempty[slot], ((it / kStreamBufs) & 1) ^ 1, p.status) &&
             wait_on(&full[stage], phase, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t at = base + stage * kStage;
          const uint64_t ad = umma_sdesc_sw128(at);
          const uint64_t bd = umma_sdesc_sw128(at + 128 * kBlockK);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_e4m3(tmem + slot * kT, ad + 2 * kk, bd + 2 * kk, idesc, kk ? 1u : 0u);
          umma_commit(&empty[stage]);
          umma_commit(&tfull[slot]);
        }
        __syncwarp();
        if (++stage == static_cast<uint32_t>(p.n_stages)) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (lane == 0) {
      umma_commit(mdrain);
      mbar_wait_drain(mdrain, 0, p.status);
    }
  }

  // TMEM lane = feature, column = row of x
  const int et = (warp & 3) * 32 + lane;
  bool ok = true;
  float2 acc[kT / 2];
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
      for (int i = 0; i < kT / 2; ++i) acc[i] = make_float2(0.f, 0.f);
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
        ok = __all_sync(0xffffffffu,
                        wait_on(&tfull[slot], (it / kStreamBufs) & 1, p.status));
        if (!ok) break;
        tc_fence_after();
        const uint32_t ta = from + slot * kT;
#pragma unroll
        for (int c = 0; c < kT; c += 16) {
          uint32_t v[16];
          tmem_ld_32x32b_x16(ta + c, v);
          tmem_wait16(v);
          if (c + 16 == kT) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[slot]);
          }
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 g = *reinterpret_cast<const float4*>(f + c + i);
            float2* a = acc + (c + i) / 2;
            a[0] = __ffma2_rn(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])),
                              make_float2(g.x, g.y), a[0]);
            a[1] = __ffma2_rn(make_float2(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3])),
                              make_float2(g.z, g.w), a[1]);
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
            if (j < tile.count) *dst = float_to_bf16_bits(j & 1 ? acc[j / 2].y : acc[j / 2].x);
            dst += p.out_pitch;
          }
        }
      } else {
        // (every copy and product of this CTA is done: the stages are free)
        float* part = reinterpret_cast<float*>(smem) + et;
#pragma unroll
        for (int j = 0; j < kT; ++j) part[j * 128] = j & 1 ? acc[j / 2].y : acc[j / 2].x;
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
  griddep_launch_dependents();
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

template <int kN>
int run_tiles(Linear p, const void* x, const void* w, int k, cudaStream_t st) {
  p.n_tiles = (p.n + kN - 1) / kN;
  const int tail = kStoreBytes + 5 * 8 + 4 + groups_bytes(p.groups);
  p.n_stages = (kSmemLimit - 1024 - tail) / (tile_stage_bytes<kN>() + 16);
  if (p.n_stages > 8) p.n_stages = 8;
  const int smem = 1024 + p.n_stages * (tile_stage_bytes<kN>() + 16) + tail;
  CUtensorMap mx, mw;
  int rc = make_map(&mx, x, k, p.n_src, p.rows ? 1 : kTileRows);
  if (!rc) rc = make_map(&mw, w, k, static_cast<long long>(p.groups) * p.n, kN);
  static std::atomic<uint64_t> ready{0};
  if (!rc)
    rc = kv4::smem_limit_once(&ready, reinterpret_cast<const void*>(tile_kernel<kN>), kSmemLimit,
                              kRegsStart);
  if (rc) return rc;
  const int nsm = current_num_sms();
  if (nsm <= 0) return DFLASH_E_CUDA;
  const long long tiles = most_tiles(p, kTileRows, kN);
  if (tiles > 0x7FFFFFFF - 256ll * kBand) return DFLASH_E_UNSUPPORTED;
  const int grid = tiles < nsm ? static_cast<int>(tiles) : nsm;
  return launch(tile_kernel<kN>, dim3(grid), dim3(kTileWarps * 32), smem, st, mx, mw, p);
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
  const int rows = (p.m + p.groups - 1) / p.groups;
  if (rows <= 16) return run_stream<16>(p, x, w, k, st);
  if (rows <= 32) return run_stream<32>(p, x, w, k, st);
  if (rows <= 64) return run_stream<64>(p, x, w, k, st);
  if (p.n > 128) return run_tiles<256>(p, x, w, k, st);
  return run_tiles<128>(p, x, w, k, st);
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
