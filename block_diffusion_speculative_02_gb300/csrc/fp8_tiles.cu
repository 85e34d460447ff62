// 8-bit products of many rows: tiles of 128 rows (or, of a pair of CTAs, 256) x kN features.
//
// A thread for each half of the features issues the products, of a pair (kPair) for both SMs: each
// SM holds 128 rows of x and half of the weights, and gets the sums of its own rows.  Per block of
// K a pair of SMs moves and reads half as many bytes of weights as two single ones.
//
// A block's sums leave TMEM in the time of the next block's products (512 cycles at 256
// features): 16 warps take a quarter of the features of 32 rows each, so that four warps of
// a scheduler cover each other's waits.  (8191 rows x 24576 x 4096 in a burst: 504 us, 655 with 8
// warps of twice the features.)  They wait at named barriers, where a warp takes no turn: one more
// warp watches the accumulators' mbarriers for them.  (With all of them trying an mbarrier 640 us: a
// try took the warps that issue the products 400 clocks and more.)
//
// A burst is twenty copies of one call in a graph, too short for the power limit, on tensors that
// stay in L2 as far as they fit.  It compares two forms of a kernel; in continuous use, each call
// with weights of its own, this one takes 606 to 610 us.
//
// What bounds it: a block of a pair takes some 640 clocks, of which its products take 513.  That is
// what shared memory needs for them (48 KB read, the rows twice, once for each half of the
// features, and 32 KB written by the copies, at 128 bytes a clock).  Products of all 256 features
// at once read 16 KB less, but leave the epilogue half the time: 536 us.  The rest is power:
// zeros as operands take 440 us, in a burst, too.
#include "fp8_linear.cuh"
#include "per_device.h"

namespace dflash {
namespace fp8 {
namespace {

constexpr int kTileRows = 128;
// Warps: 0 copies, 1 and 3 products, 2 scales, 4 and 5 watch, 6 and 7 rows
// of x by index, 16 of the epilogue.
constexpr int kTileWarps = 24;
constexpr int kEpiWarp = 8, kEpiWarps = 16;
// Registers a thread: 80 at the start; the epilogue's warps take from the others, within the
// block's 768 x 80.
constexpr int kRegsStart = 80, kRegsRest = 32, kRegsEpi = 104;
static_assert(kEpiWarp * kRegsRest + kEpiWarps * kRegsEpi <= kTileWarps * kRegsStart,
              "register split");
constexpr int kScaleRow = kTileRows + 2;        // of the rows, then of the weights
constexpr int kSmemLimit = 227 * 1024;

// Accumulators of each half of the features (all that TMEM holds: 512 rows x 12288 x 4096 in tiles
// of 128 features take 30.5 us with four, 32.2 with two, in a burst), and blocks whose scales are in shared
// memory.
template <int kN>
__host__ __device__ constexpr int slots() {
  return 512 / kN;
}
template <int kN>
__host__ __device__ constexpr int ring() {
  return 4 * slots<kN>();
}

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
    // (eight rows at a time, so that their loads are on their way together: 2000 rows x 4095
    // features of 512 in 13.4 us, one at a time 14.2)
    uint16_t* dst = p.out + static_cast<long long>(row) * p.out_pitch + col + lane;
#pragma unroll 1
    for (int r0 = 0; r0 < most; r0 += 8) {
      uint16_t v[8][kW / 32];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int h = 0; h < kW / 32; ++h)
          v[i][h] = *reinterpret_cast<const uint16_t*>(at(r0 + i, (lane >> 3) + 4 * h) +
                                                       (lane & 7) * 2);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int h = 0; h < kW / 32; ++h)
          if (r0 + i < most && col + lane + 32 * h < p.n) dst[32 * h] = v[i][h];
        dst += p.out_pitch;
      }
    }
  }
  __syncwarp();
}

// kSend: of an epilogue warp's features, those on their way out at a time.
template <bool kPair, int kN, bool kIndex, int kSend>
__global__ void __launch_bounds__(kTileWarps * 32, 1)
tile_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
            const __grid_constant__ CUtensorMap map_out, const Linear p) {
  static_assert(!(kPair && kIndex), "rows by index: tiles of single CTAs");
  constexpr int kCtas = kPair ? 2 : 1;
  constexpr int kRows = kTileRows * kCtas;
  constexpr int kStage = tile_stage_bytes<kPair, kN>();
  constexpr int kHalf = kN / 2;          // features of a product
  constexpr int kShare = kHalf / kCtas;  // of these, features whose weights this CTA holds
  constexpr int kOwn = kN / 4;           // features of an epilogue warp
  constexpr int kStore = 32 * kSend * 2;
  constexpr int kSlots = slots<kN>(), kRing = ring<kN>();
  constexpr int kCols = kSlots * kN;     // TMEM columns
  constexpr int kBlocksN = kN / kBlockK;
  const int rank = kPair ? static_cast<int>(cluster_ctarank()) : 0;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  uint8_t* store = smem + p.n_stages * kStage;
  float* scales =                        // [kRing][128 rows, weights]
      reinterpret_cast<float*>(store + kEpiWarps * kStore);
  int4* tiles = reinterpret_cast<int4*>(scales + kRing * kScaleRow);  // [kInfo] tiles' places
  uint32_t* sources = reinterpret_cast<uint32_t*>(tiles + kInfo);     // [kInfo][128]
  uint64_t* full = reinterpret_cast<uint64_t*>(sources + kInfo * kTileRows);
  uint64_t* empty = full + p.n_stages;
  uint64_t* tfull = empty + p.n_stages;  // [2 halves][kSlots] accumulators are there
  uint64_t* tempty = tfull + 2 * kSlots;   // likewise: read (of a pair: in the first CTA)
  uint64_t* mdrain = tempty + 2 * kSlots;  // [2 halves]
  uint64_t* sfull = mdrain + 2;          // [kRing] scales are there
  uint64_t* sempty = sfull + kRing;      // [kRing] both halves' sums of that block are there
  uint64_t* ifull = sempty + kRing;      // [kInfo] a tile's place is written down
  uint64_t* iempty = ifull + kInfo;      // [kInfo] and read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(iempty + kInfo);
  const Groups groups = groups_at(reinterpret_cast<uint8_t*>(tmem_slot + 1), p.groups);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int t_first = blockIdx.x / kCtas, t_step = gridDim.x / kCtas;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.n_stages; ++i) {
      mbar_init(&full[i], 1 + (kIndex ? 64 : 0));
      mbar_init(&empty[i], 2);           // the products of both halves
    }
    for (int i = 0; i < kInfo; ++i) {
      mbar_init(&ifull[i], 1);
      mbar_init(&iempty[i], 1 + (kIndex ? 2 : 0) + kEpiWarps);
    }
    for (int i = 0; i < 2 * kSlots; ++i) {
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
  fill_groups(p, groups, kRows, kTileWarps * 32);
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();             // the other CTA's barriers are there
  griddep_launch_dependents();           // (the next grid's CTAs take TMEM only after this one's)
  tc_fence_after();
  const uint32_t tmem = same(*tmem_slot);
  const int total = groups.tiles[p.groups] * p.n_tiles;   // (below 2^31: the host)
  if (warp < kEpiWarp) kv4::regs_down<kRegsRest>();

  if (warp == 0) {
    const uint64_t pol = l2_policy_evict_normal();
    uint32_t stage = 0, phase = 0, in = 0;
    int issued = 0;
    bool ok = true;
    for (int t = t_first; all(ok && t < total); t += t_step, ++in) {
      int4 place;
      if (in == 0) {                     // (the first is not waited for)
        const Tile tile = tile_at<kRows>(p, groups, t);
        place = make_int4(tile.row, tile.count, tile.n, tile.e * p.n + tile.n * kN);
      } else {
        ok = all(wait_on(&ifull[in % kInfo], (in / kInfo) & 1, p.status));
        if (!ok) break;
        place = tiles[in % kInfo];
      }
      const int x_row = same(place.x) + rank * kTileRows;
      const int w_row = same(place.w) + rank * kShare;
      // (a CTA of a pair without any rows multiplies what the stage held)
      const int x_boxes = kIndex ? 0 : kPair && same(place.x) + kTileRows < p.m ? 2 : 1;
      const uint32_t bytes = kCtas * 2 * kShare * kBlockK + x_boxes * p.box_rows * kBlockK;
      if (elect_one()) mbar_arrive(&iempty[in % kInfo]);
#pragma unroll 1
      for (int b = 0; b < p.k_blocks; ++b) {
        ok = all(wait_on(&empty[stage], phase ^ 1, p.status));
        if (!ok) break;
        uint8_t* a = smem + stage * kStage;
        const uint32_t bar = first_cta<kPair>(&full[stage]);
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], bytes);
          if (!kIndex && x_row < p.m)
            tma_box<kPair>(a, &map_x, bar, b * kBlockK, x_row, pol);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            tma_box<kPair>(a + (kTileRows + h * kShare) * kBlockK, &map_w, bar, b * kBlockK,
                           w_row + h * kHalf, pol);
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
      const uint32_t acc = tmem + half * kSlots * kHalf;
      uint64_t* done = tfull + kSlots * half;
      uint64_t* read = tempty + kSlots * half;
      uint32_t stage = 0, phase = 0, slot = 0, tphase = 0;
      bool ok = true;
      for (int t = t_first; all(ok && t < total); t += t_step) {
#pragma unroll 1
        for (int b = 0; b < p.k_blocks; ++b) {
          // (the wait for a phase before the first passes at once)
          ok = wait_both(&read[slot], tphase ^ 1, &full[stage], phase, p.status);
          if (!ok) break;
          tc_fence_after();
          if (kIndex) fence_proxy_async_smem();
          if (elect_one()) {
            const uint64_t ad = a_desc + stage * (kStage >> 4), bd = b_desc + stage * (kStage >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_e4m3<kPair>(acc + slot * kHalf, ad + 2 * kk, bd + 2 * kk, idesc, kk ? 1u : 0u);
            mma_done<kPair>(&done[slot]);
            mma_done<kPair>(&empty[stage]);
          }
          if (++slot == kSlots) {
            slot = 0;
            tphase ^= 1;
          }
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
    // Writes down the tiles' places and copies the scales, kRing - kSlots blocks ahead of the sums:
    // that those of a block are there says that those of kSlots blocks before were read, their
    // scales too.
    uint32_t it = 0, in = 0;
    bool ok = true;
    for (int t = t_first; all(ok && t < total); t += t_step, ++in) {
      const Tile tile = tile_at<kRows>(p, groups, t);
      // (the wait for a phase before the first passes at once)
      ok = all(wait_on(&iempty[in % kInfo], ((in / kInfo) & 1) ^ 1, p.status));
      if (!ok) break;
      // the scales of four rows to a lane, and of the tile's blocks of features
      const float* xs[4];
      uint32_t x_size[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int src = source_row(p, tile, rank * kTileRows + lane + 32 * i);
        x_size[i] = src >= 0 ? 4 : 0;                           // none: a zero
        xs[i] = p.xs + max(src, 0);
        if (kIndex)
          sources[in % kInfo * kTileRows + place_of<kTileRows>(lane + 32 * i)] =
              src >= 0 ? static_cast<uint32_t>(src) * (p.k / 16) : kNoRow;
      }
      if (lane == 0)
        tiles[in % kInfo] = make_int4(tile.row, tile.count, tile.n, tile.e * p.n + tile.n * kN);
      __syncwarp();
      if (elect_one()) mbar_arrive(&ifull[in % kInfo]);
      const int nb = tile.n * kBlocksN + lane;
      const uint32_t w_size = lane < kBlocksN && nb < p.n_blocks ? 4 : 0;
      const float* ws =
          p.ws + (static_cast<long long>(tile.e) * p.n_blocks + (w_size ? nb : 0)) * p.k_blocks;
#pragma unroll 1
      for (int b = 0; b < p.k_blocks; ++b, ++it) {
        if (it >= kRing - kSlots) {
          const uint32_t seen = it - (kRing - kSlots);
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
    // Watches the accumulators of half of the features, and the scales, for the epilogue, which goes
    // through its blocks to the end also when a wait gave up.
    const int half = warp & 1;
    bool ok = true;
    uint32_t it = 0;
    for (int t = t_first; all(t < total); t += t_step) {
#pragma unroll 1
      for (int b = 0; b < p.k_blocks; ++b, ++it) {
        const uint32_t slot = kSlots * half + it % kSlots;
        ok = hand_over(ok, &tfull[slot], (it / kSlots) & 1, &sfull[it % kRing], (it / kRing) & 1,
                       1 + slot, 32 * (kEpiWarps / 2 + 1), p.status);
        if (elect_one()) mbar_arrive(&sempty[it % kRing]);
      }
    }
  } else if (warp == 6 || warp == 7) {
    if (kIndex) {                        // half of the CTA's rows of x to a warp
      const int first = (warp - 6) * 64;
      RowCopies copies;
      uint32_t in = 0;
      bool ok = true;
      for (int t = t_first; all(ok && t < total); t += t_step, ++in) {
        ok = all(wait_on(&ifull[in % kInfo], (in / kInfo) & 1, p.status));
        if (!ok) break;
        ok = copies.tile<64, kTileRows>(p, smem, kStage, empty, full, 0, p.k_blocks,
                                        sources + in % kInfo * kTileRows, first, lane);
        __syncwarp();
        if (elect_one()) mbar_arrive(&iempty[in % kInfo]);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else if (warp >= kEpiWarp) {
    kv4::regs_up<kRegsEpi>();
    const int quad = warp & 3, part = (warp - kEpiWarp) >> 2;
    uint8_t* buf = store + (warp - kEpiWarp) * kStore;
    const int half = part >> 1;
    const uint32_t from = tmem + (static_cast<uint32_t>(quad * 32) << 16) +
                          half * kSlots * kHalf + (part & 1) * kOwn;
    const float* x_scale = scales + quad * 32 + lane;
    const float* w_scale = scales + kTileRows + part * kOwn / kBlockK;
    const uint32_t read = first_cta<kPair>(tempty + kSlots * half);
    uint32_t it = 0, in = 0;
    bool known = true;
    for (int t = t_first; t < total; t += t_step) {
      uint64_t acc[kOwn / 2];
#pragma unroll
      for (int i = 0; i < kOwn / 2; ++i) acc[i] = 0;
#pragma unroll 1
      for (int b = 0; b < p.k_blocks; ++b, ++it) {
        const uint32_t slot = it % kSlots;
        named_bar_sync(1 + kSlots * half + slot, 32 * (kEpiWarps / 2 + 1));
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
      // (given up: nothing is stored, but the barriers are gone through together to the end)
      known = known && all(wait_on(&ifull[in % kInfo], (in / kInfo) & 1, p.status));
      const int4 tile = tiles[in % kInfo];               // first row, rows, feature tile
      __syncwarp();
      if (elect_one()) mbar_arrive(&iempty[in % kInfo]);
      ++in;
      if (!known) continue;
      const int at = rank * kTileRows + quad * 32;
#pragma unroll
      for (int c = 0; c < kOwn; c += kSend)
        store_rows<kSend>(p, &map_out, acc + c / 2, buf, tile.x + at, tile.y - at,
                          tile.z * kN + part * kOwn + c, lane);
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

template <bool kPair, int kN, bool kIndex, int kSend = kN / 4>
int run(Linear p, cudaStream_t st) {
  constexpr int kCtas = kPair ? 2 : 1;
  constexpr int kStage = tile_stage_bytes<kPair, kN>();
  p.n_tiles = (p.n + kN - 1) / kN;
  p.box_rows = p.n_src < kTileRows ? p.n_src : kTileRows;
  constexpr int kStoreBytes = kEpiWarps * 32 * kSend * 2;
  constexpr int kRing = ring<kN>();
  const int tail = kStoreBytes + kRing * kScaleRow * 4 + kInfo * (16 + kTileRows * 4) +
                   (4 * slots<kN>() + 2 + 2 * kRing + 2 * kInfo) * 8 + 4 + groups_bytes(p.groups);
  p.n_stages = (kSmemLimit - 1024 - tail) / (kStage + 16);
  if (p.n_stages > kMaxStages) p.n_stages = kMaxStages;
  const int smem = 1024 + p.n_stages * (kStage + 16) + tail;
  CUtensorMap mx, mw, mo = {};
  int rc = make_map(&mx, p.x, p.k, p.n_src, p.box_rows);
  if (!rc) rc = make_map(&mw, p.w, p.k, static_cast<long long>(p.groups) * p.n, kN / 2 / kCtas);
  if (!rc && p.vector)
    rc = make_tmap_2d_store_bf16(&mo, p.out, p.n, p.m, p.out_pitch * 2, kSend, 32);
  const auto kernel = tile_kernel<kPair, kN, kIndex, kSend>;
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
  // clusters that fit at once (one CTA to an SM)
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DFLASH_E_CUDA;
  static PerDevice fit;
  const int most = fit.get(dev, [&] {
    cudaLaunchConfig_t q = cfg;
    q.gridDim = dim3(p.sms / kCtas * kCtas);
    q.dynamicSmemBytes = kSmemLimit;
    int n = 0;
    return cudaOccupancyMaxActiveClusters(&n, kernel, &q) == cudaSuccess ? n : 0;
  });
  if (most < 1) return DFLASH_E_CUDA;
  const long long tiles = most_tiles(p, kTileRows * kCtas, kN);
  if (tiles > 0x7FFFFFFF - 256ll * kBand) return DFLASH_E_UNSUPPORTED;
  cfg.gridDim = dim3(static_cast<unsigned>(tiles < most ? tiles : most) * kCtas);
  cfg.numAttrs = 2;
  return cuda_err(cudaLaunchKernelEx(&cfg, kernel, mx, mw, mo, p));
}

}  // namespace

int run_tiles(const Linear& p, Choice tile, cudaStream_t st) {
  if (p.rows) return run<false, 256, true>(p, st);
  if (tile.features == 128) return run<false, 128, false>(p, st);
  if (tile.rows == 128) return run<false, 256, false>(p, st);
  // Few tiles of many blocks: the way out in two halves leaves shared memory for a fifth stage.  In
  // continuous use, each call with weights of its own, 512 rows x 24576 x 4096 take 46.5 us, 47.3 with
  // four stages; between a norm and a silu_mul, all three, 53.1 and 55.4 (700 x 12288 x 4096 37.7 and
  // 39.3, 1024 x 4096 x 12288 54.5 and 59.0); in a burst 41 and 45.  No size tried was slower, nor
  // did K of 1408 to 2048 gain.  Else at once (in bursts): 4000 x 12288 x 768 40 us, 43.5 in halves,
  // 2000 x 12288 x 256 13.2 and 14.5; 8191 x 24576 x 4096 alike, 601 and 607 at the power limit.
  return p.k_blocks >= 32 && most_tiles(p, 256, 256) <= 2ll * p.sms
             ? run<true, 256, false, 32>(p, st) : run<true, 256, false>(p, st);
}

}  // namespace fp8
}  // namespace dflash
