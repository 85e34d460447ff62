// 8-bit products of few rows: the weights streamed once.
//
// The operands change places: 128 features are the product's M, kT rows its N, so that a step
// moves 16 KB of weights for each 128 kT bytes of x and the tensor cores are not kept busy with
// rows that are not there.  Bound by the weights.  Two CTAs share an SM, so that one's start and
// end hide behind the other's stream.  Where there are fewer tiles than that, the CTAs of a
// cluster take a share of K each; they add their sums through distributed shared memory, in the
// order of the shares.
#include <algorithm>
#include <cmath>

#include "fp8_linear.cuh"

namespace dflash {
namespace fp8 {
namespace {

// Warps: 0 copies, 1 products, 2 to 5 epilogue, 6 places of tiles and scales, 7 rows of x by index.
constexpr int kStreamThreads = 256;
constexpr int kStreamBufs = 4;           // accumulators in TMEM
constexpr int kMaxSplit = 8;             // CTAs that share a tile's K
constexpr int kFactors = 8;              // blocks whose scales are in shared memory
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

// This CTA's rows of a tile, every kSplit-th: the sums of the kSplit CTAs, in their order.  32
// loads are on their way at a time: with two rows' the joining of 128 rows x 2560 features in two
// shares took 4 us.
template <int kSplit>
__device__ __forceinline__ void join_shares(const Linear& p, uint32_t part, int row, int rows,
                                            int n, int rank) {
  constexpr int kAtOnce = 32 / kSplit;
  for (int j = rank; j < rows; j += kAtOnce * kSplit) {
    float v[kAtOnce][kSplit];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
      for (int r = 0; r < kSplit; ++r)
        v[i][r] = j + i * kSplit < rows ? ld_cluster(part + (j + i * kSplit) * 512, r) : 0.f;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (j + i * kSplit >= rows) break;
      float sum = v[i][0];
#pragma unroll
      for (int r = 1; r < kSplit; ++r) sum += v[i][r];
      if (n < p.n)
        p.out[static_cast<long long>(row + j + i * kSplit) * p.out_pitch + n] =
            float_to_bf16_bits(sum);
    }
  }
}

template <int kT, bool kIndex>
__global__ void __launch_bounds__(kStreamThreads, 2)
stream_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
              const Linear p, const int split) {
  constexpr int kStage = stream_stage_bytes<kT>();
  constexpr int kCols = kStreamBufs * kT;
  constexpr int kScales = (kT + 31) / 32;          // rows of x to a lane
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  float* factors = reinterpret_cast<float*>(smem + p.n_stages * kStage);   // [kFactors][kT]
  int4* tiles = reinterpret_cast<int4*>(factors + kFactors * kT);          // [kInfo]
  uint32_t* sources = reinterpret_cast<uint32_t*>(tiles + kInfo);          // [kInfo][kT]
  uint64_t* full = reinterpret_cast<uint64_t*>(sources + kInfo * kT);
  uint64_t* empty = full + p.n_stages;
  uint64_t* tfull = empty + p.n_stages;            // [kStreamBufs]
  uint64_t* tempty = tfull + kStreamBufs;
  uint64_t* ffull = tempty + kStreamBufs;          // [kFactors]
  uint64_t* fempty = ffull + kFactors;
  uint64_t* ifull = fempty + kFactors;             // [kInfo]
  uint64_t* iempty = ifull + kInfo;
  uint64_t* mdrain = iempty + kInfo;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mdrain + 1);
  const Groups groups = groups_at(reinterpret_cast<uint8_t*>(tmem_slot + 1), p.groups);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int b_first = static_cast<int>(static_cast<long long>(p.k_blocks) * rank / split);
  const int b_last = static_cast<int>(static_cast<long long>(p.k_blocks) * (rank + 1) / split);
  const int t_first = blockIdx.x / split, t_step = gridDim.x / split;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.n_stages; ++i) {
      mbar_init(&full[i], 1 + (kIndex ? 32 : 0));
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kFactors; ++i) {
      mbar_init(&ffull[i], 1);
      mbar_init(&fempty[i], 4);
    }
    for (int i = 0; i < kInfo; ++i) {
      mbar_init(&ifull[i], 1);
      mbar_init(&iempty[i], kIndex ? 6 : 5);
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
  fill_groups(p, groups, kT, kStreamThreads);
  tc_fence_before();
  __syncthreads();
  griddep_launch_dependents();           // (the next grid's CTAs take TMEM only after this one's)
  tc_fence_after();
  const uint32_t tmem = same(*tmem_slot);
  const int total = groups.tiles[p.groups] * p.n_tiles;

  if (warp == 0) {
    const uint64_t pol = l2_policy_evict_normal();
    const uint32_t bytes = (128 + (kIndex ? 0 : p.box_rows)) * kBlockK;
    uint32_t stage = 0, phase = 0, in = 0;
    int issued = 0;
    bool ok = true;
    for (int t = t_first; all(ok && t < total); t += t_step, ++in) {
      int4 place;
      if (in == 0) {                     // (the first is not waited for)
        const Tile tile = tile_at<kT>(p, groups, t);
        place = make_int4(tile.row, tile.count, tile.n, tile.e * p.n + tile.n * 128);
      } else {
        ok = all(wait_on(&ifull[in % kInfo], (in / kInfo) & 1, p.status));
        if (!ok) break;
        place = tiles[in % kInfo];
      }
      const int x_row = same(place.x), w_row = same(place.w);
      if (elect_one()) mbar_arrive(&iempty[in % kInfo]);
#pragma unroll 1
      for (int b = b_first; b < b_last; ++b) {
        ok = all(wait_on(&empty[stage], phase ^ 1, p.status));
        if (!ok) break;
        uint8_t* a = smem + stage * kStage;
        if (elect_one()) {
          mbar_arrive_expect_tx(&full[stage], bytes);
          tma_load_2d(a, &map_w, &full[stage], b * kBlockK, w_row, pol);
          if (!kIndex)
            tma_load_2d(a + 128 * kBlockK, &map_x, &full[stage], b * kBlockK, x_row, pol);
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
        if (kIndex) fence_proxy_async_smem();
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
  } else if (warp == 6) {
    // Goes through the CTA's blocks kAhead ahead of what it hands over: writes down the places of
    // the tiles it comes to, reads the scales, and stores their products in the ring.
    constexpr int kAhead = 4;
    const uint32_t kbs = b_last - b_first;
    const uint32_t blocks = t_first < total ? ((total - 1 - t_first) / t_step + 1) * kbs : 0;
    float x[kAhead][kScales], w[kAhead];
    int src[kScales] = {};
    const float* ws = p.ws;
    int t = t_first, b = b_first;
    uint32_t in = 0, read = 0;
    bool ok = true;
    const auto load = [&](float (&x)[kScales], float& w) {
      if (read == blocks) return;
      if (b == b_first) {
        const Tile tile = tile_at<kT>(p, groups, t);
        // (the wait for a phase before the first passes at once)
        ok = ok && all(wait_on(&iempty[in % kInfo], ((in / kInfo) & 1) ^ 1, p.status));
#pragma unroll
        for (int i = 0; i < kScales; ++i) {
          src[i] = lane + 32 * i < kT ? source_row(p, tile, lane + 32 * i) : -1;
          if (kIndex && lane + 32 * i < kT)
            sources[in % kInfo * kT + place_of<kT>(lane + 32 * i)] =
                src[i] >= 0 ? static_cast<uint32_t>(src[i]) * (p.k / 16) : kNoRow;
        }
        if (lane == 0)
          tiles[in % kInfo] = make_int4(tile.row, tile.count, tile.n, tile.e * p.n + tile.n * 128);
        __syncwarp();
        if (elect_one()) mbar_arrive(&ifull[in % kInfo]);
        ++in;
        ws = p.ws + (static_cast<long long>(tile.e) * p.n_blocks + tile.n) * p.k_blocks;
      }
#pragma unroll
      for (int i = 0; i < kScales; ++i)
        x[i] = src[i] >= 0 ? p.xs[static_cast<long long>(b) * p.n_src + src[i]] : 0.f;
      w = ws[b];
      ++read;
      if (++b == b_last) {
        b = b_first;
        t += t_step;
      }
    };
#pragma unroll
    for (int j = 0; j < kAhead; ++j) load(x[j], w[j]);
    for (uint32_t it0 = 0; all(ok && it0 < blocks); it0 += kAhead) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const uint32_t it = it0 + j;
        if (it >= blocks) break;
        ok = ok && all(wait_on(&fempty[it % kFactors], ((it / kFactors) & 1) ^ 1, p.status));
        if (!ok) break;
        float* f = factors + it % kFactors * kT + lane;
#pragma unroll
        for (int i = 0; i < kScales; ++i)
          if (lane + 32 * i < kT) f[32 * i] = x[j][i] * w[j];
        __syncwarp();
        if (elect_one()) mbar_arrive(&ffull[it % kFactors]);
        load(x[j], w[j]);
      }
    }
  } else if (warp == 7) {
    if (kIndex) {
      RowCopies copies;
      uint32_t in = 0;
      bool ok = true;
      for (int t = t_first; all(ok && t < total); t += t_step, ++in) {
        ok = all(wait_on(&ifull[in % kInfo], (in / kInfo) & 1, p.status));
        if (!ok) break;
        ok = copies.tile<kT, kT>(p, smem + 128 * kBlockK, kStage, empty, full, b_first, b_last,
                                 sources + in % kInfo * kT, 0, lane);
        __syncwarp();
        if (elect_one()) mbar_arrive(&iempty[in % kInfo]);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  }

  // TMEM lane = feature, column = row of x
  const int et = (warp & 3) * 32 + lane;
  bool ok = true;
  uint64_t acc[kT / 2];
  int4 tile = {};                                   // first row, rows, feature tile
  if (warp >= 2 && warp < 6) {
    const uint32_t from = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    uint32_t it = 0, in = 0;
    for (int t = t_first; all(ok && t < total); t += t_step, ++in) {
      ok = all(wait_on(&ifull[in % kInfo], (in / kInfo) & 1, p.status));
      if (!ok) break;
      tile = tiles[in % kInfo];
      __syncwarp();
      if (elect_one()) mbar_arrive(&iempty[in % kInfo]);
#pragma unroll
      for (int i = 0; i < kT / 2; ++i) acc[i] = 0;
#pragma unroll 1
      for (int b = b_first; b < b_last; ++b, ++it) {
        const uint32_t slot = it % kStreamBufs;
        ok = wait_both(&tfull[slot], (it / kStreamBufs) & 1, &ffull[it % kFactors],
                       (it / kFactors) & 1, p.status);
        if (!ok) break;
        tc_fence_after();
        const float* f = factors + it % kFactors * kT;
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
        __syncwarp();
        if (elect_one()) mbar_arrive(&fempty[it % kFactors]);
      }
      if (!ok) break;
      const int n = tile.z * 128 + et;
      if (split == 1) {
        if (n < p.n) {
          uint16_t* dst = p.out + static_cast<long long>(tile.x) * p.out_pitch + n;
#pragma unroll
          for (int j = 0; j < kT; ++j) {
            if (j < tile.y)
              *dst = float_to_bf16_bits(j & 1 ? halves(acc[j / 2]).y : halves(acc[j / 2]).x);
            dst += p.out_pitch;
          }
        }
      } else {
        // (every copy and product of this CTA is done: the stages are free)
        float* part = reinterpret_cast<float*>(smem) + et;
#pragma unroll
        for (int j = 0; j < kT; ++j)
          part[j * 128] = j & 1 ? halves(acc[j / 2]).y : halves(acc[j / 2]).x;
      }
    }
  }
  if (split > 1) {
    __syncwarp();
    cluster_sync();
    if (warp >= 2 && warp < 6 && ok && t_first < total) {
      const int n = tile.z * 128 + et;
      const uint32_t part = smem_u32(smem) + et * 4;
      if (split == 2)
        join_shares<2>(p, part, tile.x, tile.y, n, rank);
      else if (split == 4)
        join_shares<4>(p, part, tile.x, tile.y, n, rank);
      else
        join_shares<8>(p, part, tile.x, tile.y, n, rank);
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

// CTAs that share a tile's K, and about how many us the call takes.  A CTA takes some 0.2 us a
// block (0.33 with 64 rows) where the memory has time for it, a quarter more with another on its
// SM; all together 2.4 ns a block of weights at the memory's rate, 0.4 where another tile's rows
// need the same weights.  A tile ends in 0.4 us, or 1.1 where two on an SM end together; shares of
// K are joined in 1 to 2 us, more where an SM has two clusters' CTAs with many rows (192 rows x
// 4096 x 4096 in two shares of 96 tiles take 14 us), and a second wave of them costs 4 more: 16
// rows x 4096 x 4096 (32 tiles of 32 blocks) take 7.4, 6.6, 6.3 us in two, four, eight shares, 64
// rows 8.2, 8.2, 13.2; 16 rows x 49152 x 4096 (384 tiles) 34 us whole and 43 in two shares.  (Bursts
// of one call: the 17 MB of 4096 x 4096 weights come from L2; from memory, as a layer finds its own,
// 16 rows take 7.1 us.)
double stream_split(const Linear& p, int tile_rows, double tiles, int* split) {
  const double experts = p.start ? std::min(p.groups, p.m) : 1;
  const double first = experts * ((p.n + 127) / 128);                     // tiles of these
  const double block = 0.16 + tile_rows * (p.rows ? 0.0036 : 0.0026), join = 1.0 + tile_rows / 64.0;
  const double memory = (0.0024 * first + 0.0004 * (tiles - first)) * p.k_blocks;
  double cost = 0;
  for (int s = 1; s <= kMaxSplit && s <= p.k_blocks; s *= 2) {
    const double ctas = tiles * s, waves = std::ceil(ctas / (2 * p.sms));
    const bool two = ctas > p.sms;                                        // CTAs on an SM
    const double work = waves * (((p.k_blocks + s - 1) / s) * block * (two ? 1.25 : 1.0) +
                                 (two ? 1.1 : 0.4));
    // (fewer than three CTAs to two SMs do not draw all that the memory gives)
    const double drawn = memory * (ctas * 2 < 3 * p.sms ? 1.15 : 1.0) + 0.4;
    double c = 2.6 + std::max(work, drawn);
    if (s > 1)
      c += join + 4.0 * (waves - 1) + (two ? 1.5 * tile_rows * tile_rows / 4096.0 : 0.0);
    if (s == 1 || c < cost) {
      *split = s;
      cost = c;
    }
  }
  return cost;
}

template <int kT, bool kIndex>
int run(Linear p, cudaStream_t st) {
  p.n_tiles = (p.n + 127) / 128;
  p.box_rows = p.n_src < kT ? p.n_src : kT;
  const int tail = kFactors * kT * 4 + kInfo * (16 + kT * 4) +
                   (2 * kStreamBufs + 2 * kFactors + 2 * kInfo + 1) * 8 + 4 +
                   groups_bytes(p.groups);
  p.n_stages = (kStreamSmem - 1024 - tail) / (stream_stage_bytes<kT>() + 16);
  if (p.n_stages > kMaxStages) p.n_stages = kMaxStages;
  const int smem = 1024 + p.n_stages * (stream_stage_bytes<kT>() + 16) + tail;
  CUtensorMap mx, mw;
  int rc = make_map(&mx, p.x, p.k, p.n_src, p.box_rows);
  if (!rc) rc = make_map(&mw, p.w, p.k, static_cast<long long>(p.groups) * p.n, 128);
  static std::atomic<uint64_t> ready{0};
  const void* kernel = reinterpret_cast<const void*>(stream_kernel<kT, kIndex>);
  if (!rc) rc = kv4::smem_limit_once(&ready, kernel, kStreamSmem);
  if (rc) return rc;
  const int nsm = p.sms;
  const long long tiles = most_tiles(p, kT, 128);
  if (tiles > 0x7FFFFFFF / 16) return DFLASH_E_UNSUPPORTED;
  const int split = stream_shares(p, kT);
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
  return cuda_err(cudaLaunchKernelEx(&cfg, stream_kernel<kT, kIndex>, mx, mw, p, split));
}

}  // namespace

int stream_shares(const Linear& p, int rows) {
  int split;
  stream_split(p, rows, static_cast<double>(most_tiles(p, rows, 128)), &split);
  return split;
}

double stream_cost(const Linear& p, int rows) {
  int split;
  return stream_split(p, rows, row_tiles(p, rows) * ((p.n + 127) / 128), &split);
}

int run_stream(const Linear& p, int rows, cudaStream_t st) {
  const bool index = p.rows != nullptr;
#define DFLASH_RUN(kT) (index ? run<kT, true>(p, st) : run<kT, false>(p, st))
  return rows == 16 ? DFLASH_RUN(16) : rows == 32 ? DFLASH_RUN(32) : DFLASH_RUN(64);
#undef DFLASH_RUN
}

}  // namespace fp8
}  // namespace dflash
