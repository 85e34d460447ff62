// Attention of a ragged batch's rows over a KV cache held in 4 bits.
//
// "DFlash双实现对比" (hotelren.com) §2 and "dflash-mlx" (dpshk.com) 单次前向验证 ⑤:
// the drafter's block attends to its context and itself, the target's verify
// forward to the cache and, causally, to the block.  Here the new rows are in the
// cache already, so both are one product over its rows:
//   out[t, h] = softmax(q[t, h] K^T scale) V over the rows below
//   m = L - T + t + 1 (causal) or L.
//
// Work.  A unit is one KV head of one sequence with a tile of up to NQ query rows
// (its G query heads times some of its T rows); its keys come in tiles of 128.
// The tiles of all units, in order, are cut into one equal run per CTA (one CTA
// per SM), whatever the lengths are; the plan is made on the device from the
// lengths.  A unit that lies in one CTA is written out by it; the pieces of a cut
// one go to the workspace as (O, max, sum) and a second kernel joins them in order,
// so results do not depend on timing.
//
// Products.  Both run on the tensor cores with the keys or dims as the 128 rows
// and the query rows as the columns, so that few query rows cost little:
//   S^T [128 keys x NQ]  = K [128 x D] Q^T         A = K  from TMEM, B = Q  (shared)
//   O^T [D x NQ]        += V^T [D x 128] P^T       A = V^T from TMEM, B = P (shared)
// The 4-bit values never pass through shared memory again after they came: the
// threads of one role expand a key's row of K each, those of another two dims of V^T
// at a time (the cell keeps V's 16 rows side by side for that), to fp16 (exact:
// 6 significant bits) straight into TMEM.  With them in shared memory its traffic,
// not DRAM, would bound the kernel: 128 KB written and read a tile of 18 KB.
// Q is kept in fp16, where need be times a power of two (exact for bf16 values down to
// 2^-15 of the unit's largest at least, 2^-23 of it off for smaller ones); P in fp16
// (half a step is 2^-11 of its value), O, the maximum and the sum in fp32.
// Softmax: a thread owns a key and walks the query columns.  The running maximum m
// of a column only moves when a tile passes it by 2^8, which one vote per tile
// finds out; until then exp2(x - m) needs no reduction over keys at all, and the
// column sums stay in registers until the unit ends.
//
// What bounds it.  Per tile of 128 keys the instruction slots: 4,900 warp instructions at
// 64 query columns (K and V^T expansion 800 and 1,100, softmax 2,000, waits and
// hand-overs the rest) and 7,500 at 128, so 1,230 and 1,870 clocks of the SM's four slots
// against 1,700 and 2,450 measured; the products themselves take 512 and 1,024.  Beside the
// tiles a unit costs three to five tiles' time: its first maxima, the drain of O, code that
// is fetched anew.  Measured: 32 blocks of 16 rows over 512 to 16,384 keys (32 + 8 heads of
// 128 dims) 118 us, 2.7 TB/s of cells and 600 TFLOP/s (109 us at 64 dims); 4 blocks at 32,768
// keys, 64 heads (128 columns), 84 to 88 us over several runs, 780 to 820 TFLOP/s; prompt chunks of
// 257 to 1,024 rows 158 to 170 us, 690 to 740 TFLOP/s (148 us at 64 dims).  The registers of a
// role are few: some 40 bytes of a thread go to local memory at 64 columns, 130 at 128 (one warp
// instruction in 100 there loads from it).
// Tried and slower: two warpgroups that expand V at 128 columns (the registers of the
// softmax), a second S buffer at 128 in place of those of K and V (201 us against 188 then),
// one copy of the code that reads the scores (195 against 187: the loop costs more than the
// instruction cache gains), scalar instead of packed products (175 against 169).
#include <cmath>

#include "kv4_attention.cuh"

namespace dflash {
namespace kv4 {
namespace {

template <int D, int NQ>
struct Cfg {
  static constexpr int kCell = Cell<D>::kBytes;
  static constexpr int kStage = kGran * kCell;
  // Warpgroups of each role.  A lane of the first three holds a key or a dim in TMEM, so
  // a role grows by sharing out dims (K), cells (V^T) or query columns (softmax).  Up to 32
  // query rows leave the expansion of K and V as the longest step: two each then (at 64
  // columns a second one for V is no faster).
  static constexpr int kKWgs = NQ <= 32 ? 2 : 1;
  static constexpr int kVWgs = NQ <= 32 ? 2 : 1;
  static constexpr int kSoftWgs = NQ <= 32 ? 1 : NQ / 32;
  static constexpr int kCols = NQ / kSoftWgs;          // query columns of a softmax warpgroup
  static constexpr int kVWarps = D / 32;               // warps of it that hold rows of V^T
  // First warps of the roles.
  static constexpr int kMisc = 0, kSoft = 4, kV = kSoft + 4 * kSoftWgs, kK = kV + 4 * kVWgs;
  static constexpr int kThreads = 32 * (kK + 4 * kKWgs);
  // Registers: the launch's share, and what the roles make of it.  The softmax holds
  // scores, sums and maxima of its columns.
  static constexpr int kRegsSoft = NQ == 128 ? 80 : 128;
  static constexpr int kRegsRest = 56;
  static constexpr int kRegsLaunch = 65536 / kThreads / 8 * 8;
  static_assert(kRegsSoft * 128 * kSoftWgs + kRegsRest * (kThreads - 128 * kSoftWgs) <=
                    kRegsLaunch * kThreads,
                "register split");
  static constexpr bool kKeepMax = NQ <= 64;           // the columns' maxima in registers too
  // TMEM columns
  static constexpr int kKCols = D / 2, kVCols = kTile / 2;
  static constexpr int kSBufs = NQ <= 64 ? 2 : 1;
  static constexpr int kV0 = 2 * kKCols, kS0 = kV0 + 2 * kVCols, kO0 = kS0 + kSBufs * NQ;
  static_assert(kO0 + NQ <= 512, "TMEM columns");
  // shared memory
  static constexpr int kPBytes = (NQ + 63) / 64 * kTile * 128;
  static constexpr int kQBytes = NQ * D * 2;
  static constexpr int kVGran = kGran / kVWgs;          // cells of a V warpgroup
  static constexpr int kFixed = 2 * kPBytes + 2 * kQBytes;
  static constexpr int kTables = 12 * 1024;
  static constexpr int kFit = (226 * 1024 - kFixed - kTables) / kStage;
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  static constexpr int kSmem = 1024 + kFixed + kTables + kStages * kStage;
  static_assert(kStages >= 3, "shared memory");
  // The record of tile j replaces that of j - kRing once the K and V warps let go of the cells
  // of tile j - kStages, and with them of its record.  The V warps began it after the product P V
  // of two tiles before, which the MMA warp issues after it read the record of the tile between.
  static constexpr int kRing = 16;
  static_assert(kRing > kStages, "tile records");
};

// Which key of a tile lies in TMEM lane r of S^T (and is r in the second product's k index), and
// which dim in lane r of O^T.
__device__ __forceinline__ int lane_key(int r) {
  return (r & ~15) | (r & 6) << 1 | (r >> 2 & 2) | (r & 1);
}
__device__ __forceinline__ int lane_dim(int r) { return (r & ~15) | (r & 7) << 1 | (r >> 3 & 1); }

template <int D, int NQ>
__global__ void __launch_bounds__(Cfg<D, NQ>::kThreads, 1)
    kv4_attention_kernel(const Kv4AttnParams p) {
  using C = Cfg<D, NQ>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  uint8_t* pbuf = smem;
  uint8_t* qbuf = pbuf + 2 * C::kPBytes;
  uint8_t* stages = qbuf + 2 * C::kQBytes;
  uint8_t* tables = stages + C::kStages * C::kStage;
  int* col_vis = reinterpret_cast<int*>(tables);           // [2][NQ] keys a column sees
  int* col_row = col_vis + 2 * NQ;                         // [2][NQ] row of q and out
  float* col_nm = reinterpret_cast<float*>(col_row + 2 * NQ);  // [NQ] kLift - running maximum
  float* col_f = col_nm + NQ;                              // [NQ] rescale factor, then 1 / sum
  float* red = col_f + NQ;                                 // [4][NQ]
  uint2* v_scales = reinterpret_cast<uint2*>(red + 4 * NQ);  // [8 kGran * 4] of the V warps
  Piece* piece = reinterpret_cast<Piece*>(v_scales + 32 * kGran);   // [2]
  Seg* segs = reinterpret_cast<Seg*>(piece + 2);           // [2] for the query rows
  Tile* tiles = reinterpret_cast<Tile*>(segs + 2);         // [kRing]
  uint64_t* bars = reinterpret_cast<uint64_t*>(tiles + C::kRing);
  uint64_t* full = bars;
  uint64_t* empty = full + C::kStages;
  uint64_t* kd_full = empty + C::kStages;  // [2] K tile in TMEM
  uint64_t* kd_empty = kd_full + 2;        // [2] S product done (with one S buffer)
  uint64_t* s_full = kd_empty + 2;         // [kSBufs] S in TMEM
  uint64_t* s_empty = s_full + 2;          // S read
  uint64_t* pv_full = s_empty + 1;         // [2] V^T tile in TMEM, P in shared memory
  uint64_t* pv_done = pv_full + 2;         // [2] P V product done
  uint64_t* q_full = pv_done + 2;          // [2] query rows and tables of a segment
  uint64_t* q_empty = q_full + 2;          // [2] read
  uint64_t* o_empty = q_empty + 2;         // O of a segment read
  uint64_t* seg_full = o_empty + 1;        // [2] segs
  uint64_t* seg_empty = seg_full + 2;      // [2]
  uint64_t* planned = seg_empty + 2;       // *any is there
  uint64_t* mdrain = planned + 1;
  uint32_t* q_max = reinterpret_cast<uint32_t*>(mdrain + 1);   // [2]
  uint32_t* tmem_slot = q_max + 2;
  volatile int* any = reinterpret_cast<volatile int*>(tmem_slot + 1);  // this CTA has tiles

  // (the shuffle tells the compiler that the index is the same all over the warp)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  constexpr int kProducer = C::kMisc, kMma = kProducer + 1, kQuery = kMma + 1;
  if (threadIdx.x == 0) {
#pragma unroll 1
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4 * C::kKWgs + C::kVWarps * C::kVWgs);
    }
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      mbar_init(&kd_full[i], 4 * C::kKWgs);
      mbar_init(&kd_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&pv_full[i], C::kVWarps * C::kVWgs + 4 * C::kSoftWgs);
      mbar_init(&pv_done[i], 1);
      mbar_init(&q_full[i], 2);
      mbar_init(&q_empty[i], 4 * C::kSoftWgs);
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_empty[i], 2);
    }
    mbar_init(s_empty, 4 * C::kSoftWgs);
    mbar_init(o_empty, 4 * C::kSoftWgs);
    mbar_init(planned, 1);
    mbar_init(mdrain, 1);
    fence_mbar_init();
  }
  if (warp == kMma) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp < C::kSoft || warp >= C::kV) regs_down<C::kRegsRest>();
  griddep_wait();
  Waiter wait{p.status, false};
  const int G = p.group;
  constexpr uint32_t tmem = 0;   // all 512 columns are this CTA's: they start at 0

  if (warp == kProducer) {
    // ---------------- the run, and the cells of its tiles, one bulk copy each ----------------
    const int per_slab = p.s.slab_rows / kCellRows;
    Walk walk(p);
    Seg g = {};
    bool have_seg = walk.next(p, &g);
    if (lane == 0) {
      *any = have_seg;
      segs[0] = g;
    }
    __syncwarp();
    if (have_seg) warp_arrive(&seg_full[0]);
    warp_arrive(planned);
    // lane: page (or sequence) of cell `lane` of the four tiles from `tile` on; nothing looks
    // at it before those tiles' turn
    auto slab_at = [&](int tile) {
      const int key16 = tile * kGran + lane;
      if (!p.paged) return g.b;
      if (key16 >= (g.end + kCellRows - 1) / kCellRows) return -1;
      return p.page_table[static_cast<size_t>(g.b) * p.max_pages +
                          (per_slab == 1 ? key16 : key16 / per_slab)];
    };
    int ahead = slab_at(g.tile);
    if (lane == 0) *reinterpret_cast<int4*>(p.meta + 4 * blockIdx.x) = make_int4(-1, 0, 0, 0);
    griddep_launch_dependents();
    // (a cache that several units of a sequence read stays in L2)
    const uint64_t pol =
        p.max_tokens > p.tile_rows ? l2_policy_evict_normal() : l2_policy_evict_first();
    int j = 0;
    bool go = true;
#pragma unroll 1
    for (int seg = 0; go && have_seg; ++seg) {
      if (g.tile == 0 && g.n < g.nt && lane == 0)     // the rest of this unit is others'
        *reinterpret_cast<int4*>(p.meta + 4 * blockIdx.x) =
            make_int4(walk.owner(walk.here + g.nt - g.n - 1), g.lo + g.t0,
                      min(p.tile_rows, g.T - g.t0) * G, g.h);
      const int look = min(3, g.n - 1), next_par = (seg + 1) & 1;
      const uint8_t* src = nullptr;        // this lane's cell of four tiles
      uint32_t have = 0, miss = 0;
#pragma unroll 1
      for (int i = 0; i < g.n; ++i, ++j) {
        const int st = j % C::kStages, l0 = (i & 3) * kGran, at = lane - l0;
        if (l0 == 0) {
          const int key16 = (g.tile + i) * kGran + lane;
          const bool use = key16 < (g.end + kCellRows - 1) / kCellRows;
          const bool there = ahead >= 0 && ahead < p.s.n_slabs;
          const int row16 = p.paged && per_slab > 1 ? key16 % per_slab : p.paged ? 0 : key16;
          src = p.s.cells +
                static_cast<size_t>((ahead * p.s.n_kv_heads + g.h) * per_slab + row16) * C::kCell;
          have = __ballot_sync(0xffffffffu, use && there);
          miss = __ballot_sync(0xffffffffu, use && !there);
          ahead = slab_at(g.tile + i + 4);
        }
        go = go && wait_on<true>(&empty[st], ((j / C::kStages) & 1) ^ 1, p.status);
        if (!__all_sync(0xffffffffu, go)) {
          go = false;
          break;
        }
        uint8_t* dst = stages + st * C::kStage;
        if (miss >> l0 & ((1u << kGran) - 1)) {     // pages that are missing read as zeros
          if (lane == 0) set_status(p.status, DFLASH_ST_PAGE_MISSING);
#pragma unroll 1
          for (int o = lane * 16; o < C::kStage; o += 512)
            if (miss >> (l0 + o / C::kCell) & 1)
              *reinterpret_cast<uint4*>(dst + o) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();        // (before the copies that come here next)
          __syncwarp();
        }
        if (at == 0) {
          Tile t = {g.end - (g.tile + i) * kTile,
                    (i == 0 ? kFirst : 0) | (i + 1 == g.n && g.final ? kFinal : 0)};
          tiles[j % C::kRing] = t;
          mbar_arrive_expect_tx(&full[st],
                                __popc(have >> l0 & ((1u << kGran) - 1)) * C::kCell);
        }
        __syncwarp();
        // (eight lanes at once: a copy from each takes the warp 60 to 80 clocks, copies from
        // one lane 150 each)
        if (at >= 0 && at < kGran && have >> lane & 1)
          bulk_load(dst + at * C::kCell, src, C::kCell, &full[st], pol);
        if (i == look) {
          // the next segment goes out while this one is read, so that its query rows are ready
          // in time (128 of them take as long as six tiles)
          Seg next = {};
          have_seg = walk.next(p, &next);
          if (have_seg) {
            if (seg >= 1)
              go = wait_on<true>(&seg_empty[next_par], (((seg + 1) >> 1) - 1) & 1, p.status);
            if (lane == 0) segs[next_par] = next;
            warp_arrive(&seg_full[next_par]);
          }
        }
      }
      if (!go) break;
      if (!have_seg) break;
      g = segs[next_par];
      ahead = slab_at(g.tile);
    }
    // no copy may still be landing when the CTA exits
#pragma unroll 1
    for (int st = 0; st < C::kStages && st < j; ++st) {
      const int last = st + (j - 1 - st) / C::kStages * C::kStages;
      mbar_wait_drain(&full[st], (last / C::kStages) & 1, p.status);
    }
    goto done;
  }
  wait(planned, 0);
  griddep_launch_dependents();
  if (wait.gave_up() || *any == 0) goto done;
  if (warp == kMma) {
    // ---------------- the products ----------------
    // The whole warp runs the loop and one elected lane issues, so that the operands stay
    // in uniform registers: 23 clocks an instruction, against 46 when one lane runs alone.
    constexpr uint32_t idesc_s = umma_idesc_f16(128, NQ, false);
    constexpr uint32_t idesc_o = umma_idesc_f16(128, NQ, true);
    const uint64_t q_desc = umma_sdesc_sw128(smem_u32(qbuf));
    const uint64_t p_desc = umma_sdesc_sw128_mn(smem_u32(pbuf), kTile * 128, 1024);
    bool ok = true;
    auto need = [&](uint64_t* bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, ok && wait_on(bar, parity, p.status));
    };
    auto issue_pv = [&](int j, bool first, int seg) {
      if (!ok) return;
      need(&pv_full[j & 1], (j >> 1) & 1);
      if (first && seg > 0) need(o_empty, (seg - 1) & 1);
      if (!ok) return;
      // P came through the generic proxy.  Its fence stands here, between the wait and the
      // products, once a tile: in the softmax warps it took 400 clocks of each.
      fence_proxy_async_smem();
      tc_fence_after();
      const uint32_t par = j & 1;
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < kTile / 16; ++ks)
          umma_f16_ts(C::kO0, C::kV0 + par * C::kVCols + ks * 8,
                      p_desc + ((par * C::kPBytes + ks * 2048) >> 4), idesc_o, !first || ks > 0);
        umma_commit(&pv_done[par]);
      }
    };
    int seg = -1, flags = 0;
    bool opened = false;
#pragma unroll 1
    for (int j = 0;; ++j) {
      const uint32_t sb = j % C::kSBufs, par = j & 1;
      need(&kd_full[par], (j >> 1) & 1);
      if (!ok) break;
      // (votes, so that what follows from the flags is the same all over the warp)
      flags = tiles[j % C::kRing].flags;
      const bool opens = __any_sync(0xffffffffu, flags & kFirst);
      const bool final = __any_sync(0xffffffffu, flags & kFinal);
      const int qs = opens ? seg + 1 : seg;
      if (opens) need(&q_full[qs & 1], (qs >> 1) & 1);
      // (two buffers: S of two tiles back was read before its P came, waited for already)
      if (C::kSBufs == 1) need(s_empty, (j & 1) ^ 1);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t q0 = q_desc + ((qs & 1) * C::kQBytes >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          umma_f16_ts(C::kS0 + sb * NQ, par * C::kKCols + ks * 8,
                      q0 + (((ks >> 2) * NQ * 128 + (ks & 3) * 32) >> 4), idesc_s, ks > 0);
        umma_commit(&s_full[sb]);
        if (C::kSBufs == 1) umma_commit(&kd_empty[par]);
      }
      if (j > 0) issue_pv(j - 1, opened, seg);
      seg = qs;
      opened = opens;
      if (final) {
        issue_pv(j, opened, seg);
        break;
      }
    }
    if (elect_one()) umma_commit(mdrain);
    if (lane == 0) mbar_wait_drain(mdrain, 0, p.status);
    __syncwarp();
  } else if (warp < C::kSoft) {
    // ---------------- query rows of a unit, D / 8 lanes a row ----------------
    // Converted as they are if the largest finite magnitude lies in [2^-2, 2^15): then
    // fp16 holds them to 2^-23 of it.  Else a second time, with a power of two that
    // brings it to [2^14, 2^15).
    constexpr int kPer = D / 8, kItems = NQ * kPer / 64, kLoads = 8;
    const int tid = threadIdx.x - 32 * kQuery;
    const int pc = tid % kPer;
    bool go = true;
#pragma unroll 1
    for (int seg = 0; go; ++seg) {
      const int par = seg & 1;
      wait(&seg_full[par], (seg >> 1) & 1);
      if (bar_or(15, 64, wait.dead)) break;                      // (and q_max is read)
      const Seg g = segs[par];
      go = !g.final;
      warp_arrive(&seg_empty[par]);
      const int rows = min(p.tile_rows, g.T - g.t0) * G;
      const int row0 = (g.lo + g.t0) * p.n_q_heads + g.h * G;
      uint8_t* qs = qbuf + par * C::kQBytes;
      auto load = [&](int q) {           // 8 dims of query row q
        uint4 x = make_uint4(0, 0, 0, 0);
        if (q < rows)
          x = *reinterpret_cast<const uint4*>(
              p.q +
              static_cast<size_t>(row0 + q + (q * p.group_inv >> 16) * (p.n_q_heads - G)) * D +
              8 * pc);
        return x;
      };
      float f = 1.f;
      int ex = 0;
      bool again = true;
#pragma unroll 1
      for (int pass = 0; again; ++pass) {
        constexpr uint32_t kAbs = 0x7FFF7FFFu;
        uint32_t m2 = 0;                 // largest magnitudes of the even and of the odd dims
#pragma unroll 1
        for (int it0 = 0; it0 < kItems; it0 += kLoads) {
          uint4 x[kLoads];
#pragma unroll
          for (int u = 0; u < kLoads; ++u) x[u] = load(((it0 + u) * 64 + tid) / kPer);
          if (pass == 0 && it0 == 0) {
            if (seg >= 2) wait.on<true>(&q_empty[par], ((seg >> 1) - 1) & 1);
#pragma unroll 1
            for (int q = tid; q < NQ; q += 64) {
              const int t = q * p.group_inv >> 16;
              col_row[par * NQ + q] = row0 + q + t * (p.n_q_heads - G);
              col_vis[par * NQ + q] =
                  p.causal && q < rows ? max(0, min(g.len, g.len - g.T + g.t0 + t + 1)) : g.len;
            }
          }
#pragma unroll
          for (int u = 0; u < kLoads; ++u) {
            const int q = ((it0 + u) * 64 + tid) / kPer;
            const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
            uint32_t y[4];
            m2 = __vimax3_u16x2(m2, w[0] & kAbs, w[1] & kAbs);
            m2 = __vimax3_u16x2(m2, w[2] & kAbs, w[3] & kAbs);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              y[e] = pack_f16(__uint_as_float(w[e] << 16) * f,
                              __uint_as_float(w[e] & 0xFFFF0000u) * f);
            *reinterpret_cast<uint4*>(qs + (pc >> 3) * NQ * 128 + q * 128 +
                                      (((pc & 7) ^ (q & 7)) << 4)) =
                make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
        again = false;
        if (pass == 0) {
          uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xFFFFu, m2 >> 16));
          if (m >= 0x7F80u) {            // infinities or NaN: the largest finite one
            m = 0;
#pragma unroll 1
            for (int it = 0; it < kItems; ++it) {
              const uint4 x = load((it * 64 + tid) / kPer);
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t a = w[e] & 0x7FFFu, c = w[e] >> 16 & 0x7FFFu;
                m = max(m, max(a < 0x7F80u ? a : 0u, c < 0x7F80u ? c : 0u));
              }
            }
            m = __reduce_max_sync(0xffffffffu, m);
          }
          if (lane == 0) q_max[warp - kQuery] = m;
          named_bar_sync(15, 64);
          const int most = static_cast<int>(max(q_max[0], q_max[1])), e = most >> 7;
          if (most != 0 && (e < 125 || e > 141)) {                        // e: exponent + 127
            ex = max(-126, min(126, 141 - e));
            f = pow2(ex);
            again = true;
          }
        }
      }
      if (tid == 0) {
        Piece pc = {g.tile, g.n, g.nt, p.causal ? max(0, g.len - g.T + g.t0 + 1) : g.len,
                    rows | (go ? 0 : kFinalPiece),
                    times_pow2(p.scale_log2, gain_exp(p.s.k_exp, g.h) - ex),
                    pow2(gain_exp(p.s.v_exp, g.h))};
        piece[par] = pc;
      }
      fence_proxy_async_smem();
      warp_arrive(&q_full[par]);
    }
  } else if (warp >= C::kK) {
    // ---------------- K to fp16: a thread expands its key's row ----------------
    const int r = threadIdx.x & 127, wg = (warp - C::kK) >> 2;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    bool go = true;
#pragma unroll 1
    for (int j = 0; go; ++j) {
      const int st = j % C::kStages;
      wait.on<true>(&full[st], (j / C::kStages) & 1);
      wait.on<true>(&(C::kSBufs == 2 ? s_full : kd_empty)[j & 1], ((j >> 1) & 1) ^ 1);
      if (wait.gave_up()) break;
      go = !(tiles[j % C::kRing].flags & kFinal);
      tc_fence_after();
      const uint8_t* cell = stages + st * C::kStage + (r / kCellRows) * C::kCell;
      const int rr = lane_key(r) % kCellRows;
      constexpr int kParts = D / 32 / C::kKWgs;          // of 32 dims, a round each
#pragma unroll 1
      for (int c = wg * kParts; c < (wg + 1) * kParts; ++c) {
        const uint4 w = *reinterpret_cast<const uint4*>(cell + Cell<D>::k_codes(rr, 2 * c));
        const uint32_t s2 = e4m3x2_to_f16x2(
            *reinterpret_cast<const uint16_t*>(cell + Cell<D>::k_scale(rr, 2 * c)));
        const uint32_t s_lo = __byte_perm(s2, 0, 0x1010), s_hi = __byte_perm(s2, 0, 0x3232);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        uint32_t o[16];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // (bytes 0 and 2 convert as they lie; 1 and 3 would take a shift each)
          const uint32_t sc = e < 2 ? s_lo : s_hi, up = u[e] >> 8;
          o[4 * e] = hmul2(e2m1x2_to_f16x2<0>(u[e]), sc);
          o[4 * e + 1] = hmul2(e2m1x2_to_f16x2<0>(up), sc);
          o[4 * e + 2] = hmul2(e2m1x2_to_f16x2<2>(u[e]), sc);
          o[4 * e + 3] = hmul2(e2m1x2_to_f16x2<2>(up), sc);
        }
        tmem_st_32x32b_x16(lane_base + (j & 1) * C::kKCols + c * 16, o);
      }
      warp_arrive(&empty[st]);
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(&kd_full[j & 1]);
    }
  } else if (warp >= C::kV) {
    // ---------------- V^T to fp16: a thread expands two dims of every fourth key pair -------
    // A byte of V holds two dims of one key, so a thread that takes both uses every bit of
    // its words.  The store that puts row g of sixteen lanes, and row g + 8, in lanes 4 g ..
    // 4 g + 3 fits: TMEM lane 16 i + g is dim 16 i + 2 g, lane 16 i + 8 + g the next one, and
    // the 16 keys of a cell go to the columns in the order of lane_key().
    if ((warp & 3) < C::kVWarps) {
      const int w4 = warp & 3, wg = (warp - C::kV) >> 2, g0 = wg * C::kVGran;
      const int t = lane & 3;
      const uint32_t lane_base =
          tmem + (static_cast<uint32_t>(w4 * 32) << 16) + C::kV0 + g0 * 8;
      uint2* scales = v_scales + (warp - C::kV) * 8 * C::kVGran;   // [16 dims][cell][4 keys]
      bool go = true;
#pragma unroll 1
      for (int j = 0; go; ++j) {
        const int st = j % C::kStages;
        wait(&full[st], (j / C::kStages) & 1);
        wait(&pv_done[j & 1], ((j >> 1) & 1) ^ 1);
        if (wait.gave_up()) break;
        const Tile tile = tiles[j % C::kRing];
        go = !(tile.flags & kFinal);
        tc_fence_after();
        const uint8_t* base = stages + st * C::kStage + g0 * C::kCell;
        // keys in use from this warpgroup's first cell on
        const int left = tile.left - g0 * kCellRows;
        // the scales to fp16 once for the sixteen that share one, 0 past the length (codes are
        // finite whatever they hold)
#pragma unroll
        for (int u = lane; u < 8 * C::kVGran; u += 32) {
          const int c = u / 4 % C::kVGran, i = u / (4 * C::kVGran), key = 4 * (u & 3);
          const int in = left - c * kCellRows - key;              // of these four keys
          const uint32_t w = *reinterpret_cast<const uint32_t*>(
                                 base + c * C::kCell + Cell<D>::v_scale(key, 2 * w4 + i)) &
                             (in >= 4 ? ~0u : in > 0 ? (1u << 8 * in) - 1u : 0u);
          scales[u] = make_uint2(e4m3x2_to_f16x2(w), e4m3x2_to_f16x2(w >> 16));
        }
        __syncwarp();
        const uint8_t* code = base + Cell<D>::v_codes(4 * t, 16 * w4 + (lane >> 2));
#pragma unroll 2
        for (int c = 0; c < C::kVGran; ++c) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w =
                *reinterpret_cast<const uint32_t*>(code + c * C::kCell + i * 8 * kCellRows);
            const uint2 f = scales[(i * C::kVGran + c) * 4 + t];
            // low (even dim) and high nibbles of two keys to a byte, bytes 0 and 2
            const uint32_t x4 = w >> 4, x8 = w >> 8;
            const uint32_t lo = (w & 0x000F000Fu) | (x4 & ~0x000F000Fu);
            const uint32_t hi = (x4 & 0x000F000Fu) | (x8 & ~0x000F000Fu);
            tmem_st_16x128b_x2(lane_base + (static_cast<uint32_t>(16 * i) << 16) +
                                   (j & 1) * C::kVCols + c * 8,
                               hmul2(e2m1x2_to_f16x2<0>(lo), f.x),
                               hmul2(e2m1x2_to_f16x2<0>(hi), f.x),
                               hmul2(e2m1x2_to_f16x2<2>(lo), f.y),
                               hmul2(e2m1x2_to_f16x2<2>(hi), f.y));
          }
        }
        warp_arrive(&empty[st]);
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&pv_full[j & 1]);
      }
    }
  } else {
    // ---------------- softmax: a thread owns a key ----------------
    regs_up<C::kRegsSoft>();
    constexpr int CW = C::kCols;
    constexpr bool kKeepMax = C::kKeepMax;
    const int wg = (warp - C::kSoft) >> 2, q4 = warp & 3;
    const int r = q4 * 32 + lane, col0 = wg * CW, d = lane_dim(r), my_key = lane_key(r);
    const uint32_t bar = 1 + wg;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
    float* nm = col_nm + col0;
    float* fac = col_f + col0;
    int j = 0;
    bool go = true;
#pragma unroll 1
    for (int seg = 0; go; ++seg) {
      const int par = seg & 1;
      const int* vis = col_vis + par * NQ + col0;
      // the segment's tables are there (that a product is done would not order their writes)
      wait(&q_full[par], (seg >> 1) & 1);
      if (bar_or(bar, 128, wait.dead)) break;
      const int n = piece[par].n, tile0 = piece[par].tile, sure = piece[par].sure;
      const float scale = piece[par].scale;
      float2 l[CW / 2], mr[kKeepMax ? CW / 2 : 1];        // sums; kLift - maxima
#pragma unroll
      for (int c = 0; c < CW / 2; ++c) l[c] = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int i = 0; i < n; ++i, ++j) {
        const int sb = j % C::kSBufs;
        const uint32_t s_addr = lane_base + C::kS0 + sb * NQ + col0;
        const int key = (tile0 + i) * kTile + my_key;
        const bool masked = (tile0 + i + 1) * kTile > sure;
        wait(&s_full[sb], (j / C::kSBufs) & 1);
        __syncwarp();
        tc_fence_after();
        // 16 columns of this key's scores in log2 units, minus the running maxima if `sub`
        auto scores = [&](const uint32_t (&v)[16], int c0, bool sub, float* x) {
          const float2 s2 = make_float2(scale, scale);
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            float2 m0 = make_float2(0.f, 0.f), m1 = m0;
            if (sub) {
              if (kKeepMax) {
                m0 = mr[kKeepMax ? (c0 + e) / 2 : 0];
                m1 = mr[kKeepMax ? (c0 + e) / 2 + 1 : 0];
              } else {
                const float4 m = *reinterpret_cast<const float4*>(nm + c0 + e);
                m0 = make_float2(m.x, m.y);
                m1 = make_float2(m.z, m.w);
              }
            }
            const float2 a = __ffma2_rn(
                make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), s2, m0);
            const float2 b = __ffma2_rn(
                make_float2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])), s2, m1);
            x[e] = a.x;
            x[e + 1] = a.y;
            x[e + 2] = b.x;
            x[e + 3] = b.y;
          }
          if (masked) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (key >= vis[c0 + e]) x[e] = -INFINITY;
          }
        };
        float x[CW];
        auto load_all = [&] {
          uint32_t v[CW / 16][16];
#pragma unroll
          for (int c = 0; c < CW / 16; ++c) tmem_ld_32x32b_x16(s_addr + c * 16, v[c]);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < CW / 16; ++c) scores(v[c], c * 16, true, x + c * 16);
        };
        bool move = i == 0;
        if (i > 0) {
          load_all();
          float mx = x[0];
#pragma unroll
          for (int e = 1; e < CW; ++e) mx = fmaxf(mx, x[e]);
          move = bar_or(bar, 128, wait.dead || mx > kMoveLog2 + kLift);
        }
        if (move) {
          if (i > 0 && bar_or(bar, 128, wait.dead)) goto done;
          // the columns' maxima over the tile (lane c: column c), and new running maxima
          float mine = -INFINITY;
#pragma unroll 1
          for (int c0 = 0; c0 < CW; c0 += 16) {
            uint32_t v[16];
            float y[16];
            tmem_ld_32x32b_x16(s_addr + c0, v);
            tmem_ld_wait();
            scores(v, c0, false, y);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float m = warp_max(y[e]);
              if (lane == c0 + e) mine = m;
            }
          }
          if (lane < CW) red[q4 * NQ + col0 + lane] = mine;
          named_bar_sync(bar, 128);
          if (r < CW) {
            const float* m4 = red + col0 + r;
            const float was = i == 0 ? kNoMax : kLift - nm[r];
            const float now =
                fmaxf(fmaxf(fmaxf(m4[0], m4[NQ]), fmaxf(m4[2 * NQ], m4[3 * NQ])), was);
            fac[r] = ex2(was - now);
            nm[r] = kLift - now;
          }
          named_bar_sync(bar, 128);
          if (i > 0) {
            wait(&pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1);
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < CW; c0 += 16) {
              uint32_t v[16];
              tmem_ld_32x32b_x16(lane_base + C::kO0 + col0 + c0, v);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e)
                v[e] = __float_as_uint(__uint_as_float(v[e]) * fac[c0 + e]);
              tmem_st_32x32b_x16(lane_base + C::kO0 + col0 + c0, v);
            }
            tmem_st_wait();
#pragma unroll
            for (int c = 0; c < CW / 2; ++c)
              l[c] = __fmul2_rn(l[c], *reinterpret_cast<const float2*>(fac + 2 * c));
          }
          if (kKeepMax) {
#pragma unroll
            for (int c = 0; c < (kKeepMax ? CW / 2 : 0); ++c)
              mr[c] = *reinterpret_cast<const float2*>(nm + 2 * c);
          }
          load_all();
        }
        if (C::kSBufs == 1) {
          tc_fence_before();
          warp_arrive(s_empty);
        }
        // (the P buffer is free: the products run in order, and S of this tile came after
        // the P V of two tiles back)
        uint8_t* prow = pbuf + (j & 1) * C::kPBytes + (col0 / 64) * kTile * 128 + r * 128;
#pragma unroll
        for (int c0 = 0; c0 < CW; c0 += 8) {
          uint32_t pk[4];
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float a = ex2(x[c0 + e]), b = ex2(x[c0 + e + 1]);
            l[(c0 + e) / 2] = __fadd2_rn(l[(c0 + e) / 2], make_float2(a, b));
            pk[e / 2] = pack_f16(a, b);
          }
          const int ch = (col0 % 64 + c0) / 8;
          *reinterpret_cast<uint4*>(prow + ((ch ^ (r & 7)) << 4)) =
              make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
        tc_fence_before();
        warp_arrive(&pv_full[j & 1]);              // (the reader fences the proxies)
      }
      // ---- the unit's (or piece's) result ----
      go = !(piece[par].rows & kFinalPiece);
      // column sums over the warp's keys: half of the columns change hands at each step,
      // so lane c ends with column c
      {
        float y[CW];
#pragma unroll
        for (int c = 0; c < CW; ++c) y[c] = c & 1 ? l[c / 2].y : l[c / 2].x;
#pragma unroll
        for (int n = CW / 2; n; n >>= 1) {
          const bool up = lane & n;
#pragma unroll
          for (int c = 0; c < n; ++c) {
            const float other = __shfl_xor_sync(0xffffffffu, up ? y[c] : y[c + n], n);
            y[c] = (up ? y[c + n] : y[c]) + other;
          }
        }
        if (lane < CW) red[q4 * NQ + col0 + lane] = y[0];
      }
      named_bar_sync(bar, 128);
      const bool whole = tile0 == 0 && n == piece[par].nt;
      const int slot = 2 * static_cast<int>(blockIdx.x) + (tile0 == 0 ? 1 : 0);
      if (r < CW) {
        const float* s4 = red + col0 + r;
        const float sum = (s4[0] + s4[NQ]) + (s4[2 * NQ] + s4[3 * NQ]);
        // a row that sees nothing is zero (its sum is 0; NaN for a row with NaN)
        fac[r] = whole ? (sum == 0.f ? 0.f : piece[par].v_gain / sum) : 1.f;
        if (!whole) {
          float* ml = p.part_ml + (static_cast<size_t>(slot) * NQ + col0 + r) * 2;
          ml[0] = -nm[r];
          ml[1] = sum;
        }
      }
      named_bar_sync(bar, 128);
      const int* row = col_row + par * NQ + col0;
      const int rows = min(CW, (piece[par].rows & ~kFinalPiece) - col0);    // of this warpgroup
      wait(&pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1);
      __syncwarp();
      tc_fence_after();
#pragma unroll 1
      for (int c0 = 0; c0 < rows; c0 += 16) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(lane_base + C::kO0 + col0 + c0, v);
        tmem_ld_wait();
        if (r >= D) continue;
        if (whole) {                       // (O is 0 where the sum is)
          // lanes r and r + 8 hold dims d and d + 1: of two columns each takes one, both dims
          const int odd = r >> 3 & 1;
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float a = __uint_as_float(v[e]), b = __uint_as_float(v[e + 1]);
            const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
            const float f = fac[c0 + e + odd];
            const uint32_t y = pack_bf16((odd ? got : a) * f, (odd ? b : got) * f);
            if (c0 + e + odd < rows)
              *reinterpret_cast<uint32_t*>(p.out + static_cast<size_t>(row[c0 + e + odd]) * D +
                                           (d & ~1)) = y;
          }
        } else {
          float* po = p.part_o + (static_cast<size_t>(slot) * NQ + col0 + c0) * D + d;
#pragma unroll
          for (int e = 0; e < 16; ++e) po[e * D] = __uint_as_float(v[e]);
        }
      }
      tc_fence_before();
      warp_arrive(o_empty);
      warp_arrive(&q_empty[par]);
      named_bar_sync(bar, 128);                    // nm, fac and red are read
    }
  }
done:
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) tmem_dealloc(*tmem_slot, 512);
}

// Joins the pieces of the unit that starts in CTA blockIdx.x of the kernel above and ends in a
// later one, in their order: a warp takes kR query rows and reads 4 or 8 pieces at a time.
// (Joined by whichever CTA writes the last piece, a block at 8192 keys, 19 pieces a unit, took
// 23 us in place of 18: one SM then reads them all.)
template <int NQ, int kR>
constexpr int kJoinWarps = NQ / kR < 8 ? NQ / kR : 8;

template <int D, int NQ, int kR>
__global__ void __launch_bounds__(32 * kJoinWarps<NQ, kR>) kv4_join_kernel(const Kv4AttnParams p) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int kV = D / 32, kAhead = kR == 1 ? 8 : 4;
  const int c0 = blockIdx.x, lane = threadIdx.x & 31;
  const int4 meta = *reinterpret_cast<const int4*>(p.meta + 4 * c0);
  const int c1 = meta.x, row0 = meta.y, rows = meta.z, h = meta.w;
  const int q0 = (blockIdx.y * kJoinWarps<NQ, kR> + (threadIdx.x >> 5)) * kR;
  if (c1 < 0 || q0 >= rows) return;
  const float gain = pow2(gain_exp(p.s.v_exp, h));
  auto slot = [&](int c) { return static_cast<size_t>(2 * c + (c == c0 ? 1 : 0)) * NQ + q0; };
  auto ml_of = [&](int c, int u) {
    return *reinterpret_cast<const float2*>(p.part_ml + 2 * (slot(c) + u));
  };
  float o[kR][kV], L[kR], M[kR];
#pragma unroll
  for (int u = 0; u < kR; ++u) {
    L[u] = 0.f;
    M[u] = kNoMax;
#pragma unroll
    for (int e = 0; e < kV; ++e) o[u][e] = 0.f;
  }
#pragma unroll 1
  for (int c = c0 + lane; c <= c1; c += 32)
#pragma unroll
    for (int u = 0; u < kR; ++u) M[u] = fmaxf(M[u], ml_of(c, u).x);
#pragma unroll
  for (int u = 0; u < kR; ++u) M[u] = warp_max(M[u]);
#pragma unroll 1
  for (int cb = c0; cb <= c1; cb += 32) {
    float w[kR];                           // of piece cb + lane
#pragma unroll
    for (int u = 0; u < kR; ++u) {
      const float2 ml = cb + lane <= c1 ? ml_of(cb + lane, u) : make_float2(kNoMax, 0.f);
      w[u] = cb + lane <= c1 ? ex2(ml.x - M[u]) : 0.f;
      L[u] += w[u] * ml.y;
    }
    const int n = min(32, c1 - cb + 1);
#pragma unroll 1
    for (int i = 0; i < n; i += kAhead) {
      float x[kAhead][kR][kV];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (i + k >= n) break;
        const float* src = p.part_o + slot(cb + i + k) * D + lane * kV;
#pragma unroll
        for (int u = 0; u < kR; ++u) {
          if (kV == 4)
            *reinterpret_cast<float4*>(x[k][u]) = *reinterpret_cast<const float4*>(src + u * D);
          else
            *reinterpret_cast<float2*>(x[k][u]) = *reinterpret_cast<const float2*>(src + u * D);
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (i + k >= n) break;
#pragma unroll
        for (int u = 0; u < kR; ++u) {
          const float f = __shfl_sync(0xffffffffu, w[u], i + k);
#pragma unroll
          for (int e = 0; e < kV; ++e) o[u][e] += f * x[k][u][e];
        }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kR; ++u) {
    const int q = q0 + u, t = q * p.group_inv >> 16;
    if (q >= rows) break;
#pragma unroll
    for (int x = 16; x; x >>= 1) L[u] += __shfl_xor_sync(0xffffffffu, L[u], x);
    const float f = L[u] == 0.f ? 0.f : gain / L[u];     // (O is 0 where the sum is)
    uint32_t y[kV / 2];
#pragma unroll
    for (int e = 0; e < kV / 2; ++e) y[e] = pack_bf16(o[u][2 * e] * f, o[u][2 * e + 1] * f);
    uint16_t* out =
        p.out +
        (static_cast<size_t>(row0 + t) * p.n_q_heads + h * p.group + q - t * p.group) * D +
        lane * kV;
    if (kV == 4)
      *reinterpret_cast<uint2*>(out) = make_uint2(y[0], y[kV / 2 - 1]);
    else
      *reinterpret_cast<uint32_t*>(out) = y[0];
  }
}

template <int D, int NQ, int kR>
int launch_join(const Kv4AttnParams& p, int ctas, cudaStream_t st) {
  constexpr int kWarps = kJoinWarps<NQ, kR>;
  return launch(kv4_join_kernel<D, NQ, kR>, dim3(ctas, NQ / kR / kWarps), dim3(32 * kWarps), 0, st,
                p);
}

// Four rows a warp; one where a unit is small, or cut into eight pieces or more on the average over
// the units (their lengths are on the device and not looked at: one long unit among many short
// ones has the four-row join, which is slower and no less right).  Measured with
// one and four: a block at 8192 keys (19 pieces) 16.5 and 18.8 us, single rows (units of 16)
// 83.2 and 83.7; four blocks at 32,768 keys (5 pieces) 87.0 and 85.8, prompt chunks (2 to 3)
// 167.1 and 163.5: there CTAs without work cost more than they save.
template <int D, int NQ>
int run_join(const Kv4AttnParams& p, int ctas, cudaStream_t st) {
  const long long units = static_cast<long long>(p.batch) * p.s.n_kv_heads *
                          ((p.max_tokens - 1) / p.tile_rows + 1);
  return NQ == 16 || units * 8 <= ctas ? launch_join<D, NQ, 1>(p, ctas, st)
                                       : launch_join<D, NQ, 4>(p, ctas, st);
}

// Query columns of a unit: the fewest that hold the rows of the longest sequence, for every unit of
// the batch.  So a prompt among tokens puts the tokens' units into 128 columns too: one prompt
// of 1,024 rows among 63 tokens over 512 to 16,384 keys takes 343 us, in two calls the prompt 34
// and the tokens 154.  Units of 9 to 16 rows (32 x 4 rows, 32 + 8 heads, same keys) take 77 us by the
// kernel for few rows and 103 through 32 columns at 64 dims, 118 and 109 at 128; 17 to 32 rows
// (32 x 8) 104 and 110 us.
int query_columns(const dflash_kv4_dims& d) {
  const long long rows =
      static_cast<long long>(d.max_tokens) * (d.n_q_heads / d.n_kv_heads);
  return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
}

struct AttnLayout {
  int ctas, nq;
  size_t off_ml, off_o, total;
};

AttnLayout attn_layout(const dflash_kv4_dims& d) {
  AttnLayout a = {};
  a.ctas = current_num_sms();
  a.nq = query_columns(d);
  const size_t rows = 2 * static_cast<size_t>(a.ctas) * a.nq;
  a.off_ml = (16 * static_cast<size_t>(a.ctas) + 255) / 256 * 256;
  a.off_o = a.off_ml + (8 * rows + 255) / 256 * 256;
  a.total = a.ctas > 0 ? a.off_o + 4 * rows * d.head_dim : 0;
  return a;
}

template <int D, int NQ>
int run(const Kv4AttnParams& p, int ctas, cudaStream_t st) {
  using C = Cfg<D, NQ>;
  static std::atomic<uint64_t> ready{0};
  int rc = smem_limit_once(&ready, reinterpret_cast<const void*>(kv4_attention_kernel<D, NQ>),
                           C::kSmem, C::kRegsLaunch);
  if (rc) return rc;
  if ((rc = launch(kv4_attention_kernel<D, NQ>, dim3(ctas), dim3(C::kThreads), C::kSmem, st, p)))
    return rc;
  return run_join<D, NQ>(p, ctas, st);
}

}  // namespace
}  // namespace kv4

size_t kv4_attention_bytes(const dflash_kv4_dims& d) { return kv4::attn_layout(d).total; }

}  // namespace dflash

using namespace dflash;
using namespace dflash::kv4;

extern "C" int dflash_kv4_attention(const dflash_kv4_dims* dims, const void* q,
                                    const int32_t* start, const dflash_kv4_view* cache,
                                    float scale, int causal, void* out, void* ws,
                                    size_t ws_bytes, dflash_stream_t stream) {
  DFLASH_ENTRY("dflash_kv4_attention");
  int rc = check_kv4_dims(dims);
  if (rc) return rc;
  if (!q || !start || !out || !cache || !cache->kv.seq_len || !std::isfinite(scale))
    return DFLASH_E_ARG;
  Kv4AttnParams p = {};
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
  if (!std::isfinite(p.scale_log2)) return DFLASH_E_ARG;
  if ((rc = kv4_store(*dims, cache, &p.s))) return rc;
  if (!aligned16(q) || !aligned16(out)) return DFLASH_E_ALIGN;
  Kv4Plan plan;
  if ((rc = make_kv4_plan(*dims, &plan))) return rc;
  if (!ws || ws_bytes < plan.total) return DFLASH_E_WORKSPACE;
  if (!aligned16(ws)) return DFLASH_E_ALIGN;
  const AttnLayout a = attn_layout(*dims);
  if (static_cast<long long>(dims->n_tokens) * dims->n_q_heads > INT32_MAX)
    return DFLASH_E_UNSUPPORTED;
  p.batch = dims->batch;
  p.n_tokens = dims->n_tokens;
  p.max_tokens = dims->max_tokens;
  p.n_q_heads = dims->n_q_heads;
  p.group = dims->n_q_heads / dims->n_kv_heads;
  p.causal = causal != 0;
  p.tile_rows = a.nq / p.group;
  p.group_inv = (65536 + p.group - 1) / p.group;
  // Measured in tiles: with 2, 3, 4, 5, 6 of them prompt chunks (128 columns) took 261, 201,
  // 186, 168, 171 us and a prompt of 4096 rows 325, 277, 229, 208, 209 (with 4 and 5 and today's
  // drain of O 174, 158 and 212, 193), four blocks at 32K (128 columns too, units of equal
  // length) 88.0, 86.9, 87.0, 87.6, 88.0; at batch 32 over 512 to 16,384 keys blocks of 16 rows
  // (64 columns) 118.1, 118.3, 119.4, 119.8, 122.0, of 8 rows (32 columns) 109.3, 110.0, 111.0,
  // 111.3, 113.8, of 4 (the kernel for few rows) 121.1, 117.8, 118.1, 118.8, 119.6, single rows
  // 86.8, 86.6, 83.3, 83.2, 83.5.  (At 64 dims 8 rows 103.3 to 106.8, in the same order.)
  p.unit_cost = a.nq == 128 ? 5 : a.nq == 16 ? 4 : 3;
  p.paged = cache->kv.page_table != nullptr;
  p.page_size = cache->kv.page_size;
  p.max_pages = cache->kv.max_pages;
  p.limit = p.paged ? p.max_pages * p.page_size : cache->kv.capacity;
  p.seq_len = cache->kv.seq_len;
  p.start = start;
  p.page_table = cache->kv.page_table;
  p.q = static_cast<const uint16_t*>(q);
  p.out = static_cast<uint16_t*>(out);
  p.status = ws_at<uint32_t>(ws, plan.off_status);
  p.meta = ws_at<int>(ws, plan.off_att);
  p.part_ml = ws_at<float>(ws, plan.off_att + a.off_ml);
  p.part_o = ws_at<float>(ws, plan.off_att + a.off_o);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool wide = dims->head_dim == 128;
  switch (a.nq) {
    case 16: {
      const int tiles = static_cast<long long>(p.max_tokens) * p.group <= 8 ? 1 : 2;
      if ((rc = launch_rows(p, dims->head_dim, tiles, a.ctas, st))) return rc;
      return wide ? run_join<128, 16>(p, a.ctas, st) : run_join<64, 16>(p, a.ctas, st);
    }
    case 32: return wide ? run<128, 32>(p, a.ctas, st) : run<64, 32>(p, a.ctas, st);
    case 64: return wide ? run<128, 64>(p, a.ctas, st) : run<64, 64>(p, a.ctas, st);
    default: return wide ? run<128, 128>(p, a.ctas, st) : run<64, 128>(p, a.ctas, st);
  }
}
