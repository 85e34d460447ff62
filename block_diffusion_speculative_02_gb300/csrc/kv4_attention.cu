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
// The 4-bit values never pass through shared memory again after they came: each
// thread of one warpgroup expands its key's row of K, each of another its dim's
// row of V^T (the cell keeps V's 16 rows side by side for that), to fp16 (exact:
// 6 significant bits) straight into TMEM.  With them in shared memory its traffic,
// not DRAM, would bound the kernel: 128 KB written and read a tile of 18 KB.
// Q is scaled by a power of two to [1, 2) per row and kept in fp16 (11 bits: exact
// for bf16 values within 2^-7 of the row's largest, 2^-25 of it for smaller ones);
// P in fp16 (2^-12 of its value), O, the maximum and the sum in fp32.
// Softmax: a thread owns a key and walks the query columns.  The running maximum m
// of a column only moves when a tile passes it by 2^8, which one vote per tile
// finds out; until then exp2(x - m) needs no reduction over keys at all, and the
// column sums stay in registers until the unit ends.
#include <cuda_fp16.h>

#include <cmath>

#include "kv4.cuh"

namespace dflash {
namespace {

constexpr int kTile = 128;              // keys
constexpr int kGran = kTile / kCellRows;
// P = 2^(x - m + kLift): 2^7 at the maximum, so that fp16 keeps probabilities down to 2^-31
// of it, and below 2^15 until the maximum moves.
constexpr float kLift = 7.0f;
constexpr float kMoveLog2 = 8.0f;       // a column passes its maximum by so much before it moves
constexpr float kNoMax = -1.0e30f;      // running maximum of a column that has seen nothing

template <int D, int NQ>
struct Cfg {
  static constexpr int kCell = Cell<D>::kBytes;
  static constexpr int kStage = kGran * kCell;
  static constexpr int kSoftWgs = NQ >= 32 ? 2 : 1;
  static constexpr int kCols = NQ / kSoftWgs;          // query columns of a softmax warpgroup
  static constexpr int kVWarps = D / 32;               // warps that hold rows of V^T
  static constexpr int kThreads = 32 * (8 + 4 * kSoftWgs + 4);
  // TMEM columns
  static constexpr int kKCols = D / 2, kVCols = kTile / 2;
  static constexpr int kSBufs = NQ <= 64 ? 2 : 1;
  static constexpr int kV0 = 2 * kKCols, kS0 = kV0 + 2 * kVCols, kO0 = kS0 + kSBufs * NQ;
  static_assert(kO0 + NQ <= 512, "TMEM columns");
  // shared memory
  static constexpr int kPBytes = (NQ + 63) / 64 * kTile * 128;
  static constexpr int kQBytes = NQ * D * 2;
  static constexpr int kVScale = kTile * (D / 16) * 2;  // fp16 scales of a V tile
  static constexpr int kFixed = 2 * kPBytes + 2 * kQBytes + 2 * kVScale;
  static constexpr int kTables = 12 * 1024;
  static constexpr int kFit = (226 * 1024 - kFixed - kTables) / kStage;
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  static constexpr int kSmem = 1024 + kFixed + kTables + kStages * kStage;
  static_assert(kStages >= 3, "shared memory");
};

struct Kv4AttnParams {
  Kv4Store s;
  int batch, n_tokens, max_tokens, n_q_heads, group, causal;
  int tile_rows;             // rows of a sequence in one unit
  int paged, page_size, max_pages, limit;
  const int32_t* seq_len;
  const int32_t* start;
  const int32_t* page_table;
  const uint16_t* q;
  uint16_t* out;
  float scale_log2;
  uint32_t* status;
  int* meta;                 // [CTAs][4]: the unit that starts in a CTA and ends in a later one
  float* part_ml;            // [2 CTAs][NQ][2]
  float* part_o;             // [2 CTAs][NQ][D]
};

// ----------------------------------------------------------------------------
// plan: which tiles this CTA takes
// ----------------------------------------------------------------------------
struct Seq {
  int lo, T, len, n_qt;      // first row, rows, length, units per head (0: nothing to do)
};

__device__ __forceinline__ Seq load_seq(const Kv4AttnParams& p, int b, bool* bad = nullptr) {
  Seq s = {0, 0, 0, 0};
  const int lo = p.start[b], hi = p.start[b + 1], len = p.seq_len[b];
  if (lo < 0 || hi < lo || hi > p.n_tokens || hi - lo > p.max_tokens || len < 0 ||
      len > p.limit) {
    if (bad) *bad = true;
    return s;
  }
  s.lo = lo;
  s.T = hi - lo;
  s.len = len;
  s.n_qt = (s.T + p.tile_rows - 1) / p.tile_rows;
  return s;
}

// Keys that some row of unit qt sees, and its tiles (at least one: its rows are written).
__device__ __forceinline__ int unit_end(const Kv4AttnParams& p, const Seq& s, int qt) {
  if (!p.causal) return s.len;
  return max(0, min(s.len, s.len - s.T + min(s.T, (qt + 1) * p.tile_rows)));
}
__device__ __forceinline__ int unit_tiles(int end) { return max(1, (end + kTile - 1) / kTile); }

// A unit also costs kUnitCost tiles of time that are not tiles (its query rows, the
// drain of its O); the run of a CTA is cut from tiles plus those.
constexpr int kUnitCost = 2;

__device__ __forceinline__ long long seq_cost(const Kv4AttnParams& p, const Seq& s) {
  long long n = 0;
  if (!p.causal) {
    n = static_cast<long long>(s.n_qt) * unit_tiles(s.len);
  } else {
    for (int i = 0; i < s.n_qt; ++i) n += unit_tiles(unit_end(p, s, i));
  }
  return (n + static_cast<long long>(s.n_qt) * kUnitCost) * p.s.n_kv_heads;
}

struct Start {
  long long left;            // cost of this CTA's run
  Seq s;                     // sequence of its first unit
  int b, qt, h;
  long long off;             // cost of that unit before the run
  int tiles;                 // of the run
};

// One segment: consecutive tiles of one unit.
struct Seg {
  int b, h, t0, lo, T, len, end, tile, n, nt;
};

// What the softmax needs of a segment, left in shared memory beside its query rows.
struct Piece {
  int tile, n, nt, sure, rows, h;   // sure: keys that every row sees
};

struct Walk {
  long long left, off;
  int b, qt, h, end, nt;
  Seq s;
  __device__ __forceinline__ Walk(const Kv4AttnParams& p, const Start& st)
      : left(st.left), off(st.off), b(st.b), qt(st.qt), h(st.h), s(st.s) {
    end = unit_end(p, s, qt);
    nt = unit_tiles(end);
  }
  __device__ __forceinline__ bool next(const Kv4AttnParams& p, Seg* g) {
    while (left > 0) {
      if (off == nt + kUnitCost) {        // the unit after this one
        off = 0;
        if (++h == p.s.n_kv_heads) {
          h = 0;
          ++qt;
          while (qt >= s.n_qt) {
            qt = 0;
            if (++b >= p.batch) return false;
            s = load_seq(p, b);
          }
          end = unit_end(p, s, qt);
          nt = unit_tiles(end);
        }
      }
      const int o = static_cast<int>(off);
      const int take = static_cast<int>(min(left, static_cast<long long>(nt + kUnitCost - o)));
      off += take;
      left -= take;
      const int from = max(0, o - kUnitCost), to = o + take - kUnitCost;
      if (to <= from) continue;
      g->b = b;
      g->h = h;
      g->t0 = qt * p.tile_rows;
      g->lo = s.lo;
      g->T = s.T;
      g->len = s.len;
      g->end = end;
      g->tile = from;
      g->nt = nt;
      g->n = to - from;
      return true;
    }
    return false;
  }
};

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// By one warp.  CTA c of n takes [W c / n, W (c + 1) / n) of the cost W of all units.
__device__ void make_start(const Kv4AttnParams& p, Start* out) {
  const int lane = lane_id();
  long long all = 0, mine = 0;
  Seq s = {0, 0, 0, 0};      // of sequence `lane` of a group of 32
  bool bad = false;
  for (int b0 = 0; b0 < p.batch; b0 += 32) {
    if (b0 + lane < p.batch) s = load_seq(p, b0 + lane, &bad);
    mine = b0 + lane < p.batch ? seq_cost(p, s) : 0;
    all += mine;
  }
  if (bad && blockIdx.x == 0) set_status(p.status, DFLASH_ST_CAPACITY);
  const long long W = warp_sum(all);
  const long long n = min(static_cast<long long>(gridDim.x), W), c = blockIdx.x;
  Start st = {};
  long long first = 0;
  if (c < n) {
    first = W * c / n;
    st.left = W * (c + 1) / n - first;
  }
  if (st.left > 0) {
    long long before = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      if (p.batch > 32) {
        if (b0 + lane < p.batch) s = load_seq(p, b0 + lane);
        mine = b0 + lane < p.batch ? seq_cost(p, s) : 0;
      }
      long long inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, before + inc > first);
      if (hit) {
        const int l = __ffs(hit) - 1;
        st.b = b0 + l;
        st.s.lo = __shfl_sync(0xffffffffu, s.lo, l);
        st.s.T = __shfl_sync(0xffffffffu, s.T, l);
        st.s.len = __shfl_sync(0xffffffffu, s.len, l);
        st.s.n_qt = __shfl_sync(0xffffffffu, s.n_qt, l);
        before += __shfl_sync(0xffffffffu, inc - mine, l);
        break;
      }
      before += __shfl_sync(0xffffffffu, inc, 31);
    }
    long long rem = first - before;
    int cost = unit_tiles(unit_end(p, st.s, 0)) + kUnitCost;
    while (rem >= static_cast<long long>(cost) * p.s.n_kv_heads) {
      rem -= static_cast<long long>(cost) * p.s.n_kv_heads;
      cost = unit_tiles(unit_end(p, st.s, ++st.qt)) + kUnitCost;
    }
    st.h = static_cast<int>(rem / cost);
    st.off = rem - static_cast<long long>(st.h) * cost;
  }
  // the segments once over: their tiles, and the unit that is left unfinished
  int meta[4] = {-1, 0, 0, 0};
  Seg g = {};
  Walk w(p, st);
  while (w.next(p, &g)) {
    st.tiles += g.n;
    if (g.tile == 0 && g.n < g.nt) {   // its last tile ends where the run does plus the rest
      const long long end = first + st.left + (g.nt - g.n);
      meta[0] = static_cast<int>((end * n - 1) / W);
      meta[1] = g.lo + g.t0;
      meta[2] = min(p.tile_rows, g.T - g.t0) * p.group;
      meta[3] = g.h;
    }
  }
  if (lane == 0) {
    *out = st;
    *reinterpret_cast<int4*>(p.meta + 4 * blockIdx.x) =
        make_int4(meta[0], meta[1], meta[2], meta[3]);
  }
}

// ----------------------------------------------------------------------------
// small device pieces
// ----------------------------------------------------------------------------
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Named barrier of n threads that also ORs a flag over them.
__device__ __forceinline__ bool bar_or(uint32_t id, uint32_t n, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %1, 0;\n\t"
      "barrier.cta.red.or.pred b, %2, %3, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1], %2, [%3], %4;" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// D[tmem] (+)= A[tmem] * B[smem]^T, fp16 operands, issued by one thread.
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor, kind::f16: A = B = fp16, D = fp32; b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t umma_idesc_f16(int M, int N, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// A wait of a role that goes on regardless: once one gave up, the rest are skipped, so
// every role still runs its loops to their end (named barriers included).
// (The loop is kept out of line: five roles share the instruction cache.  Reading the
// global timer takes longer than most waits, so the bounded wait comes after some tries.)
__device__ __noinline__ bool slow_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                       uint32_t* status) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait(bar, parity, abort_flag, status);
}

__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                        uint32_t* status) {
  return mbar_try_wait(bar, parity) || slow_wait(bar, parity, abort_flag, status);
}

struct Waiter {
  volatile int* abort_flag;
  uint32_t* status;
  bool dead;
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
    if (!dead) dead = !wait_on(bar, parity, abort_flag, status);
    __syncwarp();
  }
};

__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if (lane_id() == 0) mbar_arrive(bar);
}

// ----------------------------------------------------------------------------
// the kernel
// ----------------------------------------------------------------------------
template <int D, int NQ>
__global__ void __launch_bounds__(Cfg<D, NQ>::kThreads, 1)
    kv4_attention_kernel(const Kv4AttnParams p) {
  using C = Cfg<D, NQ>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  uint8_t* pbuf = smem;
  uint8_t* qbuf = pbuf + 2 * C::kPBytes;
  uint8_t* vscale = qbuf + 2 * C::kQBytes;
  uint8_t* stages = vscale + 2 * C::kVScale;
  uint8_t* tables = stages + C::kStages * C::kStage;
  float* col_sc = reinterpret_cast<float*>(tables);        // [2][NQ] log2 units per score
  int* col_vis = reinterpret_cast<int*>(col_sc + 2 * NQ);  // [2][NQ] keys a column sees
  int* col_row = col_vis + 2 * NQ;                         // [2][NQ] row of q and out
  float* col_nm = reinterpret_cast<float*>(col_row + 2 * NQ);  // [NQ] kLift - running maximum
  float* col_f = col_nm + NQ;                              // [NQ] rescale factor, then 1 / sum
  float* red = col_f + NQ;                                 // [4][NQ]
  Piece* piece = reinterpret_cast<Piece*>(red + 4 * NQ);   // [2]
  uint64_t* bars = reinterpret_cast<uint64_t*>(piece + 2);
  uint64_t* full = bars;
  uint64_t* empty = full + C::kStages;
  uint64_t* kd_full = empty + C::kStages;  // [2] K tile in TMEM
  uint64_t* kd_empty = kd_full + 2;        // [2] S product done
  uint64_t* vd_full = kd_empty + 2;        // [2] V^T tile in TMEM
  uint64_t* s_full = vd_full + 2;          // [kSBufs] S in TMEM
  uint64_t* s_empty = s_full + 2;          // [kSBufs] S read
  uint64_t* p_full = s_empty + 2;          // [2] P in shared memory
  uint64_t* pv_done = p_full + 2;          // [2] P V product done
  uint64_t* q_full = pv_done + 2;          // [2] query rows and tables of a segment
  uint64_t* q_empty = q_full + 2;          // [2] read
  uint64_t* o_empty = q_empty + 2;         // O of a segment read
  uint64_t* mdrain = o_empty + 1;
  Start* start = reinterpret_cast<Start*>(mdrain + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(start + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kProducer = 8 + 4 * C::kSoftWgs, kMma = kProducer + 1, kQuery = kMma + 1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4 + C::kVWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&kd_full[i], 4);
      mbar_init(&kd_empty[i], 1);
      mbar_init(&vd_full[i], C::kVWarps);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 4 * C::kSoftWgs);
      mbar_init(&p_full[i], 4 * C::kSoftWgs);
      mbar_init(&pv_done[i], 1);
      mbar_init(&q_full[i], 2);
      mbar_init(&q_empty[i], 4 * C::kSoftWgs);
    }
    mbar_init(o_empty, 4 * C::kSoftWgs);
    mbar_init(mdrain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMma) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  griddep_wait();
  if (warp == kProducer) make_start(p, start);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_launch_dependents();
  constexpr uint32_t tmem = 0;   // all 512 columns are this CTA's: they start at 0
  const int G = p.group;
  Walk walk(p, *start);
  Seg g;
  Waiter wait{abort_flag, p.status, false};

  if (warp == kProducer) {
    // ---------------- cells of a tile, one bulk copy each ----------------
    // (a cache that several units of a sequence read stays in L2)
    const uint64_t pol =
        p.max_tokens > p.tile_rows ? l2_policy_evict_normal() : l2_policy_evict_first();
    int j = 0;
    bool go = true;
    // lane: page of cell `lane` of the four tiles from `tile` on
    auto pages = [&](int tile) {
      const int key = tile * kTile + lane * kCellRows;
      int slab = g.b;
      if (p.paged && key < g.end) {
        slab = p.page_table[static_cast<size_t>(g.b) * p.max_pages + key / p.page_size];
        if (slab >= p.s.n_slabs) slab = -1;
      }
      return slab;
    };
    while (go && walk.next(p, &g)) {
      int slab4 = 0, ahead = pages(g.tile);
      for (int i = 0; i < g.n; ++i, ++j) {
        const int st = j % C::kStages;
        if ((i & 3) == 0) {
          slab4 = ahead;
          ahead = pages(g.tile + i + 4);
        }
        const int slab = __shfl_sync(0xffffffffu, slab4, (i & 3) * kGran + (lane & (kGran - 1)));
        const int key = (g.tile + i) * kTile + lane * kCellRows;
        const bool use = lane < kGran && key < g.end;
        const uint32_t have = __ballot_sync(0xffffffffu, use && slab >= 0);
        const uint32_t miss = __ballot_sync(0xffffffffu, use && slab < 0);
        if (!wait_on(&empty[st], ((j / C::kStages) & 1) ^ 1, abort_flag, p.status)) go = false;
        if (!__all_sync(0xffffffffu, go)) {
          go = false;
          break;
        }
        uint8_t* dst = stages + st * C::kStage;
        if (miss) {                                 // pages that are missing read as zeros
          if (lane == 0) set_status(p.status, DFLASH_ST_PAGE_MISSING);
          for (int c = 0; c < kGran; ++c)
            if (miss >> c & 1)
              for (int o = lane * 16; o < C::kCell; o += 512)
                *reinterpret_cast<uint4*>(dst + c * C::kCell + o) = make_uint4(0, 0, 0, 0);
          __syncwarp();
        }
        if (lane == 0) mbar_arrive_expect_tx(&full[st], __popc(have) * C::kCell);
        __syncwarp();
        if (have >> lane & 1) {
          const int row = p.paged ? key % p.page_size : key;
          bulk_load(dst + lane * C::kCell, p.s.cells + cell_index(p.s, slab, g.h, row) * C::kCell,
                    C::kCell, &full[st], pol);
        }
      }
    }
    // no copy may still be landing when the CTA exits
    for (int st = 0; st < C::kStages && st < j; ++st) {
      const int last = st + (j - 1 - st) / C::kStages * C::kStages;
      mbar_wait_drain(&full[st], (last / C::kStages) & 1, p.status);
    }
  } else if (warp == kMma) {
    // ---------------- the products ----------------
    // The whole warp runs the loop and one elected lane issues, so that the operands stay
    // in uniform registers: 23 clocks an instruction, against 46 when one lane runs alone.
    constexpr uint32_t idesc_s = umma_idesc_f16(128, NQ, false);
    constexpr uint32_t idesc_o = umma_idesc_f16(128, NQ, true);
    const uint64_t q_desc = umma_sdesc_sw128(smem_u32(qbuf));
    const uint64_t p_desc = umma_sdesc_sw128_mn(smem_u32(pbuf), kTile * 128, 1024);
    bool ok = true;
    auto need = [&](uint64_t* bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, ok && wait_on(bar, parity, abort_flag, p.status));
    };
    auto issue_pv = [&](int j, bool first, int seg) {
      need(&p_full[j & 1], (j >> 1) & 1);
      need(&vd_full[j & 1], (j >> 1) & 1);
      if (first && seg > 0) need(o_empty, (seg - 1) & 1);
      if (!ok) return;
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
    int j = 0, seg = 0, last_seg = 0;
    bool last_first = false;
    while (ok && walk.next(p, &g)) {
      for (int i = 0; ok && i < g.n; ++i, ++j) {
        const uint32_t sb = j % C::kSBufs, par = j & 1, qpar = seg & 1;
        need(&kd_full[par], (j >> 1) & 1);
        if (i == 0) need(&q_full[qpar], (seg >> 1) & 1);
        if (j >= C::kSBufs) need(&s_empty[sb], (j / C::kSBufs - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            umma_f16_ts(C::kS0 + sb * NQ, par * C::kKCols + ks * 8,
                        q_desc + ((qpar * C::kQBytes + (ks >> 2) * NQ * 128 + (ks & 3) * 32) >> 4),
                        idesc_s, ks > 0);
          umma_commit(&s_full[sb]);
          umma_commit(&kd_empty[par]);
        }
        if (j > 0) issue_pv(j - 1, last_first, last_seg);
        last_first = i == 0;
        last_seg = seg;
      }
      ++seg;
    }
    if (ok && j > 0) issue_pv(j - 1, last_first, last_seg);
    if (elect_one()) umma_commit(mdrain);
    if (lane == 0) mbar_wait_drain(mdrain, 0, p.status);
    __syncwarp();
  } else if (warp >= kQuery) {
    // ---------------- query rows of a unit, D / 8 lanes a row ----------------
    constexpr int kPer = D / 8, kItems = NQ * kPer / 64, kLoads = kItems < 8 ? kItems : 8;
    const int tid = threadIdx.x - 32 * kQuery;
    for (int seg = 0; walk.next(p, &g); ++seg) {
      const int par = seg & 1;
      const int rows = min(p.tile_rows, g.T - g.t0) * G;
      const int row0 = (g.lo + g.t0) * p.n_q_heads + g.h * G;
      const float kx = p.scale_log2 * pow2(gain_exp(p.s.k_exp, g.h));
      uint8_t* qs = qbuf + par * C::kQBytes;
#pragma unroll 1
      for (int it0 = 0; it0 < kItems; it0 += kLoads) {
        uint4 x[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          const int q = ((it0 + u) * 64 + tid) / kPer, t = q / G;
          x[u] = make_uint4(0, 0, 0, 0);
          if (q < rows)
            x[u] = *reinterpret_cast<const uint4*>(
                p.q + static_cast<size_t>(row0 + t * p.n_q_heads + q - t * G) * D +
                8 * (tid % kPer));
        }
        if (it0 == 0 && seg >= 2) wait(&q_empty[par], ((seg >> 1) - 1) & 1);
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          const int q = ((it0 + u) * 64 + tid) / kPer, pc = tid % kPer, t = q / G;
          const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
          uint32_t m = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            m = max(m, max(w[e] & 0x7FFFu, w[e] >> 16 & 0x7FFFu));
#pragma unroll
          for (int o = kPer / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          const int ex = max(-126, min(126, 127 - static_cast<int>(m >> 7)));
          const float f = pow2(ex);
          uint32_t y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            y[e] = pack_f16(__uint_as_float(w[e] << 16) * f,
                            __uint_as_float(w[e] & 0xFFFF0000u) * f);
          *reinterpret_cast<uint4*>(qs + (pc >> 3) * NQ * 128 + q * 128 +
                                    (((pc & 7) ^ (q & 7)) << 4)) =
              make_uint4(y[0], y[1], y[2], y[3]);
          if (pc == 0) {
            col_sc[par * NQ + q] = kx * pow2(-ex);
            col_row[par * NQ + q] = row0 + t * p.n_q_heads + q - t * G;
            col_vis[par * NQ + q] =
                p.causal && q < rows ? max(0, min(g.len, g.len - g.T + g.t0 + t + 1)) : g.len;
          }
        }
      }
      if (tid == 0) {
        Piece pc = {g.tile, g.n, g.nt, p.causal ? max(0, g.len - g.T + g.t0 + 1) : g.len, rows,
                    g.h};
        piece[par] = pc;
      }
      fence_proxy_async_smem();
      warp_arrive(&q_full[par]);
    }
  } else if (warp < 4) {
    // ---------------- K to fp16: a thread expands its key's row ----------------
    const int r = threadIdx.x;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    int j = 0;
    while (walk.next(p, &g)) {
      for (int i = 0; i < g.n; ++i, ++j) {
        const int st = j % C::kStages;
        wait(&full[st], (j / C::kStages) & 1);
        if (j >= 2) wait(&kd_empty[j & 1], ((j >> 1) - 1) & 1);
        tc_fence_after();
        const uint8_t* cell = stages + st * C::kStage + (r / kCellRows) * C::kCell;
        const int rr = r % kCellRows;
#pragma unroll 1
        for (int c2 = 0; c2 < D / 64; ++c2) {          // 64 dims a round
          const uint4 wa = *reinterpret_cast<const uint4*>(cell + Cell<D>::k_codes(rr, 4 * c2));
          const uint4 wb = *reinterpret_cast<const uint4*>(cell + Cell<D>::k_codes(rr, 4 * c2 + 2));
          const uint32_t sc = *reinterpret_cast<const uint32_t*>(cell + Cell<D>::k_scale(rr, 4 * c2));
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t s2 = e4m3x2_to_f16x2(c ? sc >> 16 : sc);
            const uint32_t s_lo = __byte_perm(s2, 0, 0x1010), s_hi = __byte_perm(s2, 0, 0x3232);
            const uint32_t u[4] = {c ? wb.x : wa.x, c ? wb.y : wa.y, c ? wb.z : wa.z,
                                   c ? wb.w : wa.w};
            uint32_t o[16];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t f[4];
              e2m1x8_to_f16x2(u[e], f);
#pragma unroll
              for (int x = 0; x < 4; ++x) o[4 * e + x] = hmul2(f[x], e < 2 ? s_lo : s_hi);
            }
            tmem_st_32x32b_x16(lane_base + (j & 1) * C::kKCols + c2 * 32 + c * 16, o);
          }
        }
        warp_arrive(&empty[st]);
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&kd_full[j & 1]);
      }
    }
  } else if (warp < 8) {
    // ---------------- V^T to fp16: a thread expands its dim's row ----------------
    // The 16 threads of a group of dims share their scales, so each scale is turned to
    // fp16 once, by all threads together, and read back.
    if (warp - 4 < C::kVWarps) {
      constexpr int kN = 32 * C::kVWarps;
      const int d = threadIdx.x - 128;
      const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp - 4) * 32) << 16) + C::kV0;
      const int shift = 4 * (d & 1);
      int j = 0;
      while (walk.next(p, &g)) {
        for (int i = 0; i < g.n; ++i, ++j) {
          const int st = j % C::kStages;
          wait(&full[st], (j / C::kStages) & 1);
          const uint8_t* base = stages + st * C::kStage;
          uint8_t* vsc = vscale + (j & 1) * C::kVScale;
          {  // 8 scales a thread: half the rows of a cell, one group of dims
            const int c = d / (D / 8), x = d % (D / 8);
            const uint2 s8 = *reinterpret_cast<const uint2*>(base + c * C::kCell +
                                                             Cell<D>::v_scale(0, 0) + x * 8);
            *reinterpret_cast<uint4*>(vsc + d * 16) =
                make_uint4(e4m3x2_to_f16x2(s8.x), e4m3x2_to_f16x2(s8.x >> 16),
                           e4m3x2_to_f16x2(s8.y), e4m3x2_to_f16x2(s8.y >> 16));
          }
          if (j >= 2) wait(&pv_done[j & 1], ((j >> 1) - 1) & 1);
          tc_fence_after();
          named_bar_sync(3, kN);
          const int left = g.end - (g.tile + i) * kTile;     // keys in use from here on
          const uint8_t* code = base + Cell<D>::v_codes(0, d / 2);
          const uint4* scl = reinterpret_cast<const uint4*>(vsc + d / 16 * 32);
#pragma unroll 2
          for (int c = 0; c < kGran; ++c) {
            const uint4 w4 = *reinterpret_cast<const uint4*>(code + c * C::kCell);
            const uint4 sa = scl[c * (D / 8)], sb = scl[c * (D / 8) + 1];
            const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
            const uint32_t s[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              // this dim's nibbles of four keys, two to a byte
              const uint32_t u = w[e] >> shift;
              const uint32_t x = (u & 0x000F000Fu) | (u >> 4 & 0x00F000F0u);
              o[2 * e] = hmul2(e2m1x2_to_f16x2<0>(x), s[2 * e]);
              o[2 * e + 1] = hmul2(e2m1x2_to_f16x2<2>(x), s[2 * e + 1]);
            }
            if (left < (c + 1) * kCellRows) {                // rows past the length count as 0
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int key = c * kCellRows + 2 * e;
                if (key >= left) o[e] = 0;
                else if (key + 1 >= left) o[e] &= 0xFFFFu;
              }
            }
            tmem_st_32x32b_x8(lane_base + (j & 1) * C::kVCols + c * 8, o);
          }
          warp_arrive(&empty[st]);
          tmem_st_wait();
          tc_fence_before();
          warp_arrive(&vd_full[j & 1]);
        }
      }
    }
  } else {
    // ---------------- softmax: a thread owns a key ----------------
    constexpr int CW = C::kCols;
    constexpr bool kKeep = CW <= 32;       // the tile's scores stay in registers
    const int wg = (warp - 8) >> 2, q4 = warp & 3;
    const int r = q4 * 32 + lane, col0 = wg * CW;
    const uint32_t bar = 1 + wg;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
    float* nm = col_nm + col0;
    float* fac = col_f + col0;
    const int total = start->tiles;
    for (int j = 0, seg = 0; j < total; ++seg) {
      const int par = seg & 1;
      const float* sc = col_sc + par * NQ + col0;
      const int* vis = col_vis + par * NQ + col0;
      wait(&s_full[j % C::kSBufs], (j / C::kSBufs) & 1);     // the segment's tables are there
      const int n = piece[par].n, tile0 = piece[par].tile, sure = piece[par].sure;
      float2 l[CW / 2];
#pragma unroll
      for (int c = 0; c < CW / 2; ++c) l[c] = make_float2(0.f, 0.f);
      if (r < CW) nm[r] = kLift - kNoMax;
      named_bar_sync(bar, 128);
      for (int i = 0; i < n; ++i, ++j) {
        const int sb = j % C::kSBufs;
        const uint32_t s_addr = lane_base + C::kS0 + sb * NQ + col0;
        const int key = (tile0 + i) * kTile + r;
        const bool masked = (tile0 + i + 1) * kTile > sure;
        wait(&s_full[sb], (j / C::kSBufs) & 1);
        tc_fence_after();
        // 16 columns of S times their scale, minus the running maximum
        auto scores = [&](const uint32_t (&v)[16], int c0, float* x) {
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 a = *reinterpret_cast<const float4*>(sc + c0 + e);
            const float4 b = *reinterpret_cast<const float4*>(nm + c0 + e);
            const float2 lo = __ffma2_rn(
                make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])),
                make_float2(a.x, a.y), make_float2(b.x, b.y));
            const float2 hi = __ffma2_rn(
                make_float2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])),
                make_float2(a.z, a.w), make_float2(b.z, b.w));
            x[e] = lo.x;
            x[e + 1] = lo.y;
            x[e + 2] = hi.x;
            x[e + 3] = hi.y;
          }
          if (masked) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (key >= vis[c0 + e]) x[e] = -INFINITY;
          }
        };
        float x[kKeep ? CW : 16], mx = -INFINITY;
        auto load_all = [&] {
          uint32_t v[CW / 16][16];
#pragma unroll
          for (int c = 0; c < CW / 16; ++c) tmem_ld_32x32b_x16(s_addr + c * 16, v[c]);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < CW / 16; ++c) scores(v[c], c * 16, x + c * 16);
        };
        if (kKeep) {
          load_all();
#pragma unroll
          for (int e = 0; e < (kKeep ? CW : 0); ++e) mx = fmaxf(mx, x[e]);
        } else if (i > 0) {
#pragma unroll 1
          for (int c0 = 0; c0 < CW; c0 += 16) {
            uint32_t v[16];
            tmem_ld_32x32b_x16(s_addr + c0, v);
            tmem_ld_wait();
            scores(v, c0, x);
#pragma unroll
            for (int e = 0; e < 16; ++e) mx = fmaxf(mx, x[e]);
          }
        }
        if (bar_or(bar, 128, i == 0 || mx > kMoveLog2 + kLift)) {
          // the columns' maxima over the tile, and new running maxima
#pragma unroll 1
          for (int c0 = 0; c0 < CW; c0 += 16) {
            uint32_t v[16];
            tmem_ld_32x32b_x16(s_addr + c0, v);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float y = __uint_as_float(v[e]) * sc[c0 + e];
              const float m = warp_max(masked && key >= vis[c0 + e] ? -INFINITY : y);
              if (lane == e) red[q4 * NQ + col0 + c0 + e] = m;
            }
          }
          named_bar_sync(bar, 128);
          if (r < CW) {
            const float* m4 = red + col0 + r;
            const float was = kLift - nm[r];
            const float now = fmaxf(fmaxf(fmaxf(m4[0], m4[NQ]), fmaxf(m4[2 * NQ], m4[3 * NQ])), was);
            fac[r] = i == 0 ? 0.f : ex2(was - now);
            nm[r] = kLift - now;
          }
          named_bar_sync(bar, 128);
          if (i > 0) {
            wait(&pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1);
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
          if (kKeep) load_all();
        }
        if (kKeep) {
          tc_fence_before();
          warp_arrive(&s_empty[sb]);
        }
        if (j >= 2) wait(&pv_done[j & 1], ((j >> 1) - 1) & 1);     // P buffer free
        uint8_t* prow = pbuf + (j & 1) * C::kPBytes + (col0 / 64) * kTile * 128 + r * 128;
#pragma unroll
        for (int c0 = 0; c0 < CW; c0 += 16) {
          float* xc = kKeep ? x + c0 : x;
          if (!kKeep) {
            uint32_t v[16];
            tmem_ld_32x32b_x16(s_addr + c0, v);
            tmem_ld_wait();
            if (c0 + 16 == CW) {
              tc_fence_before();
              warp_arrive(&s_empty[sb]);
            }
            scores(v, c0, xc);
          }
          uint32_t pk[8];
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float a = ex2(xc[e]), b = ex2(xc[e + 1]);
            l[(c0 + e) / 2] = __fadd2_rn(l[(c0 + e) / 2], make_float2(a, b));
            pk[e / 2] = pack_f16(a, b);
          }
#pragma unroll
          for (int c8 = 0; c8 < 2; ++c8) {
            const int ch = (col0 % 64 + c0) / 8 + c8;
            *reinterpret_cast<uint4*>(prow + ((ch ^ (r & 7)) << 4)) =
                make_uint4(pk[4 * c8], pk[4 * c8 + 1], pk[4 * c8 + 2], pk[4 * c8 + 3]);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        warp_arrive(&p_full[j & 1]);
      }
      // ---- the unit's (or piece's) result ----
      // column sums over the warp's keys: halves of the columns change hands at each
      // step, so lane x ends with column x (of the first 32, then of the next)
      {
        float* lf = reinterpret_cast<float*>(l);
#pragma unroll
        for (int c32 = 0; c32 < CW; c32 += 32) {
          constexpr int kN = CW < 32 ? CW : 32;
          float* y = lf + c32;
#pragma unroll
          for (int n = kN / 2; n; n >>= 1) {
            const bool up = lane & n;
#pragma unroll
            for (int c = 0; c < n; ++c) {
              const float other = __shfl_xor_sync(0xffffffffu, up ? y[c] : y[c + n], n);
              y[c] = (up ? y[c + n] : y[c]) + other;
            }
          }
          if (kN == 16) y[0] += __shfl_xor_sync(0xffffffffu, y[0], 16);
          if (lane < kN) red[q4 * NQ + col0 + c32 + lane] = y[0];
        }
      }
      named_bar_sync(bar, 128);
      const bool whole = tile0 == 0 && n == piece[par].nt;
      const int slot = 2 * static_cast<int>(blockIdx.x) + (tile0 == 0 ? 1 : 0);
      if (r < CW) {
        const float* s4 = red + col0 + r;
        const float sum = (s4[0] + s4[NQ]) + (s4[2 * NQ] + s4[3 * NQ]);
        // a row that sees nothing is zero (its sum is 0; NaN for a row with NaN)
        fac[r] = whole ? (sum == 0.f ? 0.f : pow2(gain_exp(p.s.v_exp, piece[par].h)) / sum) : 1.f;
        if (!whole) {
          float* ml = p.part_ml + (static_cast<size_t>(slot) * NQ + col0 + r) * 2;
          ml[0] = -nm[r];
          ml[1] = sum;
        }
      }
      named_bar_sync(bar, 128);
      const int* row = col_row + par * NQ + col0;
      const int rows = piece[par].rows - col0;                      // of this warpgroup
      wait(&pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1);
      tc_fence_after();
#pragma unroll 1
      for (int c0 = 0; c0 < CW; c0 += 16) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(lane_base + C::kO0 + col0 + c0, v);
        tmem_ld_wait();
        if (r < D && c0 < rows) {
          float* po = p.part_o + (static_cast<size_t>(slot) * NQ + col0 + c0) * D + r;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float f = fac[c0 + e];
            const float y = f == 0.f ? 0.f : __uint_as_float(v[e]) * f;
            if (whole) {
              if (c0 + e < rows)
                p.out[static_cast<size_t>(row[c0 + e]) * D + r] = float_to_bf16_bits(y);
            } else {
              po[e * D] = y;
            }
          }
        }
      }
      tc_fence_before();
      warp_arrive(o_empty);
      warp_arrive(&q_empty[par]);
      named_bar_sync(bar, 128);                    // nm, fac and red are read
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) tmem_dealloc(*tmem_slot, 512);
}

// Joins the pieces of the unit that starts in CTA blockIdx.x of the kernel above
// and ends in a later one: a warp per query row.
template <int D, int NQ>
__global__ void __launch_bounds__(128) kv4_join_kernel(const Kv4AttnParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int c0 = blockIdx.x, lane = threadIdx.x & 31;
  const int4 meta = *reinterpret_cast<const int4*>(p.meta + 4 * c0);
  const int c1 = meta.x, row0 = meta.y, h = meta.w;
  const int q = blockIdx.y * 4 + (threadIdx.x >> 5);
  if (c1 < 0 || q >= meta.z) return;
  constexpr int kV = D / 32;
  float o[kV], L = 0.f, M = kNoMax;
#pragma unroll
  for (int e = 0; e < kV; ++e) o[e] = 0.f;
  auto slot = [&](int c) { return static_cast<size_t>(2 * c + (c == c0 ? 1 : 0)) * NQ + q; };
  for (int c = c0 + lane; c <= c1; c += 32) M = fmaxf(M, p.part_ml[2 * slot(c)]);
  M = warp_max(M);
  for (int cb = c0; cb <= c1; cb += 32) {
    float w = 0.f;
    if (cb + lane <= c1) {
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * slot(cb + lane));
      w = ex2(ml.x - M);
      L += w * ml.y;
    }
#pragma unroll 4
    for (int i = 0; i < min(32, c1 - cb + 1); ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const float* src = p.part_o + slot(cb + i) * D + lane * kV;
      if (kV == 4) {
        const float4 x = *reinterpret_cast<const float4*>(src);
        o[0] += wi * x.x;
        o[1] += wi * x.y;
        o[2 % kV] += wi * x.z;
        o[3 % kV] += wi * x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(src);
        o[0] += wi * x.x;
        o[1] += wi * x.y;
      }
    }
  }
#pragma unroll
  for (int x = 16; x; x >>= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
  const float f = L == 0.f ? 0.f : pow2(gain_exp(p.s.v_exp, h)) / L;
  const int t = q / p.group;
  uint16_t* out =
      p.out + (static_cast<size_t>(row0 + t) * p.n_q_heads + h * p.group + q - t * p.group) * D +
      lane * kV;
  uint32_t y[kV / 2];
#pragma unroll
  for (int e = 0; e < kV / 2; ++e)
    y[e] = L == 0.f ? 0u
                    : static_cast<uint32_t>(float_to_bf16_bits(o[2 * e] * f)) |
                          static_cast<uint32_t>(float_to_bf16_bits(o[2 * e + 1] * f)) << 16;
  if (kV == 4)
    *reinterpret_cast<uint2*>(out) = make_uint2(y[0], y[kV / 2 - 1]);
  else
    *reinterpret_cast<uint32_t*>(out) = y[0];
}

// Query columns of a unit: the fewest that hold the rows of the longest sequence.
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
  int rc = set_smem_limit(reinterpret_cast<const void*>(kv4_attention_kernel<D, NQ>), C::kSmem);
  if (rc) return rc;
  if ((rc = launch(kv4_attention_kernel<D, NQ>, dim3(ctas), dim3(C::kThreads), C::kSmem, st, p)))
    return rc;
  return launch(kv4_join_kernel<D, NQ>, dim3(ctas, NQ / 4), dim3(128), 0, st, p);
}

}  // namespace

size_t kv4_attention_bytes(const dflash_kv4_dims& d) { return attn_layout(d).total; }

}  // namespace dflash

using namespace dflash;

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
  p.paged = cache->kv.page_table != nullptr;
  p.page_size = cache->kv.page_size;
  p.max_pages = cache->kv.max_pages;
  p.limit = p.paged ? p.max_pages * p.page_size : cache->kv.capacity;
  p.seq_len = cache->kv.seq_len;
  p.start = start;
  p.page_table = cache->kv.page_table;
  p.q = static_cast<const uint16_t*>(q);
  p.out = static_cast<uint16_t*>(out);
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
  p.status = ws_at<uint32_t>(ws, plan.off_status);
  p.meta = ws_at<int>(ws, plan.off_att);
  p.part_ml = ws_at<float>(ws, plan.off_att + a.off_ml);
  p.part_o = ws_at<float>(ws, plan.off_att + a.off_o);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool wide = dims->head_dim == 128;
  switch (a.nq) {
    case 16: return wide ? run<128, 16>(p, a.ctas, st) : run<64, 16>(p, a.ctas, st);
    case 32: return wide ? run<128, 32>(p, a.ctas, st) : run<64, 32>(p, a.ctas, st);
    case 64: return wide ? run<128, 64>(p, a.ctas, st) : run<64, 64>(p, a.ctas, st);
    default: return wide ? run<128, 128>(p, a.ctas, st) : run<64, 128>(p, a.ctas, st);
  }
}
