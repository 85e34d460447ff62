// What the kernels of the attention over a 4-bit cache share: their parameters, the plan
// (which tiles of which units a CTA takes), waits and small device pieces.
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "kv4.cuh"

namespace dflash {
namespace kv4 {

constexpr int kTile = 128;              // keys
constexpr int kGran = kTile / kCellRows;
// P = 2^(x - m + kLift): 2^7 at the maximum, so that fp16 keeps probabilities down to 2^-31
// of it, and below 2^15 until the maximum moves.
constexpr float kLift = 7.0f;
constexpr float kMoveLog2 = 8.0f;       // a column passes its maximum by so much before it moves
constexpr float kNoMax = -1.0e30f;      // running maximum of a column that has seen nothing

struct Kv4AttnParams {
  Kv4Store s;
  int batch, n_tokens, max_tokens, n_q_heads, group, causal;
  int tile_rows;             // rows of a sequence in one unit
  // A unit also costs some tiles' time that is not tiles (its query rows, the first
  // maxima, the drain of its O): the runs are cut from tiles plus those.
  int unit_cost;
  int group_inv;             // ceil(2^16 / group): x * group_inv >> 16 = x / group, x < 128
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

__device__ __forceinline__ long long seq_cost(const Kv4AttnParams& p, const Seq& s) {
  long long n = 0;
  if (!p.causal) {
    n = static_cast<long long>(s.n_qt) * unit_tiles(s.len);
  } else {
#pragma unroll 1
    for (int i = 0; i < s.n_qt; ++i) n += unit_tiles(unit_end(p, s, i));
  }
  return (n + static_cast<long long>(s.n_qt) * p.unit_cost) * p.s.n_kv_heads;
}

// One segment: consecutive tiles of one unit.
struct Seg {
  int b, h, t0, lo, T, len, end, tile, n, nt;
  int final;                 // the last of the CTA
};

// A tile, as the warps that work on it read it.
struct Tile {
  int left;                  // keys in use from its first one on
  int flags;                 // the first of its segment; the last of the CTA
};
constexpr int kFirst = 1, kFinal = 2, kFinalPiece = 256;

// What the softmax needs of a segment, left in shared memory beside its query rows.
struct Piece {
  int tile, n, nt, sure;            // sure: keys that every row sees
  int rows;                         // and kFinalPiece, if it is the last of the CTA
  float scale, v_gain;              // log2 units per score; 2^exp of V's head
};

// The run of this CTA, by one warp.  With W the cost of all units, every CTA takes W / n
// (the first W % n one more), n = min(CTAs, W).
struct Walk {
  int left, off;             // cost left, and of the unit at hand before that
  int b, qt, h, end, nt;
  Seq s;
  int per, rem, here;        // shares; where the run stands among all costs

  __device__ __forceinline__ void unit(const Kv4AttnParams& p) {
    end = unit_end(p, s, qt);
    nt = unit_tiles(end);
  }
  __device__ __forceinline__ int owner(int pos) const {
    const int big = rem * (per + 1);
    return pos < big ? pos / (per + 1) : rem + (pos - big) / per;
  }

  __device__ __forceinline__ explicit Walk(const Kv4AttnParams& p)
      : left(0), off(0), b(0), qt(0), h(0), end(0), nt(0), per(0), rem(0), here(0) {
    const int lane = lane_id();
    long long all = 0, mine = 0;
    Seq t = {0, 0, 0, 0};    // of sequence `lane` of a group of 32
    bool bad = false;
#pragma unroll 1
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      mine = 0;
      if (b0 + lane < p.batch) {
        t = load_seq(p, b0 + lane, &bad);
        mine = seq_cost(p, t);
      }
      all += mine;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    if (all > INT32_MAX) bad = true;
    if (bad && blockIdx.x == 0) set_status(p.status, DFLASH_ST_CAPACITY);
    if (all > INT32_MAX) return;
    const int W = static_cast<int>(all), n = min(static_cast<int>(gridDim.x), W);
    const int c = blockIdx.x;
    if (c >= n) return;
    per = W / n;
    rem = W - per * n;
    here = c * per + min(c, rem);
    left = per + (c < rem ? 1 : 0);
    int before = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      if (p.batch > 32) {
        mine = 0;
        if (b0 + lane < p.batch) {
          t = load_seq(p, b0 + lane);
          mine = seq_cost(p, t);
        }
      }
      int inc = static_cast<int>(mine);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, before + inc > here);
      if (hit) {
        const int l = __ffs(hit) - 1;
        b = b0 + l;
        s.lo = __shfl_sync(0xffffffffu, t.lo, l);
        s.T = __shfl_sync(0xffffffffu, t.T, l);
        s.len = __shfl_sync(0xffffffffu, t.len, l);
        s.n_qt = __shfl_sync(0xffffffffu, t.n_qt, l);
        before += __shfl_sync(0xffffffffu, inc - static_cast<int>(mine), l);
        break;
      }
      before += __shfl_sync(0xffffffffu, inc, 31);
    }
    off = here - before;
    unit(p);
#pragma unroll 1
    while (off >= (nt + p.unit_cost) * p.s.n_kv_heads) {
      off -= (nt + p.unit_cost) * p.s.n_kv_heads;
      ++qt;
      unit(p);
    }
    h = off / (nt + p.unit_cost);
    off -= h * (nt + p.unit_cost);
  }

  // Whether next() will find another segment: what is left is more than the part of the
  // next unit's cost that is not tiles.
  __device__ __forceinline__ bool more(const Kv4AttnParams& p) const {
    return left > p.unit_cost;
  }

  __device__ __forceinline__ bool next(const Kv4AttnParams& p, Seg* g) {
#pragma unroll 1
    while (left > 0) {
      if (off == nt + p.unit_cost) {        // the unit after this one
        off = 0;
        if (++h == p.s.n_kv_heads) {
          h = 0;
          ++qt;
#pragma unroll 1
          while (qt >= s.n_qt) {
            if (++b >= p.batch) return false;
            qt = 0;
            s = load_seq(p, b);
          }
          unit(p);
        }
      }
      const int take = min(left, nt + p.unit_cost - off);
      const int from = max(0, off - p.unit_cost), to = off + take - p.unit_cost;
      off += take;
      left -= take;
      here += take;
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
      g->final = !more(p);
      return true;
    }
    return false;
  }
};

// ----------------------------------------------------------------------------
// small device pieces
// ----------------------------------------------------------------------------
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// s 2^e, |e| <= 190; half of the power at a time, so that nothing overflows or vanishes on the way
// to a result that does not.
__device__ __forceinline__ float times_pow2(float s, int e) {
  return s * pow2(e / 2) * pow2(e - e / 2);
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

// Rows g (a, c) and g + 8 (b, d) of sixteen lanes, columns t and t + 4, g = lane / 4, t = lane % 4.
__device__ __forceinline__ void tmem_st_16x128b_x2(uint32_t taddr, uint32_t a, uint32_t b,
                                                   uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// Registers per thread of this warpgroup from here on.
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
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

// The bounded wait of these kernels: it gives up once kWaitLimitNs have passed by the clock, read
// after every four tries or nap.  A try by a whole warp sleeps up to 4 us (measured), so a wait that
// is over soon never reads it.  The loop is small and holds one register, because five roles
// share the instruction cache and the softmax has none to spare (with a counter of tries
// beside the clock it spilled 300 bytes at 128 columns); a call would rule out the register split.
template <bool kNap = false>
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, uint32_t* status) {
  static_assert(kWaitLimitNs < 1ull << 32, "the low word of the clock");
#define DFLASH_TRY "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra done;\n\t"
// (t0: the low word of the clock at the first reading, 0 before it)
#define DFLASH_LOOP(body)                                                              \
  asm volatile("{\n\t.reg .pred p, q;\n\t.reg .u32 t, t0;\n\tmov.u32 t0, 0;\n\tagain:\n\t" body \
               "mov.u32 t, %%globaltimer_lo;\n\tsetp.eq.u32 q, t0, 0;\n\t"            \
               "@q mov.u32 t0, t;\n\tsub.u32 t, t, t0;\n\tsetp.lt.u32 q, t, %3;\n\t"  \
               "@q bra again;\n\tdone:\n\tselp.u32 %0, 1, 0, p;\n\t}\n"             \
               : "=r"(ok)                                                              \
               : "r"(smem_u32(bar)), "r"(parity), "n"(kWaitLimitNs)                    \
               : "memory")
  uint32_t ok;
  __syncwarp();  // (a warp that is not together does not sleep in a try)
  if (kNap)      // where 100 ns late costs nothing
    DFLASH_LOOP(DFLASH_TRY "nanosleep.u32 60;\n\t");
  else
    DFLASH_LOOP(DFLASH_TRY DFLASH_TRY DFLASH_TRY DFLASH_TRY);
#undef DFLASH_TRY
#undef DFLASH_LOOP
  if (ok) return true;
  set_status(status, DFLASH_ST_TIMEOUT);
  return false;
}

// A wait of a warp; once one gave up the rest are skipped.  Warps that meet at named
// barriers vote there on who gave up, and leave their loops together.
struct Waiter {
  uint32_t* status;
  bool dead;
  template <bool kNap = false>
  __device__ __forceinline__ void on(uint64_t* bar, uint32_t parity) {
    if (!dead) dead = !wait_on<kNap>(bar, parity, status);
  }
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
    on(bar, parity);
  }
  __device__ __forceinline__ bool gave_up() {     // by the whole warp
    dead = __any_sync(0xffffffffu, dead);
    return dead;
  }
};

__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if (elect_one()) mbar_arrive(bar);
}

// set_smem_limit, the first time on each device (a bit of *ready; past 64 every time).  A
// kernel that takes registers from one role for another is refused unless it was compiled to
// start with at least `regs` a thread: it would wait for the rest for ever.
inline int smem_limit_once(std::atomic<uint64_t>* ready, const void* kernel, int bytes,
                           int regs = 0) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DFLASH_E_CUDA;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (ready->load(std::memory_order_acquire) & bit) return DFLASH_OK;
  cudaFuncAttributes at;
  if (cudaFuncGetAttributes(&at, kernel) != cudaSuccess) return DFLASH_E_CUDA;
  if (at.numRegs < regs) return DFLASH_E_UNSUPPORTED;
  const int rc = set_smem_limit(kernel, bytes);
  if (rc == DFLASH_OK) ready->fetch_or(bit, std::memory_order_release);
  return rc;
}

// The kernel for units of at most 8 * tiles query rows (kv4_rows.cu), tiles 1 or 2.
int launch_rows(const Kv4AttnParams& p, int head_dim, int tiles, int ctas, cudaStream_t st);

}  // namespace kv4
}  // namespace dflash
