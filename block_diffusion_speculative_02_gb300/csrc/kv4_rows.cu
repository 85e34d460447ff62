// Attention over a 4-bit cache for few query rows: single tokens, at most 16 rows to a unit
// (kv4_attention.cu has the sums, the units and the plan).
//
// With so few rows the tensor cores have little to do and the way through TMEM costs
// more than the products: every hand-over between roles is paid per tile, whatever the rows
// are.  Here a warp does all of it for a cell at a time, alone: its own copies into its
// own ring, K and V expanded in registers as the fragments of m16n8k16 products, its own
// maximum, sum and O; the warps of a CTA meet at the end of a segment only, where their
// results are joined in order.
//
// The products are turned round, S^T = K Q^T and O^T = V^T P^T, so that the expanded
// fragments serve every eight query rows (kTiles of them) and few rows cost little.
// Which dim is the products' k index and which key is a row of S^T is free as long as both
// factors agree, so each is chosen to make a thread's part of the cell a 32-bit word
// (g = lane / 4, t = lane % 4):
//   S^T   row g is key 4 (g / 2) + g % 2, row g + 8 the key two further; steps 2 p, 2 p + 1
//         take the dims 32 p + 8 t .. + 7, one word of codes of one key
//   O^T   k 2 t, 2 t + 1, 2 t + 8, 2 t + 9 are then the keys 4 t .. 4 t + 3, and P^T comes
//         from S^T by an 8 x 8 transpose; rows g and g + 8 of tile i are the dims 16 i + 2 g
//         and 16 i + 2 g + 1: one word holds both for four keys, under one scale for each key
//
// What bounds it: some 400 instructions a cell (about 100 to expand K, 120 for V, 40 for the
// softmax), 58% of the issue slots and 54% of the integer pipe in use.  Measured: one token
// of each of 32 sequences over 512 to 16,384 keys (32 + 8 heads of 128 dims) 84 us, 3.7 TB/s
// of cells (61 us at 64 dims); with 15 or 17 warps on cells 86 and 90 us, by the tensor kernel
// with units of 16 columns 108 us at best.  Four rows each (kTiles = 2) 118 us, 77 at 64 dims.
#include "kv4_attention.cuh"

namespace dflash {
namespace kv4 {
namespace {

template <int D, int kTiles>
struct RowsCfg {
  static constexpr int kWarps = kTiles == 1 ? 19 : 14;   // and one that plans
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kRows = 8 * kTiles;
  static constexpr int kStages = 3;    // cells of a warp's ring
  static constexpr int kCell = Cell<D>::kBytes;
  static constexpr int kRing = kWarps * kStages * kCell;
  static constexpr int kPitch = D + 4;                   // floats, of a row of `join`
  static constexpr int kJoin = kWarps * kRows * kPitch * 4;
  static constexpr int kSegs = 4;
  static constexpr int kQuery = kTiles * (D / 32) * 512; // fragments of the query rows
  static constexpr int kSmem = 128 + kRing + kQuery + kJoin + kWarps * kRows * 8 + kRows * 8 +
                               64 * kSegs + 8 * (kWarps * kStages + 2 * kSegs) + 64;
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct RowSeg {
  int b, h, row0, T, len, end, t0, cell0, cells, rows, whole, slot, final;
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t word(const uint8_t* p) {
  return *reinterpret_cast<const uint32_t*>(p);
}

template <int D, int kTiles>
__global__ void __launch_bounds__(RowsCfg<D, kTiles>::kThreads, 1)
    kv4_rows_kernel(const Kv4AttnParams p) {
  using C = RowsCfg<D, kTiles>;
  constexpr int kP = D / 32, kI = D / 16;          // pieces of K, tiles of O^T
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((128 - (smem_u32(smem_raw) & 127)) & 127);
  uint4* qf = reinterpret_cast<uint4*>(smem + C::kRing);   // [tile][piece][lane]
  float* join = reinterpret_cast<float*>(smem + C::kRing + C::kQuery);  // [warp][row][kPitch]
  float2* wml = reinterpret_cast<float2*>(join + C::kWarps * C::kRows * C::kPitch);
                                                           // [warp][row] maximum, sum
  float* row_sc = reinterpret_cast<float*>(wml + C::kWarps * C::kRows);  // [row]
  RowSeg* segs = reinterpret_cast<RowSeg*>(row_sc + 2 * C::kRows);
  uint64_t* full = reinterpret_cast<uint64_t*>(segs + C::kSegs);       // [warp][stage]
  uint64_t* seg_full = full + C::kWarps * C::kStages;
  uint64_t* seg_empty = seg_full + C::kSegs;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < C::kWarps * C::kStages; i += C::kThreads) mbar_init(&full[i], 1);
  if (threadIdx.x < C::kSegs) {
    mbar_init(&seg_full[threadIdx.x], 1);
    mbar_init(&seg_empty[threadIdx.x], C::kWarps);
  }
  fence_mbar_init();
  __syncthreads();
  griddep_wait();
  Waiter wait{p.status, false};
  const int G = p.group;

  if (warp == C::kWarps) {
    // ---------------- the segments of this CTA ----------------
    Walk walk(p);
    Seg g = {};
    bool more = walk.next(p, &g);
    const bool any = more;
    if (lane == 0) *reinterpret_cast<int4*>(p.meta + 4 * blockIdx.x) = make_int4(-1, 0, 0, 0);
#pragma unroll 1
    for (int s = 0; more || s == 0; ++s) {
      if (s >= C::kSegs) wait.on<true>(&seg_empty[s % C::kSegs], ((s / C::kSegs) & 1) ^ 1);
      if (wait.gave_up()) break;
      RowSeg r = {};
      r.final = 1;
      if (any) {
        const int rows = min(p.tile_rows, g.T - g.t0) * G;
        const int cells = (g.end + kCellRows - 1) / kCellRows;     // of the unit
        if (g.tile == 0 && g.n < g.nt && lane == 0)   // the rest of this unit is others'
          *reinterpret_cast<int4*>(p.meta + 4 * blockIdx.x) = make_int4(
              walk.owner(walk.here + g.nt - g.n - 1), g.lo + g.t0, rows, g.h);
        r.b = g.b;
        r.h = g.h;
        r.row0 = (g.lo + g.t0) * p.n_q_heads + g.h * G;
        r.T = g.T;
        r.len = g.len;
        r.end = g.end;
        r.t0 = g.t0;
        r.cell0 = g.tile * kGran;
        r.cells = max(0, min(g.n * kGran, cells - r.cell0));
        r.rows = rows;
        r.whole = g.tile == 0 && g.n == g.nt;
        r.slot = 2 * static_cast<int>(blockIdx.x) + (g.tile == 0 ? 1 : 0);
        r.final = g.final;
        more = walk.next(p, &g);
      } else {
        r.b = -1;
      }
      if (lane == 0) segs[s % C::kSegs] = r;
      warp_arrive(&seg_full[s % C::kSegs]);
    }
    griddep_launch_dependents();
    return;
  }

  const int gl = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kCell;
  uint64_t* mine = full + warp * C::kStages;
  const uint64_t pol =
      p.max_tokens > p.tile_rows ? l2_policy_evict_normal() : l2_policy_evict_first();
  const int per_slab = p.s.slab_rows / kCellRows;
  // the cell that is copied next: segment ls (at hand or the one after), its cell lc
  int ls = 0, lc = warp, issued = 0;
  bool known = false;                  // segment ls is out (and read below)
  int l_b = 0, l_h = 0, l_cell0 = 0, l_cells = 0, l_final = 0;
  // copies ahead of cell number `done` of this warp, as far as the ring and the segments go
  auto issue = [&](int done, int seg) {
#pragma unroll 1
    while (issued < done + C::kStages) {
      if (!known) {
        if (ls > seg + 1 ||
            !__all_sync(0xffffffffu, mbar_try_wait(&seg_full[ls % C::kSegs], (ls / C::kSegs) & 1)))
          return;
        const RowSeg& r = segs[ls % C::kSegs];
        l_b = r.b;
        l_h = r.h;
        l_cell0 = r.cell0;
        l_cells = r.cells;
        l_final = r.final;
        known = true;
      }
      if (lc >= l_cells) {
        if (l_final) return;
        ++ls;
        lc = warp;
        known = false;
        continue;
      }
      const int key16 = l_cell0 + lc;
      int slab = l_b, row16 = key16;
      if (p.paged) {
        const int page = per_slab == 1 ? key16 : key16 / per_slab;
        row16 = key16 - page * per_slab;
        slab = p.page_table[static_cast<size_t>(l_b) * p.max_pages + page];
      }
      const int st = issued % C::kStages;
      const uint32_t dst = ring + st * C::kCell;
      if (slab < 0 || slab >= p.s.n_slabs) {        // a page that is missing reads as zeros
        if (lane == 0) set_status(p.status, DFLASH_ST_PAGE_MISSING);
        for (int o = lane * 16; o < C::kCell; o += 512)
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + o), "r"(0)
                       : "memory");
        fence_proxy_async_smem();                   // (before the copy that comes here next)
        warp_arrive(&mine[st]);
      } else if (lane == 0) {
        mbar_arrive_expect_tx(&mine[st], C::kCell);
        const size_t cell = (slab * p.s.n_kv_heads + l_h) * per_slab + row16;
        bulk_load(smem + (dst - smem_u32(smem)), p.s.cells + cell * C::kCell, C::kCell, &mine[st],
                  pol);
      }
      ++issued;
      lc += C::kWarps;
    }
  };

  int done = 0;
  bool go = true;
#pragma unroll 1
  for (int seg = 0; go; ++seg) {
    wait(&seg_full[seg % C::kSegs], (seg / C::kSegs) & 1);
    if (bar_or(1, 32 * C::kWarps, wait.dead)) break;
    issue(done, seg);
    const RowSeg r = segs[seg % C::kSegs];
    go = !r.final;
    if (r.b < 0) break;
    // ---- query rows as fragments, each scaled to [1, 2) by a power of two ----
    if (warp < kTiles) {
      const int row = gl + 8 * warp, tq = row * p.group_inv >> 16;
      uint4 v[kP];
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kP; ++i) {
        v[i] = make_uint4(0, 0, 0, 0);
        if (row < r.rows)
          v[i] = *reinterpret_cast<const uint4*>(
              p.q + static_cast<size_t>(r.row0 + tq * p.n_q_heads + row - tq * G) * D + 32 * i +
              8 * t);
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t a = w[e] & 0x7FFFu, b = w[e] >> 16 & 0x7FFFu;
          m = max(m, max(a < 0x7F80u ? a : 0u, b < 0x7F80u ? b : 0u));
        }
      }
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int ex = max(-126, min(126, 127 - static_cast<int>(m >> 7)));
      const float f = pow2(ex);
#pragma unroll
      for (int i = 0; i < kP; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          y[e] = pack_f16(__uint_as_float(w[e] << 16) * f, __uint_as_float(w[e] & 0xFFFF0000u) * f);
        qf[(warp * kP + i) * 32 + lane] = make_uint4(y[0], y[1], y[2], y[3]);
      }
      if (t == 0) {
        // (never 0, so that a masked score stays minus infinity: 2^-149 leaves every finite
        // score below 2^-100)
        const float y = times_pow2(p.scale_log2, gain_exp(p.s.k_exp, r.h) - ex);
        row_sc[row] = y == 0.f ? __int_as_float(1) : y;
      }
    }
    named_bar_sync(1, 32 * C::kWarps);
    float sc[kTiles][2];               // of rows 8 x + 2 t, 8 x + 2 t + 1, as all below
    int vis[kTiles][2];
#pragma unroll
    for (int x = 0; x < kTiles; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int mr = 8 * x + 2 * t + e;
        sc[x][e] = row_sc[mr];
        vis[x][e] = p.causal && mr < r.rows
                        ? max(0, min(r.len, r.len - r.T + r.t0 + (mr * p.group_inv >> 16) + 1))
                        : r.len;
      }
    const int sure = p.causal ? max(0, r.len - r.T + r.t0 + 1) : r.len;
    float o[kI][kTiles][4], l[kTiles][2], nm[kTiles][2];   // nm: kLift - running maximum
#pragma unroll
    for (int x = 0; x < kTiles; ++x) {
#pragma unroll
      for (int i = 0; i < kI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][x][e] = 0.f;
      l[x][0] = l[x][1] = 0.f;
      nm[x][0] = nm[x][1] = kLift - kNoMax;
    }
    const int kr = 4 * (gl >> 1) + (gl & 1);                // S^T rows g, g + 8: keys kr, kr + 2
    // this warp's slice of `join`, free until the segment ends: [group][key], [group][key / 2]
    uint32_t* k_sc = reinterpret_cast<uint32_t*>(join + warp * C::kRows * C::kPitch);
    uint32_t* v_sc = k_sc + D;
#pragma unroll 1
    for (int c = warp; c < r.cells; c += C::kWarps, ++done) {
      const int st = done % C::kStages;
      wait(&mine[st], (done / C::kStages) & 1);
      if (wait.gave_up()) break;
      const uint8_t* cell = smem + (warp * C::kStages + st) * C::kCell;
      const int key0 = (r.cell0 + c) * kCellRows;
      // ---- scores of 16 keys: element e is key kr + 2 (e >> 1), row 2 t + (e & 1) ----
      float s[kTiles][4], s_odd[kTiles][4];                 // (two chains of products)
#pragma unroll
      for (int x = 0; x < kTiles; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[x][e] = s_odd[x][e] = 0.f;
      // every scale to fp16 once, by all lanes, for the eight that share it: those of K
      // doubled, those of V in pairs of keys (0 past the length; codes are finite
      // whatever they hold)
      const int left = r.end - key0;
#pragma unroll
      for (int i = 0; i < D / 128 + (D < 128); ++i) {
        const int w = i * 32 + lane;                        // four scales each
        if (w < D / 4) {
          const uint32_t ks = word(cell + Cell<D>::kKScale + 4 * w);
          const uint32_t a = e4m3x2_to_f16x2(ks), b = e4m3x2_to_f16x2(ks >> 16);
          constexpr int kW = D / 64;                        // words of a key
          uint32_t* to = k_sc + w % kW * 64 + w / kW;
          to[0] = __byte_perm(a, 0, 0x1010);
          to[16] = __byte_perm(a, 0, 0x3232);
          to[32] = __byte_perm(b, 0, 0x1010);
          to[48] = __byte_perm(b, 0, 0x3232);
          const int in = left - 4 * (w & 3);                // of these four keys
          const uint32_t vs = word(cell + Cell<D>::kVScale + 4 * w) &
                              (in >= 4 ? ~0u : in > 0 ? (1u << 8 * in) - 1u : 0u);
          *reinterpret_cast<uint2*>(v_sc + 2 * w) =
              make_uint2(e4m3x2_to_f16x2(vs), e4m3x2_to_f16x2(vs >> 16));
        }
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kP; ++i) {
        uint32_t a[2][4];                                   // step; a0 .. a3
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t w = word(cell + i * 256 + (kr + 2 * u) * 16 + 4 * t);
          const uint32_t up = w >> 8;
          const uint32_t f = k_sc[(2 * i + (t >> 1)) * 16 + kr + 2 * u];
          a[0][u] = hmul2(e2m1x2_to_f16x2<0>(w), f);
          a[0][2 + u] = hmul2(e2m1x2_to_f16x2<0>(up), f);
          a[1][u] = hmul2(e2m1x2_to_f16x2<2>(w), f);
          a[1][2 + u] = hmul2(e2m1x2_to_f16x2<2>(up), f);
        }
#pragma unroll
        for (int x = 0; x < kTiles; ++x) {
          const uint4 q = qf[(x * kP + i) * 32 + lane];
          mma16816(s[x], a[0][0], a[0][1], a[0][2], a[0][3], q.x, q.y);
          mma16816(s_odd[x], a[1][0], a[1][1], a[1][2], a[1][3], q.z, q.w);
        }
      }
#pragma unroll
      for (int x = 0; x < kTiles; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[x][e] += s_odd[x][e];
      // ---- probabilities ----
      if (key0 + kCellRows > sure) {   // (a masked score is minus infinity whatever its scale)
#pragma unroll
        for (int x = 0; x < kTiles; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (key0 + kr + (e & 2) >= vis[x][e & 1])
              s[x][e] = sc[x][e & 1] < 0.f ? INFINITY : -INFINITY;
      }
      float pr[kTiles][4];
      float mx = -INFINITY;
#pragma unroll
      for (int x = 0; x < kTiles; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          pr[x][e] = fmaf(s[x][e], sc[x][e & 1], nm[x][e & 1]);
          mx = fmaxf(mx, pr[x][e]);
        }
      if (__any_sync(0xffffffffu, mx > kMoveLog2 + kLift)) {
#pragma unroll
        for (int x = 0; x < kTiles; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float y = fmaxf(s[x][e] * sc[x][e], s[x][e + 2] * sc[x][e]);
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, w));
            const float was = kLift - nm[x][e], now = fmaxf(was, y);
            const float f = ex2(was - now);
            nm[x][e] = kLift - now;
            l[x][e] *= f;
#pragma unroll
            for (int i = 0; i < kI; ++i) {
              o[i][x][e] *= f;
              o[i][x][e + 2] *= f;
            }
            pr[x][e] = fmaf(s[x][e], sc[x][e], nm[x][e]);
            pr[x][e + 2] = fmaf(s[x][e + 2], sc[x][e], nm[x][e]);
          }
      }
      uint32_t b[kTiles][2];
#pragma unroll
      for (int x = 0; x < kTiles; ++x)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float p0 = ex2(pr[x][2 * u]), p1 = ex2(pr[x][2 * u + 1]);
          l[x][0] += p0;
          l[x][1] += p1;
          asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;"
                       : "=r"(b[x][u])
                       : "r"(pack_f16(p0, p1)));
        }
      // ---- O^T += V^T P^T ----
#pragma unroll
      for (int i = 0; i < kI; ++i) {
        const uint32_t w = word(cell + Cell<D>::kV + (8 * i + gl) * 16 + 4 * t);
        const uint2 f = *reinterpret_cast<const uint2*>(v_sc + 8 * i + 2 * t);
        const uint32_t f0 = f.x, f1 = f.y;
        // low (even dim) and high nibbles of two keys to a byte, bytes 0 and 2
        const uint32_t w4 = w >> 4, w8 = w >> 8;
        const uint32_t lo = (w & 0x000F000Fu) | (w4 & ~0x000F000Fu);
        const uint32_t hi = (w4 & 0x000F000Fu) | (w8 & ~0x000F000Fu);
        const uint32_t a[4] = {hmul2(e2m1x2_to_f16x2<0>(lo), f0),
                               hmul2(e2m1x2_to_f16x2<0>(hi), f0),
                               hmul2(e2m1x2_to_f16x2<2>(lo), f1),
                               hmul2(e2m1x2_to_f16x2<2>(hi), f1)};
#pragma unroll
        for (int x = 0; x < kTiles; ++x)
          mma16816(o[i][x], a[0], a[1], a[2], a[3], b[x][0], b[x][1]);
      }
      __syncwarp();
      issue(done + 1, seg);
    }
    // ---- the warps' results, joined in order ----
#pragma unroll
    for (int x = 0; x < kTiles; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * x + 2 * t + e;
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[x][e] += __shfl_xor_sync(0xffffffffu, l[x][e], w);
        if (gl == 0) wml[warp * C::kRows + row] = make_float2(-nm[x][e], l[x][e]);
        float* dst = join + (warp * C::kRows + row) * C::kPitch + 2 * gl;
#pragma unroll
        for (int i = 0; i < kI; ++i)
          *reinterpret_cast<float2*>(dst + 16 * i) = make_float2(o[i][x][e], o[i][x][e + 2]);
      }
    if (bar_or(1, 32 * C::kWarps, wait.gave_up())) break;
    if (!go) griddep_launch_dependents();
    const int n_el = min(r.rows, C::kRows) * (D / 4);
#pragma unroll 1
    for (int i = threadIdx.x; i < n_el; i += 32 * C::kWarps) {
      const int row = i / (D / 4), d = i % (D / 4) * 4;
      float M = 2.f * kNoMax, L = 0.f;
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) M = fmaxf(M, wml[w * C::kRows + row].x);
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < C::kWarps; ++w) {
        const float2 ml = wml[w * C::kRows + row];
        const float f = ex2(ml.x - M);
        const float4 v =
            *reinterpret_cast<const float4*>(join + (w * C::kRows + row) * C::kPitch + d);
        L += f * ml.y;
        y.x += f * v.x;
        y.y += f * v.y;
        y.z += f * v.z;
        y.w += f * v.w;
      }
      if (r.whole) {
        const float f = L == 0.f ? 0.f : pow2(gain_exp(p.s.v_exp, r.h)) / L;
        const int tq = row * p.group_inv >> 16;
        uint2 u = make_uint2(0, 0);
        if (L != 0.f) {
          u.x = static_cast<uint32_t>(float_to_bf16_bits(y.x * f)) |
                static_cast<uint32_t>(float_to_bf16_bits(y.y * f)) << 16;
          u.y = static_cast<uint32_t>(float_to_bf16_bits(y.z * f)) |
                static_cast<uint32_t>(float_to_bf16_bits(y.w * f)) << 16;
        }
        *reinterpret_cast<uint2*>(
            p.out + static_cast<size_t>(r.row0 + tq * p.n_q_heads + row - tq * G) * D + d) = u;
      } else {
        *reinterpret_cast<float4*>(p.part_o + (static_cast<size_t>(r.slot) * 16 + row) * D + d) = y;
        if (d == 0) {
          float* ml = p.part_ml + (static_cast<size_t>(r.slot) * 16 + row) * 2;
          ml[0] = M;
          ml[1] = L;
        }
      }
    }
    warp_arrive(&seg_empty[seg % C::kSegs]);
    named_bar_sync(1, 32 * C::kWarps);              // join and wml are read
  }
  // no copy may still be landing when the CTA exits
#pragma unroll 1
  for (int k = done; k < issued; ++k)
    mbar_wait_drain(&mine[k % C::kStages], (k / C::kStages) & 1, p.status);
}

template <int D, int kTiles>
int run_rows(const Kv4AttnParams& p, int ctas, cudaStream_t st) {
  using C = RowsCfg<D, kTiles>;
  static std::atomic<uint64_t> ready{0};
  int rc = smem_limit_once(&ready, reinterpret_cast<const void*>(kv4_rows_kernel<D, kTiles>),
                           C::kSmem);
  if (rc) return rc;
  return launch(kv4_rows_kernel<D, kTiles>, dim3(ctas), dim3(C::kThreads), C::kSmem, st, p);
}

}  // namespace

int launch_rows(const Kv4AttnParams& p, int head_dim, int tiles, int ctas, cudaStream_t st) {
  if (tiles == 1)
    return head_dim == 128 ? run_rows<128, 1>(p, ctas, st) : run_rows<64, 1>(p, ctas, st);
  return head_dim == 128 ? run_rows<128, 2>(p, ctas, st) : run_rows<64, 2>(p, ctas, st);
}

}  // namespace kv4
}  // namespace dflash
