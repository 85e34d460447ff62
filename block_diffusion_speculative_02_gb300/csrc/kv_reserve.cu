// Block tables and slot maps from lengths, on the device.
//
// "dflash-mlx" (dpshk.com) 保证三: the caches grow by the rows of a step and are
// cut back to the committed length; with paged caches that takes pages from the
// pool and gives them back (the crop).
//
// Small batches (at most 256 sequences and 8192 rows) take one CTA, a warp to a sequence:
// the pages that the new rows lack are counted, the counts added up, the pages taken and
// the maps written in one launch, whose time is launch and latency (32 sequences of 16 new
// rows 5.2 us in a graph, 15 us with a Python call each).  The rows of a sequence are its warp's
// alone: a single prompt of 8192 rows takes 41 us in a graph.
// Larger ones take two launches.  The first counts, one CTA per sequence, the pages the new rows
// lack; the second adds up the counts of the sequences before its own (that,
// not an atomic counter, decides which page of the free list a row gets, so
// the tables depend on the lengths alone), takes the pages, and writes the
// maps of its rows.  When the pool does not cover the whole batch the second
// walks the counts in order and serves what fits.
#include "kv4.cuh"

namespace dflash {
namespace {

constexpr int kThreads = 256;
constexpr int kInvalid = -1;   // need[b] of a sequence that cannot be served

struct ReserveParams {
  int batch, n_tokens, max_tokens, limit;
  int paged, page_size, max_pages, n_pages;
  const int32_t* seq_len;
  const int32_t* n_new;
  int32_t* page_table;
  const int32_t* free_list;
  int32_t* free_count;
  int32_t* start;
  int32_t* pos;
  int32_t* slot;
  int32_t* new_len;
  int32_t* need;        // [B], then the free count of before the call
  uint32_t* status;
};

// Sum over the CTA; every thread gets it.
__device__ __forceinline__ long long cta_sum(long long v, long long* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  long long t = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) t += red[i];
  return t;
}

// Rows of the batch before sequence b.
__device__ __forceinline__ long long rows_before(const ReserveParams& p, int b, long long* red) {
  long long v = 0;
  for (int j = threadIdx.x; j < b; j += kThreads) v += max(p.n_new[j], 0);
  return cta_sum(v, red);
}

__global__ void __launch_bounds__(kThreads) reserve_count_kernel(const ReserveParams p) {
  __shared__ long long red[kThreads / 32];
  griddep_wait();
  const int b = blockIdx.x;
  const long long first = rows_before(p, b, red);
  const int n = p.n_new[b], len = p.seq_len[b];
  const bool ok = n >= 0 && n <= p.max_tokens && len >= 0 && len <= p.limit &&
                  n <= p.limit - len && first + n <= p.n_tokens;
  int missing = 0;
  if (ok && n > 0 && p.paged) {
    const int32_t* row = p.page_table + static_cast<size_t>(b) * p.max_pages;
    const int last = (len + n - 1) / p.page_size;
    for (int pg = len / p.page_size + threadIdx.x; pg <= last; pg += kThreads)
      missing += row[pg] < 0;
  }
  const long long need = cta_sum(missing, red);
  if (threadIdx.x == 0) {
    p.need[b] = ok ? static_cast<int>(need) : kInvalid;
    if (b == 0 && p.paged) p.need[p.batch] = max(0, min(*p.free_count, p.n_pages));
    if (!ok) set_status(p.status, DFLASH_ST_CAPACITY);
  }
  griddep_launch_dependents();
}

__global__ void __launch_bounds__(kThreads) reserve_assign_kernel(const ReserveParams p) {
  __shared__ long long red[kThreads / 32];
  __shared__ int warp_cnt[kThreads / 32];
  __shared__ int s_base, s_total, s_served;
  griddep_wait();
  const int b = blockIdx.x, tid = threadIdx.x;
  const long long first = rows_before(p, b, red);
  const long long rows = rows_before(p, p.batch, red);
  const int need_b = p.need[b];
  const int n = need_b == kInvalid ? 0 : p.n_new[b], len = p.seq_len[b];
  const int avail = p.paged ? p.need[p.batch] : 0;
  // pages taken by the sequences before b, and by all
  long long v = 0, w = 0;
  for (int j = tid; j < p.batch; j += kThreads) {
    const int x = max(p.need[j], 0);
    w += x;
    if (j < b) v += x;
  }
  v = cta_sum(v, red);
  w = cta_sum(w, red);
  if (tid == 0) {
    s_base = static_cast<int>(v);
    s_total = static_cast<int>(w);
    s_served = need_b != kInvalid;
    if (w > avail) {
      int used = 0;
      for (int j = 0; j < p.batch; ++j) {
        const int x = max(p.need[j], 0);
        if (j == b) {
          s_base = used;
          if (x > avail - used) {
            s_served = 0;
            set_status(p.status, DFLASH_ST_POOL_EMPTY);
          }
        }
        if (x <= avail - used) used += x;
      }
      s_total = used;
    }
  }
  __syncthreads();
  const bool served = s_served != 0;
  if (served && n > 0 && p.paged) {
    int32_t* row = p.page_table + static_cast<size_t>(b) * p.max_pages;
    const int last = (len + n - 1) / p.page_size;
    int taken = s_base;
    for (int pg0 = len / p.page_size; pg0 <= last; pg0 += kThreads) {
      const int pg = pg0 + tid;
      const bool miss = pg <= last && row[pg] < 0;
      const uint32_t votes = __ballot_sync(0xffffffffu, miss);
      __syncthreads();
      if ((tid & 31) == 0) warp_cnt[tid >> 5] = __popc(votes);
      __syncthreads();
      int before = __popc(votes & ((1u << (tid & 31)) - 1u)), all = 0;
#pragma unroll
      for (int i = 0; i < kThreads / 32; ++i) {
        if (i < (tid >> 5)) before += warp_cnt[i];
        all += warp_cnt[i];
      }
      if (miss) row[pg] = p.free_list[avail - 1 - (taken + before)];
      taken += all;
    }
    __syncthreads();
  }
  // the maps of this sequence's rows (those that fit the arrays)
  const long long n_rows = max(p.n_new[b], 0);
  for (long long i = tid; i < n_rows && first + i < p.n_tokens; i += kThreads) {
    int pos = -1, slot = -1;
    if (served) {
      pos = len + static_cast<int>(i);
      slot = p.paged ? p.page_table[static_cast<size_t>(b) * p.max_pages + pos / p.page_size] *
                               p.page_size +
                           pos % p.page_size
                     : b * p.limit + pos;
    }
    p.pos[first + i] = pos;
    p.slot[first + i] = slot;
  }
  // rows behind the last sequence, shared out over the CTAs
  for (long long i = rows + static_cast<long long>(b) * kThreads + tid; i < p.n_tokens;
       i += static_cast<long long>(p.batch) * kThreads) {
    p.pos[i] = -1;
    p.slot[i] = -1;
  }
  if (tid == 0) {
    p.start[b] = static_cast<int>(min(first, static_cast<long long>(INT32_MAX)));
    p.new_len[b] = served ? len + n : len;
    if (b == p.batch - 1) {
      p.start[p.batch] = static_cast<int>(min(rows, static_cast<long long>(INT32_MAX)));
      if (p.paged) *p.free_count = avail - s_total;
    }
  }
  griddep_launch_dependents();
}

// ---- small batches: everything in one CTA ----
constexpr int kSmallThreads = 1024;
constexpr int kSmallBatch = 256;
constexpr int kSmallRows = 8192;

__global__ void __launch_bounds__(kSmallThreads) reserve_small_kernel(const ReserveParams p) {
  __shared__ int first[kSmallBatch + 1];   // rows before the sequence
  __shared__ int base[kSmallBatch];        // pages taken before it; -1: not served
  __shared__ int need[kSmallBatch];
  __shared__ int s_avail;
  griddep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 0) {                         // rows: an exclusive sum over the sequences
    long long at = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      const int b = b0 + lane;
      const long long n = b < p.batch ? max(p.n_new[b], 0) : 0;
      long long inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      if (b < p.batch)
        first[b] = static_cast<int>(min(at + inc - n, static_cast<long long>(INT32_MAX)));
      at += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) {
      first[p.batch] = static_cast<int>(min(at, static_cast<long long>(INT32_MAX)));
      s_avail = p.paged ? max(0, min(*p.free_count, p.n_pages)) : 0;
    }
  }
  __syncthreads();
  for (int b = warp; b < p.batch; b += kSmallThreads / 32) {
    const int n = p.n_new[b], len = p.seq_len[b];
    const bool ok = n >= 0 && n <= p.max_tokens && len >= 0 && len <= p.limit &&
                    n <= p.limit - len && first[b] <= p.n_tokens - n;
    int missing = 0;
    if (ok && n > 0 && p.paged) {
      const int32_t* row = p.page_table + static_cast<size_t>(b) * p.max_pages;
      const int last = (len + n - 1) / p.page_size;
      for (int pg = len / p.page_size + lane; pg <= last; pg += 32) missing += row[pg] < 0;
#pragma unroll
      for (int o = 16; o; o >>= 1) missing += __shfl_xor_sync(0xffffffffu, missing, o);
    }
    if (lane == 0) {
      need[b] = ok ? missing : kInvalid;
      if (!ok) set_status(p.status, DFLASH_ST_CAPACITY);
    }
  }
  __syncthreads();
  if (warp == 0) {                         // pages: in order, what fits
    const int avail = s_avail;
    int at = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      const int b = b0 + lane, x = b < p.batch ? max(need[b], 0) : 0;
      int inc = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      const int all = __shfl_sync(0xffffffffu, inc, 31);
      if (!p.paged || all <= avail - at) {
        if (b < p.batch) base[b] = need[b] == kInvalid ? -1 : at + inc - x;
        at += all;
      } else {                             // one by one
        for (int l = 0; l < 32 && b0 + l < p.batch; ++l) {
          const int y = __shfl_sync(0xffffffffu, x, l);
          const bool fits = y <= avail - at;
          if (lane == l) {
            base[b] = need[b] == kInvalid || !fits ? -1 : at;
            if (!fits) set_status(p.status, DFLASH_ST_POOL_EMPTY);
          }
          if (fits) at += y;
        }
      }
    }
    if (lane == 0 && p.paged) *p.free_count = avail - at;
  }
  __syncthreads();
  for (int b = warp; b < p.batch; b += kSmallThreads / 32) {
    const bool served = base[b] >= 0;
    const int n = max(p.n_new[b], 0), len = p.seq_len[b], row0 = first[b];
    int32_t* row = p.page_table + static_cast<size_t>(b) * p.max_pages;
    if (served && n > 0 && p.paged) {
      const int last = (len + n - 1) / p.page_size;
      int taken = base[b];
      for (int pg0 = len / p.page_size; pg0 <= last; pg0 += 32) {
        const int pg = pg0 + lane;
        const bool miss = pg <= last && row[pg] < 0;
        const uint32_t votes = __ballot_sync(0xffffffffu, miss);
        if (miss)
          row[pg] = p.free_list[s_avail - 1 - (taken + __popc(votes & ((1u << lane) - 1u)))];
        taken += __popc(votes);
      }
      __syncwarp();
    }
    for (int i = lane; i < min(n, p.n_tokens - row0); i += 32) {   // (row0 may be near 2^31)
      int pos = -1, slot = -1;
      if (served) {
        pos = len + i;
        slot = p.paged ? row[pos / p.page_size] * p.page_size + pos % p.page_size
                       : b * p.limit + pos;
      }
      p.pos[row0 + i] = pos;
      p.slot[row0 + i] = slot;
    }
    __syncwarp();                          // (new_len may be seq_len)
    if (lane == 0) {
      p.start[b] = row0;
      p.new_len[b] = served ? len + n : len;
    }
  }
  for (long long i = static_cast<long long>(first[p.batch]) + tid; i < p.n_tokens;
       i += kSmallThreads) {
    p.pos[i] = -1;                         // rows behind the last sequence
    p.slot[i] = -1;
  }
  if (tid == 0) p.start[p.batch] = first[p.batch];
  griddep_launch_dependents();
}

}  // namespace

int check_kv4_dims(const dflash_kv4_dims* d) {
  if (!d) return DFLASH_E_ARG;
  if (d->batch < 1 || d->n_tokens < 1 || d->max_tokens < 1 || d->n_kv_heads < 1)
    return DFLASH_E_ARG;
  if (d->batch > kMaxKv4Batch) return DFLASH_E_UNSUPPORTED;
  if (d->head_dim != 64 && d->head_dim != 128) return DFLASH_E_UNSUPPORTED;
  if (d->n_q_heads < d->n_kv_heads || d->n_q_heads % d->n_kv_heads ||
      d->n_q_heads / d->n_kv_heads > kMaxKv4Group || d->n_kv_heads > 65535)
    return DFLASH_E_UNSUPPORTED;
  return DFLASH_OK;
}

int make_kv4_plan(const dflash_kv4_dims& d, Kv4Plan* p) {
  const int rc = check_kv4_dims(&d);
  if (rc) return rc;
  const size_t att = kv4_attention_bytes(d);
  if (!att) return DFLASH_E_CUDA;
  p->off_status = 0;
  p->off_need = 256;
  p->off_att = 256 + (sizeof(int32_t) * (d.batch + 1) + 255) / 256 * 256;
  p->total = p->off_att + att;
  return DFLASH_OK;
}

}  // namespace dflash

using namespace dflash;

extern "C" size_t dflash_kv4_workspace_bytes(const dflash_kv4_dims* dims) {
  Kv4Plan p;
  if (check_kv4_dims(dims) || make_kv4_plan(*dims, &p)) return 0;
  return p.total;
}

extern "C" int dflash_kv_reserve(const dflash_kv4_dims* dims, const dflash_kv_view* cache,
                                 const int32_t* n_new, int32_t* start, int32_t* pos,
                                 int32_t* slot, int32_t* new_len, void* ws, size_t ws_bytes,
                                 dflash_stream_t stream) {
  DFLASH_ENTRY("dflash_kv_reserve");
  int rc = check_kv4_dims(dims);
  if (rc) return rc;
  if (!cache || !cache->seq_len || !n_new || !start || !pos || !slot || !new_len)
    return DFLASH_E_ARG;
  ReserveParams p = {};
  p.paged = cache->page_table != nullptr;
  long long limit = cache->capacity, rows;
  if (p.paged) {
    if (!cache->free_list || !cache->free_count || cache->page_size < 1 ||
        cache->max_pages < 1 || cache->n_pages < 1)
      return DFLASH_E_ARG;
    limit = static_cast<long long>(cache->max_pages) * cache->page_size;
    rows = static_cast<long long>(cache->n_pages) * cache->page_size;
  } else {
    if (cache->capacity < 1) return DFLASH_E_ARG;
    rows = limit * dims->batch;
  }
  if (limit > INT32_MAX || rows > INT32_MAX) return DFLASH_E_UNSUPPORTED;  // slots are int32
  Kv4Plan plan;
  if ((rc = make_kv4_plan(*dims, &plan))) return rc;
  if (!ws || ws_bytes < plan.off_att) return DFLASH_E_WORKSPACE;
  p.batch = dims->batch;
  p.n_tokens = dims->n_tokens;
  p.max_tokens = dims->max_tokens;
  p.limit = static_cast<int>(limit);
  p.page_size = cache->page_size;
  p.max_pages = cache->max_pages;
  p.n_pages = cache->n_pages;
  p.seq_len = cache->seq_len;
  p.n_new = n_new;
  p.page_table = cache->page_table;
  p.free_list = cache->free_list;
  p.free_count = cache->free_count;
  p.start = start;
  p.pos = pos;
  p.slot = slot;
  p.new_len = new_len;
  p.need = ws_at<int32_t>(ws, plan.off_need);
  p.status = ws_at<uint32_t>(ws, plan.off_status);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (p.batch <= kSmallBatch && p.n_tokens <= kSmallRows)
    return launch(reserve_small_kernel, dim3(1), dim3(kSmallThreads), 0, st, p);
  if ((rc = launch(reserve_count_kernel, dim3(p.batch), dim3(kThreads), 0, st, p))) return rc;
  return launch(reserve_assign_kernel, dim3(p.batch), dim3(kThreads), 0, st, p);
}
