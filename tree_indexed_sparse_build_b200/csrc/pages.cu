// Paged KV cache: pages given out, forked, copied, freed, compacted and gathered on the device.
//
// K and V live in the caller's pools [num_pages, kv_heads, page, head_dim]; a sequence is a row
// of page ids and a length.  All bookkeeping stays in device memory, so every call is
// asynchronous and can be captured into a graph and replayed with lengths that move on.
//
// Results do not depend on timing: new pages are the lowest free ones (a bitmap with one bit
// per page, searched by one CTA with a prefix sum over popcounts), handed out in the order of
// the call's list; counts change by integer atomics whose order cannot be seen.
//
// A page that is only partly filled always belongs to one sequence (a fork copies it), so
// appending never has to look whether somebody else reads the page.
//
// Calls that hand out pages have two steps: a plan (one CTA checks the list, finds the
// pages, and either commits all of the call's bookkeeping or none of it) and the rows.  In a small call
// that CTA goes on with the rows; a large one is two launches, the second of which starts while the
// first drains (programmatic launch).
#include <cstdint>
#include <cstdlib>

#include "device_common.cuh"
#include "pages.h"

using namespace zha;

namespace {

enum PlanMode { kAppend = 0, kFork = 1, kCopy = 2 };

constexpr int kPlanThreads = 1024;
constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kGroups = kPlanThreads / kRowThreads;  // groups of kRowThreads threads in the plan's CTA
// Bytes that a small call moves at most.  A CTA moves 64 KB in about the 1.5 us of GPU time, and 2.5 us of the host's,
// that a second launch costs (a cluster of eight CTAs as one launch took as long as the two launches).
constexpr long long kSmallBytes = 64 * 1024;

// Table entries that a free goes through entry by entry at most (one launch); above, by columns (two).
constexpr long long kFewPages = 32 * 1024;

// A group of kRowThreads threads: the x-th of nx that share some work.
struct Group {
  int x, nx, tid;
  __device__ __forceinline__ int thread() const { return x * kRowThreads + tid; }
  __device__ __forceinline__ int threads() const { return nx * kRowThreads; }
  __device__ __forceinline__ int warp() const { return x * kRowWarps + (tid >> 5); }
  __device__ __forceinline__ int warps() const { return nx * kRowWarps; }
  __device__ static Group of_grid() { return {(int)blockIdx.x, (int)gridDim.x, (int)threadIdx.x}; }
  // In a small call: this thread's group among the CTA's.
  __device__ static Group of_cta() {
    return {(int)(threadIdx.x / kRowThreads), kGroups, (int)(threadIdx.x % kRowThreads)};
  }
};

__device__ __forceinline__ int ceil_shift(int x, int shift) { return (int)(((unsigned)x + (1u << shift) - 1u) >> shift); }

// Exclusive prefix sum of x over the CTA's 1,024 threads; *total is the sum.  sums: 32 of them.
template <typename T>
__device__ __forceinline__ T cta_scan(T x, T* sums, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();  // the last scan's readers of `sums` are done
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    T s = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    sums[lane] = s;
  }
  __syncthreads();
  *total = sums[31];
  return v - x + (warp ? sums[warp - 1] : T(0));
}

// ---------------------------------------------------------------- plan

// Checks list entry i and says how many pages it needs.  Returns error bits.
__device__ unsigned plan_entry(const PagesView& d, const PagesView& s, const int* src, const int* dst,
                               const int* counts, int T, int mode, int i, int* slot, int* len, int* cnt, int* need) {
  *slot = dst[i];
  *len = *cnt = *need = 0;
  if ((unsigned)*slot >= (unsigned)d.max_seqs) {
    *slot = -1;
    return kDevErrBadSeq;
  }
  if (mode == kAppend) {
    *len = d.lens[*slot];
    *cnt = counts ? counts[i] : T;
    if (*cnt < 0 || *cnt > T) {
      *cnt = 0;
      return kDevErrBadSeq;
    }
    if ((long long)*len + *cnt > (long long)d.width << d.shift) return kDevErrPool;
    *need = ceil_shift(*len + *cnt, d.shift) - ceil_shift(*len, d.shift);
    return 0;
  }
  const int from = src[i];
  if ((unsigned)from >= (unsigned)s.max_seqs) return kDevErrBadSeq;
  if (d.lens[*slot] != 0) return kDevErrBadSeq;  // the destination must be empty
  *len = s.lens[from];
  if ((long long)*len > (long long)d.width << d.shift) return kDevErrPool;
  *need = mode == kCopy ? ceil_shift(*len, d.shift) : ((*len & (d.page - 1)) != 0);
  return 0;
}

// The plan of a call, by one CTA of kPlanThreads threads.  Bound: latency of a few dependent loads and two
// scans for any list of up to 1,024 entries (one round); pages are found 32,768 at a time.
__device__ void plan_body(const PagesView& d, const PagesView& s, const int* src, const int* dst, const int* counts, int n,
                          int T, int mode) {
  __shared__ int sums[32];
  __shared__ long long wide_sums[32];
  __shared__ unsigned bad;
  const int tid = threadIdx.x;
  if (tid == 0) bad = 0;
  // (used below; loaded with the lists)
  const int free_pages = *d.free_pages;
  unsigned word = tid < d.words ? d.used[tid] : ~0u;
  __syncthreads();
  long long total = 0;  // 64 bits: a list may ask for more pages than 31 bits count
  int slot = -1, len = 0, cnt = 0;  // of the last round's entry
  // what each entry needs, and which entry names a slot first
  for (int at = 0; at < n; at += kPlanThreads) {
    const int i = at + tid;
    int need = 0;
    slot = -1;
    if (i < n) {
      const unsigned e = plan_entry(d, s, src, dst, counts, T, mode, i, &slot, &len, &cnt, &need);
      if (e) atomicOr(&bad, e);
      if (slot >= 0) atomicMin(&d.claim[slot], i);
      if (mode == kFork && (unsigned)src[i] < (unsigned)s.max_seqs) {
        atomicAdd(&d.mult[src[i]], 1);
        atomicMin(&d.lead[src[i]], i);
      }
    }
    long long sum;
    const long long base = cta_scan<long long>(need, wide_sums, &sum);
    if (i < n) {
      d.plan_len[i] = len;
      d.plan_cnt[i] = cnt;
      d.plan_base[i] = (int)(total + base);  // (past 31 bits only in a call that is refused)
    }
    total += sum;
  }
  __syncthreads();
  const bool one_round = n <= kPlanThreads;
  for (int i = tid; i < n; i += kPlanThreads) {
    const int x = one_round ? slot : dst[i];
    if ((unsigned)x < (unsigned)d.max_seqs && __ldcg(&d.claim[x]) != i) atomicOr(&bad, kDevErrBadSeq);
  }
  if (tid == 0 && total > free_pages) atomicOr(&bad, kDevErrPool);
  if (mode == kFork)
    for (int i = tid; i < n; i += kPlanThreads) {
      const int from = src[i];
      const bool first = (unsigned)from < (unsigned)s.max_seqs && __ldcg(&d.lead[from]) == i;
      d.plan_mult[i] = first ? __ldcg(&d.mult[from]) : 0;
    }
  __syncthreads();
  if (mode == kFork)
    for (int i = tid; i < n; i += kPlanThreads) {
      const int from = src[i];
      if ((unsigned)from >= (unsigned)s.max_seqs) continue;
      d.mult[from] = 0;
      d.lead[from] = kNoClaim;
    }
  const unsigned error = bad;
  for (int i = tid; i < n; i += kPlanThreads) {
    const int x = one_round ? slot : dst[i];
    if ((unsigned)x >= (unsigned)d.max_seqs) continue;
    d.claim[x] = kNoClaim;
    if (!error) d.lens[x] = one_round ? len + cnt : d.plan_len[i] + d.plan_cnt[i];
  }
  if (tid == 0) {
    if (error) atomicOr(d.err, error);
    *d.ok = !error;
    if (!error && total) *d.free_pages = free_pages - (int)total;
  }
  if (error) return;
  // the lowest free pages
  int given = 0;
  for (int at = 0; given < total && at < d.words; at += kPlanThreads) {
    const int w = at + tid;
    const unsigned next = w + kPlanThreads < d.words ? d.used[w + kPlanThreads] : ~0u;
    unsigned open = ~word;
    int sum;
    int rank = given + cta_scan(__popc(open), sums, &sum);
    unsigned mark = 0;
    while (open && rank < total) {
      const int bit = __ffs(open) - 1;
      const int page = w * 32 + bit;
      open &= open - 1;
      mark |= 1u << bit;
      d.fresh[rank++] = page;
      d.refs[page] = 1;
    }
    if (mark) d.used[w] = word | mark;
    given += sum;
    word = next;
  }
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PagesView d, PagesView s, const int* src, const int* dst,
                                                            const int* counts, int n, int T, int mode) {
  pdl_wait();
  pdl_release();
  plan_body(d, s, src, dst, counts, n, T, mode);
}

// ---------------------------------------------------------------- rows

// The row kernels move bytes and are bound by them where there are many: each vector is read and written once, eight
// loads in flight per thread.  At 8 KV heads of 128 in bf16, bytes read and written: 36,000 ragged tokens appended in
// 54 us (5.5 TB/s; the plan before takes 5 us) and gathered in 51 us (5.8), 125,000 tokens copied in 168 us (6.1) and compacted
// in 165 us (6.2).

// One warp copies n 16-byte vectors of K and of V; eight loads in flight per lane.
__device__ __forceinline__ void warp_copy(const uint4* ks, const uint4* vs, uint4* kd, uint4* vd, int n, int lane) {
  constexpr int U = 4;
  int i = lane;
  for (; i + (U - 1) * 32 < n; i += U * 32) {
    uint4 a[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) a[u] = __ldcg(ks + i + u * 32);
#pragma unroll
    for (int u = 0; u < U; ++u) b[u] = __ldcg(vs + i + u * 32);
#pragma unroll
    for (int u = 0; u < U; ++u) kd[i + u * 32] = a[u];
#pragma unroll
    for (int u = 0; u < U; ++u) vd[i + u * 32] = b[u];
  }
  for (; i < n; i += 32) {
    const uint4 a = __ldcg(ks + i), b = __ldcg(vs + i);
    kd[i] = a;
    vd[i] = b;
  }
}

// First vector of row 0 of (page, head).
__device__ __forceinline__ size_t page_vec(const PagesView& v, int page, int head) {
  return ((size_t)page * v.heads + head) * ((size_t)v.page * v.row_vecs);
}

// Rows of entry i's new tokens go to their pages; the entry's new pages enter its table row.  A lane group of
// row_vecs lanes moves one row of K and of V.
__device__ __forceinline__ void append_rows(const PagesView& d, int i, const Group& g, const int* dst, int T, const uint4* Kn,
                                            const uint4* Vn, uint4* K, uint4* V) {
  const int slot = dst[i], len = d.plan_len[i], cnt = d.plan_cnt[i], base = d.plan_base[i];
  const int old = ceil_shift(len, d.shift), more = ceil_shift(len + cnt, d.shift) - old;
  int* row = d.table + (size_t)slot * d.width;
  for (int j = g.thread(); j < more; j += g.threads()) row[old + j] = d.fresh[base + j];
  const int vecs = d.row_vecs, at_once = kRowThreads / vecs;  // rows per pass of the group
  const int col = g.tid % vecs, lane_row = g.tid / vecs;
  const unsigned rows = (unsigned)d.heads * (unsigned)cnt;
  constexpr int U = 4;
  for (unsigned r0 = g.x * (at_once * U); r0 < rows; r0 += g.nx * (at_once * U)) {
    uint4 a[U], b[U];
    size_t to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const unsigned r = r0 + u * at_once + lane_row;
      to[u] = ~(size_t)0;
      if (r < rows) {
        const unsigned h = r / (unsigned)cnt, t = r - h * cnt;
        const int p = len + (int)t, c = p >> d.shift;
        const int page = c < old ? row[c] : d.fresh[base + c - old];
        const size_t from = (((size_t)i * d.heads + h) * T + t) * vecs + col;
        a[u] = __ldg(Kn + from);
        b[u] = __ldg(Vn + from);
        if ((unsigned)page < (unsigned)d.num_pages)
          to[u] = page_vec(d, page, h) + (size_t)(p & (d.page - 1)) * vecs + col;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (to[u] != ~(size_t)0) {
        K[to[u]] = a[u];
        V[to[u]] = b[u];
      }
  }
}

// Entry i shares the source's full pages; a partial last page gets the entry's new page and its rows copied.
// A page's count grows once for all the entries of its source.
__device__ __forceinline__ void fork_rows(const PagesView& d, int i, const Group& g, const int* src, const int* dst, uint4* K,
                                          uint4* V) {
  const int len = d.plan_len[i], full = len >> d.shift, rest = len & (d.page - 1), forks = d.plan_mult[i];
  const int* from = d.table + (size_t)src[i] * d.width;
  int* row = d.table + (size_t)dst[i] * d.width;
  for (int j = g.thread(); j < full; j += g.threads()) {
    const int page = from[j];
    row[j] = page;
    if (forks && (unsigned)page < (unsigned)d.num_pages) atomicAdd(&d.refs[page], forks);
  }
  if (rest) {
    const int a = from[full], b = d.fresh[d.plan_base[i]];
    if (g.thread() == 0) row[full] = b;
    if ((unsigned)a >= (unsigned)d.num_pages) return;
    for (int h = g.warp(); h < d.heads; h += g.warps()) {
      const size_t x = page_vec(d, a, h), y = page_vec(d, b, h);
      warp_copy(K + x, V + x, K + y, V + y, rest * d.row_vecs, g.tid & 31);
    }
  }
}

// Every page of entry i's source is copied into a new one (rows past the length are left alone); a warp takes
// one (page, head) at a time.
__device__ __forceinline__ void copy_rows(const PagesView& d, const PagesView& s, int i, const Group& g, const int* src,
                                          const int* dst, const uint4* Ks, const uint4* Vs, uint4* K, uint4* V) {
  const int len = d.plan_len[i], pages = ceil_shift(len, d.shift);
  const int* from = s.table + (size_t)src[i] * s.width;
  const int* fresh = d.fresh + d.plan_base[i];
  int* row = d.table + (size_t)dst[i] * d.width;
  for (int j = g.thread(); j < pages; j += g.threads()) row[j] = fresh[j];
  const long long items = (long long)pages * d.heads;
  for (long long x = g.warp(); x < items; x += g.warps()) {
    const int j = (int)(x / d.heads), h = (int)(x - (long long)j * d.heads);
    const int a = from[j], b = fresh[j];
    if ((unsigned)a >= (unsigned)s.num_pages) continue;
    const size_t p = page_vec(s, a, h), q = page_vec(d, b, h);
    warp_copy(Ks + p, Vs + p, K + q, V + q, min(d.page, len - (j << d.shift)) * d.row_vecs, g.tid & 31);
  }
}

struct RowArgs {
  PagesView d, s;       // the cache, and the one copied from
  const int *src, *dst, *counts;
  int n, T;
  const uint4 *Kfrom, *Vfrom;  // new tokens, or the pools copied from
  uint4 *K, *V;
};

template <int MODE>
__device__ __forceinline__ void entry_rows(const RowArgs& x, int i, const Group& g) {
  if constexpr (MODE == kAppend)
    append_rows(x.d, i, g, x.dst, x.T, x.Kfrom, x.Vfrom, x.K, x.V);
  else if constexpr (MODE == kFork)
    fork_rows(x.d, i, g, x.src, x.dst, x.K, x.V);
  else
    copy_rows(x.d, x.s, i, g, x.src, x.dst, x.Kfrom, x.Vfrom, x.K, x.V);
}

// blockIdx.y: list entry.
template <int MODE>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const __grid_constant__ RowArgs x) {
  pdl_wait();
  pdl_release();
  if (!*x.d.ok) return;
  entry_rows<MODE>(x, blockIdx.y, Group::of_grid());
}

// Plan and rows of a small call, one CTA.
template <int MODE>
__global__ void __launch_bounds__(kPlanThreads) small_kernel(const __grid_constant__ RowArgs x) {
  pdl_wait();
  pdl_release();
  plan_body(x.d, x.s, x.src, x.dst, x.counts, x.n, x.T, MODE);
  __syncthreads();
  if (!*x.d.ok) return;
  Group g = Group::of_cta();
  const int each = max(1, kGroups / x.n), sets = kGroups / each, set = g.x / each;  // each: groups per entry
  g.x %= each;
  g.nx = each;
  if (set < sets)
    for (int i = set; i < x.n; i += sets) entry_rows<MODE>(x, i, g);
}

// blockIdx.y: list entry.  Rows [0, len) of the sequence to the dense cache.
__global__ void __launch_bounds__(kRowThreads) gather_kernel(PagesView s, const int* seqs, long long capacity, const uint4* K,
                                                             const uint4* V, uint4* Kd, uint4* Vd) {
  pdl_wait();
  pdl_release();
  const int i = blockIdx.y, slot = seqs[i];
  if ((unsigned)slot >= (unsigned)s.max_seqs) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(s.err, kDevErrBadSeq);
    return;
  }
  const int len = s.lens[slot];
  if (len > capacity) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(s.err, kDevErrPool);
    return;
  }
  const int pages = ceil_shift(len, s.shift);
  const int* row = s.table + (size_t)slot * s.width;
  const int lane = threadIdx.x & 31;
  const long long items = (long long)pages * s.heads;
  for (long long x = blockIdx.x * kRowWarps + (threadIdx.x >> 5); x < items; x += (long long)gridDim.x * kRowWarps) {
    const int h = (int)(x / pages), j = (int)(x - (long long)h * pages);
    const int a = row[j];
    if ((unsigned)a >= (unsigned)s.num_pages) continue;
    const size_t p = page_vec(s, a, h);
    const size_t q = (((size_t)i * s.heads + h) * (size_t)capacity + ((size_t)j << s.shift)) * s.row_vecs;
    warp_copy(K + p, V + p, Kd + q, Vd + q, min(s.page, len - (j << s.shift)) * s.row_vecs, lane);
  }
}

// One CTA per list entry (few pages in all).  Whoever takes the length away frees the sequence, so a slot that is
// named twice is freed once.
__global__ void __launch_bounds__(kRowThreads) free_kernel(PagesView d, const int* seqs) {
  __shared__ int s_len, s_freed;
  pdl_wait();
  pdl_release();
  const int slot = seqs[blockIdx.x];
  if ((unsigned)slot >= (unsigned)d.max_seqs) {
    if (threadIdx.x == 0) atomicOr(d.err, kDevErrBadSeq);
    return;
  }
  if (threadIdx.x == 0) {
    s_len = atomicExch(&d.lens[slot], 0);
    s_freed = 0;
  }
  __syncthreads();
  const int pages = ceil_shift(s_len, d.shift);
  int* row = d.table + (size_t)slot * d.width;
  int freed = 0;
  for (int j = threadIdx.x; j < pages; j += kRowThreads) {
    const int page = row[j];
    row[j] = -1;
    if ((unsigned)page < (unsigned)d.num_pages && atomicSub(&d.refs[page], 1) == 1) {
      atomicAnd(&d.used[page >> 5], ~(1u << (page & 31)));
      ++freed;
    }
  }
  freed = __reduce_add_sync(0xffffffffu, freed);
  if ((threadIdx.x & 31) == 0 && freed) atomicAdd(&s_freed, freed);
  __syncthreads();
  if (threadIdx.x == 0 && s_freed) atomicAdd(d.free_pages, s_freed);
}

// Many pages: the lengths first, by one CTA, into plan_len (0 for a slot that a lower entry names too) ..
__global__ void __launch_bounds__(kPlanThreads) free_plan_kernel(PagesView d, const int* seqs, int n) {
  pdl_wait();
  pdl_release();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int slot = seqs[i];
    if ((unsigned)slot < (unsigned)d.max_seqs)
      atomicMin(&d.claim[slot], i);
    else
      atomicOr(d.err, kDevErrBadSeq);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int slot = seqs[i];
    d.plan_len[i] = (unsigned)slot < (unsigned)d.max_seqs && __ldcg(&d.claim[slot]) == i ? d.lens[slot] : 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int slot = seqs[i];
    if ((unsigned)slot >= (unsigned)d.max_seqs) continue;
    d.claim[slot] = kNoClaim;
    d.lens[slot] = 0;
  }
}

// .. then the table by columns: a thread takes a column of kRun entries.  Forks hold the same page in the same column,
// so a run of equal pages changes its count once (63 forks of 8,192 pages: 5 us; page by page 41 us,
// half a million counts to 8,192 places).
constexpr int kRun = 16;

struct Columns {
  const int* row[kRun];  // table rows, null: none
  int pages[kRun], most;
};

// Fills *c (shared memory) with entries first .. of n: slot and tokens by `get(i, &slot, &len)`.
template <typename Get>
__device__ __forceinline__ void columns_of(const PagesView& d, const int* table, int first, int n, Columns* c, Get get) {
  const int i = threadIdx.x;
  if (i < kRun) {
    int slot = 0, len = 0;
    if (first + i < n) get(first + i, &slot, &len);
    c->pages[i] = ceil_shift(len, d.shift);
    c->row[i] = table + (size_t)slot * d.width;
  }
  __syncthreads();
  if (i == 0) {
    int most = 0;
    for (int k = 0; k < kRun; ++k) most = max(most, c->pages[k]);
    c->most = most;
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kRowThreads) free_columns_kernel(PagesView d, const int* seqs, int n) {
  __shared__ Columns c;
  pdl_wait();
  pdl_release();
  columns_of(d, d.table, blockIdx.y * kRun, n, &c, [&](int i, int* slot, int* len) {
    *len = d.plan_len[i];
    *slot = *len ? seqs[i] : 0;
  });
  int freed = 0;
  for (int j = blockIdx.x * kRowThreads + threadIdx.x; j < c.most; j += gridDim.x * kRowThreads) {
    int page[kRun];
#pragma unroll
    for (int k = 0; k < kRun; ++k) page[k] = j < c.pages[k] ? c.row[k][j] : -1;
#pragma unroll
    for (int k = 0; k < kRun; ++k)
      if (j < c.pages[k]) const_cast<int*>(c.row[k])[j] = -1;
    int run = 0, less[kRun], held[kRun];  // by how much each run's count falls (at its last entry)
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      less[k] = 0;
      if ((unsigned)page[k] >= (unsigned)d.num_pages) continue;
      ++run;
      bool more = false;  // the same page again, no other between
#pragma unroll
      for (int x = kRun - 1; x > k; --x)
        if (page[x] >= 0) more = page[x] == page[k];
      if (more) continue;
      less[k] = run;
      run = 0;
    }
#pragma unroll
    for (int k = 0; k < kRun; ++k) held[k] = less[k] ? atomicSub(&d.refs[page[k]], less[k]) : 0;
#pragma unroll
    for (int k = 0; k < kRun; ++k)
      if (less[k] && held[k] == less[k]) {
        atomicAnd(&d.used[page[k] >> 5], ~(1u << (page[k] & 31)));
        ++freed;
      }
  }
  freed = __reduce_add_sync(0xffffffffu, freed);
  if ((threadIdx.x & 31) == 0 && freed) atomicAdd(d.free_pages, freed);
}

// ---------------------------------------------------------------- compact

// live = pages in use; the k-th free page below `live` is to receive the k-th used page at or above it
// (there are equally many): fresh[k] = destination, plan[k] = source is kept as name[source] and
// the list of sources follows the destinations in fresh (at most num_pages / 2 each).
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(PagesView d, int* out_live) {
  __shared__ int sums[32];
  pdl_wait();
  pdl_release();
  const int tid = threadIdx.x;
  const int live = d.num_pages - *d.free_pages;
  const int half = d.num_pages / 2;
  const int edge = live >> 5;  // the word that holds page `live`
  const unsigned below = (1u << (live & 31)) - 1u;
  int holes = 0, strays = 0;
  for (int at = 0; at < d.words; at += kPlanThreads) {
    const int w = at + tid;
    const unsigned word = w < d.words ? d.used[w] : 0u;
    // bits past num_pages are marked used and are no pages
    const int first = w * 32;
    const unsigned real = w >= d.words ? 0u : d.num_pages - first >= 32 ? ~0u : (1u << (d.num_pages - first)) - 1u;
    const unsigned low = w < edge ? ~0u : w == edge ? below : 0u;
    unsigned hole = ~word & low & real, stray = word & ~low & real;
    int sum;
    int k = holes + cta_scan(__popc(hole), sums, &sum);
    holes += sum;
    for (; hole; hole &= hole - 1) d.fresh[k++] = first + __ffs(hole) - 1;
    k = strays + cta_scan(__popc(stray), sums, &sum);
    strays += sum;
    for (; stray; stray &= stray - 1) d.fresh[half + k++] = first + __ffs(stray) - 1;
    if (w < d.words) d.used[w] = low | ~real;
  }
  __syncthreads();
  for (int k = tid; k < strays; k += kPlanThreads) d.name[d.fresh[half + k]] = d.fresh[k];
  if (tid == 0) {
    *d.moves = strays;
    *d.live = live;
    if (out_live) *out_live = live;
  }
}

__global__ void __launch_bounds__(kRowThreads) compact_move_kernel(PagesView d, uint4* K, uint4* V) {
  pdl_wait();
  pdl_release();
  const int moves = *d.moves, live = *d.live, half = d.num_pages / 2;
  if (moves == 0) return;
  const int lane = threadIdx.x & 31;
  for (int k = blockIdx.x * kRowThreads + threadIdx.x; k < moves; k += gridDim.x * kRowThreads) {
    const int a = d.fresh[half + k];
    d.refs[d.fresh[k]] = d.refs[a];
    d.refs[a] = 0;
  }
  for (int s = blockIdx.x; s < d.max_seqs; s += gridDim.x) {
    const int pages = ceil_shift(d.lens[s], d.shift);
    int* row = d.table + (size_t)s * d.width;
    for (int j = threadIdx.x; j < pages; j += kRowThreads) {
      const int page = row[j];
      if (page >= live && page < d.num_pages) row[j] = d.name[page];
    }
  }
  const long long items = (long long)moves * d.heads;
  for (long long x = blockIdx.x * kRowWarps + (threadIdx.x >> 5); x < items; x += (long long)gridDim.x * kRowWarps) {
    const int k = (int)(x / d.heads), h = (int)(x - (long long)k * d.heads);
    const size_t p = page_vec(d, d.fresh[half + k], h), q = page_vec(d, d.fresh[k], h);
    warp_copy(K + p, V + p, K + q, V + q, d.page * d.row_vecs, lane);
  }
}

// ---------------------------------------------------------------- init and load

__global__ void __launch_bounds__(kRowThreads) init_kernel(PagesView d) {
  pdl_wait();
  const size_t at = (size_t)blockIdx.x * kRowThreads + threadIdx.x, step = (size_t)gridDim.x * kRowThreads;
  for (size_t i = at; i < (size_t)d.max_seqs * d.width; i += step) d.table[i] = -1;
  for (size_t i = at; i < (size_t)d.num_pages; i += step) {
    d.refs[i] = d.count[i] = d.partial[i] = 0;
  }
  for (size_t i = at; i < (size_t)d.max_seqs; i += step) {
    d.lens[i] = d.mult[i] = 0;
    d.claim[i] = d.lead[i] = kNoClaim;
  }
  for (size_t i = at; i < (size_t)d.words; i += step) {
    const long long left = (long long)d.num_pages - 32 * (long long)i;
    d.used[i] = left >= 32 ? 0u : ~((1u << left) - 1u);
  }
  if (at == 0) {
    *d.err = 0;
    *d.ok = 1;
    *d.free_pages = d.num_pages;
    *d.moves = 0;
    *d.live = 0;
    *d.load_bad = *d.ticket = 0;
  }
}

// Counts the pages' holders, by columns of kRun slots as above, and marks partly filled last pages.
__global__ void __launch_bounds__(kRowThreads) load_count_kernel(PagesView d, const int* table, const int* lens) {
  __shared__ Columns c;
  __shared__ int partial[kRun];  // the column of a slot's partial last page, or -1
  pdl_wait();
  pdl_release();
  columns_of(d, table, blockIdx.y * kRun, d.max_seqs, &c, [&](int i, int* slot, int* len) {
    *slot = i;
    *len = lens[i];
    if (*len < 0 || (long long)*len > (long long)d.width << d.shift) {
      *d.load_bad = 1;
      *len = 0;
    }
    partial[i % kRun] = *len & (d.page - 1) ? *len >> d.shift : -1;
  });
  for (int j = blockIdx.x * kRowThreads + threadIdx.x; j < c.most; j += gridDim.x * kRowThreads) {
    int page[kRun];
#pragma unroll
    for (int k = 0; k < kRun; ++k) page[k] = j < c.pages[k] ? c.row[k][j] : -1;
    int run = 0;
    bool bad = false;
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      if (j >= c.pages[k]) continue;
      if ((unsigned)page[k] >= (unsigned)d.num_pages) {
        bad = true;
        page[k] = -1;
        continue;
      }
      ++run;
      if (partial[k] == j) d.partial[page[k]] = 1;
      bool more = false;
#pragma unroll
      for (int x = kRun - 1; x > k; --x)
        if (page[x] >= 0) more = page[x] == page[k];
      if (more) continue;
      atomicAdd(&d.count[page[k]], run);
      run = 0;
    }
    if (bad) *d.load_bad = 1;
  }
}

// A partly filled last page has one holder.
__global__ void __launch_bounds__(kRowThreads) load_check_kernel(PagesView d) {
  pdl_wait();
  pdl_release();
  for (int i = blockIdx.x * kRowThreads + threadIdx.x; i < d.num_pages; i += gridDim.x * kRowThreads) {
    if (d.partial[i] && d.count[i] > 1) *d.load_bad = 1;
    d.partial[i] = 0;
  }
}

// Adopts the counted table, or leaves an empty cache when something in it did not hold.
__global__ void __launch_bounds__(kRowThreads) load_apply_kernel(PagesView d, const int* table, const int* lens) {
  pdl_wait();
  pdl_release();
  const bool ok = !*d.load_bad;
  for (int s = blockIdx.x; s < d.max_seqs; s += gridDim.x) {
    // (table and lens may be the cache's own: every entry is read and written by one thread)
    const int len = ok ? lens[s] : 0, pages = ceil_shift(len, d.shift);
    const size_t row = (size_t)s * d.width;
    constexpr int U = 4;
    for (int j0 = threadIdx.x; j0 < d.width; j0 += U * kRowThreads) {
      int page[U];
#pragma unroll
      for (int u = 0; u < U; ++u) page[u] = j0 + u * kRowThreads < pages ? table[row + j0 + u * kRowThreads] : -1;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (j0 + u * kRowThreads < d.width) d.table[row + j0 + u * kRowThreads] = page[u];
    }
    __syncthreads();  // all have read the length
    if (threadIdx.x == 0) d.lens[s] = len;
  }
  // a warp makes one word of the bitmap
  const Group g = Group::of_grid();
  const int lane = g.tid & 31;
  for (int w = g.warp(); w < d.words; w += g.warps()) {
    const int page = w * 32 + lane;
    int refs = 0;
    if (page < d.num_pages) {
      refs = ok ? d.count[page] : 0;
      d.count[page] = 0;
      d.refs[page] = refs;
    }
    const unsigned held = __ballot_sync(0xffffffffu, page >= d.num_pages || refs > 0);
    if (lane == 0) {
      const int more = __popc(d.used[w]) - __popc(held);  // pages that become free
      d.used[w] = held;
      if (more) atomicAdd(d.free_pages, more);
    }
  }
  // the last CTA to leave puts the flag back, when every thread of every CTA has looked
  __syncthreads();
  __threadfence();
  if (threadIdx.x == 0 && atomicAdd(d.ticket, 1) == (int)gridDim.x - 1) {
    *d.ticket = 0;
    *d.load_bad = 0;
    if (!ok) atomicOr(d.err, kDevErrBadSeq);
  }
}

// ---------------------------------------------------------------- host

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t elem_bytes(const zha_pages_desc* d) { return d->kv_dtype == ZHA_BF16 ? 2 : 4; }

zha_status desc_status(const zha_pages_desc* d) {
  if (!d) return ZHA_ERR_INVALID_ARG;
  if (d->kv_heads < 1 || d->kv_heads > 65535 || d->page_tokens < 1 || d->num_pages < 1 || d->max_seqs < 1 ||
      d->max_seqs > 65535 || d->max_seq_pages < 1)
    return ZHA_ERR_INVALID_ARG;
  if (d->kv_dtype != ZHA_F32 && d->kv_dtype != ZHA_BF16) return ZHA_ERR_INVALID_ARG;
  if (d->head_dim != 64 && d->head_dim != 128) return ZHA_ERR_UNSUPPORTED;
  if (d->page_tokens < 8 || d->page_tokens > 256 || (d->page_tokens & (d->page_tokens - 1))) return ZHA_ERR_UNSUPPORTED;
  // counts, lengths and (page, head) pairs fit 31 bits
  if ((long long)d->max_seqs * d->max_seq_pages > (1LL << 30) || (long long)d->max_seq_pages * d->page_tokens > (1LL << 30) ||
      (long long)d->num_pages * d->kv_heads > (1LL << 30))
    return ZHA_ERR_UNSUPPORTED;
  return ZHA_OK;
}

// Lays the workspace out; returns its size.  base may be null.
size_t layout(const zha_pages_desc* d, char* base, PagesView* v) {
  size_t at = 0;
  auto take = [&](size_t n) {
    char* p = base + at;
    at = (at + n * 4 + 255) / 256 * 256;
    return reinterpret_cast<int*>(p);
  };
  int* head = take(64);
  v->err = reinterpret_cast<unsigned*>(head);
  v->ok = head + 1;
  v->free_pages = head + 2;
  v->moves = head + 3;
  v->live = head + 4;
  v->load_bad = head + 5;
  v->ticket = head + 6;
  v->max_seqs = d->max_seqs;
  v->width = d->max_seq_pages;
  v->num_pages = d->num_pages;
  v->words = (d->num_pages + 31) / 32;
  v->page = d->page_tokens;
  v->shift = 0;
  while ((1 << v->shift) < d->page_tokens) ++v->shift;
  v->heads = d->kv_heads;
  v->row_vecs = (int)(d->head_dim * elem_bytes(d) / 16);
  v->lens = take(d->max_seqs);
  v->claim = take(d->max_seqs);
  v->plan_len = take(d->max_seqs);
  v->plan_cnt = take(d->max_seqs);
  v->plan_base = take(d->max_seqs);
  v->plan_mult = take(d->max_seqs);
  v->mult = take(d->max_seqs);
  v->lead = take(d->max_seqs);
  v->refs = take(d->num_pages);
  v->fresh = take(d->num_pages);
  v->name = take(d->num_pages);
  v->count = take(d->num_pages);
  v->partial = take(d->num_pages);
  v->used = reinterpret_cast<unsigned*>(take(v->words));
  v->table = take((size_t)d->max_seqs * d->max_seq_pages);
  return at;
}

zha_status cuda_status(cudaError_t e) { return e == cudaSuccess ? ZHA_OK : ZHA_ERR_CUDA; }

// Plan and rows of a call that hands out pages and moves at most `bytes`.
template <int MODE>
zha_status launch_rows(zha_pages* p, const RowArgs& x, long long bytes, unsigned grid_x, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (bytes <= kSmallBytes) {
    e = launch_pdl(small_kernel<MODE>, dim3(1), dim3(kPlanThreads), 0, s, x);
    count_launches(p, 1);
  } else {
    e = launch_pdl(plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, x.d, x.s, x.src, x.dst, x.counts, x.n, x.T, (int)MODE);
    if (e == cudaSuccess) e = launch_pdl(rows_kernel<MODE>, dim3(grid_x, x.n), dim3(kRowThreads), 0, s, x);
    count_launches(p, 2);
  }
  return cuda_status(e);
}

// CTAs over the columns of a table.
unsigned column_grid(const zha_pages* p) {
  const int g = (p->desc.max_seq_pages + kRowThreads - 1) / kRowThreads;
  return (unsigned)(g < 2 * p->sms ? g : 2 * p->sms);
}

// CTAs over blockIdx.x so that `entries` list entries fill the device about 16 CTAs deep, and no more than `items`
// units of work per CTA could use.  Eight of them are resident: a long entry's others take the places that short entries
// leave (nine prompts of up to 8,000 tokens appended and gathered 121 us at 8 deep, 113.5 at 16, 113 at 32, 114.6 at 64).
unsigned row_grid(const zha_pages* p, int entries, long long items, int per_cta) {
  long long g = (16LL * p->sms + entries - 1) / entries;
  const long long most = (items + per_cta - 1) / per_cta;
  if (g > most) g = most;
  return (unsigned)(g < 1 ? 1 : g);
}

// The checks that every call with a list makes.  *skip: nothing to do.
zha_status list_status(const zha_pages* p, const int* list, int n, bool* skip) {
  *skip = false;
  if (!p || n < 0 || n > p->desc.max_seqs) return ZHA_ERR_INVALID_ARG;
  if (n == 0) {
    *skip = true;
    return ZHA_OK;
  }
  if (!list || !aligned(list, 4) || !on_device(p)) return ZHA_ERR_INVALID_ARG;
  return ZHA_OK;
}

bool vectors(const void* a, const void* b) { return a && b && aligned(a, 16) && aligned(b, 16); }

}  // namespace

extern "C" {

size_t zha_pages_workspace_bytes(const zha_pages_desc* desc) {
  if (desc_status(desc) != ZHA_OK) return 0;
  PagesView v;
  return layout(desc, nullptr, &v);
}

zha_status zha_pages_init(const zha_pages_desc* desc, void* d_workspace, size_t workspace_bytes, void* stream,
                          zha_pages** out) {
  if (!out) return ZHA_ERR_INVALID_ARG;
  *out = nullptr;
  const zha_status st = desc_status(desc);
  if (st != ZHA_OK) return st;
  if (!d_workspace || !aligned(d_workspace, 256)) return ZHA_ERR_INVALID_ARG;
  if (workspace_bytes < zha_pages_workspace_bytes(desc)) return ZHA_ERR_INVALID_ARG;
  zha_pages* p = static_cast<zha_pages*>(std::calloc(1, sizeof(zha_pages)));
  if (!p) return ZHA_ERR_INVALID_ARG;
  p->desc = *desc;
  layout(desc, static_cast<char*>(d_workspace), &p->v);
  if (cudaGetDevice(&p->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&p->sms, cudaDevAttrMultiProcessorCount, p->device) != cudaSuccess ||
      launch_pdl(init_kernel, dim3(2 * p->sms), dim3(kRowThreads), 0, static_cast<cudaStream_t>(stream), p->v) !=
          cudaSuccess) {
    std::free(p);
    return ZHA_ERR_CUDA;
  }
  p->launches = 1;
  *out = p;
  return ZHA_OK;
}

zha_status zha_pages_destroy(zha_pages* p) {
  if (!p) return ZHA_ERR_INVALID_ARG;
  std::free(p);
  return ZHA_OK;
}

zha_status zha_pages_load(zha_pages* p, const int* d_table, const int* d_lens, void* stream) {
  if (!p || !d_table || !d_lens || !aligned(d_table, 4) || !aligned(d_lens, 4) || !on_device(p))
    return ZHA_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const zha_pages_desc& d = p->desc;
  const dim3 block(kRowThreads), columns(column_grid(p), (d.max_seqs + kRun - 1) / kRun);
  cudaError_t e = launch_pdl(load_count_kernel, columns, block, 0, s, p->v, d_table, d_lens);
  if (e == cudaSuccess) e = launch_pdl(load_check_kernel, dim3(p->sms), block, 0, s, p->v);
  if (e == cudaSuccess) e = launch_pdl(load_apply_kernel, dim3(4 * p->sms), block, 0, s, p->v, d_table, d_lens);
  count_launches(p, 3);
  return cuda_status(e);
}

zha_status zha_pages_append(zha_pages* p, void* d_K, void* d_V, const int* d_seqs, int n, const void* d_Knew,
                            const void* d_Vnew, int tokens, const int* d_counts, void* stream) {
  bool skip;
  const zha_status st = list_status(p, d_seqs, n, &skip);
  if (st != ZHA_OK || tokens < 0) return st != ZHA_OK ? st : ZHA_ERR_INVALID_ARG;
  if (skip || tokens == 0) return ZHA_OK;
  if (!vectors(d_K, d_V) || !vectors(d_Knew, d_Vnew) || !aligned(d_counts, 4)) return ZHA_ERR_INVALID_ARG;
  if (tokens > 1 << 30 || (long long)tokens * p->desc.kv_heads > 1LL << 30) return ZHA_ERR_UNSUPPORTED;
  const RowArgs x = {p->v, p->v, nullptr, d_seqs, d_counts, n, tokens, (const uint4*)d_Knew, (const uint4*)d_Vnew,
                     (uint4*)d_K, (uint4*)d_V};
  const long long rows = (long long)tokens * p->desc.kv_heads;
  return launch_rows<kAppend>(p, x, 32LL * n * rows * p->v.row_vecs,
                              row_grid(p, n, rows, kRowThreads / p->v.row_vecs * 4), stream);
}

zha_status zha_pages_fork(zha_pages* p, void* d_K, void* d_V, const int* d_src, const int* d_dst, int n, void* stream) {
  bool skip;
  const zha_status st = list_status(p, d_src, n, &skip);
  if (st != ZHA_OK || skip) return st;
  if (!d_dst || !aligned(d_dst, 4) || !vectors(d_K, d_V)) return ZHA_ERR_INVALID_ARG;
  const RowArgs x = {p->v, p->v, d_src, d_dst, nullptr, n, 0, nullptr, nullptr, (uint4*)d_K, (uint4*)d_V};
  const long long tail = 32LL * p->v.page * p->v.heads * p->v.row_vecs;  // K and V of a page
  return launch_rows<kFork>(p, x, n * (tail + 8LL * p->desc.max_seq_pages), row_grid(p, n, p->desc.max_seq_pages, kRowThreads),
                            stream);
}

zha_status zha_pages_copy(const zha_pages* from, const void* d_Kfrom, const void* d_Vfrom, zha_pages* p, void* d_K,
                          void* d_V, const int* d_src, const int* d_dst, int n, void* stream) {
  bool skip;
  const zha_status st = list_status(p, d_src, n, &skip);
  if (st != ZHA_OK) return st;
  if (!from || from->device != p->device || from->desc.kv_heads != p->desc.kv_heads ||
      from->desc.head_dim != p->desc.head_dim || from->desc.page_tokens != p->desc.page_tokens ||
      from->desc.kv_dtype != p->desc.kv_dtype)
    return ZHA_ERR_INVALID_ARG;
  if (skip) return ZHA_OK;
  if (!d_dst || !aligned(d_dst, 4) || !vectors(d_K, d_V) || !vectors(d_Kfrom, d_Vfrom)) return ZHA_ERR_INVALID_ARG;
  const RowArgs x = {p->v, from->v, d_src, d_dst, nullptr, n, 0, (const uint4*)d_Kfrom, (const uint4*)d_Vfrom, (uint4*)d_K,
                     (uint4*)d_V};
  const long long page = 32LL * p->v.page * p->v.heads * p->v.row_vecs;
  // (a copy moves no more pages than the pool has)
  const long long most = (long long)n * p->desc.max_seq_pages, pool = p->desc.num_pages;
  return launch_rows<kCopy>(p, x, (most < pool ? most : pool) * page,
                            row_grid(p, n, (long long)p->desc.max_seq_pages * p->desc.kv_heads, kRowWarps), stream);
}

zha_status zha_pages_free(zha_pages* p, const int* d_seqs, int n, void* stream) {
  bool skip;
  const zha_status st = list_status(p, d_seqs, n, &skip);
  if (st != ZHA_OK || skip) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((long long)n * p->desc.max_seq_pages <= kFewPages) {
    count_launches(p, 1);
    return cuda_status(launch_pdl(free_kernel, dim3(n), dim3(kRowThreads), 0, s, p->v, d_seqs));
  }
  cudaError_t e = launch_pdl(free_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, p->v, d_seqs, n);
  if (e == cudaSuccess)
    e = launch_pdl(free_columns_kernel, dim3(column_grid(p), (n + kRun - 1) / kRun), dim3(kRowThreads), 0, s, p->v, d_seqs, n);
  count_launches(p, 2);
  return cuda_status(e);
}

zha_status zha_pages_compact(zha_pages* p, void* d_K, void* d_V, int* d_live, void* stream) {
  if (!p || !vectors(d_K, d_V) || !aligned(d_live, 4) || !on_device(p)) return ZHA_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_pdl(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, p->v, d_live);
  if (e == cudaSuccess)
    e = launch_pdl(compact_move_kernel, dim3(8 * p->sms), dim3(kRowThreads), 0, s, p->v, (uint4*)d_K, (uint4*)d_V);
  count_launches(p, 2);
  return cuda_status(e);
}

zha_status zha_pages_gather(const zha_pages* p, const void* d_K, const void* d_V, const int* d_seqs, int n, void* d_Kout,
                            void* d_Vout, long long capacity_tokens, void* stream) {
  bool skip;
  const zha_status st = list_status(p, d_seqs, n, &skip);
  if (st != ZHA_OK || capacity_tokens < 1) return st != ZHA_OK ? st : ZHA_ERR_INVALID_ARG;
  if (skip) return ZHA_OK;
  if (!vectors(d_K, d_V) || !vectors(d_Kout, d_Vout)) return ZHA_ERR_INVALID_ARG;
  const dim3 grid(row_grid(p, n, (long long)p->desc.max_seq_pages * p->desc.kv_heads, kRowWarps), n);
  const cudaError_t e = launch_pdl(gather_kernel, grid, dim3(kRowThreads), 0, static_cast<cudaStream_t>(stream), p->v,
                                   d_seqs, capacity_tokens, (const uint4*)d_K, (const uint4*)d_V, (uint4*)d_Kout,
                                   (uint4*)d_Vout);
  count_launches(p, 1);
  return cuda_status(e);
}

zha_status zha_pages_check(zha_pages* p, void* stream) {
  if (!p || !on_device(p)) return ZHA_ERR_INVALID_ARG;  // (stream 0 is the current device's)
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned h = 0;
  if (cudaMemcpyAsync(&h, p->v.err, sizeof(h), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return ZHA_ERR_CUDA;
  if (h != 0 && (cudaMemsetAsync(p->v.err, 0, sizeof(unsigned), s) != cudaSuccess ||
                 cudaStreamSynchronize(s) != cudaSuccess))
    return ZHA_ERR_CUDA;
  if (h & kDevErrTimeout) return ZHA_ERR_TIMEOUT;
  if (h & kDevErrBadSeq) return ZHA_ERR_DEVICE;
  if (h & kDevErrPool) return ZHA_ERR_CAPACITY;
  return ZHA_OK;
}

const int* zha_pages_table(const zha_pages* p) { return p ? p->v.table : nullptr; }
const int* zha_pages_lens(const zha_pages* p) { return p ? p->v.lens : nullptr; }
const int* zha_pages_refs(const zha_pages* p) { return p ? p->v.refs : nullptr; }
long long zha_pages_launch_count(const zha_pages* p) { return p ? __atomic_load_n(&p->launches, __ATOMIC_RELAXED) : -1; }
int zha_pages_device(const zha_pages* p) { return p ? p->device : -1; }

zha_status zha_pages_get_desc(const zha_pages* p, zha_pages_desc* out) {
  if (!p || !out) return ZHA_ERR_INVALID_ARG;
  *out = p->desc;
  return ZHA_OK;
}

zha_status zha_pages_set_wait_limit(zha_pages* p, long long cycles) {
  if (!p || cycles < 0) return ZHA_ERR_INVALID_ARG;
  p->wait_limit = cycles;
  return ZHA_OK;
}

}  // extern "C"
