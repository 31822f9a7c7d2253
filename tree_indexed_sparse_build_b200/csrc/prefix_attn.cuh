// Work list of the shared-prefix attention: what the kernels and the join agree on.
//
// The rows of one KV head are the queries of its group: rows = q_heads / kv_heads * nq of each
// sequence.  Items are tiles of rows against a run of key tiles, in this order:
//   dual    two row tiles (each the rows of several sequences, or a slice of one's) against the shared
//           tokens (tensor kernel only: its two streams share the loads)
//   single  one row tile against the shared tokens
//   own     one sequence's rows (or a slice) against its tokens behind the prefix
// All items, laid end to end in that order, are cut into one equal share of cost per CTA, so that no CTA
// waits for a long sequence; a key tile belongs to the share in which it starts.  A CTA's part of an
// item is a segment; its result (maximum, sum and weighted values, fp32) goes to the slot item + cta,
// which is unique because both only grow along the order.  A second kernel joins a row's slots.
//
// The cut depends on lengths that only the device knows.  A CTA finds its place by a sum
// over the batch's lengths; the join finds a row's segments by arithmetic on the same sums.
#pragma once

#include <atomic>

#include "device_common.cuh"
#include "pages.h"

namespace zha {

struct PrefixShape {
  int batch, heads, rows, nq;
  int prefix;          // shared tokens
  int causal;
  int prefix_seq;
  int tile_keys;
  int prefix_tile;     // rows of a prefix row tile
  int own_tile;        // rows of an own row tile
  int seqs_per_tile;   // rows <= prefix_tile: sequences per prefix row tile (else 0)
  int tiles_per_seq;   // rows > prefix_tile: prefix row tiles per sequence
  int duals, singles;  // prefix items per head
  int own_tiles;       // own row tiles per sequence and head
  int prefix_parts;    // partial results that one stream leaves of a row of a single item
  int own_parts;       // .. of an own item
  int streams;         // streams of a single or own item's segment (1, or 2 in the tensor kernel)
  int prefix_keys;     // key tiles of the prefix
  int ctas;
  int single_cost;               // of a key tile of a single item
  int dual_total, prefix_total;  // cost of all dual items, of all prefix items
  int dual_slot_rows, single_slot_rows, own_slot_rows;
  long long single_slot0, own_slot0;   // first row of the single and of the own slots
};

struct PrefixArgs {
  PrefixShape s;
  PagesView v;
  const void* Q;
  const void* K;
  const void* V;
  const int* seqs;
  int* cum;        // [batch + 1] own cost before a sequence, per row tile, and [batch] tokens (by CTA 0, for the join)
  float2* ml;      // [slot rows] maximum (base 2, scaled) and sum
  float* acc;      // [slot rows, head_dim]
  void* O;
  float scale_log2;  // scale * log2(e)
  long long wait_cycles;
};

// Tokens of batch entry b, 0 for a bad slot; at most what its table row holds.
__device__ __forceinline__ int prefix_len(const PrefixArgs& a, int b, int* slot) {
  const int x = a.seqs[b];
  *slot = x;
  if ((unsigned)x >= (unsigned)a.v.max_seqs) return 0;
  return max(0, min(a.v.lens[x], a.v.width << a.v.shift));
}

__device__ __forceinline__ int own_key_tiles(const PrefixShape& s, int len) {
  return len > s.prefix ? (len - s.prefix + s.tile_keys - 1) / s.tile_keys : 0;
}

// Tokens that query i of a sequence of `len` tokens sees.
__device__ __forceinline__ int tokens_seen(const PrefixShape& s, int len, int i) {
  return s.causal ? len - s.nq + 1 + i : len;
}

// Costs, by what the tensor kernel takes for a bf16 output: a dual tile about 3,900 clocks, any other (its 64 KB of keys
// and values are the bound) 2,000 to 2,600, and so does the start and end of an own item.  (Tiles of 64 keys with three
// products, for an fp32 output, are weighted alike; a run of lone ones takes about 3,000 clocks each.)
constexpr int kDualCost = 2, kTileCost = 1, kOwnStart = 1;

// Where CTA c's share of the cost T starts (c == ctas: T).
__device__ __forceinline__ int share_start(int c, int T, int ctas) {
  const int each = T / ctas, more = T - each * ctas;
  return c * each + min(c, more);
}

// Of n tiles of cost w from position `at`, those that start before x.
__device__ __forceinline__ int tiles_before(int x, int at, int n, int w) {
  return max(0, min(n, (x - at + w - 1) / w));
}

enum SegmentKind { kDual = 0, kSingle = 1, kOwn = 2 };

struct Segment {
  int kind;
  int head;
  int b;        // own: sequence
  int tile;     // row tile (dual: the first of the two)
  int t0, t1;   // key tiles
  int pages;    // slot whose pages the keys are
  int len;      // tokens of that sequence that count
  long long slot;  // first row of its slot
};

// A CTA's share of the work, segment by segment.  Every warp that walks sees the same list.
struct Walk {
  int pos, hi;
  int b, n;             // own part: the sequence at pos and its key tiles
  int len, pages;       // its tokens and slot
  int next_len, next_pages;  // those of sequence b + 1, fetched ahead
  int item, at;         // its row tile (heads * own_tiles of them), and where that item's first key tile starts

  __device__ __forceinline__ void fetch(const PrefixArgs& a) {
    next_len = 0;
    if (b + 1 < a.s.batch) next_len = prefix_len(a, b + 1, &next_pages);
  }

  __device__ __forceinline__ bool next(const PrefixArgs& a, int cta, Segment* g) {
    const PrefixShape& s = a.s;
    while (pos < hi && pos < s.prefix_total) {
      const bool dual = pos < s.dual_total;
      const int w = dual ? kDualCost : s.single_cost, per_head = dual ? s.duals : s.singles, origin = dual ? 0 : s.dual_total;
      const int len_w = s.prefix_keys * w, i = (pos - origin) / len_w, start = origin + i * len_w;
      g->t0 = tiles_before(pos, start, s.prefix_keys, w);
      g->t1 = tiles_before(hi, start, s.prefix_keys, w);
      pos = start + len_w;
      if (g->t0 >= g->t1) continue;
      g->kind = dual ? kDual : kSingle;
      g->head = i / per_head;
      g->tile = dual ? 2 * (i - g->head * per_head) : 2 * s.duals + i - g->head * per_head;
      g->b = 0;
      g->pages = s.prefix_seq;
      g->len = s.prefix;
      g->slot = dual ? (long long)(i + cta) * s.dual_slot_rows : s.single_slot0 + (long long)(i + cta) * s.single_slot_rows;
      return true;
    }
    const int group = s.heads * s.own_tiles;
    while (pos < hi) {
      const int end = at + n * kTileCost;
      if (pos >= end) {  // the next item
        if (++item == group) {
          item = 0;
          do {
            ++b;
            len = next_len;
            pages = next_pages;
            n = own_key_tiles(s, len);
            fetch(a);
          } while (n == 0 && b < s.batch);
          if (b >= s.batch) return false;
        }
        at = end + kOwnStart;
        continue;
      }
      g->t0 = tiles_before(pos, at, n, kTileCost);
      g->t1 = tiles_before(hi, at, n, kTileCost);
      pos = end;
      if (g->t0 >= g->t1) continue;
      g->kind = kOwn;
      g->head = s.own_tiles == 1 ? item : item / s.own_tiles;
      g->tile = item - g->head * s.own_tiles;
      g->b = b;
      g->pages = pages;
      g->len = len;
      g->slot = s.own_slot0 + ((long long)b * group + item + cta) * s.own_slot_rows;
      return true;
    }
    return false;
  }
};

__device__ __forceinline__ int own_cost(const PrefixShape& s, int len) {
  const int n = own_key_tiles(s, len);
  return n ? n * kTileCost + kOwnStart : 0;
}

// Finds CTA `cta`'s share; all of the CTA's `threads` threads call it.  sm: at least
// threads / 32 + 4 ints.  CTA 0 also leaves the sums for the join and checks the call's slots.
__device__ __forceinline__ Walk find_share(const PrefixArgs& a, int cta, int threads, int* sm) {
  const PrefixShape& s = a.s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = threads / 32;
  const int group = s.heads * s.own_tiles;
  int* out = sm + warps;  // sequence, cost before it, its tokens and slot
  // sums of the own costs before this thread's entry of a round of `threads` (lane, then warp)
  int before = 0, total = 0;
  auto round = [&](int cost) {
    int v = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    if (lane == 31) sm[warp] = v;
    __syncthreads();
    before = total + v - cost;
    for (int i = 0; i < warps; ++i) {
      before += i < warp ? sm[i] : 0;
      total += sm[i];
    }
  };
  auto entry = [&](int b, int* slot) {
    int len = 0;
    *slot = 0;
    if (b < s.batch) {
      len = prefix_len(a, b, slot);
      if (cta == 0) {
        a.cum[s.batch + 1 + b] = len;
        if ((unsigned)*slot >= (unsigned)a.v.max_seqs) atomicOr(a.v.err, kDevErrBadSeq);
      }
    }
    return len;
  };
  // the total first: a share's borders depend on it
  int slot, len = entry(tid, &slot);
  round(own_cost(s, len));
  for (int b0 = threads; b0 < s.batch; b0 += threads) {
    int x;
    const int l = entry(b0 + tid, &x);
    __syncthreads();
    round(own_cost(s, l));
  }
  const int all = total, T = s.prefix_total + all * group;
  Walk w;
  w.pos = share_start(cta, T, s.ctas);
  w.hi = share_start(cta + 1, T, s.ctas);
  w.b = w.n = w.item = w.at = w.len = w.pages = w.next_len = w.next_pages = 0;
  if (cta == 0 && tid == 0) {
    a.cum[s.batch] = all;
    if (s.prefix > 0 && a.v.lens[s.prefix_seq] < s.prefix) atomicOr(a.v.err, kDevErrBadSeq);
  }
  // the sequence at the share's start (or the first one, if the share starts in the prefix)
  const bool find = w.pos < w.hi && w.hi > s.prefix_total;
  if (find || cta == 0) {
    const int x = max(0, w.pos - s.prefix_total);
    const bool again = s.batch > threads;  // (else the sums of the only round still stand)
    if (again) total = 0;
    for (int b0 = 0; b0 < s.batch; b0 += threads) {
      if (again) {
        len = entry(b0 + tid, &slot);
        __syncthreads();
        round(own_cost(s, len));
      }
      const int b = b0 + tid, cost = own_cost(s, len);
      if (b < s.batch) {
        if (cta == 0) a.cum[b] = before;
        if (x >= before * group && x < (before + cost) * group) {
          out[0] = b;
          out[1] = before;
          out[2] = len;
          out[3] = slot;
        }
      }
      if (cta != 0 && total * group > x) break;
    }
    __syncthreads();
    if (find) {  // (nothing is written to `out` for an empty share)
      w.b = out[0];
      w.len = out[2];
      w.pages = out[3];
      w.n = own_key_tiles(s, w.len);
      const int start = out[1] * group, cost = w.n * kTileCost + kOwnStart;
      w.item = (x - start) / cost;
      w.at = s.prefix_total + start + w.item * cost + kOwnStart;
      w.fetch(a);
    }
    __syncthreads();
  }
  return w;
}

// Launches (prefix_attn.cu, prefix_attn_tc.cu).
cudaError_t launch_prefix_tc(const zha_pages* p, const PrefixArgs& a, int head_dim, bool wide_p, cudaStream_t stream);

// Lets kernel K use `bytes` of shared memory on the device, once per device: the setting stays.  (Asking for it at every
// launch took up to 0.5 us of a call's 16 us of host time on one machine, and nothing measurable on another.)
template <auto K>
cudaError_t allow_shared(const zha_pages* p, size_t bytes) {
  static std::atomic<unsigned long long> done{0};
  const unsigned long long bit = p->device < 64 ? 1ull << p->device : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace zha
