// Work list of the shared-prefix attention: what the kernels and the join agree on.
//
// The rows of one KV head are the queries of its group: rows = q_heads / kv_heads * nq of each
// sequence.  Two kinds of items, each a tile of rows against a run of key tiles:
//   prefix  the rows of several sequences (or a slice of one's) against the shared tokens
//   own     one sequence's rows (or a slice) against its tokens behind the prefix
// All items' key tiles, laid end to end in a fixed order, are cut into one equal share of cost per
// CTA, so that no CTA waits for a long sequence.  A CTA's part of an item is a segment; its
// result (maximum, sum and weighted values, fp32) goes to the slot item + cta, which is unique
// because both only grow along the order.  A second kernel joins a row's slots.
//
// The cut depends on lengths that only the device knows.  A CTA finds its place by a sum
// over the batch's lengths; the join finds a row's segments by arithmetic on the same sums.
#pragma once

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
  int row_tiles;       // prefix row tiles per head
  int pairs;           // prefix items per head
  int duals;           // of those, items of two row tiles (tensor kernel)
  int own_tiles;       // own row tiles per sequence and head
  int streams;         // partial results an item of one row tile leaves: 1, or 2 (tensor kernel)
  int prefix_keys;     // key tiles of the prefix
  int dual_cost;       // cost of a key tile of a two-tile item (one-tile: 1)
  int ctas;
  long long head_cost; // cost of one head's prefix items
  long long prefix_cost;
  int prefix_slot_rows, own_slot_rows;
  long long own_slot0; // first row of the own slots
};

struct PrefixArgs {
  PrefixShape s;
  PagesView v;
  const void* Q;
  const void* K;
  const void* V;
  const int* seqs;
  long long* cum;  // [batch + 1] own key tiles before a sequence (written by CTA 0 for the join)
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
  return a.v.lens[x];
}

__device__ __forceinline__ int own_key_tiles(const PrefixShape& s, int len) {
  return len > s.prefix ? (len - s.prefix + s.tile_keys - 1) / s.tile_keys : 0;
}

// Tokens that query i of a sequence of `len` tokens sees.
__device__ __forceinline__ int tokens_seen(const PrefixShape& s, int len, int i) {
  return s.causal ? len - s.nq + 1 + i : len;
}

struct Segment {
  bool own;
  bool dual;
  int head;
  int b;        // own: sequence
  int tile;     // prefix: pair index; own: row tile
  int t0, t1;   // key tiles
  long long slot;  // first row of its slot
};

// A CTA's share of the work, segment by segment.  Every warp that walks sees the same list.
struct Walk {
  long long pos, hi;
  int b, n;        // own part: the sequence at pos and its key tiles
  long long cum;   // key tiles before it

  __device__ __forceinline__ bool next(const PrefixArgs& a, int cta, Segment* g) {
    const PrefixShape& s = a.s;
    while (pos < hi) {
      if (pos < s.prefix_cost) {
        const int head = (int)(pos / s.head_cost);
        long long start = head * s.head_cost;
        const long long rem = pos - start, dual = (long long)s.prefix_keys * s.dual_cost;
        int w = s.dual_cost, tile;
        if (rem < s.duals * dual) {
          tile = (int)(rem / dual);
          start += tile * dual;
        } else {
          w = 1;
          tile = s.duals + (int)((rem - s.duals * dual) / s.prefix_keys);
          start += s.duals * dual + (long long)(tile - s.duals) * s.prefix_keys;
        }
        g->t0 = (int)((pos - start + w - 1) / w);
        const long long t1 = (hi - start + w - 1) / w;
        g->t1 = t1 < s.prefix_keys ? (int)t1 : s.prefix_keys;
        pos = start + (long long)s.prefix_keys * w;
        if (g->t0 >= g->t1) continue;
        g->own = false;
        g->dual = tile < s.duals;
        g->head = head;
        g->tile = tile;
        g->b = 0;
        g->slot = ((long long)head * s.pairs + tile + cta) * s.prefix_slot_rows;
        return true;
      }
      const int group = s.heads * s.own_tiles;
      const long long x = pos - s.prefix_cost;
      while (x >= (cum + n) * group) {
        cum += n;
        ++b;
        int slot;
        n = own_key_tiles(s, prefix_len(a, b, &slot));
      }
      const long long y = x - cum * group;
      const int item = (int)(y / n);
      g->t0 = (int)(y - (long long)item * n);
      const long long left = hi - pos;
      g->t1 = n - g->t0 < left ? n : g->t0 + (int)left;
      pos += g->t1 - g->t0;
      g->own = true;
      g->dual = false;
      g->head = item / s.own_tiles;
      g->tile = item - g->head * s.own_tiles;
      g->b = b;
      g->slot = s.own_slot0 + ((long long)b * group + item + cta) * s.own_slot_rows;
      return true;
    }
    return false;
  }
};

// Finds CTA `cta`'s share; all of the CTA's `threads` threads call it.  sm: at least
// threads / 32 + 4 long longs.  CTA 0 also leaves the sums for the join and checks the call's slots.
__device__ __forceinline__ Walk find_share(const PrefixArgs& a, int cta, int threads, long long* sm) {
  const PrefixShape& s = a.s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = threads / 32;
  const int group = s.heads * s.own_tiles;
  long long* out = sm + warps;  // total, b, cum, n
  long long total = 0;
  // the total first: a share's borders depend on it
  long long mine = 0;
  for (int b = tid; b < s.batch; b += threads) {
    int slot;
    const int len = prefix_len(a, b, &slot);
    mine += own_key_tiles(s, len);
    if (cta == 0 && (unsigned)slot >= (unsigned)a.v.max_seqs) atomicOr(a.v.err, kDevErrBadSeq);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) sm[warp] = mine;
  __syncthreads();
  for (int i = 0; i < warps; ++i) total += sm[i];
  __syncthreads();
  const long long T = s.prefix_cost + total * group;
  Walk w;
  w.pos = cta * T / s.ctas;
  w.hi = (cta + 1) * T / s.ctas;
  w.b = w.n = 0;
  w.cum = 0;
  if (cta == 0 && tid == 0) {
    a.cum[s.batch] = total;
    if (s.prefix > 0 && a.v.lens[s.prefix_seq] < s.prefix) atomicOr(a.v.err, kDevErrBadSeq);
  }
  // the sequence at the share's start (or the first one, if the share starts in the prefix)
  const long long x = w.pos < s.prefix_cost ? 0 : w.pos - s.prefix_cost;
  if (w.hi > s.prefix_cost || cta == 0) {
    long long carry = 0;
    for (int b0 = 0; b0 < s.batch; b0 += threads) {
      const int b = b0 + tid;
      int slot, n = 0;
      if (b < s.batch) n = own_key_tiles(s, prefix_len(a, b, &slot));
      long long v = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
      }
      if (lane == 31) sm[warp] = v;
      __syncthreads();
      long long before = carry;
      for (int i = 0; i < warp; ++i) before += sm[i];
      for (int i = 0; i < warps; ++i) carry += sm[i];
      before += v - n;
      if (b < s.batch) {
        if (cta == 0) a.cum[b] = before;
        if (n > 0 && x >= before * group && x < (before + n) * group) {
          out[1] = b;
          out[2] = before;
          out[3] = n;
        }
      }
      __syncthreads();
      if (cta != 0 && carry * group > x) break;
    }
    if (total > 0) {
      w.b = (int)out[1];
      w.cum = out[2];
      w.n = (int)out[3];
    }
    __syncthreads();
  }
  return w;
}

// Launches (prefix_attn.cu, prefix_attn_tc.cu).
cudaError_t launch_prefix_tc(const zha_pages* p, const PrefixArgs& a, int head_dim, bool wide_p, cudaStream_t stream);

}  // namespace zha
