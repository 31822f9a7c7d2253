// Host-side state of a paged cache and the view of its workspace that kernels take.
#pragma once

#include "zha_internal.h"

namespace zha {

constexpr int kNoClaim = 0x7fffffff;

// The workspace of a paged cache (device pointers into the caller's buffer).
struct PagesView {
  unsigned* err;   // device error word
  int* ok;         // 1: the last planned call's arguments held, its row kernel may run
  int* free_pages; // pages that no sequence holds
  int* moves;      // pages that a compaction moves
  int* live;       // pages in use
  int* load_bad;   // a load met something that does not hold (0 between calls)
  int* ticket;     // CTAs of a load's last step that are done (0 between calls)
  int* lens;       // [max_seqs] tokens
  int* claim;      // [max_seqs] lowest list entry that names a slot (kNoClaim between calls)
  int* plan_len;   // [max_seqs] per list entry: tokens before the call (append) or of the source
  int* plan_cnt;   // [max_seqs] tokens the entry adds
  int* plan_base;  // [max_seqs] its first page's place in `fresh`
  int* plan_mult;  // [max_seqs] a fork's entries that name its source, at the first of them; else 0
  int* mult;       // [max_seqs] entries that name a slot as source (0 between calls)
  int* lead;       // [max_seqs] the lowest of them (kNoClaim between calls)
  int* refs;       // [num_pages] sequences that hold a page
  int* fresh;      // [num_pages] pages given out by the call / pages that a compaction moves
  int* name;       // [num_pages] a moved page's new id
  int* count;      // [num_pages] load: table entries that name a page (0 between calls)
  int* partial;    // [num_pages] load: 1 for a partly filled last page (0 between calls)
  unsigned* used;  // [words] bit p: page p is held (bits past num_pages are set)
  int* table;      // [max_seqs, width] page ids, -1 behind a sequence's last page
  int max_seqs, width, num_pages, words;
  int page, shift;  // tokens per page, a power of two
  int heads;        // KV heads
  int row_vecs;     // 16-byte vectors per row (head_dim elements)
};

}  // namespace zha

struct zha_pages {
  zha_pages_desc desc;
  zha::PagesView v;
  int sms;
  int device;
  long long launches;  // (changed by count_launches alone: calls that only read the cache may overlap)
  long long wait_limit;
};

namespace zha {

inline void count_launches(const zha_pages* p, int n) {
  __atomic_fetch_add(&const_cast<zha_pages*>(p)->launches, n, __ATOMIC_RELAXED);  // the handle is logically const
}

// True when the pages' device is the current one (launches go to the current device).
inline bool on_device(const zha_pages* p) {
  int d = -1;
  return cudaGetDevice(&d) == cudaSuccess && d == p->device;
}

}  // namespace zha
