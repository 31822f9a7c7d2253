// Shared-prefix attention on the tensor cores: bf16 queries over a bf16 paged cache.
//
// S = Q K^T and O += P V of a tile of 128 rows against 128 keys are tcgen05 MMAs with
// accumulators in TMEM.  A CTA holds two streams, each with its S (128 columns, overwritten
// in place by P) and its O: while one stream's 128 threads (one row each) form its weights,
// the other's MMAs run.  A dual item's two row tiles are the two streams over the same keys, which
// halves the key and value traffic.  The key tiles of all other segments of a CTA's share are dealt
// to the streams in turn, across segments, so that a run of short sequences keeps both busy; the
// join adds what the two streams leave of a segment.
//
//   warps 0-3, 4-7  stream 0, 1: maximum, exp2, sum, P; correction and output of O
//   warp 8, 9       TMA: queries and keys, values, page by page into a ring each.  A load for every (page,
//                   64 columns) takes the issuing warp about 100 clocks, so one warp for both was too slow
//   warp 10, 11     MMA issue (one lane) for stream 0, 1; warp 10 also holds TMEM.  Looking for the next
//                   operands takes an issuer 500 clocks, in which the other issues.  They take turns: left
//                   alone the streams fall into step, and MMAs and weights alternate instead of overlapping
//
// Up to 32 rows fill one warp's lanes.  Then the queries are loaded four times, into the lanes of each
// warp, and each weighs a quarter of the keys (P is zero elsewhere): a fourth of the
// latency per tile, for four partial results instead of one.
//
// The maximum that weights refer to moves only when a score exceeds it by more than 8 in
// base 2: weights then stay below 2^8, which costs no accuracy in floating point, and O is rarely
// rescaled.  Rows of a page past the sequence may hold anything: their scores are replaced, and
// the rows of V that an MMA step still touches are zeroed in shared memory, because 0 times NaN is NaN.
//
// Bound: a pair of dual tiles takes 3,900 clocks, 2,048 of them tensor work; the rest is the chain from scores to weights
// (2,000) to product, which two streams hide in part.  Measured with the join, 32 query and 8 KV heads of 128: 64
// sequences on a prefix of 131,072 tokens 200 us (0.69 PFLOP/s, 3.4 TB/s), 33 sequences of up to 4,000 tokens, nothing
// shared, 62 us (4.4 TB/s), eight sequences of four queries on 32,768 tokens, fp32 output, 65 us; with 64 query heads 16
// sequences on 1,048,576 tokens 775 us (5.6 TB/s).
// Twice the warps for the weights (16 rows each, 96 registers a thread) spilled and took 229 us for the first of these.
//
// Every wait is bounded; one that runs out sets an error that makes all warps leave, the
// producer waiting (bounded) for its loads and the issuer for its MMAs.
#include <cmath>

#include "prefix_attn.cuh"
#include "tcgen05.cuh"

using namespace zha;

namespace {

constexpr int kRows = 128;
// Keys of a tile.  An fp32 output wants the weights in 24 bits: three bf16 numbers each, whose three MMAs with V
// find room in S only for 64 keys.  (Two numbers for 128 keys were off by 1.5e-6 of the output.)
__host__ __device__ constexpr int keys_of(bool wide) { return wide ? 64 : 128; }
// Tiles whose products with V one sum in TMEM takes before it is added (in fp32, rounded) to the partial result in
// memory.  The tensor core cuts its sums off instead of rounding them: at each of the 12 MMAs of a tile with an fp32 output
// they lose 1.6e-8 of themselves on average.  Without end, an output over 120,000 tokens was off by 2.1e-5; with 16 tiles a
// sum 3.5e-6, with 8 1.8e-6, with 4 1.0e-6, for 61, 61, 65 and 71 us of eight sequences of four queries on 32,768 tokens.
// A bf16 output's tiles of 8 MMAs lose 1.4e-8 at each: sums of 8,192 tiles made outputs 9.4e-4 too small, those of 256
// 4.5e-5, a fiftieth of what the rounding of the weights takes off or adds at random.
__host__ __device__ constexpr int tiles_per_sum(bool wide) { return wide ? 8 : 256; }
constexpr int kThreads = 384;
constexpr int kTmemCols = 512;
constexpr int kByFma = 2;     // of 16 pairs of weights, those whose exp2 the FMA pipes compute
constexpr float kSlack = 8.f;  // base-2 growth of the maximum that is let pass

struct TcMaps {
  CUtensorMap q_prefix, q_own, k, v;
};

struct TcArgs {
  PrefixArgs a;
  TcMaps maps;
  int q_prefix_bytes, q_own_bytes;  // of one row tile's box (all of head_dim)
  int chunk, chunk_shift;           // rows a page contributes to a key tile
  int flip;                         // scale < 0: scores are negated and a.scale_log2 is its size
};

// Adds two values in memory.  (Whoever adds is the only one, so the order of the sums is the program's.)
__device__ __forceinline__ void add_to(float* p, float x, float y) {
  asm volatile("red.relaxed.gpu.global.add.v2.f32 [%0], {%1, %2};" ::"l"(p), "f"(x), "f"(y) : "memory");
}

template <int D>
struct Tc {
  static constexpr int kTile = 128 * D * 2;  // bytes of 128 rows
  static constexpr int kHalf = 128 * 128;    // bytes of 128 rows x 64 elements
  static constexpr int kKStages = D == 128 ? 2 : 5, kVStages = D == 128 ? 3 : 5;
  static constexpr size_t kSmem = 1024 + (size_t)(2 + kKStages + kVStages) * kTile + 1024;
};

struct Bars {
  uint64_t k_full[5], k_empty[5], v_full[5], v_empty[5];
  uint64_t q_full[2], q_empty[2], s_full[2], p_ready[2], o_full[2], o_free[2], turn[2], drain[2];
  int2 k_meta[5], v_meta[5];  // of a ring place: its keys, and TileFlags
  uint32_t tmem;
  int gone;  // a wait ran out
  int share[kThreads / 32 + 4];
};
static_assert(sizeof(Bars) <= 1024, "the barriers' page");

// What the issuers have to know of a tile, written by the loaders.
enum TileFlags {
  kFirst = 1,   // keys: its stream's first tile of the segment; values: of a sum
  kLast = 2,    // .. last
  kPaired = 4,  // a dual tile: both streams'
  kAlone = 8,   // keys: one stream alone uses the queries
  kLoneNext = 16,  // a dual tile that no dual tile follows
  kEnd = 32,    // no tile: the stream is done
  kQuery = 64   // keys, from here up: which query tile (mod 4)
};

// Bounded waits on the barriers of one CTA.  A whole warp waits, and all of its lanes get the same answer:
// what follows (TMEM accesses, MMA issue) needs the warp to stay together, also when it gives up.
struct Waiter {
  unsigned* err;
  volatile int* gone;

  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity, long long limit = kCopyWaitCycles) const {
    constexpr unsigned all = 0xffffffffu;
    const bool poll = limit < kPollWaitBelow;  // a test's
    if (!poll && __all_sync(all, mbar_try_wait(bar, parity))) return true;
    const long long t0 = clock64();
    while (!__all_sync(all, poll ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity))) {
      if (__any_sync(all, *gone != 0)) return false;
      if (__any_sync(all, clock64() - t0 > limit)) {
        atomicOr(err, kDevErrTimeout);
        *gone = 1;
        return false;
      }
    }
    return true;
  }
};

// The key tiles of a CTA's share, one after the other.
struct Tiles {
  Walk w;
  Segment g;
  int t;
  bool any;
  __device__ __forceinline__ Tiles(const PrefixArgs& a, const Walk& from, int cta) : w(from) {
    any = w.next(a, cta, &g);
    t = g.t0;
  }
  __device__ __forceinline__ bool dual() const { return g.kind == kDual; }
  __device__ __forceinline__ int k0(const PrefixArgs& a) const { return (g.kind == kOwn ? a.s.prefix : 0) + t * a.s.tile_keys; }
  __device__ __forceinline__ int keys(const PrefixArgs& a) const { return min(a.s.tile_keys, g.len - k0(a)); }
  __device__ __forceinline__ void step(const PrefixArgs& a, int cta) {
    if (++t == g.t1) {
      any = w.next(a, cta, &g);
      t = g.t0;
    }
  }
};

// A place in a ring and how often the ring has gone round.  Place y holds tile y.
template <int STAGES>
struct Place {
  int stage = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void add(int n) {  // n <= 2
    stage += n;
    if (stage >= STAGES) {
      stage -= STAGES;
      round ^= 1;
    }
  }
};

template <int REGS>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS)); }
template <int REGS>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS)); }

// The kernel launches with 168 registers a thread: 384 x 168 = 128 x (2 x 192 + 120).
constexpr int kStreamRegs = 192, kOtherRegs = 120;

// ---- warps 8 and 9

template <int D, bool WIDE>
struct Loader {
  using C = Tc<D>;
  const TcArgs& args;
  const PrefixArgs& a;
  Bars& bars;
  const Waiter& wait;
  uint32_t q_smem, ring;  // shared addresses of the queries and of this loader's ring
  int lane, per_tile, chunk, half;
  bool mine;
  uint32_t qc = 0, tiles = 0;  // query tiles and key tiles loaded

  __device__ __forceinline__ Loader(const TcArgs& x, Bars& b, const Waiter& w, uint32_t q, uint32_t kv)
      : args(x), a(x.a), bars(b), wait(w), q_smem(q), ring(kv), lane(threadIdx.x & 31) {
    per_tile = a.s.tile_keys >> args.chunk_shift;
    chunk = lane % per_tile;
    half = lane / per_tile;
    mine = lane < per_tile * (D / 64);
  }

  // Row tile `rt` of g to the next query buffer.
  __device__ __forceinline__ bool queries(const Segment& g, int rt) {
    const PrefixShape& s = a.s;
    const int buf = qc & 1;
    if (!wait(&bars.q_empty[buf], ((qc >> 1) & 1) ^ 1)) return false;
    const bool own = g.kind == kOwn;
    const int copies = own ? s.own_parts : g.kind == kSingle ? s.prefix_parts : 1;
    if (lane == 0) mbar_arrive_expect_tx(&bars.q_full[buf], copies * (own ? args.q_own_bytes : args.q_prefix_bytes));
    __syncwarp();
    if (lane < copies * (D / 64)) {
      const int h = lane % (D / 64), i = lane / (D / 64);
      int row = 0, b = rt * s.seqs_per_tile;
      if (own) {
        row = g.tile * s.own_tile;
        b = g.b;
      } else if (s.tiles_per_seq) {
        b = rt / s.tiles_per_seq;
        row = (rt - b * s.tiles_per_seq) * s.prefix_tile;
      }
      tma_load4(q_smem + buf * C::kTile + h * C::kHalf + i * 32 * 128, own ? &args.maps.q_own : &args.maps.q_prefix, h * 64,
                row, g.head, b, &bars.q_full[buf]);
    }
    __syncwarp();
    ++qc;
    return true;
  }

  // Page of this lane's part of the key tile (a bad id becomes one past the pool, which reads as zeros).
  __device__ __forceinline__ int page_of(const Tiles& x) const {
    const int token = x.k0(a) + (chunk << args.chunk_shift);
    if (!mine || token >= x.g.len) return -1;
    const int id = a.v.table[(size_t)x.g.pages * a.v.width + (token >> a.v.shift)];
    if ((unsigned)id < (unsigned)a.v.num_pages) return id;
    atomicOr(a.v.err, kDevErrBadSeq);
    return a.v.num_pages;
  }

  // The share's key tiles, KEYS: with the queries, else the values.
  template <bool KEYS>
  __device__ __forceinline__ bool run(const Walk& walk, int cta) {
    constexpr int kStages = KEYS ? C::kKStages : C::kVStages;
    uint64_t* const full = KEYS ? bars.k_full : bars.v_full;
    uint64_t* const empty = KEYS ? bars.k_empty : bars.v_empty;
    int2* const meta = KEYS ? bars.k_meta : bars.v_meta;
    const CUtensorMap* const map = KEYS ? &args.maps.k : &args.maps.v;
    Place<kStages> at;
    Tiles x(a, walk, cta);
    int page = x.any ? page_of(x) : -1;
    while (x.any) {
      const bool dual = x.dual();
      const int by = dual ? 1 : 2;
      const Segment g = x.g;
      const bool with_queries = KEYS && x.t == x.g.t0;
      int flags = dual ? kPaired : 0;
      const bool sums = !KEYS;  // first and last of a sum, else of the segment
      const int j = (x.t - x.g.t0) >> (by - 1);
      if (sums ? j % tiles_per_sum(WIDE) == 0 : j == 0) flags |= kFirst;
      if (x.t + by >= x.g.t1 || (sums && (j + 1) % tiles_per_sum(WIDE) == 0)) flags |= kLast;
      if (KEYS) {
        if (dual || x.g.t1 - x.g.t0 == 1) flags |= kAlone;
        flags |= ((with_queries ? qc : qc - 1 - dual) & 3) * kQuery;
      }
      const int n = x.keys(a), y = x.k0(a) & (a.v.page - 1) & ~(args.chunk - 1), z = page * a.s.heads + x.g.head;
      const bool load = page >= 0;
      x.step(a, cta);
      if (x.any) page = page_of(x);
      if (dual && !(x.any && x.dual())) flags |= kLoneNext;
      if (!wait(&empty[at.stage], at.round ^ 1)) return false;
      if (lane == 0) {
        meta[at.stage] = make_int2(n, flags);
        mbar_arrive_expect_tx(&full[at.stage], ((n + args.chunk - 1) >> args.chunk_shift) * args.chunk * D * 2);
      }
      __syncwarp();
      if (load)
        tma_load3(ring + at.stage * C::kTile + half * C::kHalf + (chunk << args.chunk_shift) * 128, map, half * 64, y, z,
                  &full[at.stage]);
      at.add(1);
      ++tiles;
      // the queries after the keys: they wait for the segment before the last, the keys need not
      if (with_queries)
        for (int i = 0; i < 1 + dual; ++i)
          if (!queries(g, g.tile + i)) return false;
    }
    if (KEYS)
      for (int i = 0; i < 2; ++i) {  // where each stream's next tile would be
        if (!wait(&empty[at.stage], at.round ^ 1)) return false;
        if (lane == 0) {
          meta[at.stage] = make_int2(0, kEnd);
          mbar_arrive(&full[at.stage]);
        }
        __syncwarp();
        at.add(1);
        ++tiles;
      }
    return true;
  }

  // After a wait that ran out: leaves no load in flight.
  template <bool KEYS>
  __device__ __forceinline__ void drain() {
    constexpr uint32_t stages = KEYS ? C::kKStages : C::kVStages;
    uint64_t* const full = KEYS ? bars.k_full : bars.v_full;
    for (uint32_t i = tiles > stages ? tiles - stages : 0; i < tiles; ++i)
      mbar_wait_bounded(&full[i % stages], (i / stages) & 1, a.v.err, kDevErrTimeout, kCopyWaitCycles);
    for (uint32_t i = qc > 2 ? qc - 2 : 0; i < qc; ++i)
      mbar_wait_bounded(&bars.q_full[i & 1], (i >> 1) & 1, a.v.err, kDevErrTimeout, kCopyWaitCycles);
  }
};

// ---- warps 10 and 11

template <int D, bool WIDE>
struct Issuer {
  using C = Tc<D>;
  const PrefixArgs& a;
  Bars& bars;
  const Waiter& wait;
  uint32_t q_smem, k_smem, v_smem, tmem;
  int st;

  __device__ __forceinline__ Issuer(const TcArgs& x, Bars& b, const Waiter& w, uint32_t q, uint32_t t, int stream)
      : a(x.a), bars(b), wait(w), q_smem(q), k_smem(q + 2 * C::kTile), v_smem(k_smem + C::kKStages * C::kTile), tmem(t), st(stream) {}

  // This stream's tiles: S of the first, then again and again O += P V of one and S of the next.  A tile's keys are
  // released by two arrivals, its queries too: one of each stream, or two of the only one that uses them.
  //
  // A stage of a ring may have held, a round before, a tile of the other stream.  A parity says that a phase is over only to somebody who knows that
  // the phase before is.  Here the turns say so: the other stream issued its scores of that tile before it gave
  // up the turn that this stream used last.
  __device__ __forceinline__ bool run(bool pairs) {
    Place<C::kKStages> kp;
    Place<C::kVStages> vp;
    if (!pairs) {  // tiles of one stream each: this one's first
      kp.add(st);
      vp.add(st);
    }
    uint32_t tiles = 0, segments = 0, turns = 0;  // phases of p_ready, o_free, turn
    const uint32_t s_tmem = same(tmem + st * 128), o_tmem = same(tmem + 256 + st * D);
    bool started = false;
    int2 v = make_int2(0, 0);
    while (true) {
      // the next keys
      if (!wait(&bars.k_full[kp.stage], kp.round, a.wait_cycles)) return false;
      const int2 k = bars.k_meta[kp.stage];
      const bool more = !(k.y & kEnd);
      const int q = (k.y / kQuery + (k.y & kPaired ? st : 0)) & 3;
      if (more && (k.y & kFirst) && !wait(&bars.q_full[q & 1], q >> 1, a.wait_cycles)) return false;
      const uint32_t kd = same((k_smem + kp.stage * C::kTile) >> 4), qd = same((q_smem + (q & 1) * C::kTile) >> 4);
      const uint32_t sd = same(mma_desc(128, (k.x + 15) & ~15, false));
      uint32_t vd = 0;
      int steps = 0;
      bool add = false;
      if (started) {  // the values of the tile before
        if (!wait(&bars.v_full[vp.stage], vp.round, a.wait_cycles)) return false;
        v = bars.v_meta[vp.stage];
        if ((v.y & kFirst) && !wait(&bars.o_free[st], (segments++ & 1) ^ 1)) return false;
        vd = same((v_smem + vp.stage * C::kTile) >> 4);
        steps = same((v.x + 15) / 16);
        add = same(!(v.y & kFirst));
      }
      if (!wait(&bars.turn[st], (turns++ & 1) ^ (st ^ 1))) return false;
      if (started && !wait(&bars.p_ready[st], tiles++ & 1)) return false;
      tc_fence_after();
      if (elect_one()) {
        if (started) {
          constexpr uint32_t od = mma_desc(128, D, true);
#pragma unroll
          for (int x = 0; x < keys_of(WIDE) / 16; ++x) {
            if (x >= steps) break;
            mma_ts(o_tmem, s_tmem + x * 8, desc_of(vd + x * 128, C::kHalf), od, add || x > 0);
            if (WIDE) {
              mma_ts(o_tmem, s_tmem + 32 + x * 8, desc_of(vd + x * 128, C::kHalf), od, true);
              mma_ts(o_tmem, s_tmem + 64 + x * 8, desc_of(vd + x * 128, C::kHalf), od, true);
            }
          }
          mma_commit(&bars.v_empty[vp.stage]);
          if (!(v.y & kPaired)) mma_commit(&bars.v_empty[vp.stage]);
          if (v.y & kLast) mma_commit(&bars.o_full[st]);
        }
        if (more) {
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            const uint32_t off = (x / 4 * C::kHalf + x % 4 * 32) >> 4;
            mma_ss(s_tmem, desc_of(qd + off, 16), desc_of(kd + off, 16), sd, x > 0);
          }
        }
        mbar_arrive(&bars.turn[st ^ 1]);
        if (more) {
          mma_commit(&bars.s_full[st]);
          mma_commit(&bars.k_empty[kp.stage]);
          if (!(k.y & kPaired)) mma_commit(&bars.k_empty[kp.stage]);
          if (k.y & kLast) {
            mma_commit(&bars.q_empty[q & 1]);
            if (k.y & kAlone) mma_commit(&bars.q_empty[q & 1]);
          }
        }
      }
      __syncwarp();
      if (started) vp.add(v.y & kPaired ? step(v) : 2);
      if (!more) return true;
      started = true;
      kp.add(k.y & kPaired ? step(k) : 2);
    }
  }
  // From a dual tile to this stream's next: the next, or behind the last of them its first lone tile.
  __device__ __forceinline__ int step(int2 m) const { return m.y & kLoneNext ? 1 + st : 1; }
};

// ---- warps 0 to 7

template <int D, bool WIDE>
struct Stream {
  using C = Tc<D>;
  const TcArgs& args;
  const PrefixArgs& a;
  Bars& bars;
  const Waiter& wait;
  char* ring;  // of values
  uint32_t ts, to;  // this warp's lanes of S and O
  int st, quarter, lane, r;
  uint32_t ns = 0, no = 0;

  __device__ __forceinline__ Stream(const TcArgs& x, Bars& b, const Waiter& w, char* kv, uint32_t tmem)
      : args(x), a(x.a), bars(b), wait(w), ring(kv) {
    const int warp = threadIdx.x >> 5;
    lane = threadIdx.x & 31;
    st = warp >> 2;
    quarter = warp & 3;
    r = quarter * 32 + lane;
    ts = tmem + ((uint32_t)quarter << 21) + st * 128;
    to = tmem + ((uint32_t)quarter << 21) + 256 + st * D;
  }

  float m, l;  // of this thread's row: what its weights refer to, their sum

  // N columns of P.
  template <int N>
  __device__ __forceinline__ void put(int col, const uint32_t* w) {
    if constexpr (N == 16)
      tmem_st16(ts + col, w);
    else
      tmem_st8(ts + col, w);
  }

  // Weights of COLS keys: scores at S columns [col, col + COLS), of which the first lim count.  O is
  // rescaled when the maximum moves (`fresh`: there is none yet).
  template <int COLS>
  __device__ __forceinline__ void weigh(int col, int lim, bool fresh) {
    const float c = a.scale_log2;
    uint32_t x[COLS];
    if constexpr (COLS == 16) {
      tmem_ld16(x, ts + col);
    } else {
#pragma unroll
      for (int q = 0; q < COLS / 32; ++q) tmem_ld32(x + 32 * q, ts + col + 32 * q);
    }
    tmem_wait_ld();
    if (args.flip) {
#pragma unroll
      for (int k = 0; k < COLS; ++k) x[k] ^= 0x80000000u;
    }
    if (__any_sync(0xffffffffu, lim < COLS)) {
#pragma unroll
      for (int k = 0; k < COLS; ++k) x[k] = k < lim ? x[k] : 0xff800000u;
    }
    float t0 = __uint_as_float(x[0]), t1 = __uint_as_float(x[1]);
#pragma unroll
    for (int k = 2; k < COLS; k += 4) {
      t0 = max3(t0, __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
      if (k + 3 < COLS) t1 = max3(t1, __uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]));
    }
    // a score that is NaN or +inf makes the row NaN, by way of the maximum
    float top = max3(t0, t1, t1) * c;
    if (top == INFINITY) top = NAN;
    float fix = 1.f;
    if (m == -INFINITY) {
      m = top;  // nothing of this row in O yet
    } else if (!(top <= m + kSlack)) {
      fix = exp2_approx(m - top);
      m = top;
    }
    if (WIDE) l *= fix;  // (a fresh sum may follow another)
    if (!fresh && __any_sync(0xffffffffu, fix != 1.f)) {
      if (!WIDE) l *= fix;
#pragma unroll
      for (int q = 0; q < D / 16; ++q) {
        uint32_t y[16];
        tmem_ld16(y, to + 16 * q);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * fix);
        tmem_st16(to + 16 * q, y);
      }
    }
    const float off = m == -INFINITY ? 0.f : -m;
    const uint64_t cc = pair(c, c), oo = pair(off, off);
    uint64_t sum = pair(0.f, 0.f);
    constexpr int G = COLS < 32 ? COLS / 2 : 16;  // packed columns at a time
#pragma unroll
    for (int q = 0; q < COLS / 2 / G; ++q) {
      uint32_t hi[G], mid[G], lo[G];
#pragma unroll
      for (int k = 0; k < G; ++k) {
        float p0, p1;
        const int at = 2 * (q * G + k);
        const uint64_t e = fma2(pair(__uint_as_float(x[at]), __uint_as_float(x[at + 1])), cc, oo);
        if (!WIDE && k < kByFma) {
          exp2_by_fma(e, &p0, &p1);
        } else {
          split(e, &p0, &p1);
          p0 = exp2_approx(p0);
          p1 = exp2_approx(p1);
        }
        sum = add2(sum, pair(p0, p1));
        hi[k] = pack_bf16(p0, p1);
        if (WIDE) {  // what a rounding leaves is exact in fp32
          p0 -= __uint_as_float(hi[k] << 16);
          p1 -= __uint_as_float(hi[k] & 0xffff0000u);
          mid[k] = pack_bf16(p0, p1);
          lo[k] = pack_bf16(p0 - __uint_as_float(mid[k] << 16), p1 - __uint_as_float(mid[k] & 0xffff0000u));
        }
      }
      put<G>(col / 2 + G * q, hi);
      if (WIDE) {
        put<G>(32 + col / 2 + G * q, mid);
        put<G>(64 + col / 2 + G * q, lo);
      }
    }
    float s0, s1;
    split(sum, &s0, &s1);
    l += s0 + s1;
  }

  // Zeros for the other warps' quarters of the keys.
  __device__ __forceinline__ void clear_others() {
    constexpr int G = keys_of(WIDE) / 8;
    const uint32_t z[16] = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q != quarter) {
        put<G>(G * q, z);
        if (WIDE) {
          put<G>(32 + G * q, z);
          put<G>(64 + G * q, z);
        }
      }
  }

  // A sum in memory, times a factor of each lane's row.
  __device__ __noinline__ void rescale(size_t slot, bool valid, float by) {
    __threadfence();
    __syncwarp();
    for (int r = 0; r < 32; ++r) {
      const float f = __shfl_sync(0xffffffffu, by, r);
      if (!__shfl_sync(0xffffffffu, valid, r)) continue;
      float* p = a.acc + (slot + r) * D;
      for (int c = lane; c < D; c += 32) __stcg(p + c, __ldcg(p + c) * f);
    }
    __threadfence();
    __syncwarp();
  }

  // Adds a bf16 output's sum, whose weights refer to m, to the one in memory, a row a thread.  Once in 256 tiles: short code
  // rather than quick.  (As the stores and reductions of segment(), or as a function to call, it cost the segments that
  // never come here more registers or instructions: 33 sequences of up to 4,000 tokens 63.5 and 65 us, this way 62.5,
  // without any of it 61.7.)
  __device__ __forceinline__ void add_sum(size_t slot, bool valid) {
    __syncwarp();  // other lanes' stores
    float by = 1.f, old = 1.f;  // what this sum is multiplied by, and the one in memory
    if (valid) {
      const float before = a.ml[slot + lane].x;
      // (up to 2^16 this sum is scaled, which leaves it finite; more is rare, and what is there is scaled)
      if (m <= before + 2 * kSlack)
        by = m == before ? 1.f : exp2_approx(m - before);
      else
        old = before == -INFINITY ? 0.f : exp2_approx(before - m);
      a.ml[slot + lane] = make_float2(old == 1.f ? before : m, l * by);
    }
    float* p = a.acc + (slot + lane) * D;
#pragma unroll 1
    for (int c = 0; c < D; c += 16) {
      __syncwarp();
      uint32_t y[16];
      tmem_ld16(y, to + c);
      tmem_wait_ld();
      if (!valid) continue;
#pragma unroll
      for (int k = 0; k < 16; k += 4) {
        float4 x = __ldcg(reinterpret_cast<float4*>(p + c + k));
        x.x = fmaf(x.x, old, __uint_as_float(y[k]) * by);
        x.y = fmaf(x.y, old, __uint_as_float(y[k + 1]) * by);
        x.z = fmaf(x.z, old, __uint_as_float(y[k + 2]) * by);
        x.w = fmaf(x.w, old, __uint_as_float(y[k + 3]) * by);
        __stcg(reinterpret_cast<float4*>(p + c + k), x);
      }
    }
    __syncwarp();
  }

  // This stream's tiles j0, j0 + by, .. of a segment that starts with the share's tile `tile0`.
  __device__ __forceinline__ bool segment(const Segment& g, int j0, int by, uint32_t tile0) {
    constexpr int kKeys = keys_of(WIDE), kQuarter = kKeys / 4;
    const PrefixShape& s = a.s;
    const int n = g.t1 - g.t0;
    const int parts = g.kind == kOwn ? s.own_parts : g.kind == kSingle ? s.prefix_parts : 1;
    const int row = parts == 4 ? lane : r;
    const int first = g.kind == kOwn ? s.prefix : 0;
    int b, rem, rows = kRows;  // rows that one partial result has
    bool valid;
    if (g.kind == kOwn) {
      b = g.b;
      rem = g.tile * s.own_tile + row;
      valid = rem < s.rows;
      rows = min(s.rows, s.own_tile);
    } else {
      const int rt = g.kind == kDual ? g.tile + st : g.tile;
      if (s.seqs_per_tile) {
        const int x = row / s.rows;
        b = rt * s.seqs_per_tile + x;
        rem = row - x * s.rows;
        valid = x < s.seqs_per_tile && b < s.batch;
      } else {
        b = rt / s.tiles_per_seq;
        rem = (rt - b * s.tiles_per_seq) * s.prefix_tile + row;
        valid = rem < s.rows;
      }
      if (parts == 4) rows = s.rows * s.batch;
    }
    int row_end = 0;
    if (valid) {
      int slot;
      const int len = g.kind == kOwn ? g.len : prefix_len(a, b, &slot);
      row_end = min(g.len, tokens_seen(s, len, s.nq == 1 ? 0 : rem % s.nq));
    }
    const bool work = __any_sync(0xffffffffu, valid);
    m = -INFINITY;
    l = 0.f;
    float put_m = -INFINITY;  // WIDE: the maximum that the sums in memory refer to
    int j = j0;
    do {
      const int sum0 = j, sum1 = min(n, j + tiles_per_sum(WIDE) * by);  // the tiles of one sum
      for (; j < sum1; j += by) {
        const int k0 = first + (g.t0 + j) * kKeys, left = min(kKeys, g.len - k0);  // first key, keys
        if (!wait(&bars.s_full[st], ns++ & 1)) return false;
        tc_fence_after();
        if (left & 15) {  // rows of V behind the sequence, up to the end of the last MMA's 16
          const uint32_t p = tile0 + j;
          const int stage = p % C::kVStages;
          if (!wait(&bars.v_full[stage], (p / C::kVStages) & 1)) return false;
          if (r >= left && r < ((left + 15) & ~15)) {
            char* v = ring + stage * C::kTile + r * 128;
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
#pragma unroll
              for (int y = 0; y < 8; ++y) *reinterpret_cast<uint4*>(v + x * C::kHalf + y * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (work) {
          if (parts == 4) {
            weigh<kQuarter>(kQuarter * quarter, row_end - k0 - kQuarter * quarter, j == (WIDE ? sum0 : j0));
            __syncwarp();
            clear_others();
          } else {
            weigh<kKeys>(0, row_end - k0, j == (WIDE ? sum0 : j0));
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_ready[st]);
      }
      if (!wait(&bars.o_full[st], no++ & 1)) return false;
      tc_fence_after();
      if (work) {
        const int part = g.kind == kDual ? st : (j0 * parts + (parts == 4 ? quarter : 0));
        const size_t slot = (size_t)g.slot + part * rows + (parts == 4 ? 0 : quarter * 32);  // of this warp's first row
        if (!WIDE && sum0 > j0) {
          add_sum(slot, valid);
        } else {
          float fix = 1.f;  // WIDE: from what this sum's weights refer to, to what the sums in memory do
          if (WIDE) {
            if (sum0 == j0) put_m = m;
            // (up to 2^16 this sum is scaled, which leaves it finite; more is rare, and what is there is scaled)
            if (__any_sync(0xffffffffu, m != put_m && !(m <= put_m + 2 * kSlack))) {
              rescale(slot, valid, put_m == -INFINITY ? 0.f : exp2_approx(put_m - m));
              put_m = m;
            }
            if (m != put_m) fix = exp2_approx(m - put_m);
          }
          if (valid) a.ml[slot + lane] = WIDE ? make_float2(put_m, l * fix) : make_float2(m, l);
          // in whole 32-byte sectors: a row a thread, 16 bytes at a time, took four times as long (13,000 clocks)
          const unsigned some = __ballot_sync(0xffffffffu, valid);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (!(some >> (16 * i) & 0xffffu)) continue;
            const int r0 = 16 * i + lane / 4;
            const float f0 = WIDE ? __shfl_sync(0xffffffffu, fix, r0) : 0.f, f1 = WIDE ? __shfl_sync(0xffffffffu, fix, r0 + 8) : 0.f;
            float* out = a.acc + (slot + r0) * D + lane % 4 * 2;
#pragma unroll
            for (int c = 0; c < D; c += 64) {
              uint32_t y[32];
              tmem_ld_blocks(y, to + (16u * i << 16) + c);
              tmem_wait_ld();
              if (WIDE && sum0 > j0) {
#pragma unroll
                for (int k = 0; k < 16; ++k)
                  if (some >> (r0 + k % 2 * 8) & 1)
                    add_to(out + k % 2 * 8 * D + c + k / 2 * 8, __uint_as_float(y[2 * k]) * (k & 1 ? f1 : f0),
                           __uint_as_float(y[2 * k + 1]) * (k & 1 ? f1 : f0));
                continue;
              }
              if (some >> r0 & 1) {
#pragma unroll
                for (int k = 0; k < 8; ++k) *reinterpret_cast<uint2*>(out + c + 8 * k) = make_uint2(y[4 * k], y[4 * k + 1]);
              }
              if (some >> (r0 + 8) & 1) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  *reinterpret_cast<uint2*>(out + 8 * D + c + 8 * k) = make_uint2(y[4 * k + 2], y[4 * k + 3]);
              }
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.o_free[st]);
    } while (j < n);
    return true;
  }

  __device__ __forceinline__ bool run(Walk walk, int cta) {
    Segment g;
    uint32_t tile = 0;
    int turn = 0;  // whose tile the next single or own one is
    while (walk.next(a, cta, &g)) {
      const bool dual = g.kind == kDual;
      const int n = g.t1 - g.t0, j0 = dual ? 0 : st ^ turn;
      if (j0 < n && !segment(g, j0, dual ? 1 : 2, tile)) return false;
      tile += n;
      if (!dual) turn ^= n & 1;
    }
    return true;
  }
};

template <int D, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1) tc_kernel(const __grid_constant__ TcArgs args) {
  extern __shared__ char raw[];
  using C = Tc<D>;
  const PrefixArgs& a = args.a;
  char* base = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  Bars& bars = *reinterpret_cast<Bars*>(base + (2 + C::kKStages + C::kVStages) * C::kTile);
  const uint32_t q_smem = smem_addr(base);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;
  const Waiter wait{a.v.err, &bars.gone};

  if (threadIdx.x == 0) {
    for (int i = 0; i < 5; ++i) {
      mbar_init(&bars.k_full[i], 1);
      mbar_init(&bars.k_empty[i], 2);
      mbar_init(&bars.v_full[i], 1);
      mbar_init(&bars.v_empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.q_full[i], 1);
      mbar_init(&bars.q_empty[i], 2);
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_ready[i], 4);
      mbar_init(&bars.o_full[i], 1);
      mbar_init(&bars.o_free[i], 4);
      mbar_init(&bars.turn[i], 1);
      mbar_init(&bars.drain[i], 1);
    }
    bars.gone = 0;
    fence_mbar_init();
  }
  if (warp == 10) tmem_alloc(&bars.tmem, kTmemCols);
  if (warp == 8 && lane < 4) prefetch_map(lane == 0 ? &args.maps.q_prefix : lane == 1 ? &args.maps.q_own : lane == 2 ? &args.maps.k : &args.maps.v);
  pdl_wait();
  pdl_release();
  const Walk walk = find_share(a, cta, kThreads, bars.share);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;

  if (warp < 8) {
    more_registers<kStreamRegs>();
    Stream<D, WIDE> s(args, bars, wait, base + (2 + C::kKStages) * C::kTile, tmem);
    s.run(walk, cta);
  } else {
    fewer_registers<kOtherRegs>();
    if (warp == 8) {
      Loader<D, WIDE> x(args, bars, wait, q_smem, q_smem + 2 * C::kTile);
      if (!x.template run<true>(walk, cta)) x.template drain<true>();
    } else if (warp == 9) {
      Loader<D, WIDE> x(args, bars, wait, q_smem, q_smem + (2 + C::kKStages) * C::kTile);
      if (!x.template run<false>(walk, cta)) x.template drain<false>();
    } else {
      Issuer<D, WIDE> x(args, bars, wait, q_smem, tmem, warp - 10);
      // (a share may start inside the last dual tile, which is the one before's)
      Walk w = walk;
      Segment first;
      x.run(w.next(a, cta, &first) && first.kind == kDual);
      // leave no MMA in flight, whatever ended the run
      if (elect_one()) mma_commit(&bars.drain[warp - 10]);
      __syncwarp();
      mbar_wait_bounded(&bars.drain[warp - 10], 0, a.v.err, kDevErrTimeout, kCopyWaitCycles);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 10) tmem_free(tmem, kTmemCols);
}

// ---------------------------------------------------------------- host

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// A bf16 tensor of `rank` dense dimensions, boxes 64 elements wide with the 128-byte swizzle.
bool encode(CUtensorMap* map, const void* p, int rank, const cuuint64_t* dims, const cuuint32_t* box) {
  const EncodeFn fn = encoder();
  if (!fn) return false;
  cuuint64_t strides[4];
  cuuint64_t bytes = 2;
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  for (int i = 0; i + 1 < rank; ++i) strides[i] = bytes *= dims[i];
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(p), dims, strides, box, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool WIDE>
cudaError_t launch(const zha_pages* p, const TcArgs& args, cudaStream_t stream) {
  const cudaError_t e = allow_shared<tc_kernel<D, WIDE>>(p, Tc<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(tc_kernel<D, WIDE>, dim3(args.a.s.ctas), dim3(kThreads), Tc<D>::kSmem, stream, args);
}

}  // namespace

namespace zha {

cudaError_t launch_prefix_tc(const zha_pages* p, const PrefixArgs& a, int head_dim, bool wide, cudaStream_t stream) {
  TcArgs x;
  x.a = a;
  const PrefixShape& s = a.s;
  const cuuint64_t d = head_dim;
  const cuuint64_t q[4] = {d, (cuuint64_t)s.rows, (cuuint64_t)s.heads, (cuuint64_t)s.batch};
  const cuuint32_t rows = s.rows < kRows ? s.rows : kRows;
  const cuuint32_t own[4] = {64, rows, 1, 1};
  const int together = s.prefix_parts == 4 ? s.batch : s.seqs_per_tile ? s.seqs_per_tile : 1;
  const cuuint32_t shared[4] = {64, rows, 1, (cuuint32_t)together};
  x.chunk = p->desc.page_tokens < s.tile_keys ? p->desc.page_tokens : s.tile_keys;
  x.chunk_shift = 0;
  while ((1 << x.chunk_shift) < x.chunk) ++x.chunk_shift;
  const cuuint64_t kv[3] = {d, (cuuint64_t)p->desc.page_tokens, (cuuint64_t)p->desc.num_pages * s.heads};
  const cuuint32_t kv_box[3] = {64, (cuuint32_t)x.chunk, 1};
  if (!encode(&x.maps.q_own, a.Q, 4, q, own) || !encode(&x.maps.q_prefix, a.Q, 4, q, shared) ||
      !encode(&x.maps.k, a.K, 3, kv, kv_box) || !encode(&x.maps.v, a.V, 3, kv, kv_box))
    return cudaErrorInvalidValue;
  x.q_own_bytes = (int)(rows * d * 2);
  x.q_prefix_bytes = (int)(rows * shared[3] * d * 2);
  x.flip = a.scale_log2 < 0.f;
  x.a.scale_log2 = fabsf(a.scale_log2);
  // a scale of zero: any size so small that every weight is 1 (0 times a masked score is NaN)
  if (x.a.scale_log2 < 1e-37f) x.a.scale_log2 = 1e-37f;
  if (head_dim == 64) return wide ? launch<64, true>(p, x, stream) : launch<64, false>(p, x, stream);
  return wide ? launch<128, true>(p, x, stream) : launch<128, false>(p, x, stream);
}

}  // namespace zha
