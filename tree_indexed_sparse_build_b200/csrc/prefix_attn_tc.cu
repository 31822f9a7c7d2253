// Shared-prefix attention on the tensor cores: bf16 queries over a bf16 paged cache.
//
// S = Q K^T and O += P V of a tile of 128 rows against 128 keys are tcgen05 MMAs with
// accumulators in TMEM.  A CTA holds two streams, each with its S (128 columns, overwritten
// in place by P) and its O: while one stream's 128 threads (one row each) form its weights,
// the other's MMAs run.  An item of two row tiles runs them as the two streams over the same
// keys, which halves the key and value traffic; an item of one row tile gives its streams alternate
// key tiles, and the join adds the two results.
//
//   warps 0-3, 4-7  stream 0, 1: maximum, exp2, sum, P; correction and output of O
//   warp 8          TMA: queries, and keys and values page by page into a ring
//   warp 9          MMA issue (one lane) and TMEM
//
// The maximum that weights refer to moves only when a score exceeds it by more than 8 in
// base 2: weights then stay below 2^8, which costs no accuracy in floating point, and O is rarely
// rescaled.  Rows of a page past the sequence may hold anything: their scores are replaced, and
// their rows of V zeroed in shared memory, because 0 times NaN is NaN.
//
// Every wait is bounded; one that runs out sets an error that makes all warps leave, the
// producer waiting (bounded) for its loads and the issuer for its MMAs.
#include <cmath>

#include "prefix_attn.cuh"
#include "tcgen05.cuh"

using namespace zha;

namespace {

constexpr int kRows = 128, kKeys = 128;
constexpr int kThreads = 320;
constexpr int kTmemCols = 512;
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

template <int D>
struct Tc {
  static constexpr int kTile = 128 * D * 2;  // bytes of 128 rows
  static constexpr int kHalf = 128 * 128;    // bytes of 128 rows x 64 elements
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr size_t kSmem = 1024 + (size_t)(2 + kStages) * kTile + 1024;
};

struct Bars {
  uint64_t full[10], empty[10], q_full[2], q_empty[2], s_full[2], p_ready[2], o_full[2], o_free[2], drain;
  uint32_t tmem;
  int gone;  // a wait ran out
  long long share[kThreads / 32 + 4];
};
static_assert(sizeof(Bars) <= 1024, "the barriers' page");

struct Waiter {
  unsigned* err;
  volatile int* gone;
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity, long long limit) const {
    if (limit >= kPollWaitBelow && mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!(limit < kPollWaitBelow ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity))) {
      if (*gone) return false;
      if (clock64() - t0 > limit) {
        atomicOr(err, kDevErrTimeout);
        *gone = 1;
        return false;
      }
    }
    return true;
  }
};

// Place in the ring, from the segment's first, of the keys and values of tile j of n.
__device__ __forceinline__ int k_at(bool dual, int j) { return dual ? 2 * j : j ? 2 * j - 1 : 0; }
__device__ __forceinline__ int v_at(bool dual, int j, int n) { return dual ? 2 * j + 1 : j < n - 1 ? 2 * j + 2 : 2 * n - 1; }

template <int D, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1) tc_kernel(const __grid_constant__ TcArgs args) {
  extern __shared__ char raw[];
  using C = Tc<D>;
  const PrefixArgs& a = args.a;
  const PrefixShape& s = a.s;
  char* base = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  Bars& bars = *reinterpret_cast<Bars*>(base + (2 + C::kStages) * C::kTile);
  const uint32_t q_smem = smem_addr(base), kv_smem = q_smem + 2 * C::kTile;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;
  const Waiter wait{a.v.err, &bars.gone};
  const long long bound = kCopyWaitCycles;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.q_full[i], 1);
      mbar_init(&bars.q_empty[i], 1);
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_ready[i], 4);
      mbar_init(&bars.o_full[i], 1);
      mbar_init(&bars.o_free[i], 4);
    }
    mbar_init(&bars.drain, 1);
    bars.gone = 0;
    fence_mbar_init();
  }
  if (warp == 9) tmem_alloc(&bars.tmem, kTmemCols);
  pdl_wait();
  pdl_release();
  Walk walk = find_share(a, cta, kThreads, bars.share);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;
  Segment g;

  if (warp == 8) {
    // ------------------------------------------------------------ loads
    uint32_t at = 0, qc = 0;  // ring position, query tiles loaded
    bool ok = true;
    const int per_tile = kKeys >> args.chunk_shift;  // chunks
    const int chunk = lane % per_tile, half = lane / per_tile;
    const bool mine = lane < per_tile * (D / 64);
    while (ok && walk.next(a, cta, &g)) {
      const int tiles_q = g.dual ? 2 : 1;
      for (int i = 0; ok && i < tiles_q; ++i, ++qc) {
        const int buf = qc & 1;
        ok = wait(&bars.q_empty[buf], ((qc >> 1) & 1) ^ 1, bound);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars.q_full[buf], g.own ? args.q_own_bytes : args.q_prefix_bytes);
          for (int h = 0; h < D / 64; ++h) {
            const uint32_t dst = q_smem + buf * C::kTile + h * C::kHalf;
            if (g.own) {
              tma_load4(dst, &args.maps.q_own, h * 64, g.tile * s.own_tile, g.head, g.b, &bars.q_full[buf]);
            } else {
              const int rt = g.dual ? 2 * g.tile + i : g.tile + s.duals;
              if (s.seqs_per_tile)
                tma_load4(dst, &args.maps.q_prefix, h * 64, 0, g.head, rt * s.seqs_per_tile, &bars.q_full[buf]);
              else
                tma_load4(dst, &args.maps.q_prefix, h * 64, rt % s.tiles_per_seq * s.prefix_tile, g.head,
                          rt / s.tiles_per_seq, &bars.q_full[buf]);
            }
          }
        }
        __syncwarp();
      }
      if (!ok) break;
      int slot = s.prefix_seq, first = 0, end = s.prefix;
      if (g.own) {
        end = prefix_len(a, g.b, &slot);
        first = s.prefix;
      }
      const int* row = a.v.table + (size_t)slot * a.v.width;
      const int n = g.t1 - g.t0;
      // page of this lane's chunk of tile j (a bad id becomes one past the pool: zeros)
      auto page_of = [&](int j) {
        const int t = first + (g.t0 + j) * kKeys + (chunk << args.chunk_shift);
        if (j >= n || !mine || t >= end) return -1;
        const int id = row[t >> a.v.shift];
        if ((unsigned)id < (unsigned)a.v.num_pages) return id;
        atomicOr(a.v.err, kDevErrBadSeq);
        return a.v.num_pages;
      };
      auto load = [&](const CUtensorMap* map, int j, int page) {
        const int stage = at % C::kStages;
        if (!wait(&bars.empty[stage], ((at / C::kStages) & 1) ^ 1, bound)) return false;
        const int k0 = first + (g.t0 + j) * kKeys;
        const int chunks = min(per_tile, (end - k0 + args.chunk - 1) >> args.chunk_shift);
        if (lane == 0) mbar_arrive_expect_tx(&bars.full[stage], chunks * args.chunk * D * 2);
        __syncwarp();
        if (page >= 0)
          tma_load3(kv_smem + stage * C::kTile + half * C::kHalf + (chunk << args.chunk_shift) * 128, map, half * 64,
                    k0 & (a.v.page - 1) & ~(args.chunk - 1), page * s.heads + g.head, &bars.full[stage]);
        ++at;
        return true;
      };
      int now = page_of(0), next = page_of(1), later;
      if (g.dual) {
        for (int j = 0; ok && j < n; ++j) {
          later = page_of(j + 2);
          ok = load(&args.maps.k, j, now) && load(&args.maps.v, j, now);
          now = next;
          next = later;
        }
      } else {
        ok = load(&args.maps.k, 0, now);
        for (int j = 0; ok && j < n; ++j) {
          later = page_of(j + 2);
          if (j + 1 < n) ok = load(&args.maps.k, j + 1, next);
          ok = ok && load(&args.maps.v, j, now);
          now = next;
          next = later;
        }
      }
    }
    if (!ok) {  // leave no load in flight
      for (uint32_t i = at > C::kStages ? at - C::kStages : 0; i < at; ++i)
        mbar_wait_bounded(&bars.full[i % C::kStages], (i / C::kStages) & 1, a.v.err, kDevErrTimeout, bound);
      for (uint32_t i = qc > 2 ? qc - 2 : 0; i < qc; ++i)
        mbar_wait_bounded(&bars.q_full[i & 1], (i >> 1) & 1, a.v.err, kDevErrTimeout, bound);
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMAs
    constexpr uint32_t qk = mma_desc(128, 128, false), pv = mma_desc(128, D, true);
    uint32_t at = 0, qc = 0, np[2] = {0, 0}, no[2] = {0, 0};
    bool ok = true;
    auto stage_wait = [&](uint32_t p) { return wait(&bars.full[p % C::kStages], (p / C::kStages) & 1, a.wait_cycles); };
    while (ok && walk.next(a, cta, &g)) {
      const int n = g.t1 - g.t0;
      const int count[2] = {g.dual ? n : (n + 1) / 2, g.dual ? n : n / 2};
      const int tiles_q = g.dual ? 2 : 1;
      for (int i = 0; ok && i < tiles_q; ++i)
        ok = wait(&bars.q_full[(qc + i) & 1], ((qc + i) >> 1) & 1, a.wait_cycles);
      auto scores = [&](int st, int i) {
        const uint32_t p = at + k_at(g.dual, g.dual ? i : 2 * i + st);
        if (!stage_wait(p)) return false;
        if (lane == 0) {
          const uint32_t q = q_smem + ((qc + (g.dual ? st : 0)) & 1) * C::kTile;
          const uint32_t k = kv_smem + p % C::kStages * C::kTile;
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            const uint32_t off = x / 4 * C::kHalf + x % 4 * 32;
            mma_ss(tmem + st * 128, smem_desc(q + off, 16, 1024), smem_desc(k + off, 16, 1024), qk, x > 0);
          }
          mma_commit(&bars.s_full[st]);
          if (!g.dual || st == 1) mma_commit(&bars.empty[p % C::kStages]);
        }
        __syncwarp();
        return true;
      };
      for (int st = 0; st < 2; ++st)
        if (ok && count[st]) ok = scores(st, 0);
      for (int i = 0; ok && i < count[0]; ++i) {
        for (int st = 0; ok && st < 2; ++st) {
          if (i >= count[st]) continue;
          const uint32_t p = at + v_at(g.dual, g.dual ? i : 2 * i + st, n);
          ok = wait(&bars.p_ready[st], np[st]++ & 1, bound) && stage_wait(p);
          if (ok && i == 0) ok = wait(&bars.o_free[st], (no[st]++ & 1) ^ 1, bound);
          if (!ok) break;
          tc_fence_after();
          if (lane == 0) {
            const uint32_t v = kv_smem + p % C::kStages * C::kTile;
#pragma unroll
            for (int x = 0; x < kKeys / 16; ++x) {
              const uint64_t desc = smem_desc(v + x * 2048, C::kHalf, 1024);
              mma_ts(tmem + 256 + st * D, tmem + st * 128 + x * 8, desc, pv, i > 0 || x > 0);
              if (WIDE) mma_ts(tmem + 256 + st * D, tmem + st * 128 + 64 + x * 8, desc, pv, true);
            }
            if (!g.dual || st == 1) mma_commit(&bars.empty[p % C::kStages]);
            if (i + 1 == count[st]) mma_commit(&bars.o_full[st]);
          }
          __syncwarp();
          if (i + 1 < count[st]) ok = scores(st, i + 1);
        }
      }
      if (ok && lane == 0)
        for (int i = 0; i < tiles_q; ++i) mma_commit(&bars.q_empty[(qc + i) & 1]);
      __syncwarp();
      at += 2 * n;
      qc += tiles_q;
    }
    if (!ok) {  // leave no MMA in flight
      if (lane == 0) mma_commit(&bars.drain);
      __syncwarp();
      mbar_wait_bounded(&bars.drain, 0, a.v.err, kDevErrTimeout, bound);
    }
  } else {
    // ------------------------------------------------------------ weights
    const int st = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // this thread's row of the tile
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t ts = tmem + lanes + st * 128, to = tmem + lanes + 256 + st * D;
    const float c = a.scale_log2;
    uint32_t at = 0, ns = 0, no = 0;
    bool ok = true;
    while (ok && walk.next(a, cta, &g)) {
      const int n = g.t1 - g.t0;
      const int count = g.dual ? n : (n + 1 - st) / 2;
      const uint32_t first_at = at;
      at += 2 * n;
      if (count == 0) continue;
      int b, rem;
      bool valid;
      if (g.own) {
        b = g.b;
        rem = g.tile * s.own_tile + r;
        valid = rem < s.rows;
      } else {
        const int rt = g.dual ? 2 * g.tile + st : g.tile + s.duals;
        if (s.seqs_per_tile) {
          const int x = r / s.rows;
          b = rt * s.seqs_per_tile + x;
          rem = r - x * s.rows;
          valid = x < s.seqs_per_tile && b < s.batch;
        } else {
          b = rt / s.tiles_per_seq;
          rem = (rt - b * s.tiles_per_seq) * s.prefix_tile + r;
          valid = rem < s.rows;
        }
      }
      int slot, row_end = 0;
      const int first = g.own ? s.prefix : 0;
      int end = s.prefix;
      if (g.own) end = prefix_len(a, g.b, &slot);
      if (valid) row_end = min(end, tokens_seen(s, prefix_len(a, b, &slot), rem % s.nq));
      const bool work = __any_sync(0xffffffffu, valid);
      float m = -INFINITY, l = 0.f;
      for (int i = 0; ok && i < count; ++i) {
        const int j = g.dual ? i : 2 * i + st;
        const int k0 = first + (g.t0 + j) * kKeys;
        ok = wait(&bars.s_full[st], ns++ & 1, bound);
        if (!ok) break;
        tc_fence_after();
        if (end - k0 < kKeys) {  // rows of V behind the sequence
          const uint32_t p = first_at + v_at(g.dual, j, n);
          ok = wait(&bars.full[p % C::kStages], (p / C::kStages) & 1, bound);
          if (!ok) break;
          if (r >= end - k0) {
            char* v = base + (2 + p % C::kStages) * C::kTile + r * 128;
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
#pragma unroll
              for (int y = 0; y < 8; ++y) *reinterpret_cast<uint4*>(v + x * C::kHalf + y * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (work) {
          uint32_t x[kKeys];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(x + 32 * q, ts + 32 * q);
          tmem_wait_ld();
          float* f = reinterpret_cast<float*>(x);
          if (args.flip) {
#pragma unroll
            for (int k = 0; k < kKeys; ++k) f[k] = -f[k];
          }
          const int lim = row_end - k0;
          if (__any_sync(0xffffffffu, lim < kKeys)) {
#pragma unroll
            for (int k = 0; k < kKeys; ++k) f[k] = k < lim ? f[k] : -INFINITY;
          }
          float t0 = f[0], t1 = f[1], t2 = f[2], t3 = f[3];
#pragma unroll
          for (int k = 4; k < kKeys; k += 4) {
            t0 = fmaxf(t0, f[k]);
            t1 = fmaxf(t1, f[k + 1]);
            t2 = fmaxf(t2, f[k + 2]);
            t3 = fmaxf(t3, f[k + 3]);
          }
          const float top = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)) * c;
          float fix = 1.f;
          if (m == -INFINITY) {
            m = top;  // nothing of this row in O yet
          } else if (top > m + kSlack) {
            fix = exp2_approx(m - top);
            m = top;
          }
          if (i > 0 && __any_sync(0xffffffffu, fix != 1.f)) {
            l *= fix;
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
              uint32_t y[32];
              tmem_ld32(y, to + 32 * q);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * fix);
              tmem_st32(to + 32 * q, y);
            }
          }
          const float off = m == -INFINITY ? 0.f : -m;
          float u0 = 0.f, u1 = 0.f;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float p0 = exp2_approx(fmaf(f[32 * q + 2 * k], c, off));
              const float p1 = exp2_approx(fmaf(f[32 * q + 2 * k + 1], c, off));
              u0 += p0;
              u1 += p1;
              hi[k] = pack_bf16(p0, p1);
              if (WIDE)
                lo[k] = pack_bf16(p0 - __uint_as_float(hi[k] << 16), p1 - __uint_as_float(hi[k] & 0xffff0000u));
            }
            tmem_st16(ts + 16 * q, hi);
            if (WIDE) tmem_st16(ts + 64 + 16 * q, lo);
          }
          l += u0 + u1;
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_ready[st]);
      }
      if (!ok) break;
      ok = wait(&bars.o_full[st], no++ & 1, bound);
      if (!ok) break;
      tc_fence_after();
      if (work) {
        const size_t out = (size_t)g.slot + (g.own ? st * (s.own_slot_rows / 2) : st * s.prefix_tile) + r;
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t y[32];
          tmem_ld32(y, to + 32 * q);
          tmem_wait_ld();
          if (valid) {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              *reinterpret_cast<uint4*>(a.acc + out * D + 32 * q + k) = make_uint4(y[k], y[k + 1], y[k + 2], y[k + 3]);
          }
        }
        if (valid) a.ml[out] = make_float2(m, l);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.o_free[st]);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_free(tmem, kTmemCols);
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
cudaError_t launch(const TcArgs& args, cudaStream_t stream) {
  auto kern = tc_kernel<D, WIDE>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Tc<D>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(args.a.s.ctas), dim3(kThreads), Tc<D>::kSmem, stream, args);
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
  const cuuint32_t shared[4] = {64, rows, 1, (cuuint32_t)(s.seqs_per_tile ? s.seqs_per_tile : 1)};
  x.chunk = p->desc.page_tokens < kKeys ? p->desc.page_tokens : kKeys;
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
  if (head_dim == 64) return wide ? launch<64, true>(x, stream) : launch<64, false>(x, stream);
  return wide ? launch<128, true>(x, stream) : launch<128, false>(x, stream);
}

}  // namespace zha
