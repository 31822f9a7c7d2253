// Attention over a shared prefix and each sequence's own pages: the plan, the fp32 kernel and the
// join of the partial results.  (bf16 queries over a bf16 cache: prefix_attn_tc.cu.)
#include <cmath>
#include <cstdint>

#include "prefix_attn.cuh"

using namespace zha;

namespace {

constexpr int kThreads = 256;
constexpr int kKeys = 32;  // keys per tile of the fp32 kernel

// ---------------------------------------------------------------- fp32 kernel
//
// A tile of RT rows against 32 keys at a time, everything in fp32 on the FMA pipes: thread
// (ty, tx) forms the scores of rows ty * RT/16 .. and keys tx, tx + 16, keeps those rows'
// running maximum and sum (the 16 threads of a row agree on them by shuffles) and
// accumulates columns 4 tx .. of the same rows.  The next tile's keys and values are on their way in registers,
// and the page ids of the one after, while a tile is computed; two CTAs share an SM.  (64 keys a tile and one
// buffer for K and V in turn, loads exposed: 16 sequences of 1,400 tokens 27 us.)  Bound: latency: a small call's CTAs have a
// tile or two each, and finding them (dependent loads and sums over the batch) takes as long.  16 sequences of up to 700 own
// tokens on 1,008 shared, 8 query and 2 KV heads of 128: 24 us with the join, which takes 9.
template <int D, typename TQ, typename TKV>
struct Fp32Tile {
  static constexpr int kStride = D + 4;  // 16 rows apart by 4 banks: float4 reads without conflicts
  static constexpr int kPStride = kKeys + 4;
  static constexpr int kVec = 16 / sizeof(TKV), kPer = D / kVec;      // values and vectors of a load, of a row
  static constexpr int kLoads = (kKeys * kPer + kThreads - 1) / kThreads;  // of a thread, for K and for V

  // The next tiles of one segment.
  struct Ahead {
    uint4 k[kLoads], v[kLoads];
    int page[kLoads];  // -1: a row behind the sequence (or a page that is none)

    __device__ __forceinline__ static int row(int i) { return (threadIdx.x + i * kThreads) / kPer; }

    __device__ __forceinline__ void find(const PagesView& v, const int* pages, int t0, int end) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int t = t0 + row(i);
        page[i] = row(i) < kKeys && t < end ? pages[t >> v.shift] : -1;
      }
    }
    __device__ __forceinline__ void load(const PagesView& w, const TKV* K, const TKV* V, int head, int t0) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        k[i] = v[i] = make_uint4(0, 0, 0, 0);
        if (page[i] == -1) continue;
        if ((unsigned)page[i] >= (unsigned)w.num_pages) {
          atomicOr(w.err, kDevErrBadSeq);
          continue;
        }
        const int t = t0 + row(i), c = (threadIdx.x + i * kThreads) % kPer;
        const size_t at = (((size_t)page[i] * w.heads + head) * w.page + (t & (w.page - 1))) * D + c * kVec;
        k[i] = *reinterpret_cast<const uint4*>(K + at);
        v[i] = *reinterpret_cast<const uint4*>(V + at);
      }
    }
    __device__ __forceinline__ static void put(const uint4& x, float* sm) {
      float f[kVec];
      Vec16<TKV>::to_f32(x, f);
#pragma unroll
      for (int q = 0; q < kVec; q += 4) *reinterpret_cast<float4*>(sm + q) = make_float4(f[q], f[q + 1], f[q + 2], f[q + 3]);
    }
    __device__ __forceinline__ void store(float* ks, float* vs) const {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        if (row(i) >= kKeys) continue;
        const int at = row(i) * kStride + (threadIdx.x + i * kThreads) % kPer * kVec;
        put(k[i], ks + at);
        put(v[i], vs + at);
      }
    }
  };

  template <int RT>
  __device__ static void segment(const PrefixArgs& a, const Segment& g, float* smem) {
    constexpr int R = RT / 16, C = D / 64;
    const PrefixShape& s = a.s;
    float* qs = smem;
    float* ks = qs + 64 * kStride;
    float* vs = ks + kKeys * kStride;
    float* ps = vs + kKeys * kStride;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;

    // row r of the tile -> (sequence, row within it)
    auto place = [&](int r, int* b, int* rem) {
      if (g.kind == kOwn) {
        *b = g.b;
        *rem = g.tile * s.own_tile + r;
        return *rem < s.rows && r < s.own_tile;
      }
      if (s.seqs_per_tile) {
        *b = g.tile * s.seqs_per_tile + r / s.rows;
        *rem = r % s.rows;
        return r < s.seqs_per_tile * s.rows && *b < s.batch;
      }
      *b = g.tile / s.tiles_per_seq;
      *rem = (g.tile % s.tiles_per_seq) * s.prefix_tile + r;
      return *rem < s.rows;
    };

    const int first = g.kind == kOwn ? s.prefix : 0, end = g.len;
    const int* pages = a.v.table + (size_t)g.pages * a.v.width;
    const TKV* K = static_cast<const TKV*>(a.K);
    const TKV* V = static_cast<const TKV*>(a.V);
    Ahead next;
    next.find(a.v, pages, first + g.t0 * kKeys, end);
    next.load(a.v, K, V, g.head, first + g.t0 * kKeys);
    next.find(a.v, pages, first + (g.t0 + 1) * kKeys, end);

    __syncthreads();  // the last segment is done with shared memory
    constexpr int qvec = 16 / sizeof(TQ), qper = D / qvec;
    for (int i = tid; i < RT * qper; i += kThreads) {
      const int r = i / qper, c = i % qper;
      int b, rem;
      float f[qvec];
      if (place(r, &b, &rem)) {
        const TQ* src = static_cast<const TQ*>(a.Q) + (((size_t)b * s.heads + g.head) * s.rows + rem) * D + c * qvec;
        Vec16<TQ>::to_f32(*reinterpret_cast<const uint4*>(src), f);
      } else {
#pragma unroll
        for (int k = 0; k < qvec; ++k) f[k] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < qvec; ++k) qs[r * kStride + c * qvec + k] = f[k];
    }

    // what each of this thread's rows sees
    bool valid[R];
    int seen[R];
    float m[R], l[R], acc[R][4 * C];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      int b = 0, rem = 0, slot;
      valid[i] = place(ty * R + i, &b, &rem);
      seen[i] = valid[i] ? tokens_seen(s, prefix_len(a, b, &slot), rem % s.nq) : 0;
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < 4 * C; ++c) acc[i][c] = 0.f;
    }
    for (int t = g.t0; t < g.t1; ++t) {
      const int k0 = first + t * kKeys, n = min(kKeys, end - k0);
      __syncthreads();
      next.store(ks, vs);
      __syncthreads();
      if (t + 1 < g.t1) {
        next.load(a.v, K, V, g.head, k0 + kKeys);
        next.find(a.v, pages, k0 + 2 * kKeys, end);
      }
      constexpr int J = kKeys / 16;
      float sc[R][J];
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j) sc[i][j] = 0.f;
#pragma unroll 4
      for (int c = 0; c < D; c += 4) {
        float4 q[R], k[J];
#pragma unroll
        for (int i = 0; i < R; ++i) q[i] = *reinterpret_cast<const float4*>(&qs[(ty * R + i) * kStride + c]);
#pragma unroll
        for (int j = 0; j < J; ++j) k[j] = *reinterpret_cast<const float4*>(&ks[(tx + 16 * j) * kStride + c]);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int j = 0; j < J; ++j) {
            sc[i][j] = fmaf(q[i].x, k[j].x, sc[i][j]);
            sc[i][j] = fmaf(q[i].y, k[j].y, sc[i][j]);
            sc[i][j] = fmaf(q[i].z, k[j].z, sc[i][j]);
            sc[i][j] = fmaf(q[i].w, k[j].w, sc[i][j]);
          }
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float top = m[i];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int key = tx + 16 * j;
          sc[i][j] = key < n && k0 + key < seen[i] ? sc[i][j] * a.scale_log2 : -INFINITY;
          top = fmaxf(top, sc[i][j]);
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float base = top == -INFINITY ? 0.f : top;  // a row that has seen nothing yet
        const float fix = exp2f(m[i] - base);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const float p = exp2f(sc[i][j] - base);
          ps[(ty * R + i) * kPStride + tx + 16 * j] = p;
          sum += p;
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l[i] = l[i] * fix + sum;
        m[i] = top;
#pragma unroll
        for (int c = 0; c < 4 * C; ++c) acc[i][c] *= fix;
      }
      __syncwarp();  // a row's weights are written and read by the same half of a warp
#pragma unroll 4
      for (int key = 0; key < kKeys; ++key) {
        float p[R];
#pragma unroll
        for (int i = 0; i < R; ++i) p[i] = ps[(ty * R + i) * kPStride + key];
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const float4 x = *reinterpret_cast<const float4*>(&vs[key * kStride + 64 * c + 4 * tx]);
#pragma unroll
          for (int i = 0; i < R; ++i) {
            acc[i][4 * c + 0] = fmaf(p[i], x.x, acc[i][4 * c + 0]);
            acc[i][4 * c + 1] = fmaf(p[i], x.y, acc[i][4 * c + 1]);
            acc[i][4 * c + 2] = fmaf(p[i], x.z, acc[i][4 * c + 2]);
            acc[i][4 * c + 3] = fmaf(p[i], x.w, acc[i][4 * c + 3]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (!valid[i]) continue;
      const size_t r = (size_t)g.slot + ty * R + i;
#pragma unroll
      for (int c = 0; c < C; ++c)
        *reinterpret_cast<float4*>(a.acc + r * D + 64 * c + 4 * tx) =
            make_float4(acc[i][4 * c], acc[i][4 * c + 1], acc[i][4 * c + 2], acc[i][4 * c + 3]);
      if (tx == 0) a.ml[r] = make_float2(m[i], l[i]);
    }
  }

  static constexpr size_t kSmem = ((64 + 2 * kKeys) * kStride + 64 * kPStride) * sizeof(float);
};

template <int D, typename TQ, typename TKV>
__global__ void __launch_bounds__(kThreads, 2) fp32_kernel(const __grid_constant__ PrefixArgs a) {
  extern __shared__ float smem[];
  __shared__ int share[kThreads / 32 + 4];
  pdl_wait();
  pdl_release();
  using Tile = Fp32Tile<D, TQ, TKV>;
  Walk w = find_share(a, blockIdx.x, kThreads, share);
  Segment g;
  while (w.next(a, blockIdx.x, &g)) {
    if ((g.kind == kOwn ? a.s.own_tile : a.s.prefix_tile) == 16)
      Tile::template segment<16>(a, g, smem);
    else
      Tile::template segment<64>(a, g, smem);
  }
}

// ---------------------------------------------------------------- join
//
// One CTA for up to four rows of a sequence and head: its warps take the rows' partial results in turn (finding one
// takes longer than reading it, and it is found for all the rows at once), rescale by the maxima and
// add (fp32); the order is fixed, so the result does not depend on timing.  Bound: latency of a row's parts, which the
// warps read two at a time each, after the division that finds them.  An item leaves one part for each CTA that it is cut
// over, times streams and quarters (8) for up to 32 rows on the tensor cores: 30 or so where there are many items, but 148 x 8
// for one.  2,048 rows of 128 on a 131,072-token prefix: 14 of 200 us; one sequence of 131,072 tokens on one KV head (4 rows,
// one CTA here): 85 us in all, where its keys and values take 10.
constexpr int kJoinWarps = 8, kJoinRows = 4, kAtOnce = 2;

template <int D>
struct Joined {
  static constexpr int N = D / 32;  // columns of a lane
  float m = -INFINITY, l = 0.f, acc[N];
  __device__ __forceinline__ Joined() {
#pragma unroll
    for (int c = 0; c < N; ++c) acc[c] = 0.f;
  }
  template <int K>
  __device__ __forceinline__ void add(const float2 (&ml)[K], const float (&x)[K][N]) {
    float top = m;
#pragma unroll
    for (int k = 0; k < K; ++k) top = fmaxf(top, ml[k].x);
    // (not left out if it is -inf: the sum of scores that are all NaN is NaN, and has to come through)
    const float base = top == -INFINITY ? 0.f : top;
    float f = exp2f(m - base);
    m = top;
    l *= f;
#pragma unroll
    for (int c = 0; c < N; ++c) acc[c] *= f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      f = exp2f(ml[k].x - base);
      l += ml[k].y * f;
#pragma unroll
      for (int c = 0; c < N; ++c) acc[c] += x[k][c] * f;
    }
  }
};

// The CTA whose share of T holds position x.
__device__ __forceinline__ int cta_of(int x, int T, int ctas) {
  const int each = T / ctas, more = T - each * ctas, bent = more * (each + 1);
  return x < bent ? x / (each + 1) : more + (x - bent) / each;
}

template <int D, typename TO>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ PrefixArgs a) {
  using J = Joined<D>;
  __shared__ float s_acc[kJoinRows][kJoinWarps][D];
  __shared__ float2 s_ml[kJoinRows][kJoinWarps];
  pdl_wait();
  pdl_release();
  const PrefixShape& s = a.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunks = (s.rows + kJoinRows - 1) / kJoinRows;
  const int bh = blockIdx.x / chunks, head = bh % s.heads, b = bh / s.heads;
  const int rem = (blockIdx.x - bh * chunks) * kJoinRows, rows = min(kJoinRows, s.rows - rem);  // row tiles are multiples of 4 rows
  const int group = s.heads * s.own_tiles;
  const int before = a.cum[b], all = a.cum[s.batch], len = a.cum[s.batch + 1 + b];
  const bool lost = (*a.v.err & kDevErrTimeout) != 0;
  const int T = s.prefix_total + all * group;
  J sum[kJoinRows];
  // the partial results of the segments of an item of n key tiles of cost w from `start`: `parts` rows
  // `step` apart of each stream that took part
  auto item = [&](int start, int n, int w, int streams, int parts, long long slot0, int slot_rows, int step) {
    const int c0 = cta_of(start, T, s.ctas), c1 = cta_of(start + (n - 1) * w, T, s.ctas);
    const int each = streams * parts, count = (c1 - c0 + 1) * each;
    for (int i0 = warp; i0 < count; i0 += kJoinWarps * kAtOnce) {
      float2 ml[kJoinRows][kAtOnce];
      float x[kJoinRows][kAtOnce][J::N];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int i = i0 + u * kJoinWarps, y = i / each, c = c0 + y, k = i - y * each;
        const int lo = share_start(c, T, s.ctas), hi = share_start(c + 1, T, s.ctas);
        const bool there = i < count && tiles_before(hi, start, n, w) - tiles_before(lo, start, n, w) > (parts == 1 ? k : k / parts);
        const long long row = slot0 + (long long)c * slot_rows + k * step;
#pragma unroll
        for (int r = 0; r < kJoinRows; ++r) {
          ml[r][u] = make_float2(-INFINITY, 0.f);
#pragma unroll
          for (int q = 0; q < J::N; ++q) x[r][u][q] = 0.f;
          if (!there || r >= rows) continue;
          ml[r][u] = a.ml[row + r];
          const float* p = a.acc + (row + r) * D + J::N * lane;
          if constexpr (D == 128) {
            const float4 z = *reinterpret_cast<const float4*>(p);
            x[r][u][0] = z.x, x[r][u][1] = z.y, x[r][u][2] = z.z, x[r][u][3] = z.w;
          } else {
            const float2 z = *reinterpret_cast<const float2*>(p);
            x[r][u][0] = z.x, x[r][u][1] = z.y;
          }
        }
      }
#pragma unroll
      for (int r = 0; r < kJoinRows; ++r) sum[r].add(ml[r], x[r]);
    }
  };
  if (s.prefix > 0) {
    int rt, r;
    if (s.seqs_per_tile) {
      rt = b / s.seqs_per_tile;
      r = b % s.seqs_per_tile * s.rows + rem;
    } else {
      rt = b * s.tiles_per_seq + rem / s.prefix_tile;
      r = rem % s.prefix_tile;
    }
    if (rt < 2 * s.duals) {
      const int x = head * s.duals + (rt >> 1);
      item(x * s.prefix_keys * kDualCost, s.prefix_keys, kDualCost, 1, 1, (long long)x * s.dual_slot_rows + (rt & 1) * s.prefix_tile + r, s.dual_slot_rows, 0);
    } else {
      const int x = head * s.singles + rt - 2 * s.duals;
      item(s.dual_total + x * s.prefix_keys * s.single_cost, s.prefix_keys, s.single_cost, s.streams, s.prefix_parts, s.single_slot0 + (long long)x * s.single_slot_rows + r, s.single_slot_rows,
           s.single_slot_rows / (s.streams * s.prefix_parts));
    }
  }
  const int n = own_key_tiles(s, len);
  if (n > 0) {
    const int x = head * s.own_tiles + rem / s.own_tile;
    item(s.prefix_total + before * group + x * own_cost(s, len) + kOwnStart, n, kTileCost, s.streams, s.own_parts,
         s.own_slot0 + ((long long)b * group + x) * s.own_slot_rows + rem % s.own_tile, s.own_slot_rows,
         s.own_slot_rows / (s.streams * s.own_parts));
  }
#pragma unroll
  for (int r = 0; r < kJoinRows; ++r) {
    if (lane == 0) s_ml[r][warp] = make_float2(sum[r].m, sum[r].l);
#pragma unroll
    for (int c = 0; c < J::N; ++c) s_acc[r][warp][lane * J::N + c] = sum[r].acc[c];
  }
  __syncthreads();
  if (warp >= rows) return;
  float2 ml[kJoinWarps];
  float x[kJoinWarps][J::N];
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) {
    ml[i] = s_ml[warp][i];
#pragma unroll
    for (int c = 0; c < J::N; ++c) x[i][c] = s_acc[warp][i][lane * J::N + c];
  }
  J row;
  row.add(ml, x);
  const bool sees = tokens_seen(s, len, (rem + warp) % s.nq) > 0;
  TO* O = static_cast<TO*>(a.O) + ((size_t)bh * s.rows + rem + warp) * D + lane * J::N;
#pragma unroll
  for (int c = 0; c < J::N; ++c) {
    const float y = lost ? NAN : sees ? row.acc[c] / row.l : 0.f;
    if constexpr (sizeof(TO) == 2)
      O[c] = f32_to_bf16_bits(y);
    else
      O[c] = y;
  }
}

// ---------------------------------------------------------------- host

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

template <int D, typename TQ, typename TKV>
cudaError_t launch_fp32(const zha_pages* p, const PrefixArgs& a, cudaStream_t s) {
  const size_t smem = Fp32Tile<D, TQ, TKV>::kSmem;
  const cudaError_t e = allow_shared<fp32_kernel<D, TQ, TKV>>(p, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(fp32_kernel<D, TQ, TKV>, dim3(a.s.ctas), dim3(kThreads), smem, s, a);
}

template <int D>
cudaError_t launch_fp32_types(const zha_pages* p, const PrefixArgs& a, zha_dtype q, zha_dtype kv, cudaStream_t s) {
  if (q == ZHA_F32) return kv == ZHA_F32 ? launch_fp32<D, float, float>(p, a, s) : launch_fp32<D, float, uint16_t>(p, a, s);
  return launch_fp32<D, uint16_t, float>(p, a, s);
}

template <int D>
cudaError_t launch_join(const PrefixArgs& a, zha_dtype o, cudaStream_t s) {
  const dim3 grid((unsigned)((long long)a.s.batch * a.s.heads * ceil_div(a.s.rows, kJoinRows))), block(kJoinWarps * 32);
  return o == ZHA_BF16 ? launch_pdl(join_kernel<D, uint16_t>, grid, block, 0, s, a)
                       : launch_pdl(join_kernel<D, float>, grid, block, 0, s, a);
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The cut of a call.  Returns false on sizes outside the kernels' index ranges.
// wide: tensor kernel with an fp32 output.
bool plan(const zha_pages* p, int batch, int q_heads, int nq, long long prefix, bool tensor, bool wide, PrefixShape* s) {
  const int heads = p->desc.kv_heads;
  if (batch < 1 || nq < 1 || q_heads < 1 || q_heads % heads) return false;
  const long long rows = (long long)(q_heads / heads) * nq;
  if (rows > 1 << 20 || (long long)batch * heads * rows > 1LL << 30 || batch > 1 << 20) return false;
  *s = PrefixShape{};
  s->batch = batch;
  s->heads = heads;
  s->rows = (int)rows;
  s->nq = nq;
  s->prefix = (int)prefix;
  s->tile_keys = !tensor ? kKeys : wide ? 64 : 128;
  // fp32: 16 rows at a time where there are no more, else 64 (the arithmetic is per tile row)
  s->prefix_tile = tensor ? 128 : rows * batch <= 16 ? 16 : 64;
  s->own_tile = tensor ? 128 : rows <= 16 ? 16 : 64;
  int row_tiles;
  if (rows <= s->prefix_tile) {
    s->seqs_per_tile = s->prefix_tile / (int)rows;
    row_tiles = ceil_div(batch, s->seqs_per_tile);
  } else {
    s->tiles_per_seq = ceil_div(rows, s->prefix_tile);
    row_tiles = batch * s->tiles_per_seq;
  }
  s->duals = tensor ? row_tiles / 2 : 0;
  s->singles = row_tiles - 2 * s->duals;
  s->streams = tensor ? 2 : 1;
  s->own_tiles = ceil_div(rows, s->own_tile);
  s->prefix_keys = ceil_div(prefix, s->tile_keys);
  // up to 32 rows fill one warp's lanes of TMEM; the tensor kernel then lets each of a stream's four
  // warps weigh a quarter of the keys and leaves four partial results
  s->prefix_parts = tensor && rows * batch <= 32 ? 4 : 1;
  s->own_parts = tensor && rows <= 32 ? 4 : 1;
  s->ctas = tensor ? p->sms : 2 * p->sms;
  // all costs, sequences as long as they may be, are counted in 31 bits
  const long long most = (long long)p->desc.max_seq_pages * p->desc.page_tokens;
  // fp32: the arithmetic of 64 rows takes about three times that of 16
  s->single_cost = !tensor && s->prefix_tile > s->own_tile ? 3 * kTileCost : kTileCost;
  if ((long long)heads * row_tiles * s->prefix_keys * (kDualCost + s->single_cost) +
          (long long)batch * heads * s->own_tiles * (ceil_div(most, s->tile_keys) * kTileCost + kOwnStart) > 0x7fffffffLL)
    return false;
  s->dual_total = heads * s->duals * s->prefix_keys * kDualCost;
  s->prefix_total = s->dual_total + heads * s->singles * s->prefix_keys * s->single_cost;
  s->dual_slot_rows = 2 * s->prefix_tile;
  const int single_rows = s->prefix_parts == 4 ? (int)rows * batch : s->prefix_tile;
  s->single_slot_rows = s->streams * s->prefix_parts * single_rows;
  s->own_slot_rows = s->streams * s->own_parts * (int)(rows < s->own_tile ? rows : s->own_tile);
  const long long shared = prefix > 0;
  s->single_slot0 = shared && s->duals ? ((long long)s->duals * heads + s->ctas) * s->dual_slot_rows : 0;
  s->own_slot0 = s->single_slot0 + (shared && s->singles ? ((long long)s->singles * heads + s->ctas) * s->single_slot_rows : 0);
  return true;
}

// bf16 against bf16 runs on the tensor cores at any size: their tiles cost less than the bytes even when
// a tile is mostly empty.
bool tensor_path(const zha_pages* p, zha_dtype q) { return q == ZHA_BF16 && p->desc.kv_dtype == ZHA_BF16; }

struct Scratch {
  size_t cum, ml, acc, bytes;
};

Scratch scratch_of(const zha_pages* p, const PrefixShape& s) {
  const long long rows =
      s.own_slot0 + ((long long)s.batch * s.heads * s.own_tiles + s.ctas) * s.own_slot_rows;
  Scratch x;
  x.cum = 0;
  x.ml = ((size_t)(2 * s.batch + 1) * 4 + 255) / 256 * 256;
  x.acc = x.ml + ((size_t)rows * 8 + 255) / 256 * 256;
  x.bytes = x.acc + (size_t)rows * p->desc.head_dim * 4;
  return x;
}

}  // namespace

extern "C" {

size_t zha_prefix_attn_scratch_bytes(const zha_pages* p, int batch, int q_heads, int nq, long long prefix_tokens) {
  if (!p || prefix_tokens < 0 || prefix_tokens > 1LL << 30) return 0;
  PrefixShape s;
  size_t most = 0;
  for (int kind = 0; kind < 3; ++kind) {  // whatever the queries' and the output's type, if they can be planned
    if (kind && p->desc.kv_dtype != ZHA_BF16) break;
    if (!plan(p, batch, q_heads, nq, prefix_tokens, kind > 0, kind > 1, &s)) continue;
    const size_t n = scratch_of(p, s).bytes;
    if (n > most) most = n;
  }
  return most;
}

zha_status zha_prefix_attn_decode(const zha_pages* p, const void* d_Q, zha_dtype q_dtype, int batch, int q_heads, int nq,
                                  const void* d_K, const void* d_V, const int* d_seqs, int prefix_seq,
                                  long long prefix_tokens, int causal, float scale, void* d_O, zha_dtype o_dtype,
                                  void* d_scratch, size_t scratch_bytes, void* stream) {
  if (!p || batch < 0 || q_heads < 1 || nq < 0) return ZHA_ERR_INVALID_ARG;
  if ((q_dtype != ZHA_F32 && q_dtype != ZHA_BF16) || (o_dtype != ZHA_F32 && o_dtype != ZHA_BF16))
    return ZHA_ERR_INVALID_ARG;
  if (q_heads % p->desc.kv_heads != 0 || !std::isfinite(scale)) return ZHA_ERR_INVALID_ARG;
  if (prefix_tokens < 0 || prefix_tokens % p->desc.page_tokens != 0) return ZHA_ERR_INVALID_ARG;
  if (prefix_tokens > (long long)p->desc.max_seq_pages * p->desc.page_tokens) return ZHA_ERR_CAPACITY;
  if (prefix_tokens > 0 && (prefix_seq < 0 || prefix_seq >= p->desc.max_seqs)) return ZHA_ERR_INVALID_ARG;
  if (!on_device(p)) return ZHA_ERR_INVALID_ARG;
  if (batch == 0 || nq == 0) return ZHA_OK;
  if (!d_Q || !d_K || !d_V || !d_seqs || !d_O || !d_scratch) return ZHA_ERR_INVALID_ARG;
  if (!aligned(d_Q, 16) || !aligned(d_K, 16) || !aligned(d_V, 16) || !aligned(d_O, 16) || !aligned(d_seqs, 4) ||
      !aligned(d_scratch, 16))
    return ZHA_ERR_INVALID_ARG;
  PrefixArgs a;
  const bool tensor = tensor_path(p, q_dtype);
  if (!plan(p, batch, q_heads, nq, prefix_tokens, tensor, o_dtype == ZHA_F32, &a.s)) return ZHA_ERR_UNSUPPORTED;
  const Scratch x = scratch_of(p, a.s);  // of the plan that will run
  if (scratch_bytes < x.bytes) return ZHA_ERR_INVALID_ARG;
  char* base = static_cast<char*>(d_scratch);
  a.s.causal = causal != 0;
  a.s.prefix_seq = prefix_tokens > 0 ? prefix_seq : 0;
  a.v = p->v;
  a.Q = d_Q;
  a.K = d_K;
  a.V = d_V;
  a.seqs = d_seqs;
  a.cum = reinterpret_cast<int*>(base + x.cum);
  a.ml = reinterpret_cast<float2*>(base + x.ml);
  a.acc = reinterpret_cast<float*>(base + x.acc);
  a.O = d_O;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.wait_cycles = p->wait_limit > 0 ? p->wait_limit : kCopyWaitCycles;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int d = p->desc.head_dim;
  cudaError_t e = tensor    ? launch_prefix_tc(p, a, d, o_dtype == ZHA_F32, s)
                  : d == 64 ? launch_fp32_types<64>(p, a, q_dtype, p->desc.kv_dtype, s)
                            : launch_fp32_types<128>(p, a, q_dtype, p->desc.kv_dtype, s);
  if (e == cudaSuccess) e = d == 64 ? launch_join<64>(a, o_dtype, s) : launch_join<128>(a, o_dtype, s);
  count_launches(p, 2);
  return e == cudaSuccess ? ZHA_OK : ZHA_ERR_CUDA;
}

}  // extern "C"
