// tcgen05 (5th-generation tensor core) and tiled TMA wrappers: one-CTA MMAs on bf16 operands with
// fp32 accumulators in TMEM, operands in shared memory with the 128-byte swizzle, or A in TMEM.
// No cluster multicast anywhere.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "device_common.cuh"

namespace zha {

__device__ __forceinline__ void tmem_alloc(uint32_t* smem_out, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(smem_out)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Arrives on `bar` when every MMA this thread has issued so far is complete.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// One lane of the warp; the compiler knows that the branch it guards is taken by one.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// Lane 0's x: a value that all lanes hold anyway, in a form that can live in a uniform register, which
// is what MMA operands are read from.
template <typename T>
__device__ __forceinline__ T same(T x) { return __shfl_sync(0xffffffffu, x, 0); }

// 128-byte-swizzled operand in shared memory at 16 times addr16.  K-major: rows of 128 bytes (64 elements along
// K) in groups of 8, 1,024 bytes apart; lbo unused.  MN-major: 64 elements along MN by 8 along K
// make a group; lbo is the stride to the next 64 along MN, 1,024 that to the next 8 along K.
__device__ __forceinline__ uint64_t desc_of(uint32_t addr16, uint32_t lbo) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(addr16 | (lbo >> 4) << 16), "r"((1024u >> 4) | (1u << 14) | (2u << 29)));
  return d;
}
// bf16 x bf16 -> fp32, M x N; b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t mma_desc(int m, int n, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}

#define ZHA_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define ZHA_W8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])

// 32 columns of this warp's 32 lanes (lane i of the warp: its own row).
__device__ __forceinline__ void tmem_ld32(uint32_t* r, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : ZHA_R8(r, 0), ZHA_R8(r, 8), ZHA_R8(r, 16), ZHA_R8(r, 24)
      : "r"(addr));
}
// 64 columns of 16 lanes from `addr`'s on, as 8 blocks of 8 columns: block j of thread t is columns 8 j + 2 (t % 4) + 0, 1 of
// lane t / 4 (r[4 j], r[4 j + 1]) and of lane t / 4 + 8 (r[4 j + 2], r[4 j + 3]); four threads hold 32 bytes of a lane.
__device__ __forceinline__ void tmem_ld_blocks(uint32_t* r, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : ZHA_R8(r, 0), ZHA_R8(r, 8), ZHA_R8(r, 16), ZHA_R8(r, 24)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t* r, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : ZHA_R8(r, 0), ZHA_R8(r, 8)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(addr),
      ZHA_W8(r, 0), ZHA_W8(r, 8)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), ZHA_W8(r, 0)
               : "memory");
}
#undef ZHA_R8
#undef ZHA_W8

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// Tiled loads (x times the element size is a multiple of 16 bytes at every call).
__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load4(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kExp2C0 = 0.999924541f, kExp2C1 = 0.693136752f, kExp2C2 = 0.242639482f, kExp2C3 = 0.0558382832f;
// The largest of three, NaN if one of them is.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split(uint64_t x, float* lo, float* hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// 2^x of two floats on the FMA pipes, for x <= 8 or so: x is split into the nearest integer n, read off the low
// bits of x + 1.5 * 2^23, and the rest f in [-1/2, 1/2]; 2^f is a cubic through Chebyshev nodes of
// that interval, off by less than 1.1e-4 of itself; n is added to the exponent.  x below -125 (a masked score) counts as
// -125, and what that gives is taken off all results: exactly zero for those, nothing that others see.  A NaN
// is lost here; the caller's maximum keeps it.
__device__ __forceinline__ void exp2_by_fma(uint64_t x, float* lo, float* hi) {
  float a, b;
  split(x, &a, &b);
  x = pair(fmaxf(a, -125.f), fmaxf(b, -125.f));
  const uint64_t n = add2(x, pair(12582912.f, 12582912.f));
  const uint64_t f = fma2(add2(n, pair(-12582912.f, -12582912.f)), pair(-1.f, -1.f), x);
  uint64_t p = fma2(f, pair(kExp2C3, kExp2C3), pair(kExp2C2, kExp2C2));
  p = fma2(f, p, pair(kExp2C1, kExp2C1));
  p = fma2(f, p, pair(kExp2C0, kExp2C0));
  float na, nb, pa, pb;
  split(n, &na, &nb);
  split(p, &pa, &pb);
  pa = __uint_as_float(__float_as_uint(pa) + (__float_as_uint(na) << 23));
  pb = __uint_as_float(__float_as_uint(pb) + (__float_as_uint(nb) << 23));
  constexpr float least = kExp2C0 * 0x1p-125f;
  split(add2(pair(pa, pb), pair(-least, -least)), lo, hi);
}
// Two floats to bf16 (nearest even): lo in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace zha
