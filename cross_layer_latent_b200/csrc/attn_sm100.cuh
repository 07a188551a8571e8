// attn_sm100.cuh -- tensor-memory and matrix-descriptor pieces that the
// attention kernels share.
#pragma once

#include <cuda_bf16.h>

#include "sm100.cuh"

namespace li {

// Shared-memory operands are 128-byte swizzled, in two orders.  K-major: an
// atom is 8 rows of 64 bf16, 1024 bytes (sbo) apart along the rows, lbo
// unused.  MN-major: an atom is 8 rows of K, each 64 bf16 along MN; 1024 bytes
// (sbo) step along K, `lbo` bytes to the next 64 along MN.
// Instruction descriptor bits of operands stored with MN contiguous.
constexpr uint32_t kMajorMnA = 1u << 15, kMajorMnB = 1u << 16;

// Descriptor words of a 128-byte-swizzled operand: the low word holds the
// address (in 16-byte units) and lbo, the high word the rest, which is the
// same for every tile.  Steps within a tile add to the low word alone, which
// keeps the issuing thread's work per MMA to a few instructions.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr >> 4) & 0x3FFFu) | (((lbo >> 4) & 0x3FFFu) << 16);
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);   // sbo 1024, version 1, 128-byte swizzle

// D += A B over STEPS steps of 16 along K, both operands in shared memory;
// a_step and b_step are the steps of the low words.  The first step of all
// overwrites D where `accumulate` is 0.
template <int STEPS, int A_STEP, int B_STEP>
__device__ __forceinline__ void umma_ss_steps(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo + k * A_STEP), "r"(b_lo + k * B_STEP), "r"(idesc), "r"(k == 0 ? accumulate : 1u), "n"(kDescHi)
        : "memory");
  }
}

// The same with A in tensor memory (8 columns of packed pairs a step).
template <int STEPS, int B_STEP>
__device__ __forceinline__ void umma_ts_steps(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "mov.b64 b, {%2, %5};\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem + k * 8), "r"(b_lo + k * B_STEP), "r"(idesc), "r"(k == 0 ? accumulate : 1u), "n"(kDescHi)
        : "memory");
  }
}

// ---- pairs of CTAs (cta_group::2): one MMA over both SMs' tensor cores.  The
// M rows of A and D are split between the pair, B's N rows likewise, each CTA
// holding its part at the same shared- and tensor-memory addresses; the even
// CTA issues.

template <int STEPS, int A_STEP, int B_STEP>
__device__ __forceinline__ void umma2_ss_steps(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo + k * A_STEP), "r"(b_lo + k * B_STEP), "r"(idesc), "r"(k == 0 ? accumulate : 1u), "n"(kDescHi)
        : "memory");
  }
}

template <int STEPS, int B_STEP>
__device__ __forceinline__ void umma2_ts_steps(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "mov.b64 b, {%2, %5};\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem + k * 8), "r"(b_lo + k * B_STEP), "r"(idesc), "r"(k == 0 ? accumulate : 1u), "n"(kDescHi)
        : "memory");
  }
}

// Arrive on the barrier at this offset in both CTAs when every MMA issued so
// far has completed.
__device__ __forceinline__ void umma2_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_addr(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
__device__ __forceinline__ void tmem2_alloc(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst_smem)), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem2_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// All threads of both CTAs, their earlier shared-memory operations on each
// other included.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Barriers of the pair live in the even CTA; `bar` is a shared::cluster
// address (cluster_addr).  Arrivals that hand over nothing but tensor memory
// (ordered by the tcgen05 fences) or byte counts are relaxed: a release at
// cluster scope takes about 1300 cycles.
__device__ __forceinline__ void mbar_arrive_relaxed_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_release_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx_at(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// Tile loads into this CTA's memory that complete on a barrier of the pair.
__device__ __forceinline__ void tma2_load_2d(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void tma2_load_3d(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// bounded_wait on a barrier that the other CTA arrives on too.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool bounded_wait_cluster(uint64_t* bar, uint32_t parity, const WaitCtl& w) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = cycles();
  for (;;) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if (*w.abort_flag) return false;
    if (cycles() - t0 > w.limit_ns * kCyclesPerNs) return give_up(w);
  }
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// C consecutive fp32 columns of this warp's 32 lanes; tmem_wait_ld() before
// the registers are used.
template <int C>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[C]) {
  static_assert(C == 8 || C == 16 || C == 32, "8, 16 or 32 columns");
  if constexpr (C == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
  } else if constexpr (C == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
  }
}

template <int C>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[C]) {
  static_assert(C == 8 || C == 16 || C == 32, "8, 16 or 32 columns");
  if constexpr (C == 8) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
  } else if constexpr (C == 16) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
  } else {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
  }
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Largest value over the warp's lanes.
__device__ __forceinline__ float warp_max_f32(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// 2^x to 2^-22 of the value (one special-function instruction; -inf gives 0).
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Paired fp32 arithmetic (one instruction for two IEEE operations).
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The larger of two values, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 2^x of a pair on the FMA pipes, for x <= 100: x = n + r with |r| <= 1/2, a
// polynomial for 2^r and n added to its exponent.  The coefficients are the
// best of degree 4 for the relative error on [-1/2, 1/2] (a Remez exchange):
// 2.7e-6 at most, 1.6e-6 on average, a thousandth of the rounding to bf16 that
// follows.  x below -126 counts as -126.  NaN gives 3.4e38: the exponent that is
// added to the canonical NaN 0x7FFFFFFF is its own lowest bits.
__device__ __forceinline__ float2 exp2_poly(uint64_t x) {
  float2 v = unpair(x);
  const uint64_t y = pair(max_nan(v.x, -126.f), max_nan(v.y, -126.f));
  const uint64_t big = pair(12582912.f, 12582912.f), less = pair(-12582912.f, -12582912.f);   // 1.5 * 2^23: rounds to whole
  const uint64_t n = add2(y, big);
  const uint64_t whole = add2(n, less);
  const uint64_t r = fma2(whole, pair(-1.f, -1.f), y);
  uint64_t p = fma2(pair(0.009570102207362652f, 0.009570102207362652f), r, pair(0.05591785907745361f, 0.05591785907745361f));
  p = fma2(p, r, pair(0.240247443318367f, 0.240247443318367f));
  p = fma2(p, r, pair(0.6931217908859253f, 0.6931217908859253f));
  p = fma2(p, r, pair(0.9999992847442627f, 0.9999992847442627f));
  const float2 m = unpair(p), e = unpair(n);
  return make_float2(__int_as_float(__float_as_int(m.x) + (__float_as_int(e.x) << 23)),
                     __int_as_float(__float_as_int(m.y) + (__float_as_int(e.y) << 23)));
}

// At least `ns` nanoseconds on an SM.
__device__ __forceinline__ void delay_ns(uint64_t ns) {
  const uint64_t t0 = cycles();
  while (cycles() - t0 < ns * kCyclesPerNs) __nanosleep(1000);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Whether `x` holds in any of the `count` threads of named barrier `id`.
__device__ __forceinline__ bool named_bar_any(int id, int count, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(count), "r"(static_cast<uint32_t>(x))
      : "memory");
  return r != 0;
}

}  // namespace li
