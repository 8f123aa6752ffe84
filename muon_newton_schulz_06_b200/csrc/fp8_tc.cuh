// Tensor-core primitives of the block-scaled 8-bit products (tcgen05 kind::mxf8f6f4 with
// scales in tensor memory), shared by the kernels of k_fp8_gemm.cu.
//
// The instruction multiplies A (rows x 32 codes) and B (columns x 32 codes) and scales
// each row's and column's 32-code product by 2^(byte - 127), one byte each.  A block of
// 128 of the format is four such steps with the same bytes.  A 32-bit word of tensor
// memory holds four bytes per row, and the instruction descriptor picks one of them: here
// byte q of the word is the scale of the q-th block of 128 within a group of 512 codes,
// so scales move to tensor memory once per 512 codes.
//
// 128 rows of words are 512 bytes: row r at lane r % 32, word r / 32, copied from shared
// memory as 32 lanes x 16 bytes and replicated to the four lane quadrants.
#pragma once

#include "fp8_internal.h"
#include "tc_primitives.cuh"

namespace muon {
namespace {

constexpr int kF8K = 128;        // k-block: one scale block, one 128-byte swizzle row
constexpr int kF8Group = 4;      // k-blocks per word of scales
constexpr uint32_t kF8SfBytes = 512;  // words of 128 rows

// Instruction descriptor: D f32, UE8M0 scales; the scale bytes' index goes in per step.
__host__ __device__ constexpr uint32_t f8_idesc(bool a_e5m2, bool b_e5m2, bool a_mn, bool b_mn, int m, int n) {
  return ((a_e5m2 ? 1u : 0u) << 7) | ((b_e5m2 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(m >> 7) << 27);
}
__device__ __forceinline__ uint32_t f8_idesc_sf(uint32_t idesc, int q) {
  return idesc | ((uint32_t)q << 4) | ((uint32_t)q << 29);
}

// Shared-memory descriptor of a block of scale words: 32 rows of 16 bytes, no swizzle,
// 128 bytes per group of 8 rows.
__device__ __forceinline__ uint64_t f8_sf_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(128u >> 4) << 16;
  d |= (uint64_t)(128u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  return d;
}

__device__ __forceinline__ void f8_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                       uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate));
}

// 512 bytes of scale words to 4 columns of tensor memory, in all four lane quadrants.
__device__ __forceinline__ void f8_copy_sf(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

__device__ __forceinline__ void tma_load_2d_local(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y)
      : "memory");
}

// The forms for a pair of CTAs (one instruction works on both; scale words and code tiles are
// read from each CTA's own shared memory at the same offsets).
__device__ __forceinline__ void f8_mma_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate));
}
__device__ __forceinline__ void f8_copy_sf_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// Copy into this CTA's shared memory, counted on the barrier at `bar_cluster_addr` (the
// leader CTA's).  No multicast.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar_cluster_addr,
                                                 int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster_addr), "r"(x), "r"(y)
      : "memory");
}
// 32 lanes x 32 columns of tensor memory <- registers (tmem_ld32's layout), complete on return.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float* v) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]));
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Waits of the loops that feed the tensor cores.  One thread issues everything for a k-block
// whose products take 512 clocks (pair kernel), so its own instructions count: the test of a
// barrier that is already complete is inlined and takes shared-memory addresses, and only a
// real wait is a call.  (Through the general mbar_wait, with descriptors built per
// instruction, an iteration took 1050 clocks and the tensor cores waited for it.)
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
constexpr long long kF8WaitClocks = 4000000000ll;  // about 2 s at full clock
__device__ __noinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                           long long limit = kF8WaitClocks) {
  const long long t0 = clock64();
  uint32_t n = 0;
  while (true) {
    if (bar_try(bar, parity)) return true;
    if ((++n & 63u) == 0) {
      if (abort_flag != nullptr && *abort_flag) return false;
      if (clock64() - t0 > limit) return false;
    }
  }
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return bar_try(bar, parity) || bar_wait_slow(bar, parity, abort_flag);
}

// Records a wait that ran out: `status` is a page-locked host word.
__device__ __forceinline__ void f8_record_timeout(int* status) {
  *reinterpret_cast<volatile int*>(status) = kDevTimeout;
  __threadfence_system();
}

// Arrives on a barrier of either CTA of the pair to hand over tensor memory that has been
// read.  No release at cluster scope: that waits for the thread's global stores (1,200 clocks
// in the epilogue), which the reader of this barrier does not look at.
__device__ __forceinline__ void arrive_tmem_free(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Commits by shared-memory address: on this CTA's barrier, or at the same offset in both CTAs.
__device__ __forceinline__ void f8_commit_at(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void f8_commit_both_at(uint32_t bar) {
  const uint16_t mask = 0x3;
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}
__device__ __forceinline__ void expect_tx_at(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// True in one lane of the warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok));
  return ok != 0;
}

// Scale words of 128 rows from r0 on, for k-blocks kb0 .. kb0 + 3, four rows per lane; rows and
// k-blocks out of range take 2^0 (their codes are zero).  f8_sf_load issues the loads,
// f8_sf_store puts the words where the copy to tensor memory expects them (512 bytes at dst).
// Lane l has rows l + 32 j, or, where all 128 rows exist (`quads`), rows 4 l + j: their four
// bytes lie together, in one aligned word or two, in the place of four loads (f8_read4).
struct F8SfWords {
  uint32_t w[4];
  bool quads;
};
__device__ __forceinline__ F8SfWords f8_sf_load(const F8Scales& s, int r0, int rows, int kb0, int nkb, int lane) {
  F8SfWords f;
  f.quads = false;
  if (!s.by_row) {
    const uint8_t* p = s.s + (int64_t)(r0 / kFp8Block) * s.s_r + (int64_t)kb0 * s.s_k;
    uint32_t word = 0;
#pragma unroll
    for (int q = 0; q < kF8Group; ++q)
      word |= (uint32_t)((r0 < rows && kb0 + q < nkb) ? p[(int64_t)q * s.s_k] : 127) << (8 * q);
    f.w[0] = f.w[1] = f.w[2] = f.w[3] = word;
    return f;
  }
  const uint8_t* p = s.s + r0 + (int64_t)kb0 * s.s_k;  // s_r is 1
  f.quads = r0 + kFp8Block <= rows;
  if (f.quads) {
    uint32_t x[4];
    const uintptr_t lo = reinterpret_cast<uintptr_t>(s.s), hi = lo + (uintptr_t)((int64_t)nkb * s.s_k);
#pragma unroll
    for (int q = 0; q < kF8Group; ++q) {
      x[q] = 0x7f7f7f7fu;
      if (kb0 + q < nkb)
        x[q] = f8_read4(
            reinterpret_cast<uintptr_t>(p + (int64_t)q * s.s_k + 4 * lane), lo, hi,
            [](uintptr_t a) { return *reinterpret_cast<const uint32_t*>(a); },
            [](uintptr_t a) { return (uint32_t)*reinterpret_cast<const uint8_t*>(a); });
    }
    // byte j of the four loads makes row j's word
    const uint32_t a = __byte_perm(x[0], x[1], 0x5140), b = __byte_perm(x[2], x[3], 0x5140);
    const uint32_t c = __byte_perm(x[0], x[1], 0x7362), d = __byte_perm(x[2], x[3], 0x7362);
    f.w[0] = __byte_perm(a, b, 0x5410);
    f.w[1] = __byte_perm(a, b, 0x7632);
    f.w[2] = __byte_perm(c, d, 0x5410);
    f.w[3] = __byte_perm(c, d, 0x7632);
    return f;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = lane + 32 * j;
    f.w[j] = 0;
#pragma unroll
    for (int q = 0; q < kF8Group; ++q)
      f.w[j] |= (uint32_t)((r0 + r < rows && kb0 + q < nkb) ? p[(int64_t)q * s.s_k + r] : 127) << (8 * q);
  }
  return f;
}
__device__ __forceinline__ void f8_sf_store(uint8_t* dst, const F8SfWords& f, int lane) {
  if (f.quads) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 4 * lane + j;
      *reinterpret_cast<uint32_t*>(dst + (r & 31) * 16 + (r >> 5) * 4) = f.w[j];
    }
  } else {
    *reinterpret_cast<uint4*>(dst + lane * 16) = make_uint4(f.w[0], f.w[1], f.w[2], f.w[3]);
  }
}

// Brings a tensor map (a kernel parameter) into the cache ahead of its first copy.
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

}  // namespace
}  // namespace muon
