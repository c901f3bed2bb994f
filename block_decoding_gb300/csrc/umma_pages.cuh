// What the attention kernels over the paged cache use of barriers, asynchronous
// copies and tensor cores beside umma.cuh.
#pragma once

#include "umma.cuh"

namespace dllm {

// named_bar_sync that tells whether `pred` holds for any of the threads.
__device__ __forceinline__ bool bar_any(uint32_t id, uint32_t count, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(count), "r"(static_cast<uint32_t>(pred))
      : "memory");
  return r != 0;
}

// Give up or take registers, for a whole warpgroup: N a thread afterwards.
// The groups' shares must not add up to more than the launch gave the CTA.
template <int N>
__device__ __forceinline__ void reg_dealloc() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_alloc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// mbar_wait by a whole warp that has to stay together.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}

// Bounded wait that no abort cuts short: for copies already in flight.
__device__ __forceinline__ void mbar_drain(uint64_t *bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity) && clock64() - t0 < kWaitLimitCycles) {
  }
}

// The 128-byte line at p into L2.
__device__ __forceinline__ void l2_prefetch_line(const void *p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<uint64_t>(p)));
}

// Untiled load of `bytes` (a multiple of 16; both addresses 16-byte aligned).
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// 16 bytes of shared memory, loaded where this stands among other such
// statements (the compiler does not bring it forward).
__device__ __forceinline__ float4 load_shared4(const float4 *p) {
  float4 f;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w)
               : "r"(smem_u32(p)));
  return f;
}

// 4-D tiled load of the box at (0, 0, 0, w).
__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %2, %2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// 16 bytes from global to shared memory without registers (zeros if !there);
// copies_wait: the thread's copies have landed.
__device__ __forceinline__ void copy16(void *dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
               :: "r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}
// copies_arrive: one arrival on `bar` when they have (the barrier's count
// includes it).
__device__ __forceinline__ void copies_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// True in one lane of the (converged) warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// D[tmem] (+)= A[smem] * B[smem]^T, kind::f8f6f4 (8-bit floats in, fp32
// accumulate), K = 32 per instruction.
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// Descriptor of an operand written by threads without swizzle: 128-byte core
// matrices of 8 rows x 16 bytes.
//   K-major operand : row = one M/N index, 16 bytes along K; the next 16 bytes
//                     of K are LBO away, the next 8 M/N indices SBO.
//   MN-major operand: row = one K index, 16 bytes along M/N; the next 8 K
//                     indices are LBO away, the next 16 bytes of M/N SBO.
__device__ __forceinline__ uint64_t plain_desc(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
  return sw128_desc(saddr, lbo_bytes, sbo_bytes) & ~(7ull << 61);
}

// The same as sw128_desc for rows of 64 bytes under the 64-byte swizzle
// (atoms of 8 rows x 64 bytes, 512-byte aligned).
__device__ __forceinline__ uint64_t sw64_desc(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
  return plain_desc(saddr, lbo_bytes, sbo_bytes) | (4ull << 61);
}

// Instruction descriptor of tcgen05.mma kind::f8f6f4: 8-bit A and B of the
// given formats, fp32 D, operand majorness (0 = K-major, 1 = MN-major).
constexpr uint32_t kE4M3 = 0, kE5M2 = 1;
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, uint32_t a_type, uint32_t b_type, int a_mn, int b_mn) {
  return (1u << 4) | (a_type << 7) | (b_type << 10) | (static_cast<uint32_t>(a_mn) << 15) |
         (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Tensor map over the rows of a page pool (`rows` rows of `dh` elements of
// `elem_bytes` = 1 or 2; rows a multiple of 8): one box is `box_rows` rows,
// laid out in shared memory as 8-row groups, each holding its 128-byte column
// pieces (8 rows x 128 bytes, swizzled) one after the other. The last
// coordinate counts 8-row groups; groups beyond the pool read as zeros.
bool make_tmap_page_rows(CUtensorMap *map, const void *base, uint64_t rows, int dh, int elem_bytes, uint32_t box_rows);

// Tensor map over query rows [rows][heads][dh] bf16, `stride` elements (a
// multiple of 8) from row to row: one box is 64 elements of `box_heads` heads of
// `box_rows` rows, laid out in shared memory as one 128-byte row (swizzled) per
// head after the other. Rows beyond the last read as zeros.
bool make_tmap_query_rows(CUtensorMap *map, const void *q, uint64_t rows, int heads, int dh, long long stride,
                          uint32_t box_heads, uint32_t box_rows);

}  // namespace dllm
