// The paged K/V cache as the kernels see it: page and slot of a position,
// argument checks shared by the entry points, and the 8-bit row format.
#pragma once

#include "common.cuh"

namespace dllm {

uint32_t status_kv(bool clear);
uint32_t status_paged(bool clear);
uint32_t status_rope(bool clear);
uint32_t status_tree(bool clear);
uint32_t status_mass(bool clear);
uint32_t status_evict(bool clear);

struct KvPages {
  uint8_t *k, *v;                  // [num_pages][heads][page_size][dh], bf16 or e4m3
  uint8_t *k_scale, *v_scale;      // [num_pages][heads][page_size], or null (bf16)
  int num_pages, heads, page_shift;
  const int32_t *table;            // [B][max_pages]
  int max_pages;
};

// Cache row of head 0 at position u of request i, as an index over
// [num_pages][heads][page_size] (the row of head h: + h << page_shift);
// -1 when the table or the pool does not hold it.
__device__ __forceinline__ int page_row(const KvPages &c, int i, int u) {
  const int n = u >> c.page_shift;
  if (u < 0 || n >= c.max_pages) return -1;
  const int page = c.table[static_cast<size_t>(i) * c.max_pages + n];
  if (page < 0 || page >= c.num_pages) return -1;
  return ((page * c.heads) << c.page_shift) + (u & ((1 << c.page_shift) - 1));
}

inline dllm_status check_pages(const dllm_kv_pages *p) {
  if (!p) return DLLM_ERR_INVALID_ARG;
  if (p->type != DLLM_KV_BF16 && p->type != DLLM_KV_E4M3) return DLLM_ERR_UNSUPPORTED;
  if (p->dh != 64 && p->dh != 128) return DLLM_ERR_UNSUPPORTED;
  if (p->page_size != 16 && p->page_size != 32 && p->page_size != 64 && p->page_size != 128)
    return DLLM_ERR_UNSUPPORTED;
  if (p->num_pages < 1 || p->heads < 1) return DLLM_ERR_INVALID_ARG;
  if (p->heads > 256) return DLLM_ERR_UNSUPPORTED;
  if (static_cast<long long>(p->num_pages) * p->heads * p->page_size >= (1ll << 31)) return DLLM_ERR_UNSUPPORTED;
  return DLLM_OK;
}

inline dllm_status check_page_pointers(const dllm_kv_pages *p) {
  if (!p->k || !p->v || !aligned16(p->k) || !aligned16(p->v)) return DLLM_ERR_INVALID_ARG;
  if (p->type == DLLM_KV_E4M3 && (!p->k_scale || !p->v_scale || !aligned16(p->k_scale) || !aligned16(p->v_scale)))
    return DLLM_ERR_INVALID_ARG;
  return DLLM_OK;
}

inline KvPages device_pages(const dllm_kv_pages *p, const int32_t *table, int max_pages) {
  KvPages c{};
  c.k = static_cast<uint8_t *>(p->k);
  c.v = static_cast<uint8_t *>(p->v);
  c.k_scale = p->type == DLLM_KV_E4M3 ? p->k_scale : nullptr;
  c.v_scale = p->type == DLLM_KV_E4M3 ? p->v_scale : nullptr;
  c.num_pages = p->num_pages;
  c.heads = p->heads;
  c.page_shift = p->page_size == 16 ? 4 : p->page_size == 32 ? 5 : p->page_size == 64 ? 6 : 7;
  c.table = table;
  c.max_pages = max_pages;
  return c;
}

// Two e4m3 codes (low byte first) -> two floats, exactly.
__device__ __forceinline__ float2 e4m3x2_to_f32(uint16_t v) {
  uint32_t h;   // f16x2 holds every e4m3 value
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  float2 f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// Two floats -> two e4m3 codes (nearest even, clamped to +-448; NaN stays NaN).
__device__ __forceinline__ uint16_t f32_to_e4m3x2(float a, float b) {
  uint16_t p;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(p) : "f"(b), "f"(a));
  return p;
}

// The scale that a byte stands for: 2^(byte - 127), and NaN for 255.
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float((byte << 23) | (byte == 255 ? 0x400000u : 0u)); }

// Four codes (lowest byte first) -> four bf16 in the order 0, 2, 1, 3, exactly
// (NaN codes, which no row holds, become +-480). A code's exponent and
// mantissa bits are put where bf16 has its lowest exponent and highest
// mantissa bits; the product with 2^120 makes up for the exponent bias and
// turns subnormal codes into normal numbers. Nine integer and packed-half
// operations: conversions through half and float cost twice the time.
__device__ __forceinline__ uint2 e4m3x4_to_bf16_0213(uint32_t w) {
  uint32_t even = ((w << 4) & 0x07f007f0u) | ((w << 8) & 0x80008000u);
  uint32_t odd = ((w >> 4) & 0x07f007f0u) | (w & 0x80008000u);
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(even) : "r"(0x7b807b80u));
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(odd) : "r"(0x7b807b80u));
  return make_uint2(even, odd);
}

// Exponent byte of a row with the largest magnitude bits `a` (finite bf16):
// the least e >= -117 with |x| <= 448 * 2^e, + 127. 448 = 1.75 * 2^8, and
// |x| = (1 + m / 128) * 2^((a >> 7) - 127).
__device__ __forceinline__ int scale_byte(uint32_t a) {
  const int b = static_cast<int>(a >> 7) - 8 + ((a & 127) > 96 ? 1 : 0);
  return min(max(b, 10), 247);
}

// Largest magnitude bits among eight bf16 and the halves of m.
__device__ __forceinline__ uint32_t max_mag(const uint4 &u, uint32_t m) {
  m = __vmaxu2(m, u.x & 0x7fff7fffu);
  m = __vmaxu2(m, u.y & 0x7fff7fffu);
  m = __vmaxu2(m, u.z & 0x7fff7fffu);
  return __vmaxu2(m, u.w & 0x7fff7fffu);
}

// Eight bf16 of a row whose largest magnitude has the bits m, scaled by a
// power of two into (224, 448], as two e4m3 parts: hi = rn(x), lo = rn(x - hi).
// Returns the byte of the power of two that undoes the scaling.
__device__ __forceinline__ int split_e4m3(const uint4 &u, uint32_t m, uint2 &hi, uint2 &lo) {
  const int byte = scale_byte(m);
  const float f = __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);
  float x[8];
  unpack8(u, x);
  uint32_t h[4], r[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float p = x[2 * e] * f, q = x[2 * e + 1] * f;
    const uint16_t hh = f32_to_e4m3x2(p, q);
    const float2 b = e4m3x2_to_f32(hh);
    h[e] = hh;
    r[e] = f32_to_e4m3x2(p - b.x, q - b.y);
  }
  hi = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  lo = make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
  return byte;
}

// Packed bf16 product, and a value that bf16 holds in both halves.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
  return a;
}
__device__ __forceinline__ uint32_t bf16x2_of(float f) {
  const uint32_t b = __float_as_uint(f) >> 16;
  return b | (b << 16);
}

// The lowest n bits (none for n <= 0, all from 32 on).
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

}  // namespace dllm
