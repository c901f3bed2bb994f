// Rows on their way into the pages of the cache: the request of a row, and the
// 8-bit form of a row that a few neighbouring lanes hold.
#pragma once

#include "pages.cuh"

namespace dllm {

// Request that holds row r (the last i with off[i] <= r), or -1.
__device__ __forceinline__ int request_of(const int32_t *off, int B, int r) {
  int lo = 0, hi = B;   // off[lo] <= r < off[hi]
  if (r < off[0] || r >= off[B]) return -1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= r) lo = mid; else hi = mid;
  }
  return lo;
}

// Eight bf16 -> eight e4m3 codes of x * f.
__device__ __forceinline__ uint2 quantise8(const uint4 &u, float f) {
  // (a product with a power of two is exact in bf16 too, but for what is far
  // below the least code)
  const uint32_t f2 = bf16x2_of(f), x[4] = {u.x, u.y, u.z, u.w};
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t y = mul_bf16x2(x[i], f2);
    w[i] = f32_to_e4m3x2(__uint_as_float(y << 16), __uint_as_float(y & 0xffff0000u));
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// Codes above 240 (they would stand for 2^128 with the largest scale) -> 240.
__device__ __forceinline__ uint32_t cap240(uint32_t w) {
  uint32_t r = 0;
  for (int i = 0; i < 4; ++i) {
    uint32_t c = (w >> (8 * i)) & 0xffu;
    if ((c & 0x7fu) > 0x77u) c = (c & 0x80u) | 0x77u;
    r |= c << (8 * i);
  }
  return r;
}

// Quantise one row held by LPR lanes (chunks a, b of this lane); returns the
// scale byte.
template <int LPR>
__device__ __forceinline__ int quantise_row(const uint4 &a, const uint4 &b, uint2 &qa, uint2 &qb) {
  const uint32_t m2 = max_mag(b, max_mag(a, 0));
  uint32_t m = max(m2 & 0xffffu, m2 >> 16);
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const int byte = scale_byte(m);
  const float f = __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);
  qa = quantise8(a, f);
  qb = quantise8(b, f);
  if (byte == 247) {
    qa = make_uint2(cap240(qa.x), cap240(qa.y));
    qb = make_uint2(cap240(qb.x), cap240(qb.y));
  }
  return m >= 0x7f80u ? 255 : byte;
}

}  // namespace dllm
