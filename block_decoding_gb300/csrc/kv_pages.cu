// Writing new K/V rows into the pages of the cache (in bf16 as they are, or
// in 8 bits with one power-of-two scale per row and head) and reading rows
// back as contiguous bf16. Both move each byte once: memory bound.
//
// One row of one head is handled by dh / 16 neighbouring lanes, 16 elements
// of K and 16 of V each: two 16-byte chunks half a row apart, so that the
// lanes of a row read and write contiguous runs. A block takes neighbouring
// rows of up to four neighbouring heads: runs of several rows on the pages'
// side, of several heads on the other.
// Measured (dh 128, 32 heads, e4m3): 10 k rows written in 54.6 us (4.7 TB/s, 69 %
// of a copy's rate; short of issue slots: 57.3 us when every thread looked its
// row's place up and multiplied in fp32), 19 k rows read in 79.8 us (6.0 TB/s,
// 89 %); 64 single tokens (8 heads) written in 3.1 us, of which nearly all is the
// launch and the chain request -> page -> store. Writing loads its rows before it
// looks their places up (3 us less). Blocks of 64 or 256 threads and of 2 or 8
// heads: within 3 %. Several rows per thread: 4.4 us for the 64 tokens; a
// persistent grid that loads its next rows ahead: slower.
#include "page_rows.cuh"

namespace dllm {

DLLM_DEFINE_STATUS(kv)

namespace {

constexpr int kThreads = 128;
constexpr int kHeads = 4;   // heads of one block, at most

struct MoveArgs {
  KvPages c;
  uint16_t *k, *v;             // the contiguous side
  long long k_stride, v_stride;
  int rows, B;
  int hb, per;                 // heads and rows of a block
  int run;                     // blocks until the slower of row and head moves
  uint32_t inv;                // n / hb = n * inv >> 16 for n < 256
  const int32_t *off, *pos0;
  unsigned int *status;
};

// The block's first row, and this thread's row in the block and head: unit u
// (LPR lanes each) of a block has head h0 + u % hb of row r0 + u / hb. Returns
// whether there is such a unit. Neighbouring blocks have neighbouring rows of
// the same heads where rows are written (54.6 us; heads first: 55.5), and the
// heads of the same rows where they are read (79.8; rows first: 82.6).
template <int LPR, bool ROWS_FIRST>
__device__ __forceinline__ bool place_of(const MoveArgs &g, int &r0, int &n, int &h) {
  const int u = threadIdx.x / LPR, slow = blockIdx.x / g.run, fast = blockIdx.x - slow * g.run;
  r0 = (ROWS_FIRST ? fast : slow) * g.per;
  n = static_cast<int>(u * g.inv >> 16);
  h = (ROWS_FIRST ? slow : fast) * g.hb + u - n * g.hb;
  return n < g.per && h < g.c.heads;
}

// Cache row of row r for head 0: -1 when it is in no request, -2 when it has
// no place (reported).
__device__ __forceinline__ int find_row(const MoveArgs &g, int r) {
  if (r >= g.rows) return -1;
  const int i = request_of(g.off, g.B, r);
  if (i < 0) return -1;
  const long long u = static_cast<long long>(g.pos0[i]) + (r - g.off[i]);
  const int row = u < 0 || u > 0x7fffffffll ? -1 : page_row(g.c, i, static_cast<int>(u));
  if (row < 0) {
    atomicOr(g.status, DLLM_DEV_PAGE);
    return -2;
  }
  return row;
}

template <int DH, bool FP8>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const MoveArgs g) {
  constexpr int LPR = DH / 16;
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x + threadIdx.x == 0 && (g.off[0] < 0 || g.off[g.B] > g.rows)) atomicOr(g.status, DLLM_DEV_OFFSETS);
  __shared__ int s_row[kThreads / LPR];
  const int l = threadIdx.x % LPR;
  int r0, n, h;
  const bool live = place_of<LPR, true>(g, r0, n, h);
  const int r = r0 + n;
  uint4 ka = make_uint4(0, 0, 0, 0), kb = ka, va = ka, vb = ka;
  if (live && r < g.rows) {
    const uint4 *ks = reinterpret_cast<const uint4 *>(g.k + r * g.k_stride + h * DH);
    const uint4 *vs = reinterpret_cast<const uint4 *>(g.v + r * g.v_stride + h * DH);
    ka = __ldg(ks + l); kb = __ldg(ks + l + LPR);
    va = __ldg(vs + l); vb = __ldg(vs + l + LPR);
  }
  // the places of the block's rows, found once while the rows are on their way
  // (the kernel is short of issue slots; reading, which has to wait for them
  // before its loads, every thread finds its own: 81 us, this way 84)
  if (threadIdx.x < g.per) s_row[threadIdx.x] = find_row(g, r0 + threadIdx.x);
  __syncthreads();
  const int row = live ? s_row[n] : -1;
  const size_t at = static_cast<size_t>(max(row, 0)) + (static_cast<size_t>(h) << g.c.page_shift);
  if constexpr (FP8) {
    uint2 qa, qb;
    const int kbyte = quantise_row<LPR>(ka, kb, qa, qb);
    if (row >= 0) {
      uint2 *d = reinterpret_cast<uint2 *>(g.c.k + at * DH);
      d[l] = qa; d[l + LPR] = qb;
    }
    const int vbyte = quantise_row<LPR>(va, vb, qa, qb);
    if (row >= 0) {
      uint2 *d = reinterpret_cast<uint2 *>(g.c.v + at * DH);
      d[l] = qa; d[l + LPR] = qb;
      if (l == 0) {
        g.c.k_scale[at] = static_cast<uint8_t>(kbyte);
        g.c.v_scale[at] = static_cast<uint8_t>(vbyte);
      }
    }
  } else if (row >= 0) {
    uint4 *d = reinterpret_cast<uint4 *>(g.c.k + at * (DH * 2));
    d[l] = ka; d[l + LPR] = kb;
    d = reinterpret_cast<uint4 *>(g.c.v + at * (DH * 2));
    d[l] = va; d[l + LPR] = vb;
  }
}

// Eight codes -> eight bf16 of code * 2^(byte - 127): exact (a code has four
// significant bits, and the scales keep every value normal).
__device__ __forceinline__ uint4 restore8(uint2 q, float f) {
  float x[8];
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = e4m3x2_to_f32(static_cast<uint16_t>(w[i])), b = e4m3x2_to_f32(static_cast<uint16_t>(w[i] >> 16));
    x[4 * i] = a.x * f; x[4 * i + 1] = a.y * f; x[4 * i + 2] = b.x * f; x[4 * i + 3] = b.y * f;
  }
  return pack8(x);
}

template <int DH, bool FP8>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const MoveArgs g) {
  constexpr int LPR = DH / 16;
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x + threadIdx.x == 0 && (g.off[0] < 0 || g.off[g.B] > g.rows)) atomicOr(g.status, DLLM_DEV_OFFSETS);
  const int l = threadIdx.x % LPR;
  int r0, n, h;
  if (!place_of<LPR, false>(g, r0, n, h)) return;
  const int r = r0 + n, row = find_row(g, r);
  if (row == -1) return;   // a row without a place (-2) reads as zeros
  uint4 ka = make_uint4(0, 0, 0, 0), kb = ka, va = ka, vb = ka;
  if (row >= 0) {
    const size_t at = static_cast<size_t>(row) + (static_cast<size_t>(h) << g.c.page_shift);
    if constexpr (FP8) {
      const uint2 *ks = reinterpret_cast<const uint2 *>(g.c.k + at * DH);
      const uint2 *vs = reinterpret_cast<const uint2 *>(g.c.v + at * DH);
      const uint2 qa = __ldg(ks + l), qb = __ldg(ks + l + LPR), pa = __ldg(vs + l), pb = __ldg(vs + l + LPR);
      const float kf = scale_of(g.c.k_scale[at]), vf = scale_of(g.c.v_scale[at]);
      ka = restore8(qa, kf); kb = restore8(qb, kf);
      va = restore8(pa, vf); vb = restore8(pb, vf);
    } else {
      const uint4 *ks = reinterpret_cast<const uint4 *>(g.c.k + at * (DH * 2));
      const uint4 *vs = reinterpret_cast<const uint4 *>(g.c.v + at * (DH * 2));
      ka = __ldg(ks + l); kb = __ldg(ks + l + LPR);
      va = __ldg(vs + l); vb = __ldg(vs + l + LPR);
    }
  }
  uint4 *d = reinterpret_cast<uint4 *>(g.k + r * g.k_stride + h * DH);
  d[l] = ka; d[l + LPR] = kb;
  d = reinterpret_cast<uint4 *>(g.v + r * g.v_stride + h * DH);
  d[l] = va; d[l + LPR] = vb;
}

dllm_status move(bool write, const dllm_kv_pages *pages, uint16_t *k, uint16_t *v, long long k_stride,
                 long long v_stride, int rows, const int32_t *off, const int32_t *pos0, const int32_t *page_table,
                 int max_pages, int B, cudaStream_t s) {
  const dllm_status st = check_pages(pages);
  if (st != DLLM_OK) return st;
  if (rows < 0 || B < 0 || max_pages < 0) return DLLM_ERR_INVALID_ARG;
  // (a block numbers its rows beyond the last one, by less than its threads)
  if (B > 4096 || rows > 0x7fffffff - kThreads) return DLLM_ERR_UNSUPPORTED;
  if (rows == 0 || B == 0) return DLLM_OK;
  const dllm_status sp = check_page_pointers(pages);
  if (sp != DLLM_OK) return sp;
  const long long d = static_cast<long long>(pages->heads) * pages->dh;
  if (!k || !v || !off || !pos0 || (!page_table && max_pages > 0)) return DLLM_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || k_stride < d || v_stride < d || k_stride % 8 || v_stride % 8)
    return DLLM_ERR_INVALID_ARG;
  MoveArgs g{};
  g.c = device_pages(pages, page_table, max_pages);
  g.k = k; g.v = v; g.k_stride = k_stride; g.v_stride = v_stride;
  g.rows = rows; g.B = B; g.off = off; g.pos0 = pos0;
  cudaError_t e = cudaGetSymbolAddress(reinterpret_cast<void **>(&g.status), g_status_kv);
  if (e != cudaSuccess) return cuda_error(e);
  g.hb = pages->heads < kHeads ? pages->heads : kHeads;
  g.per = kThreads / (pages->dh / 16) / g.hb;
  g.inv = 65536u / g.hb + 1;
  const int groups = (pages->heads + g.hb - 1) / g.hb, row_blocks = (rows - 1) / g.per + 1;
  const long long blocks = static_cast<long long>(row_blocks) * groups;
  g.run = write ? row_blocks : groups;
  if (blocks > 0x7fffffffll) return DLLM_ERR_UNSUPPORTED;
  const bool fp8 = pages->type == DLLM_KV_E4M3;
  void (*kern)(MoveArgs);
  if (write)
    kern = pages->dh == 64 ? (fp8 ? kv_write_kernel<64, true> : kv_write_kernel<64, false>)
                           : (fp8 ? kv_write_kernel<128, true> : kv_write_kernel<128, false>);
  else
    kern = pages->dh == 64 ? (fp8 ? kv_read_kernel<64, true> : kv_read_kernel<64, false>)
                           : (fp8 ? kv_read_kernel<128, true> : kv_read_kernel<128, false>);
  e = launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, s, g);
  if (e != cudaSuccess) return cuda_error(e);
  return launch_status();
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" dllm_status dllm_kv_write(const dllm_kv_pages *pages, const dllm_bf16 *k, const dllm_bf16 *v,
                                     long long k_stride, long long v_stride, int rows, const int32_t *off,
                                     const int32_t *pos0, const int32_t *page_table, int max_pages, int B,
                                     dllm_stream stream) {
  return move(true, pages, const_cast<dllm_bf16 *>(k), const_cast<dllm_bf16 *>(v), k_stride, v_stride, rows, off, pos0,
              page_table, max_pages, B, static_cast<cudaStream_t>(stream));
}

extern "C" dllm_status dllm_kv_read(const dllm_kv_pages *pages, dllm_bf16 *k, dllm_bf16 *v, int rows,
                                    const int32_t *off, const int32_t *pos0, const int32_t *page_table, int max_pages,
                                    int B, dllm_stream stream) {
  const long long d = pages ? static_cast<long long>(pages->heads) * pages->dh : 0;
  return move(false, pages, k, v, d, d, rows, off, pos0, page_table, max_pages, B, static_cast<cudaStream_t>(stream));
}
