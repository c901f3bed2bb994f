// Rotary positions on the way into the paged cache: q and k rows are turned by
// their positions on one or several axes, q goes to its own rows and k, v to
// the pages (bf16, or 8 bits with a scale per row and head), in one pass.
//
// Pair j of a head (elements j and j + rot / 2) turns by pos[axis(j)] * freq(j).
// The angle is needed modulo a turn only: freq(j) / 2 pi is kept as a 64-bit
// fraction of a turn, its product with the position wraps around by itself, and
// what is left is within 2^-64 turns per position of the exact angle, however
// far the position (a product in fp32 is off by 0.06 at position 10^6).
//
// Bound by memory: each row is read and written once. The sines and cosines of
// a row are computed once per block and serve all of its heads. One row of one
// head is handled by dh / 16 neighbouring lanes, two 16-byte chunks each: a pair's
// two halves lie in the same lane. Measured (dh 128): 7.1 k rows of 32 + 2 x 8
// heads, bf16 pages, 36 us, 4.9 TB/s and 72 % of a copy's rate; 11 k rows of 32 +
// 2 x 32 heads, e4m3 pages, 92 us, the same rate. (Blocks of 2 rows 42, of 8 40 to
// 43 us; one unit of a thread on the way 45, three or four 38 to 40: registers.
// Sines and cosines read with bank conflicts: 2 us more.) 64 single tokens: 4.6
// us, the chain offsets -> position -> page -> store.
#include "page_rows.cuh"
#include "turns.cuh"
#include "umma.cuh"

namespace dllm {

DLLM_DEFINE_STATUS(rope)

namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 4;      // rows of a block: a warp finds each one's place
constexpr int kMaxHalf = 64;     // pairs of a head
constexpr int kAhead = 2;        // units of a thread whose loads are on their way

struct RopeArgs {
  KvPages c;
  const uint16_t *q, *k, *v;
  uint16_t *q_out;
  long long q_stride, k_stride, v_stride, q_out_stride;
  const int32_t *pos;          // [axes][rows]
  int rows, B, Hq, half, per;
  const int32_t *off, *pos0;
  unsigned int *status;
  unsigned long long turns[kMaxHalf];   // of a position, in 2^-64
  uint8_t axis[kMaxHalf];
};

// Scale byte of a row whose largest magnitude has the bits `a` (finite fp32).
__device__ __forceinline__ int scale_byte_f32(uint32_t a) {
  const int b = static_cast<int>(a >> 23) - 8 + ((a & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(b, 10), 247);
}

__device__ __forceinline__ uint2 quantise8_f32(const float *x, float f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = f32_to_e4m3x2(x[2 * i] * f, x[2 * i + 1] * f);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// As quantise_row, of 16 fp32 elements a lane.
template <int LPR>
__device__ __forceinline__ int quantise_row_f32(const float (&a)[8], const float (&b)[8], uint2 &qa, uint2 &qb) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    m = max(m, max(__float_as_uint(a[e]) & 0x7fffffffu, __float_as_uint(b[e]) & 0x7fffffffu));
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const int byte = scale_byte_f32(m);
  const float f = __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);
  qa = quantise8_f32(a, f);
  qb = quantise8_f32(b, f);
  if (byte == 247) {
    qa = make_uint2(cap240(qa.x), cap240(qa.y));
    qb = make_uint2(cap240(qb.x), cap240(qb.y));
  }
  return m >= 0x7f800000u ? 255 : byte;
}

// (cos, sin) of `pos` times a 64-bit fraction of a turn.
__device__ __forceinline__ float2 turn_of(int pos, unsigned long long turns) {
  const long long t = static_cast<long long>(turns * static_cast<unsigned long long>(static_cast<long long>(pos)));
  float2 r;
  sincospif(__ll2float_rn(t) * 0x1p-63f, &r.y, &r.x);
  return r;
}

// Request that holds row r, or -1, by a whole warp: 32 offsets at a time (a
// bisection's loads wait for each other).
__device__ __forceinline__ int request_of_warp(const int32_t *off, int B, int r, int lane) {
  int lo = 0, hi = B + 1;      // off[lo] <= r, and r < off[hi] if there is one
  if (r < off[0]) return -1;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const uint32_t m = __ballot_sync(0xffffffffu, at < hi && off[at] <= r);
    lo += (31 - __clz(m)) * step;       // (lane 0's holds)
    hi = min(hi, lo + step);
  }
  return lo < B ? lo : -1;
}

template <int DH, bool FP8>
__global__ void __launch_bounds__(kThreads) rope_write_kernel(const __grid_constant__ RopeArgs g) {
  constexpr int LPR = DH / 16, kUnits = kThreads / LPR;
  __shared__ float2 s_cs[kMaxRows * kMaxHalf];
  __shared__ int s_row[kMaxRows];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, l = tid % LPR;
  if (blockIdx.x + tid == 0 && (g.off[0] < 0 || g.off[g.B] > g.rows)) atomicOr(g.status, DLLM_DEV_OFFSETS);
  const int r0 = blockIdx.x * g.per, rows = min(g.per, g.rows - r0);
  const int heads = g.c.heads, T = g.Hq + 2 * heads, half = g.half, rc = half / 8, total = rows * T;
  // this lane's chunks of a head: the halves of eight pairs, or two that are not turned
  const bool turns = l < rc;
  const int ca = turns ? l : rc + l, cb = turns ? l + rc : ca + LPR - rc;
  // Unit u of the block is head u % T of row u / T: q's heads, k's, v's. A
  // thread's units are kUnits apart, and kAhead of them are loaded at a time.
  int n = 0, t = tid / LPR;
  while (t >= T) { t -= T; ++n; }
  uint4 a[kAhead], b[kAhead];
  int un[kAhead], ut[kAhead];
  auto load = [&] {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      un[i] = n;
      ut[i] = t;
      a[i] = b[i] = make_uint4(0, 0, 0, 0);
      if (n < rows) {
        const long long r = r0 + n;
        const uint16_t *src = t < g.Hq           ? g.q + r * g.q_stride + t * DH
                              : t < g.Hq + heads ? g.k + r * g.k_stride + (t - g.Hq) * DH
                                                 : g.v + r * g.v_stride + (t - g.Hq - heads) * DH;
        a[i] = reinterpret_cast<const uint4 *>(src)[ca];
        b[i] = reinterpret_cast<const uint4 *>(src)[cb];
      }
      t += kUnits;
      while (t >= T) { t -= T; ++n; }
    }
  };
  load();
  // the rows' places, and their sines and cosines, while the first units are on their way
  if (tid / 32 < rows) {
    const int r = r0 + tid / 32, i = request_of_warp(g.off, g.B, r, tid % 32);
    int row = -1;                                   // in no request
    if (i >= 0) {
      const long long u = static_cast<long long>(g.pos0[i]) + (r - g.off[i]);
      row = u < 0 || u > 0x7fffffffll ? -1 : page_row(g.c, i, static_cast<int>(u));
      if (row < 0) {
        if (tid % 32 == 0) atomicOr(g.status, DLLM_DEV_PAGE);
        row = -2;                                   // no place
      }
    }
    if (tid % 32 == 0) s_row[tid / 32] = row;
  }
  for (int idx = tid; idx < rows * half; idx += kThreads) {
    const int m = idx / half, j = idx - m * half;
    // (lane l of a unit reads pairs 8 l .. 8 l + 7, two at a time: the l-th pairs of two of all lanes lie side by side)
    s_cs[m * kMaxHalf + j % 8 / 2 * 16 + j / 8 * 2 + j % 2] = turn_of(g.pos[static_cast<size_t>(g.axis[j]) * g.rows + r0 + m], g.turns[j]);
  }
  __syncthreads();
  // Every lane of a warp goes through the same rounds: the lanes of a row
  // exchange maxima.
  for (int u0 = 0; u0 < total; u0 += kAhead * kUnits) {
    if (u0 > 0) load();
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const bool live = un[i] < rows, is_q = ut[i] < g.Hq, is_k = !is_q && ut[i] < g.Hq + heads;
      const int row = live ? s_row[un[i]] : -1;
      const int h = is_q ? ut[i] : is_k ? ut[i] - g.Hq : ut[i] - g.Hq - heads;
      float x[8], y[8];
      unpack8(a[i], x);
      unpack8(b[i], y);
      if (turns && (is_q || is_k) && live) {
        const float4 *cs = reinterpret_cast<const float4 *>(s_cs + un[i] * kMaxHalf) + l;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float4 w = cs[e / 2 * 8];
          const float p = x[e] * w.x - y[e] * w.y, q = x[e + 1] * w.z - y[e + 1] * w.w;
          y[e] = y[e] * w.x + x[e] * w.y;
          y[e + 1] = y[e + 1] * w.z + x[e + 1] * w.w;
          x[e] = p;
          x[e + 1] = q;
        }
      }
      if (is_q && row != -1) {
        uint4 *d = reinterpret_cast<uint4 *>(g.q_out + (r0 + un[i]) * g.q_out_stride + h * DH);
        d[ca] = pack8(x);
        d[cb] = pack8(y);
      }
      const size_t at = static_cast<size_t>(max(row, 0)) + (static_cast<size_t>(h) << g.c.page_shift);
      if constexpr (FP8) {
        // (a round without rows for the pages is one for whole warps)
        if (!__any_sync(0xffffffffu, !is_q && row >= 0)) continue;
        uint2 qa, qb;
        const int byte = quantise_row_f32<LPR>(x, y, qa, qb);
        if (!is_q && row >= 0) {
          uint2 *d = reinterpret_cast<uint2 *>((is_k ? g.c.k : g.c.v) + at * DH);
          d[ca] = qa;
          d[cb] = qb;
          if (l == 0) (is_k ? g.c.k_scale : g.c.v_scale)[at] = static_cast<uint8_t>(byte);
        }
      } else if (!is_q && row >= 0) {
        uint4 *d = reinterpret_cast<uint4 *>((is_k ? g.c.k : g.c.v) + at * (DH * 2));
        d[ca] = is_k ? pack8(x) : a[i];
        d[cb] = is_k ? pack8(y) : b[i];
      }
    }
  }
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" dllm_status dllm_rope_kv_write(const dllm_kv_pages *pages, const dllm_rope *rope,
                                          const dllm_rope_write_args *a, dllm_stream stream) {
  const dllm_status st = check_pages(pages);
  if (st != DLLM_OK) return st;
  if (!rope || !a || a->rows < 0 || a->B < 0 || a->max_pages < 0 || a->Hq < 0) return DLLM_ERR_INVALID_ARG;
  if (a->B > 4096 || a->rows > 0x7fffffff - kThreads || a->Hq > 16384) return DLLM_ERR_UNSUPPORTED;
  if (rope->rot < 0 || rope->rot > pages->dh || rope->axes < 1) return DLLM_ERR_INVALID_ARG;
  if (rope->rot % 16 || rope->axes > DLLM_ROPE_AXES) return DLLM_ERR_UNSUPPORTED;
  for (int j = 0; j < rope->rot / 2; ++j) {
    if (rope->axis[j] >= rope->axes) return DLLM_ERR_INVALID_ARG;
    if (!(fabs(rope->freq[j]) <= 1024.0)) return DLLM_ERR_INVALID_ARG;      // NaN too
  }
  if (a->rows == 0 || a->B == 0) return DLLM_OK;
  const dllm_status sp = check_page_pointers(pages);
  if (sp != DLLM_OK) return sp;
  const long long d = static_cast<long long>(pages->heads) * pages->dh, dq = static_cast<long long>(a->Hq) * pages->dh;
  if (!a->k || !a->v || !a->pos || !a->off || !a->pos0 || (!a->page_table && a->max_pages > 0)) return DLLM_ERR_INVALID_ARG;
  if (!aligned16(a->k) || !aligned16(a->v) || a->k_stride < d || a->v_stride < d || a->k_stride % 8 || a->v_stride % 8)
    return DLLM_ERR_INVALID_ARG;
  if (a->Hq > 0 && (!a->q || !a->q_out || !aligned16(a->q) || !aligned16(a->q_out) || a->q_stride < dq ||
                    a->q_out_stride < dq || a->q_stride % 8 || a->q_out_stride % 8))
    return DLLM_ERR_INVALID_ARG;
  RopeArgs g{};
  g.c = device_pages(pages, a->page_table, a->max_pages);
  g.q = a->q; g.k = a->k; g.v = a->v; g.q_out = a->q_out;
  g.q_stride = a->q_stride; g.k_stride = a->k_stride; g.v_stride = a->v_stride; g.q_out_stride = a->q_out_stride;
  g.pos = a->pos; g.rows = a->rows; g.B = a->B; g.Hq = a->Hq; g.half = rope->rot / 2;
  g.off = a->off; g.pos0 = a->pos0;
  for (int j = 0; j < g.half; ++j) {
    g.turns[j] = fraction_of_turn(rope->freq[j]);
    g.axis[j] = rope->axis[j];
  }
  cudaError_t e = cudaGetSymbolAddress(reinterpret_cast<void **>(&g.status), g_status_rope);
  if (e != cudaSuccess) return cuda_error(e);
  // Blocks of four rows, or of one where there are few. (32 + 2 x 8 heads: 300
  // rows 6.3 and 4.6 us, 600 6.7 and 5.2, 1200 8.9 and 8.9, 2400 12.3 and 15.7.)
  g.per = a->rows >= 8 * num_sms() ? kMaxRows : 1;
  const bool fp8 = pages->type == DLLM_KV_E4M3;
  void (*kern)(RopeArgs) = pages->dh == 64 ? (fp8 ? rope_write_kernel<64, true> : rope_write_kernel<64, false>)
                                           : (fp8 ? rope_write_kernel<128, true> : rope_write_kernel<128, false>);
  e = launch_pdl(kern, dim3(static_cast<unsigned>((a->rows - 1) / g.per + 1)), dim3(kThreads), 0,
                 static_cast<cudaStream_t>(stream), g);
  if (e != cudaSuccess) return cuda_error(e);
  return launch_status();
}
