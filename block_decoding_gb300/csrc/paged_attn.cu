// Attention of new tokens over the paged K/V cache (bf16 or e4m3 pages):
// grouped query heads, causal or bidirectional, sliding window with the
// first tokens visible.
//
// One warp per (query row, query head): the lanes split dh, each key's score
// is a warp sum, and the softmax runs with a running maximum and sum in
// registers, one pass over the visible keys.
#include "pages.cuh"

namespace dllm {

DLLM_DEFINE_STATUS(paged)

namespace {

struct PagedArgs {
  KvPages c;
  const uint16_t *q;
  long long q_stride;
  void *out;
  int out_fp32;
  float *lse;
  const int32_t *q_off, *kv_len, *q_pos;
  int B, Hq, group, max_q, max_kv, q_rows;
  float scale;
  int left, right, sinks;
  unsigned int *status;
};

// Request i clipped to the buffers and host bounds: query rows [q0, q0 + W),
// L keys, position of the first row.
struct Extent {
  int q0, W, L, pos;
};

__device__ __forceinline__ Extent paged_extent(const PagedArgs &a, int i, bool report) {
  Extent x;
  bool bad = false;
  x.q0 = a.q_off[i];
  x.W = a.q_off[i + 1] - x.q0;
  x.L = a.kv_len[i];
  if (x.q0 < 0 || x.W < 0 || x.q0 > a.q_rows) { bad = true; x.q0 = 0; x.W = 0; }
  if (x.W > a.q_rows - x.q0) { bad = true; x.W = a.q_rows - x.q0; }
  if (x.W > a.max_q) { bad = true; x.W = a.max_q; }
  if (x.L < 0) { bad = true; x.L = 0; }
  if (x.L > a.max_kv) { bad = true; x.L = a.max_kv; }
  // positions beyond +-2^30 see nothing or everything alike
  x.pos = a.q_pos ? min(max(a.q_pos[i], -(1 << 30)), 1 << 30) : x.L - x.W;
  if (bad && report) atomicOr(a.status, DLLM_DEV_OFFSETS);
  return x;
}

// Keys [lo, hi) that a row at position p sees apart from the sinks.
__device__ __forceinline__ void visible(const PagedArgs &a, int p, int L, int &lo, int &hi) {
  hi = a.right < 0 ? L : min(L, max(p + a.right + 1, 0));
  lo = a.left < 0 ? 0 : max(p - a.left, 0);
}

template <int DH, bool FP8>
__device__ __forceinline__ void load_row(const KvPages &c, const uint8_t *pool, const uint8_t *scale, int row, int lane,
                                         float (&x)[DH / 32]) {
  constexpr int N = DH / 32;
  if (row < 0) {
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = 0.f;
    return;
  }
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    const size_t at = static_cast<size_t>(row) * DH + lane * N + e;
    if constexpr (FP8) {
      const float2 v = e4m3x2_to_f32(*reinterpret_cast<const uint16_t *>(pool + at));
      const float s = __uint_as_float(static_cast<uint32_t>(scale[row]) << 23);
      x[e] = v.x * s; x[e + 1] = v.y * s;
    } else {
      const uint32_t v = *reinterpret_cast<const uint32_t *>(pool + at * 2);
      x[e] = __uint_as_float(v << 16); x[e + 1] = __uint_as_float(v & 0xffff0000u);
    }
  }
}

template <int DH, bool FP8>
__global__ void __launch_bounds__(128) paged_attn_rows_kernel(const PagedArgs a) {
  constexpr int N = DH / 32;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, h = blockIdx.y * 4 + (threadIdx.x >> 5), i = blockIdx.z, t = blockIdx.x;
  const Extent x = paged_extent(a, i, t == 0 && blockIdx.y == 0 && threadIdx.x == 0);
  if (t >= x.W || h >= a.Hq) return;
  const int kh = h / a.group;
  const size_t r = static_cast<size_t>(x.q0) + t;
  float q[N], o[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    q[e] = bf16_to_f32(a.q[r * a.q_stride + h * DH + lane * N + e]) * a.scale;
    o[e] = 0.f;
  }
  int lo, hi;
  visible(a, x.pos + t, x.L, lo, hi);
  float m = -INFINITY, l = 0.f;
  bool bad = false;
  const int first = a.left >= 0 ? min(a.sinks, min(lo, hi)) : 0;   // sinks before the window
  for (int n = 0; n < first + max(hi - lo, 0); ++n) {
    const int u = n < first ? n : lo + n - first;
    int row = page_row(a.c, i, u);
    if (row < 0) bad = true; else row += kh << a.c.page_shift;
    float k[N], v[N];
    load_row<DH, FP8>(a.c, a.c.k, a.c.k_scale, row, lane, k);
    load_row<DH, FP8>(a.c, a.c.v, a.c.v_scale, row, lane, v);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) s = fmaf(q[e], k[e], s);
    s = warp_sum(s);
    const float mn = fmaxf(m, s);
    const float corr = m == mn ? 1.f : expf(m - mn), p = expf(s - mn);
    l = l * corr + p;
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = fmaf(p, v[e], o[e] * corr);
    m = mn;
  }
  if (bad && lane == 0) atomicOr(a.status, DLLM_DEV_PAGE);
  const float inv = l != 0.f ? 1.f / l : 0.f;   // a row that sees nothing: zeros
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const size_t at = (r * a.Hq + h) * DH + lane * N + e;
    if (a.out_fp32) static_cast<float *>(a.out)[at] = o[e] * inv;
    else static_cast<uint16_t *>(a.out)[at] = f32_to_bf16(o[e] * inv);
  }
  if (a.lse && lane == 0) a.lse[r * a.Hq + h] = l != 0.f ? m + logf(l) : -INFINITY;
}

dllm_status check_shape(const dllm_kv_pages *pages, const dllm_paged_attn_args *a) {
  const dllm_status st = check_pages(pages);
  if (st != DLLM_OK) return st;
  if (!a || a->B < 0 || a->Hq < 1 || a->max_q < 0 || a->max_kv < 0 || a->q_rows < 0 || a->max_pages < 0 || a->sinks < 0)
    return DLLM_ERR_INVALID_ARG;
  if (a->Hq % pages->heads || a->Hq / pages->heads > 64 || a->B > 4096) return DLLM_ERR_UNSUPPORTED;
  if (a->left >= (1 << 30) || a->right >= (1 << 30) || a->sinks >= (1 << 30)) return DLLM_ERR_UNSUPPORTED;
  if (a->max_kv >= (1 << 30)) return DLLM_ERR_UNSUPPORTED;
  return DLLM_OK;
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" size_t dllm_paged_attn_workspace(const dllm_kv_pages *pages, const dllm_paged_attn_args *a) {
  if (check_shape(pages, a) != DLLM_OK) return 0;
  return 0;
}

extern "C" dllm_status dllm_paged_attn(const dllm_kv_pages *pages, const dllm_paged_attn_args *a, void *ws,
                                       size_t ws_bytes, dllm_stream stream) {
  const dllm_status st = check_shape(pages, a);
  if (st != DLLM_OK) return st;
  if (a->B == 0 || a->max_q == 0 || a->q_rows == 0) return DLLM_OK;
  const dllm_status sp = check_page_pointers(pages);
  if (sp != DLLM_OK) return sp;
  if (!a->q || !a->out || !a->q_off || !a->kv_len || !a->page_table) return DLLM_ERR_INVALID_ARG;
  if (!aligned16(a->q) || !aligned16(a->out) || a->q_stride < static_cast<long long>(a->Hq) * pages->dh ||
      a->q_stride % 8)
    return DLLM_ERR_INVALID_ARG;
  PagedArgs g{};
  g.c = device_pages(pages, a->page_table, a->max_pages);
  g.q = a->q; g.q_stride = a->q_stride; g.out = a->out; g.out_fp32 = a->out_fp32; g.lse = a->lse;
  g.q_off = a->q_off; g.kv_len = a->kv_len; g.q_pos = a->q_pos;
  g.B = a->B; g.Hq = a->Hq; g.group = a->Hq / pages->heads; g.max_q = a->max_q; g.q_rows = a->q_rows;
  // keys beyond the table are not there
  const long long table = static_cast<long long>(a->max_pages) * pages->page_size;
  g.max_kv = static_cast<int>(table < a->max_kv ? table : a->max_kv);
  g.scale = a->scale;
  g.left = a->left; g.right = a->right; g.sinks = a->left >= 0 ? a->sinks : 0;
  cudaError_t e = cudaGetSymbolAddress(reinterpret_cast<void **>(&g.status), g_status_paged);
  if (e != cudaSuccess) return cuda_error(e);
  const bool fp8 = pages->type == DLLM_KV_E4M3;
  auto kern = pages->dh == 64 ? (fp8 ? paged_attn_rows_kernel<64, true> : paged_attn_rows_kernel<64, false>)
                              : (fp8 ? paged_attn_rows_kernel<128, true> : paged_attn_rows_kernel<128, false>);
  e = launch_pdl(kern, dim3(a->max_q, (a->Hq + 3) / 4, a->B), dim3(128), 0, static_cast<cudaStream_t>(stream), g);
  if (e != cudaSuccess) return cuda_error(e);
  return launch_status();
}
