// The weight that attention gave to every cached row: for each position of a
// request and cached head, the sum over query rows (and the query heads that
// share the cached head) of exp(scale <q, k> - lse), added to what the row's
// slot holds from earlier steps, times a decay.
#include <math.h>

#include "paged.cuh"

namespace dllm {

DLLM_DEFINE_STATUS(mass)

namespace {

struct MassArgs : PagedArgs {
  float *mass;
  const int32_t *fresh;
  float decay;
};

constexpr int kKeys = 128, kRows = 16;

template <int DH, bool FP8>
__global__ void __launch_bounds__(kKeys) mass_kernel(const __grid_constant__ MassArgs a) {
  __shared__ float s_q[kRows][DH];
  __shared__ float s_lse[kRows];
  __shared__ int s_hi[kRows];
  pdl_trigger();
  pdl_wait();
  const int i = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
  const Extent x = paged_extent(a, i, blockIdx.x + blockIdx.y + tid == 0);
  const int u = blockIdx.x * kKeys + tid;
  if (x.W == 0 || blockIdx.x * kKeys >= static_cast<unsigned>(x.L)) return;
  int row = -1;
  if (u < x.L) {
    row = page_row(a.c, i, u);
    if (row < 0) atomicOr(a.status, DLLM_DEV_PAGE);
  }
  const size_t at = static_cast<size_t>(max(row, 0)) + (static_cast<size_t>(h) << a.c.page_shift);
  float k[DH];
  float c = a.scale_log2;
  if constexpr (FP8) {
    if (row >= 0) c *= scale_of(a.c.k_scale[at]);
    const uint16_t *src = reinterpret_cast<const uint16_t *>(a.c.k + at * DH);
#pragma unroll
    for (int e = 0; e < DH / 2; ++e) {
      const float2 f = e4m3x2_to_f32(src[e]);
      k[2 * e] = f.x;
      k[2 * e + 1] = f.y;
    }
  } else {
    const uint4 *src = reinterpret_cast<const uint4 *>(a.c.k + at * (DH * 2));
#pragma unroll
    for (int e = 0; e < DH / 8; ++e) unpack8(src[e], k + 8 * e);
  }
  float sum = 0.f;
  const int rows = x.W * a.group;
  for (int r0 = 0; r0 < rows; r0 += kRows) {
    __syncthreads();
    for (int idx = tid; idx < kRows * DH; idx += kKeys) {
      const int n = idx / DH, e = idx % DH, r = r0 + n, t = r / a.group, g = r - t * a.group;
      s_q[n][e] = r < rows ? bf16_to_f32(a.q[(x.q0 + t) * a.q_stride + (h * a.group + g) * DH + e]) : 0.f;
      if (e == 0) {
        int lo, hi = 0;
        float lse = 0.f;
        if (r < rows) {
          visible(a, x.pos, t, x.L, lo, hi);
          lse = a.lse[static_cast<size_t>(x.q0 + t) * a.Hq + h * a.group + g];
          if (lse == -INFINITY) hi = 0;
        }
        s_lse[n] = lse * 1.4426950408889634f;
        s_hi[n] = hi;
      }
    }
    __syncthreads();
    for (int n = 0; n < kRows; ++n) {
      float d = 0.f;
#pragma unroll
      for (int e = 0; e < DH; ++e) d += s_q[n][e] * k[e];
      if (u < s_hi[n]) sum += exp2f(fmaf(d, c, -s_lse[n]));
    }
  }
  if (row >= 0) {
    const float old = a.fresh && u >= a.fresh[i] ? 0.f : a.decay * a.mass[at];
    a.mass[at] = old + sum;
  }
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" dllm_status dllm_attn_mass(const dllm_kv_pages *pages, const dllm_attn_mass_args *a, dllm_stream stream) {
  const dllm_status st = check_pages(pages);
  if (st != DLLM_OK) return st;
  if (!a || a->B < 0 || a->Hq < 1 || a->max_q < 0 || a->max_kv < 0 || a->q_rows < 0 || a->max_pages < 0) return DLLM_ERR_INVALID_ARG;
  if (!isfinite(a->decay)) return DLLM_ERR_INVALID_ARG;
  if (a->Hq % pages->heads || a->Hq / pages->heads > 64 || a->B > 4096 || a->right >= (1 << 30) || a->max_kv >= (1 << 30))
    return DLLM_ERR_UNSUPPORTED;
  if (static_cast<long long>(a->q_rows) * a->Hq >= (1ll << 30) || static_cast<long long>(a->max_q) * a->Hq >= (1ll << 30))
    return DLLM_ERR_UNSUPPORTED;
  if (a->B == 0 || a->max_q == 0 || a->q_rows == 0 || a->max_kv == 0 || a->max_pages == 0) return DLLM_OK;
  const dllm_status sp = check_page_pointers(pages);
  if (sp != DLLM_OK) return sp;
  if (!a->q || !a->lse || !a->mass || !a->q_off || !a->kv_len || !a->page_table) return DLLM_ERR_INVALID_ARG;
  if (!aligned16(a->q) || a->q_stride < static_cast<long long>(a->Hq) * pages->dh || a->q_stride % 8) return DLLM_ERR_INVALID_ARG;
  MassArgs g{};
  g.c = device_pages(pages, a->page_table, a->max_pages);
  g.q = a->q; g.q_stride = a->q_stride; g.lse = const_cast<float *>(a->lse);
  g.q_off = a->q_off; g.kv_len = a->kv_len; g.q_pos = a->q_pos;
  g.B = a->B; g.Hq = a->Hq; g.group = a->Hq / pages->heads; g.max_q = a->max_q; g.q_rows = a->q_rows;
  const long long table = static_cast<long long>(a->max_pages) * pages->page_size;   // keys beyond the table are not there
  g.max_kv = static_cast<int>(table < a->max_kv ? table : a->max_kv);
  g.scale_log2 = a->scale * 1.4426950408889634f;
  g.left = -1; g.right = a->right;
  g.mass = a->mass; g.fresh = a->fresh; g.decay = a->decay;
  cudaError_t e = cudaGetSymbolAddress(reinterpret_cast<void **>(&g.status), g_status_mass);
  if (e != cudaSuccess) return cuda_error(e);
  const bool fp8 = pages->type == DLLM_KV_E4M3;
  void (*kern)(MassArgs) = pages->dh == 64 ? (fp8 ? mass_kernel<64, true> : mass_kernel<64, false>)
                                           : (fp8 ? mass_kernel<128, true> : mass_kernel<128, false>);
  e = launch_pdl(kern, dim3((g.max_kv + kKeys - 1) / kKeys, pages->heads, a->B), dim3(kKeys), 0,
                 static_cast<cudaStream_t>(stream), g);
  if (e != cudaSuccess) return cuda_error(e);
  return launch_status();
}
