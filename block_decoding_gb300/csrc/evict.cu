// Moving rows within the paged cache, and choosing the rows that stay when a
// cache is cut down to a budget.
#include "pages.cuh"

namespace dllm {

DLLM_DEFINE_STATUS(evict)

namespace {

// ---------------------------------------------------------------------------
// selection
// ---------------------------------------------------------------------------
struct SelectArgs {
  KvPages c;
  const float *mass;
  const int32_t *kv_len;
  int32_t *new_len, *keep;     // [B], [B][heads][budget]
  int budget, max_kv, sinks, recent;
  unsigned int *status;
};

constexpr int kSelThreads = 512;

// Order of weights as unsigned numbers: -0 is 0, NaN is above everything.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// One CTA per cached head and request: radix selection of the least weight
// that stays, 8 bits at a time, then the positions in order.
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectArgs a) {
  __shared__ int s_hist[256];
  __shared__ int s_scan[kSelThreads / 32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_left;
  pdl_trigger();
  pdl_wait();
  const int h = blockIdx.x, i = blockIdx.y, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  int n = a.kv_len[i];
  if (n < 0 || n > a.max_kv) {
    if (tid + h == 0) atomicOr(a.status, DLLM_DEV_OFFSETS);
    n = min(max(n, 0), a.max_kv);
  }
  int32_t *keep = a.keep + (static_cast<size_t>(i) * a.c.heads + h) * a.budget;
  const int k = min(n, a.budget);
  if (h == 0 && tid == 0) a.new_len[i] = k;
  for (int j = tid + k; j < a.budget; j += kSelThreads) keep[j] = -1;
  if (n <= a.budget) {
    for (int j = tid; j < k; j += kSelThreads) keep[j] = j;
    return;
  }
  const int s = a.sinks, e = n - a.recent;       // [s, e) is chosen from: at least n - budget + 1 rows
  auto key = [&](int u) {
    const int row = page_row(a.c, i, u);
    if (row < 0) {
      atomicOr(a.status, DLLM_DEV_PAGE);
      return 0u;
    }
    return order_of(a.mass[row + (static_cast<size_t>(h) << a.c.page_shift)]);
  };
  int left = k - s - a.recent;                   // how many of them stay
  uint32_t prefix = 0;
  for (int shift = 24; shift >= 0 && left > 0; shift -= 8) {
    for (int b = tid; b < 256; b += kSelThreads) s_hist[b] = 0;
    __syncthreads();
    for (int u = s + tid; u < e; u += kSelThreads) {
      const uint32_t x = key(u);
      if (shift == 24 || x >> (shift + 8) == prefix >> (shift + 8)) atomicAdd(&s_hist[x >> shift & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int b = 255;
      while (s_hist[b] < left) left -= s_hist[b--];
      s_prefix = prefix | static_cast<uint32_t>(b) << shift;
      s_left = left;
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_left;
  }
  if (left <= 0) prefix = 0xffffffffu;           // none of them
  // `left` rows of weight `prefix` stay, the first ones, and all above
  int done = 0, ties = 0;                        // before this round
  for (int u0 = 0; u0 < n; u0 += kSelThreads) {
    const int u = u0 + tid;
    bool in = false, tie = false;
    if (u < n) {
      if (u < s || u >= e) in = true;
      else if (left > 0) {
        const uint32_t x = key(u);
        in = x > prefix;
        tie = x == prefix;
      }
    }
    auto rank = [&](bool p, int &total) {        // of this thread among those with p
      const uint32_t m = __ballot_sync(0xffffffffu, p);
      if (lane == 0) s_scan[warp] = __popc(m);
      __syncthreads();
      int before = __popc(m & ((1u << lane) - 1));
      total = 0;
      for (int w = 0; w < kSelThreads / 32; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
      }
      __syncthreads();
      return before;
    };
    int total;
    const int tr = rank(tie, total);
    in |= tie && ties + tr < left;
    ties += total;
    const int r = rank(in, total);
    if (in) keep[done + r] = u;
    done += total;
  }
}

// ---------------------------------------------------------------------------
// moves
// ---------------------------------------------------------------------------
struct ShiftArgs {
  KvPages c;
  const int32_t *dst_table;
  int dst_pages;
  const int32_t *src;          // [B][src_heads][max_n]
  int src_heads, max_n;
  const int32_t *count, *first;   // [B]; first may be null: 0
  float *mass;
  bool in_place;
  unsigned int *status;
};

constexpr int kMoveThreads = 256, kEach = 8;   // 16-byte pieces of a thread on the way

// One CTA per cached head, request, and K or V. Rows move in ascending order,
// a piece at a time, every row of a piece read before any is written: in place
// a row's own place is written no earlier than it is read.
template <int ROW>
__global__ void __launch_bounds__(kMoveThreads) shift_kernel(const ShiftArgs a) {
  constexpr int kChunks = ROW / 16, kRows = kMoveThreads * kEach / kChunks;
  pdl_trigger();
  pdl_wait();
  const int h = blockIdx.x, i = blockIdx.y, tid = threadIdx.x;
  const bool v = blockIdx.z;
  uint8_t *pool = v ? a.c.v : a.c.k, *scale = v ? a.c.v_scale : a.c.k_scale;
  float *mass = v ? nullptr : a.mass;
  int n = a.count[i];
  if (n < 0 || n > a.max_n) {
    if (tid == 0) atomicOr(a.status, DLLM_DEV_OFFSETS);
    n = min(max(n, 0), a.max_n);
  }
  const int first = a.first ? a.first[i] : 0;
  const int32_t *src = a.src + (static_cast<size_t>(i) * a.src_heads + (a.src_heads > 1 ? h : 0)) * a.max_n;
  KvPages to = a.c;
  to.table = a.dst_table;
  to.max_pages = a.dst_pages;
  for (int j0 = 0; j0 < n; j0 += kRows) {
    uint4 x[kEach];
    uint8_t sc[kEach];
    float m[kEach];
    long long at[kEach];
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
      const int idx = tid + q * kMoveThreads, j = j0 + idx / kChunks, c = idx % kChunks;
      at[q] = -1;
      if (j >= n) continue;
      const int u = src[j];
      const long long d = static_cast<long long>(first) + j;
      bool bad = d < 0 || d > 0x7fffffffll;
      if (a.in_place) bad |= u < d || (j > 0 && src[j - 1] >= u);
      const int from = bad ? -1 : page_row(a.c, i, u), dest = bad ? -1 : page_row(to, i, static_cast<int>(d));
      if (from < 0 || dest < 0) {
        atomicOr(a.status, DLLM_DEV_PAGE);
        continue;
      }
      const size_t s = from + (static_cast<size_t>(h) << a.c.page_shift);
      at[q] = dest + (static_cast<long long>(h) << a.c.page_shift);
      x[q] = *reinterpret_cast<const uint4 *>(pool + s * ROW + c * 16);
      if (c == 0) {
        if (scale) sc[q] = scale[s];
        if (mass) m[q] = mass[s];
      }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
      const int c = (tid + q * kMoveThreads) % kChunks;
      if (at[q] < 0) continue;
      *reinterpret_cast<uint4 *>(pool + at[q] * ROW + c * 16) = x[q];
      if (c == 0) {
        if (scale) scale[at[q]] = sc[q];
        if (mass) mass[at[q]] = m[q];
      }
    }
    __syncthreads();
  }
}

dllm_status launch_shift(const dllm_kv_pages *pages, const ShiftArgs &g, int B, cudaStream_t s) {
  const int row = pages->dh * (pages->type == DLLM_KV_E4M3 ? 1 : 2);
  void (*kern)(ShiftArgs) = row == 64 ? shift_kernel<64> : row == 128 ? shift_kernel<128> : shift_kernel<256>;
  const cudaError_t e = launch_pdl(kern, dim3(pages->heads, B, 2), dim3(kMoveThreads), 0, s, g);
  return e == cudaSuccess ? DLLM_OK : cuda_error(e);
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" dllm_status dllm_kv_move(const dllm_kv_pages *pages, const dllm_kv_move_args *a, dllm_stream stream) {
  const dllm_status st = check_pages(pages);
  if (st != DLLM_OK) return st;
  if (!a || a->B < 0 || a->max_n < 0 || a->max_pages < 0 || a->dst_pages < 0) return DLLM_ERR_INVALID_ARG;
  if (a->src_heads != 1 && a->src_heads != pages->heads) return DLLM_ERR_INVALID_ARG;
  if (a->B > 4096 || a->max_n >= (1 << 30)) return DLLM_ERR_UNSUPPORTED;
  if (a->B == 0 || a->max_n == 0) return DLLM_OK;
  const dllm_status sp = check_page_pointers(pages);
  if (sp != DLLM_OK) return sp;
  if (!a->src || !a->count || (!a->page_table && a->max_pages > 0) || (a->dst_table && a->dst_table == a->page_table && a->dst_pages != a->max_pages))
    return DLLM_ERR_INVALID_ARG;
  ShiftArgs g{};
  g.c = device_pages(pages, a->page_table, a->max_pages);
  g.in_place = !a->dst_table || a->dst_table == a->page_table;
  g.dst_table = g.in_place ? a->page_table : a->dst_table;
  g.dst_pages = g.in_place ? a->max_pages : a->dst_pages;
  g.src = a->src; g.src_heads = a->src_heads; g.max_n = a->max_n; g.count = a->count; g.first = a->first; g.mass = a->mass;
  cudaError_t e = cudaGetSymbolAddress(reinterpret_cast<void **>(&g.status), g_status_evict);
  if (e != cudaSuccess) return cuda_error(e);
  const dllm_status sl = launch_shift(pages, g, a->B, static_cast<cudaStream_t>(stream));
  return sl == DLLM_OK ? launch_status() : sl;
}

extern "C" dllm_status dllm_kv_evict(const dllm_kv_pages *pages, const dllm_kv_evict_args *a, dllm_stream stream) {
  const dllm_status st = check_pages(pages);
  if (st != DLLM_OK) return st;
  if (!a || a->B < 0 || a->max_pages < 0 || a->dst_pages < 0 || a->budget < 1 || a->max_kv < 0 || a->sinks < 0 || a->recent < 0)
    return DLLM_ERR_INVALID_ARG;
  if (a->B > 4096 || a->max_kv >= (1 << 30) || a->budget >= (1 << 30)) return DLLM_ERR_UNSUPPORTED;
  if (static_cast<long long>(a->sinks) + a->recent > a->budget) return DLLM_ERR_INVALID_ARG;
  if (a->B == 0) return DLLM_OK;
  const dllm_status sp = check_page_pointers(pages);
  if (sp != DLLM_OK) return sp;
  if (!a->mass || !a->kv_len || (!a->page_table && a->max_pages > 0) || !a->new_len || !a->keep ||
      (a->dst_table && a->dst_table == a->page_table && a->dst_pages != a->max_pages))
    return DLLM_ERR_INVALID_ARG;
  SelectArgs g{};
  g.c = device_pages(pages, a->page_table, a->max_pages);
  const long long table = static_cast<long long>(a->max_pages) * pages->page_size;   // rows beyond the table are not there
  g.mass = a->mass; g.kv_len = a->kv_len; g.new_len = a->new_len; g.keep = a->keep;
  g.budget = a->budget; g.max_kv = static_cast<int>(table < a->max_kv ? table : a->max_kv);
  g.sinks = a->sinks; g.recent = a->recent;
  cudaError_t e = cudaGetSymbolAddress(reinterpret_cast<void **>(&g.status), g_status_evict);
  if (e != cudaSuccess) return cuda_error(e);
  ShiftArgs m{};
  m.c = g.c;
  m.in_place = !a->dst_table || a->dst_table == a->page_table;
  m.dst_table = m.in_place ? a->page_table : a->dst_table;
  m.dst_pages = m.in_place ? a->max_pages : a->dst_pages;
  m.src = a->keep; m.src_heads = pages->heads; m.max_n = a->budget; m.count = a->new_len;
  m.mass = a->move_mass ? a->mass : nullptr;
  m.status = g.status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  e = launch_pdl(select_kernel, dim3(pages->heads, a->B), dim3(kSelThreads), 0, s, g);
  if (e != cudaSuccess) return cuda_error(e);
  const dllm_status sl = launch_shift(pages, m, a->B, s);
  return sl == DLLM_OK ? launch_status(2) : sl;
}
