// Trees of drafted tokens: which tokens of its request every token descends
// from, as the bits that attention over the cache takes (dllm_tree_attn), and
// how deep it lies.
//
// One CTA per request. Ancestors by pointer doubling: a token's bits cover the
// path up to, not including, the token that its jump names; taking over that
// token's bits and its jump doubles the path, so a tree of depth d takes
// log2(d) + 1 rounds. Latency bound (a request has some hundred bytes): the
// chain offsets -> parents -> rounds -> stores, 3 us for 32 requests of 64 tokens
// or fewer.
#include "pages.cuh"

namespace dllm {

DLLM_DEFINE_STATUS(tree)

namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) tree_mask_kernel(const int32_t *__restrict__ parent, const int32_t *__restrict__ off,
                                                             int rows, int max_q, uint32_t *__restrict__ mask, int stride,
                                                             int32_t *__restrict__ depth, unsigned int *status) {
  extern __shared__ uint32_t s_bits[];               // [max_q][words], then two arrays of jumps
  const int words = (max_q + 31) / 32, tid = threadIdx.x;
  int *jump = reinterpret_cast<int *>(s_bits + max_q * words), *next = jump + max_q;
  pdl_trigger();
  pdl_wait();
  const int q0 = off[blockIdx.x], given = off[blockIdx.x + 1] - q0;
  int W = given;
  if (q0 < 0 || W < 0 || q0 > rows) W = 0;
  W = min(min(W, rows - q0), max_q);
  if (W != given && tid == 0) atomicOr(status, DLLM_DEV_OFFSETS);
  for (int i = tid; i < W * words; i += kThreads) {
    const int t = i / words, w = i - t * words;
    s_bits[i] = t / 32 == w ? 1u << (t % 32) : 0u;
  }
  bool open = false;
  for (int t = tid; t < W; t += kThreads) {
    int p = parent[q0 + t];
    if (p < -1 || p >= t) {
      atomicOr(status, DLLM_DEV_TREE);
      p = -1;
    }
    jump[t] = p;
    open |= p >= 0;
  }
  while (__syncthreads_or(open)) {
    // (bits that another thread has taken over in this round already are
    // ancestors' too)
    for (int i = tid; i < W * words; i += kThreads) {
      const int t = i / words, p = jump[t];
      if (p >= 0) s_bits[i] |= s_bits[p * words + (i - t * words)];
    }
    open = false;
    for (int t = tid; t < W; t += kThreads) {
      const int p = jump[t], pp = p >= 0 ? jump[p] : -1;
      next[t] = pp;
      open |= pp >= 0;
    }
    int *const x = jump;
    jump = next;
    next = x;
  }
  for (int i = tid; i < W * words; i += kThreads) {
    const int t = i / words;
    mask[static_cast<size_t>(q0 + t) * stride + (i - t * words)] = s_bits[i];
  }
  if (depth)
    for (int t = tid; t < W; t += kThreads) {
      int n = -1;
      for (int w = 0; w < words; ++w) n += __popc(s_bits[t * words + w]);
      depth[q0 + t] = n;
    }
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" dllm_status dllm_tree_mask(const int32_t *parent, const int32_t *off, int rows, int max_q, int B, uint32_t *mask,
                                      int mask_stride, int32_t *depth, dllm_stream stream) {
  if (rows < 0 || max_q < 0 || B < 0 || mask_stride < 0) return DLLM_ERR_INVALID_ARG;
  if (max_q > DLLM_TREE_TOKENS || B > 4096) return DLLM_ERR_UNSUPPORTED;
  const int words = (max_q + 31) / 32;
  if (mask_stride < words) return DLLM_ERR_INVALID_ARG;
  if (rows == 0 || B == 0 || max_q == 0) return DLLM_OK;
  if (!parent || !off || !mask) return DLLM_ERR_INVALID_ARG;
  unsigned int *status;
  cudaError_t e = cudaGetSymbolAddress(reinterpret_cast<void **>(&status), g_status_tree);
  if (e != cudaSuccess) return cuda_error(e);
  const size_t smem = static_cast<size_t>(max_q) * (words + 2) * 4;
  if (smem > 48 * 1024) {
    e = cudaFuncSetAttribute(tree_mask_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return cuda_error(e);
  }
  e = launch_pdl(tree_mask_kernel, dim3(B), dim3(kThreads), smem, static_cast<cudaStream_t>(stream), parent, off, rows, max_q,
                 mask, mask_stride, depth, status);
  if (e != cudaSuccess) return cuda_error(e);
  return launch_status();
}
