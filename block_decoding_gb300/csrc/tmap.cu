// Host side of the TMA path: the tensor-map encoder (fetched from the driver
// at run time, so the library has no link-time driver dependency) and the
// per-device SM count used to size persistent grids.
#include <mutex>

#include "umma_pages.cuh"

namespace dllm {

namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                                  CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);

EncodeTiledFn encoder() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

}  // namespace

bool make_tmap_bf16_sw128(CUtensorMap *map, const void *base, uint64_t rows, uint64_t cols, uint64_t ld,
                          uint32_t box_rows) {
  EncodeTiledFn fn = encoder();
  if (!fn || !base || rows == 0 || cols == 0 || (ld * 2) % 16 != 0 || box_rows == 0 || box_rows > 256)
    return false;
  if (reinterpret_cast<uintptr_t>(base) % 16 != 0) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {ld * 2};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_tmap_page_rows(CUtensorMap *map, const void *base, uint64_t rows, int dh, int elem_bytes,
                         uint32_t box_rows) {
  EncodeTiledFn fn = encoder();
  if (!fn || !base || rows == 0 || rows % 8 || box_rows % 8 || reinterpret_cast<uintptr_t>(base) % 16) return false;
  const cuuint64_t row = static_cast<cuuint64_t>(dh) * elem_bytes;      // 64, 128 or 256 bytes
  const cuuint32_t piece = row < 128 ? static_cast<cuuint32_t>(row) : 128u, pieces = static_cast<cuuint32_t>(row / piece);
  cuuint64_t dims[4] = {piece / elem_bytes, 8, pieces, rows / 8};
  cuuint64_t strides[3] = {row, piece, row * 8};
  cuuint32_t box[4] = {piece / elem_bytes, 8, pieces, box_rows / 8};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, elem_bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4,
            const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            piece == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int num_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  static std::mutex mu;
  static int cache[64] = {0};
  std::lock_guard<std::mutex> lock(mu);
  if (dev >= 0 && dev < 64 && cache[dev]) return cache[dev];
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
  if (dev >= 0 && dev < 64) cache[dev] = n;
  return n;
}

namespace {
thread_local int t_sm_budget = 0;   // 0: every SM
}  // namespace

int sm_budget() {
  const int n = num_sms();
  return t_sm_budget > 0 && t_sm_budget < n ? t_sm_budget : n;
}

SmBudget::SmBudget(int sms) : prev(t_sm_budget) { t_sm_budget = sms; }
SmBudget::~SmBudget() { t_sm_budget = prev; }

}  // namespace dllm
