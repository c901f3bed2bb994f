// What the attention kernels over the paged cache share: the call as the
// device sees it, which keys a row sees, and the split of the work.
#pragma once

#include "pages.cuh"
#include "umma.cuh"

namespace dllm {

struct PagedArgs {
  KvPages c;
  const uint16_t *q;
  long long q_stride;
  void *out;
  int out_fp32;
  float *lse;
  const int32_t *q_off, *kv_len, *q_pos;
  int B, Hq, group, max_q, max_kv, q_rows;
  float scale_log2;
  int left, right, sinks;
  int uniform;      // > 0: no item is divided
  unsigned int *status;
  // partial results of items whose keys several CTAs share
  float *part_o;
  float2 *part_ml;
  int4 *join;
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
  // positions beyond +-2^30 see what the nearest one there sees
  x.pos = a.q_pos ? min(max(a.q_pos[i], -(1 << 30)), 1 << 30) : x.L - x.W;
  if (bad && report) atomicOr(a.status, DLLM_DEV_OFFSETS);
  return x;
}

// Keys [lo, hi) that a row at position p sees apart from the sinks.
__device__ __forceinline__ void visible(const PagedArgs &a, long long p, int L, int &lo, int &hi) {
  hi = a.right < 0 ? L : static_cast<int>(min(static_cast<long long>(L), max(p + a.right + 1, 0ll)));
  lo = a.left < 0 ? 0 : static_cast<int>(min(max(p - a.left, 0ll), 1ll << 30));
}

constexpr int kTile = 128;   // keys per tile

// The key tiles of one tile of query rows: `count` of them, the j-th being
// tile j for j < sink_tiles (those before the window that hold sinks) and
// window tile j - sink_tiles after. [lo, hi) is the union of its rows' keys
// apart from the sinks.
struct TileList {
  int lo, hi, sink_tiles, first, count;
  int lo_last, hi_first;   // every row sees [lo_last, hi_first)
  __device__ __forceinline__ int tile(int j) const { return j < sink_tiles ? j : first + j - sink_tiles; }
};

// Flat rows r = t * group + g of one cached head, tiles of `n` of them.
__device__ __forceinline__ TileList tile_list(const PagedArgs &a, const Extent &x, int rt, int n) {
  TileList t;
  const long long t0 = (static_cast<long long>(rt) * n) / a.group;
  const long long t1 = min((static_cast<long long>(rt + 1) * n - 1) / a.group, static_cast<long long>(x.W) - 1);
  visible(a, x.pos + t0, x.L, t.lo, t.hi_first);
  visible(a, x.pos + t1, x.L, t.lo_last, t.hi);
  const int s = min(a.sinks, t.hi);
  t.first = t.lo / kTile;
  int n_win = 0;
  if (t.hi > t.lo) {
    n_win = (t.hi + kTile - 1) / kTile - t.first;
    t.sink_tiles = min((s + kTile - 1) / kTile, t.first);
  } else {
    t.sink_tiles = (s + kTile - 1) / kTile;
  }
  t.count = t.sink_tiles + n_win;
  return t;
}

// Tiles that every row tile of the request is given (at least one, so that
// rows without keys are written too): no fewer than any of them needs. With
// `uniform` every item of the call is given that many, so that equal pieces
// of whole items divide none.
__device__ __forceinline__ int tiles_per_item(const PagedArgs &a, const Extent &x, int n) {
  if (a.uniform) return a.uniform;
  int lo, hi;
  visible(a, static_cast<long long>(x.pos) + x.W - 1, x.L, lo, hi);
  int most = (hi + kTile - 1) / kTile;
  if (a.left >= 0 && a.right >= 0) {
    // window keys of one row tile: left + right + 1 of a row, and the rows' spread
    const long long keys = static_cast<long long>(a.left) + a.right + 1 + (n - 1) / a.group + 1;
    const long long win = (keys - 1) / kTile + 2 + (min(a.sinks, hi) + kTile - 1) / kTile;
    most = static_cast<int>(min(static_cast<long long>(most), win));
  }
  return max(most, 1);
}

}  // namespace dllm
