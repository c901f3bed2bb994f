// What the attention kernels over the paged cache share: the call as the
// device sees it, which keys a row sees, and the split of the work.
#pragma once

#include "pages.cuh"
#include "umma_pages.cuh"

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
  int whole;        // no item may be divided (there is no workspace)
  unsigned int *status;
  // partial results of items whose keys several CTAs share
  float *part_o;
  float2 *part_ml;
  struct JoinJob *join;
};

// An item that several CTAs shared: its first piece, the number of pieces,
// its first flat row, the request's flat rows, first query row and the head.
struct JoinJob {
  int slot, parts, r0, rows, q0, h, pad0, pad1;
};

// Request i clipped to the buffers and host bounds: query rows [q0, q0 + W),
// L keys. The position of the first row is that of the request as it is given.
struct Extent {
  int q0, W, L, pos;
};

__device__ __forceinline__ Extent paged_extent(const PagedArgs &a, int i, bool report) {
  Extent x;
  bool bad = false;
  x.q0 = a.q_off[i];
  x.W = a.q_off[i + 1] - x.q0;
  x.L = a.kv_len[i];
  const long long last = static_cast<long long>(x.L) - x.W;   // (of W < 0 no row is left)
  if (x.q0 < 0 || x.W < 0 || x.q0 > a.q_rows) { bad = true; x.q0 = 0; x.W = 0; }
  if (x.W > a.q_rows - x.q0) { bad = true; x.W = a.q_rows - x.q0; }
  if (x.W > a.max_q) { bad = true; x.W = a.max_q; }
  if (x.L < 0) { bad = true; x.L = 0; }
  if (x.L > a.max_kv) { bad = true; x.L = a.max_kv; }
  // (what kv_len and q_off give is within 32 bits but for lengths that are out of bounds by as much)
  x.pos = a.q_pos ? a.q_pos[i] : static_cast<int>(min(max(last, -0x80000000ll), 0x7fffffffll));
  if (bad && report) atomicOr(a.status, DLLM_DEV_OFFSETS);
  return x;
}

// Keys [lo, hi) that row t of a request whose first row is at position pos sees
// apart from the sinks. (64 bits: positions are any 32-bit numbers.)
__device__ __forceinline__ void visible(const PagedArgs &a, int pos, int t, int L, int &lo, int &hi) {
  const long long p = static_cast<long long>(pos) + t;
  hi = a.right < 0 ? L : static_cast<int>(min(static_cast<long long>(L), max(p + a.right + 1, 0ll)));
  lo = a.left < 0 ? 0 : static_cast<int>(min(max(p - a.left, 0ll), 0x7fffffffll));
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
  const int t0 = rt * n / a.group, t1 = min(((rt + 1) * n - 1) / a.group, x.W - 1);   // W * group <= 2^30
  visible(a, x.pos, t0, x.L, t.lo, t.hi_first);
  visible(a, x.pos, t1, x.L, t.lo_last, t.hi);
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
// rows without keys are written too): no fewer than any of them needs.
__device__ __forceinline__ int tiles_per_item(const PagedArgs &a, const Extent &x, int n) {
  int lo, hi;
  visible(a, x.pos, x.W - 1, x.L, lo, hi);
  int most = (hi + kTile - 1) / kTile;
  if (a.left >= 0 && a.right >= 0) {
    // window keys of one row tile: left + right + 1 of a row, and the rows' spread
    const unsigned keys = static_cast<unsigned>(a.left) + a.right + 1 + (n - 1) / a.group + 1;
    const unsigned win = (keys - 1) / kTile + 2 + (min(a.sinks, hi) + kTile - 1) / kTile;
    most = static_cast<int>(min(static_cast<unsigned>(most), win));
  }
  return max(most, 1);
}

// The work is a line of all items, each as long as its tiles and kItemCost
// more for what every item costs however short it is (rows staged, results
// written: about as much as so many tiles). It is cut into gridDim.x equal
// stretches. Where it takes no longer that way, items stay whole: then every
// item is as long as the longest, and stretches are so many items. (Dividing
// costs an item's fixed part twice, and the joining about kJoinCost tiles.)
// Measured: 64 single tokens over 1 to 8192 keys (e4m3, 8 x 4 heads, dh 128)
// take 161 us with a cost of 0, 132 with 3, 124 with 6, 131 with 12; 16 blocks
// of 64 to 96 rows over 352 to 1120 keys (32 heads, bf16) 60, 54, 54, 55;
// longer items hardly differ. A join cost of 0 or 12 for 4 changes those blocks
// by 1 %; the other calls divide their items, or leave them whole, with each.
// Items that are left whole, against all of them divided: 32 tokens that see
// 4096 keys (128 items of 35 tiles) 41.8 and 42.5 us (e4m3), 50.7 and 53.0
// (bf16), that see 1024 (11 tiles) 23.5 and 24.8, 23.1 and 25.4; 2000 rows under
// windows of 256 to 4096 (128 items) 5 to 22 % longer divided.
constexpr int kItemCost = 6, kJoinCost = 4;
constexpr int kMinTiles = 4;     // fewest tiles a CTA is given: each piece costs a prologue and a join (1 or 8: the same time
                                 // for single tokens over 257 keys and 20000 to 40000)

// Where this CTA's stretch starts.
struct Start {
  long long residual;   // length of request i before it
  long long left;       // its length
  long long per;        // the length of every stretch
  int i;
  int whole;            // > 0: tiles of every item, none is divided
};

struct Scan {           // sums and maxima of the warps
  long long length[16];
  int items[16], most[16];
};

// x / y of numbers >= 0, in 32 bits where they fit: every launch begins with
// such divisions, one after another, and those in 64 bits take some 400 cycles.
__device__ __forceinline__ long long quotient(long long x, long long y) {
  if ((x | y) >> 32) return x / y;
  return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
}

// Every thread of the CTA takes part. (A single token over 257 keys takes 8.8 us
// this way, 9.1 with the warps' sums added up one after the other and 64-bit
// divisions.)
__device__ __forceinline__ void find_start(const PagedArgs &a, int n_rows, Scan *s_scan, Start *s_start) {
  const int nt = blockDim.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int chunk = (a.B + nt - 1) / nt;
  const int i0 = tid * chunk, i1 = min(a.B, i0 + chunk);
  auto request = [&](int i, bool report, int &items, int &n) {
    const Extent x = paged_extent(a, i, report);
    items = (x.W * a.group + n_rows - 1) / n_rows * a.c.heads;
    n = items ? tiles_per_item(a, x, n_rows) : 0;
  };
  long long length = 0;
  int items = 0, most = 0, k = 0, n = 0;   // (k, n: of the last request)
  for (int i = i0; i < i1; ++i) {
    request(i, blockIdx.x == 0, k, n);
    items += k;
    length += static_cast<long long>(k) * (n + kItemCost);
    most = max(most, n);
  }
  long long length_up = length;
  int items_up = items;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, length_up, o);
    const int z = __shfl_up_sync(0xffffffffu, items_up, o);
    if (lane >= o) { length_up += y; items_up += z; }
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 31) {
    s_scan->length[warp] = length_up;
    s_scan->items[warp] = items_up;
    s_scan->most[warp] = most;
  }
  if (tid == 0) s_start->left = 0;
  __syncthreads();
  // the sums of all warps, and of those before this one
  const bool has = lane < nt / 32;
  long long total = has ? s_scan->length[lane] : 0, earlier = lane < warp ? total : 0;
  const int items_of = has ? s_scan->items[lane] : 0;
  most = __reduce_max_sync(0xffffffffu, has ? s_scan->most[lane] : 0);
  const int total_items = __reduce_add_sync(0xffffffffu, items_of);
  items_up += __reduce_add_sync(0xffffffffu, lane < warp ? items_of : 0);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    earlier += __shfl_xor_sync(0xffffffffu, earlier, o);
  }
  length_up += earlier;
  const long long even = max(quotient(total + gridDim.x - 1, gridDim.x), static_cast<long long>(kMinTiles));
  const int each = (total_items + gridDim.x - 1) / gridDim.x;      // whole items of a CTA
  const bool whole = a.whole || static_cast<long long>(each) * (most + kItemCost) <= even + kItemCost + kJoinCost;
  const long long before = whole ? items_up - items : length_up - length, mine = whole ? items : length;
  const long long begin = (whole ? each : even) * blockIdx.x, end = whole ? total_items : total;
  if (begin >= before && begin < before + mine) {
    long long at = before;
    for (int i = i0; i < i1; ++i) {
      if (chunk > 1) request(i, false, k, n);
      const long long m = whole ? k : static_cast<long long>(k) * (n + kItemCost);
      if (begin < at + m) {
        const int unit = whole ? most + kItemCost : 1;
        s_start->i = i;
        s_start->residual = (begin - at) * unit;
        s_start->left = min(whole ? static_cast<long long>(each) : even, end - begin) * unit;
        s_start->per = even;
        s_start->whole = whole ? most : 0;
        break;
      }
      at += m;
    }
  }
  __syncthreads();
}

// The pieces of work of one CTA, walked by the warps that prepare them.
struct Walk {
  const PagedArgs &a;
  int n_rows, whole_tiles;
  int i, item, at;         // request, item of the request, place in the item
  long long left;          // length still to come
  Extent x;
  int n, items, row_tiles; // tiles of an item, items of the request
  // the current piece
  int h, rt, j0, j1;       // head, row tile, tiles [j0, j1) of it
  TileList t;
  __device__ __forceinline__ Walk(const PagedArgs &args, int rows, const Start &s) 
      : a(args), n_rows(rows), whole_tiles(s.whole), left(s.left) {
    if (left <= 0) return;
    i = s.i;
    load();
    item = static_cast<int>(quotient(s.residual, n + kItemCost));
    at = static_cast<int>(s.residual - static_cast<long long>(item) * (n + kItemCost));
  }
  __device__ __forceinline__ void load() {
    x = paged_extent(a, i, false);
    row_tiles = (x.W * a.group + n_rows - 1) / n_rows;
    items = row_tiles * a.c.heads;
    n = whole_tiles ? whole_tiles : items ? tiles_per_item(a, x, n_rows) : 0;
  }
  // The next piece that has tiles: a cut within an item's fixed cost leaves
  // the whole item to the CTA behind it.
  __device__ __forceinline__ bool next() {
    do {
      if (left <= 0) return false;
      while (item >= items) {
        if (++i >= a.B) return false;
        item = at = 0;
        load();
      }
      h = item / row_tiles;
      rt = item - h * row_tiles;
      const int end = static_cast<int>(min(static_cast<long long>(n + kItemCost), at + left));
      j0 = max(at - kItemCost, 0);
      j1 = max(end - kItemCost, 0);
      left -= end - at;
      if (end == n + kItemCost) { at = 0; ++item; } else { at = end; }
    } while (j1 <= j0);
    t = tile_list(a, x, rt, n_rows);
    return true;
  }
  __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == n; }
  __device__ __forceinline__ int tiles() const { return max(min(j1, t.count) - j0, 0); }   // that hold visible keys
};

// What is to join for the item that the CTA's piece `w` begins (its partial
// results in `slot`): the item's other pieces are the first slots of the next
// CTAs. Returns whether the item is divided there.
__device__ __forceinline__ bool begin_join(const PagedArgs &a, const Walk &w, const Start &s, int slot) {
  if (w.j0 != 0 || w.whole()) return false;
  const int parts = 1 + static_cast<int>((w.n - w.j1 + s.per - 1) / s.per);   // (the fixed cost lies before tile 0)
  a.join[blockIdx.x] = JoinJob{slot, parts, w.rt * w.n_rows, w.x.W * a.group, w.x.q0, w.h, 0, 0};
  return true;
}

// The query rows of the piece `w` on their way to L2, by one warp.
__device__ __forceinline__ void prefetch_rows(const PagedArgs &a, const Walk &w, int n_rows, int dh, int lane) {
  const int rows = w.x.W * a.group, lines = dh / 64;   // 128-byte lines of a row
  for (int idx = lane; idx < n_rows * lines; idx += 32) {
    const int r = w.rt * n_rows + idx / lines, t = r / a.group;
    if (r >= rows) break;
    l2_prefetch_line(a.q + (w.x.q0 + t) * a.q_stride + (w.h * a.group + r - t * a.group) * dh + idx % lines * 64);
  }
}

// The warp that loads the K and V tiles of a CTA's pieces: one box per page
// and tile, K tile n to stage n % KS, V tile n to stage KS + n % VS. A tile's
// V is asked for LEAD tiles after its K: it is read that much later, and
// until then its space would hold nothing but other loads back. With e4m3
// pages (SCALES > 0) a tile's scale bytes, K's then V's, go to a ring of
// SCALES slots with the truth of which pages the tile has.
template <int DH, int ELEM, int KS, int VS, int LEAD, int SCALES>
__device__ __forceinline__ void load_tiles(const PagedArgs &a, const Start &start, int n_rows, const CUtensorMap *tm_k,
                                           const CUtensorMap *tm_v, uint8_t *ring, uint64_t *full, uint64_t *empty,
                                           uint8_t *scales, uint32_t *pages_of, uint64_t *sc_full, volatile int *abort,
                                           int lane) {
  constexpr int kRow = DH * ELEM, kRaw = kTile * kRow;
  const int per_tile = kTile >> a.c.page_shift, page_rows = 1 << a.c.page_shift;
  const int none = static_cast<int>((static_cast<long long>(a.c.num_pages) * a.c.heads << a.c.page_shift) / 8);
  Walk w(a, n_rows, start);
  bool bad = false, ok = true;
  uint32_t nk = 0, nv = 0;     // K and V tiles asked for
  int lag[LEAD + 1];           // pages of the tiles whose V is not
  // tile n's box of this lane's page (8-row group g)
  auto load = [&](const CUtensorMap *tm, uint32_t st, uint32_t round, int g) {
    if (round > 0) ok = ok && warp_wait(&empty[st], (round - 1) & 1, abort);
    if (!ok) return;
    if (lane == 0) mbar_arrive_expect_tx(&full[st], kRaw);
    __syncwarp();
    if (lane < per_tile) tma_load_4d(ring + st * kRaw + lane * page_rows * kRow, tm, &full[st], g);
  };
  auto load_v = [&](int g) {
    load(tm_v, KS + nv % VS, nv / VS, g);
    if (ok) ++nv;
  };
  while (ok && w.next()) {
    const int nT = w.tiles();
    const int32_t *row = a.c.table + static_cast<size_t>(w.i) * a.c.max_pages;
    // 8-row group of this lane's page of tile j; pages without cached rows read as zeros
    auto group_of = [&](int j) {
      if (lane >= per_tile || j >= w.j0 + nT) return none;
      const int u = w.t.tile(j) * kTile + lane * page_rows;
      if (u >= w.x.L) return none;
      const int page = __ldg(row + (u >> a.c.page_shift));
      if (page < 0 || page >= a.c.num_pages) { bad = true; return none; }
      return ((page * a.c.heads + w.h) << a.c.page_shift) / 8;
    };
    int g = group_of(w.j0);
    for (int j = w.j0; ok && j < w.j0 + nT; ++j) {
      const int g_next = group_of(j + 1);     // its latency passes behind this tile's waits
      load(tm_k, nk % KS, nk / KS, g);
      if (!ok) break;
      if constexpr (SCALES > 0) {
        const bool live = g < none;
        const uint32_t slot = nk % SCALES, pages = __ballot_sync(0xffffffffu, live);
        if (lane == 0) {
          pages_of[slot] = pages;
          mbar_arrive_expect_tx(&sc_full[slot], __popc(pages) * page_rows * 2);
        }
        __syncwarp();
        if (live) {
          uint8_t *dst = scales + slot * (2 * kTile) + lane * page_rows;
          bulk_load(dst, a.c.k_scale + static_cast<size_t>(g) * 8, page_rows, &sc_full[slot]);
          bulk_load(dst + kTile, a.c.v_scale + static_cast<size_t>(g) * 8, page_rows, &sc_full[slot]);
        }
      }
      ++nk;
#pragma unroll
      for (int i = LEAD; i > 0; --i) lag[i] = lag[i - 1];
      lag[0] = g;
      if (nk > LEAD) load_v(lag[LEAD]);
      g = g_next;
    }
  }
#pragma unroll
  for (int i = LEAD - 1; i >= 0; --i)
    if (ok && nk - nv == static_cast<uint32_t>(i) + 1) load_v(lag[i]);
  if (bad) atomicOr(a.status, DLLM_DEV_PAGE);
  // after an abort: the loads in flight land before the CTA's memory is given up
  if (!ok) {
    if (lane < KS && lane < nk) mbar_drain(&full[lane], ((nk - 1 - lane) / KS) & 1);
    if (lane < VS && lane < nv) mbar_drain(&full[KS + lane], ((nv - 1 - lane) / VS) & 1);
    if constexpr (SCALES > 0)
      if (lane < SCALES && lane < nk) mbar_drain(&sc_full[lane], ((nk - 1 - lane) / SCALES) & 1);
  }
}

// 64 keys of a V tile of e4m3 codes (rows of DH bytes as the load lays them
// out, the first of them key 64 * piece of the tile) to bf16 rows in the
// layout of a bf16 tile, every four elements in the order 0, 2, 1, 3, by 128
// threads (t): half a row each, of key 64 * piece + t % 64. `ready` waits
// until dst may be written; `extra` multiplies four elements by the row's scale.
template <int DH, typename Ready, typename Extra>
__device__ __forceinline__ void convert_v(const uint8_t *raw, uint8_t *dst, int piece, int t, bool seen, Ready ready,
                                          Extra extra) {
  constexpr int kChunks = DH / 32;   // 16-byte pieces of codes
  const int k64 = t % 64, ch = t / 64 * kChunks, key = piece * 64 + k64;
  const uint8_t *src = raw + key * DH;
  uint8_t *out = dst + (k64 / 8) * (8 * DH * 2) + (k64 % 8) * 128;
  uint4 q[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c)   // under the load's swizzle (rows of 128 or 64 bytes)
    q[c] = *reinterpret_cast<const uint4 *>(src + (DH == 128 ? (ch + c) ^ (key & 7) : (ch + c) ^ ((key >> 1) & 3)) * 16);
  ready();
  if (!seen) {   // whatever lies there: 0 * NaN would not be 0
#pragma unroll
    for (int c = 0; c < kChunks; ++c) q[c] = make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const uint2 a0 = extra(e4m3x4_to_bf16_0213(q[c].x)), a1 = extra(e4m3x4_to_bf16_0213(q[c].y));
    const uint2 b0 = extra(e4m3x4_to_bf16_0213(q[c].z)), b1 = extra(e4m3x4_to_bf16_0213(q[c].w));
    const int o = 2 * (ch + c);       // bf16 pieces o and o + 1 of the row, eight to a 128-byte column piece
    uint8_t *d = out + (o / 8) * 1024;
    *reinterpret_cast<uint4 *>(d + ((o & 7) ^ (key & 7)) * 16) = make_uint4(a0.x, a0.y, a1.x, a1.y);
    *reinterpret_cast<uint4 *>(d + (((o + 1) & 7) ^ (key & 7)) * 16) = make_uint4(b0.x, b0.y, b1.x, b1.y);
  }
}

constexpr int kWholeTiles = 4;   // items of no more tiles are not divided
constexpr int kMaxCtas = 192;    // bound of the workspace, above any GB300's SM count
constexpr int kConvKeys = 64;    // keys of one converted V piece
constexpr float kLazy = 8.f;     // a reference maximum moves when a score passes it by more than 2^8
constexpr float kNone = -3.0e38f;   // reference of a row that has seen no key: finite, so that differences are not NaN
constexpr float kLn2 = 0.69314718055994531f;

// Launches the kernel for many rows per cached head (paged_rows.cu) with row
// tiles of n_rows = 128 or 256 on `ctas` CTAs.
dllm_status launch_paged_rows(int dh, bool fp8, int n_rows, const CUtensorMap &tk, const CUtensorMap &tv,
                              const PagedArgs &a, int ctas, cudaStream_t s);

}  // namespace dllm
