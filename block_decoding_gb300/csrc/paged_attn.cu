// Attention of new tokens over the paged K/V cache (bf16 or e4m3 pages):
// grouped query heads, causal or bidirectional, sliding window with the
// first tokens visible.
//
// The work of one (request, cached head) is S^T = K Q^T over the head's
// cached rows, with the query rows that share the head (W rows x group heads)
// as N. Keys are the M = 128 rows of the tensor-core tile, so N is as small
// as the rows are (16, 32 or 64): a single token costs a tile of 16, not of
// 128, the exponentials of one key tile spread over 128 threads (one key
// each, whatever N is), and a key's scales and visibility are one thread's
// scalars. O^T = V^T P^T accumulates in TMEM.
//
// The key tiles of all (request, head, row tile) items form one line that is
// cut into equal pieces, one per CTA: long and short requests balance, and a
// single long one spreads over the whole GPU. An item that a cut divides
// leaves partial (m, l, O) of its pieces in the workspace, and a second
// kernel joins them.
//
// Warp roles:
//   warp 0      TMA: one box per page and tile; K and V tiles alternate in one ring
//   warp 1      S^T MMAs: K tile (A) x query rows (B) into an S buffer
//   warp 2      O^T MMAs: V tile (A, transposed by its descriptor) x P (B)
//   warps 4..11 two softmax warpgroups, one key per thread
//   last four   (e4m3 pages) V codes -> bf16, 64 keys at a time
// A reference maximum per row moves only when a score passes it by more than
// 2^8 (P is bf16: no precision is lost), so most tiles need no maximum at
// all, only the vote that nobody passed it.
//
// e4m3 pages: K codes go to the tensor cores as they are, against the query
// rows split into two e4m3 parts (high + low: exact for elements within 2^-10
// of the row's largest, else 2^-19 of that off), and the key's scale is a
// factor of its thread's scores. V codes become bf16, which holds them
// exactly, and the scale enters P before its one rounding to bf16, so tail
// weights keep their relative precision however small they are.
#include "paged.cuh"

namespace dllm {

DLLM_DEFINE_STATUS(paged)

namespace {

constexpr int kPBuf = 2, kCBuf = 2;
constexpr int kConvKeys = 64;    // keys of one converted V piece
constexpr int kMinTiles = 2;     // fewest tiles a CTA is given: each piece costs a prologue and a join
constexpr int kMaxCtas = 192;    // bound of the workspace, above any GB300's SM count

template <int DH, bool FP8, int N>
struct Cfg {
  // Two softmax warpgroups. With up to 32 columns they take every other key
  // tile (each with its own references, sums and O, merged at the end): the
  // steps of one tile depend on each other, and two tiles under way hide
  // that. With 64 columns each takes 32 of them, of every tile.
  static constexpr bool kByTile = N <= 32;
  static constexpr int kCols = kByTile ? N : N / 2;             // columns of one group
  static constexpr int kSBuf = kByTile ? 4 : 3;
  static constexpr int kConvWarp0 = 12;
  static constexpr int kThreads = 32 * (kConvWarp0 + (FP8 ? 4 : 0));
  // registers a thread: what the TMA and MMA warps and the converters do not
  // need goes to the softmax groups (the sum is the launch's)
  static constexpr int kRegsIssue = FP8 ? 64 : 72, kRegsSoft = FP8 ? 176 : 216, kRegsConv = 96;
  static_assert(FP8 ? kRegsIssue + 2 * kRegsSoft + kRegsConv <= 4 * 128 : kRegsIssue + 2 * kRegsSoft <= 3 * 168, "registers");
  static constexpr int kRaw = kTile * DH * (FP8 ? 1 : 2);       // one K or V tile as it is cached
  static constexpr int kGroup8 = 8 * DH * (FP8 ? 1 : 2);        // eight cached rows
  static constexpr int kVGroup8 = 8 * DH * 2;                   // eight bf16 rows of V
  static constexpr int kP = kTile * N * 2;
  static constexpr int kQ = N * DH * 2;                         // bf16, or two e4m3 parts
  static constexpr int kConv = FP8 ? kCBuf * kConvKeys * DH * 2 : 0;
  static constexpr int kMisc = FP8 ? 12288 : 8192;              // row tables, scales, barriers, alignment
  static constexpr int kFixed = kConv + kPBuf * kP + kQ + kMisc;
  static constexpr int kMaxStages = (232448 - kFixed) / kRaw;
  // even, so that K tiles have the even stages; 192 KB in flight are enough
  static constexpr int kStages = (kMaxStages * kRaw > 196608 ? 196608 / kRaw : kMaxStages) & ~1;
  static constexpr int kOffConv = kStages * kRaw;
  static constexpr int kOffP = kOffConv + kConv;
  static constexpr int kOffQ = kOffP + kPBuf * kP;
  static constexpr int kOffMisc = kOffQ + kQ;
  static constexpr int kBytes = kOffMisc + kMisc;
  // Scales of a tile's keys. A slot is written again once the K stage of the
  // tile kStages / 2 before it is free: that tile's S^T is done, so the
  // scores and scales of every tile up to kSBuf before that one are read.
  static constexpr int kScaleSlots = FP8 ? kStages / 2 + kSBuf + 1 : 0;
  static constexpr uint32_t kTmemCols = N * (kByTile ? 8 : 4);  // S buffers and O (kSBuf + 1 or 2, a power of two)
  static_assert(kStages >= 4 && kBytes <= 232448, "shared memory");
};

// What the softmax needs to know of the row tile's rows.
template <int N>
struct RowInfo {
  int lo[N], hi[N];   // the keys the row sees, apart from the sinks
  int out[N];         // row of out [q_rows * Hq], or -1: not a query row
  float scale[N];     // e4m3 parts: what the query row was divided by
};

// The pieces of work of one CTA, walked alike by every warp.
struct Walk {
  const PagedArgs &a;
  int n_rows;
  int i, item, j;          // request, item of the request, tile of the item
  long long left;          // tiles of this CTA still to come
  Extent x;
  int n, items, row_tiles;
  // the current piece
  int h, rt, j0, j1;       // head, row tile, tiles [j0, j1) of it
  TileList t;
  __device__ __forceinline__ Walk(const PagedArgs &args, int rows) : a(args), n_rows(rows) {}
  __device__ __forceinline__ void load() {
    x = paged_extent(a, i, false);
    row_tiles = (x.W * a.group + n_rows - 1) / n_rows;
    items = row_tiles * a.c.heads;
    n = items ? tiles_per_item(a, x, n_rows) : 0;
  }
  __device__ __forceinline__ bool next() {
    if (left <= 0) return false;
    while (item >= items) {
      if (++i >= a.B) return false;
      item = 0;
      load();
    }
    h = item / row_tiles;
    rt = item - h * row_tiles;
    j0 = j;
    j1 = static_cast<int>(min(static_cast<long long>(n), j + left));
    left -= j1 - j0;
    if (j1 == n) { j = 0; ++item; } else { j = j1; }
    t = tile_list(a, x, rt, n_rows);
    return true;
  }
  __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == n; }
  __device__ __forceinline__ int tiles() const { return max(min(j1, t.count) - j0, 0); }   // that hold visible keys
};

// Where this CTA starts: the total of all items' tiles, cut into gridDim.x
// pieces. Every thread of the CTA takes part; s_scan holds 32 values.
struct Start {
  long long residual;   // tiles of request i before this CTA's first
  long long left;       // tiles of this CTA
  long long per;        // tiles of every CTA
  int i;
};

__device__ __forceinline__ long long request_tiles(const PagedArgs &a, int i, int n_rows, bool report) {
  const Extent x = paged_extent(a, i, report);
  const long long items = static_cast<long long>((static_cast<long long>(x.W) * a.group + n_rows - 1) / n_rows) * a.c.heads;
  return items ? items * tiles_per_item(a, x, n_rows) : 0;
}

__device__ void find_start(const PagedArgs &a, int n_rows, int min_tiles, long long *s_scan, Start *s_start) {
  const int nt = blockDim.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int chunk = (a.B + nt - 1) / nt;
  const int i0 = tid * chunk, i1 = min(a.B, i0 + chunk);
  long long mine = 0;
  for (int i = i0; i < i1; ++i) mine += request_tiles(a, i, n_rows, blockIdx.x == 0);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_scan[warp] = incl;
  if (tid == 0) s_start->left = 0;
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < nt / 32; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  long long per = max((total + gridDim.x - 1) / gridDim.x, static_cast<long long>(min_tiles));
  if (a.uniform) per = (per + a.uniform - 1) / a.uniform * a.uniform;
  const long long begin = per * blockIdx.x;
  const long long excl = before + incl - mine;
  if (begin >= excl && begin < excl + mine) {
    long long at = excl;
    for (int i = i0; i < i1; ++i) {
      const long long m = request_tiles(a, i, n_rows, false);
      if (begin < at + m) {
        s_start->i = i;
        s_start->residual = begin - at;
        s_start->left = min(per, total - begin);
        s_start->per = per;
        break;
      }
      at += m;
    }
  }
  __syncthreads();
}

// v[k] of every lane reduced over the warp's lanes, for CNT values: lane c
// (mod CNT) ends with the result of value c. CNT - 1 shuffles (+ 1 for 16).
template <int CNT, typename Op>
__device__ __forceinline__ float reduce_columns(float (&v)[CNT], int lane, Op op) {
#pragma unroll
  for (int o = CNT / 2; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int k = 0; k < o; ++k) {
      const float send = up ? v[k] : v[k + o], keep = up ? v[k + o] : v[k];
      v[k] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
    }
  }
  float r = v[0];
#pragma unroll
  for (int o = CNT; o < 32; o <<= 1) r = op(r, __shfl_xor_sync(0xffffffffu, r, o));
  return r;
}

// Scores of a key at position u in the columns whose rows do not see it.
template <int CNT>
__device__ __forceinline__ void mask_columns(float (&x)[CNT], const int *lo, const int *hi, int u, int sinks) {
#pragma unroll
  for (int e = 0; e < CNT; ++e)
    if (!(u < hi[e] && (u >= lo[e] || u < sinks))) x[e] = -INFINITY;
}

template <int CNT>
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[CNT]) {
  if constexpr (CNT == 32) tmem_ld32(addr, r);
  else if constexpr (CNT == 16) tmem_ld16(addr, r);
  else tmem_ld8(addr, r);
}
template <int CNT>
__device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t (&r)[CNT]) {
  if constexpr (CNT == 32) tmem_st32(addr, r); else tmem_st16(addr, r);
}

// Query rows [c0, c0 + COLS) of the row tile into shared memory as the B
// operand of S^T (core matrices along K, row groups of 8), by 128 threads,
// with what the softmax needs to know of each row.
template <int DH, bool FP8, int N, int COLS>
__device__ __forceinline__ void stage_queries(const PagedArgs &a, const Walk &w, uint8_t *sq, RowInfo<N> &info, int c0, int tid) {
  const int rows = w.x.W * a.group;
  constexpr int kChunks = DH / 8;                  // 16-byte chunks of a bf16 row
  constexpr int kPieces = COLS * kChunks;
#pragma unroll
  for (int it = 0; it < (kPieces + 127) / 128; ++it) {
    const int idx = it * 128 + tid;
    if (kPieces % 128 && idx >= kPieces) break;    // whole warps
    const int n = c0 + idx / kChunks, c = idx % kChunks;
    const int r = w.rt * N + n, t = r / a.group, g = r - t * a.group;
    const bool live = r < rows;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (live)
      u = *reinterpret_cast<const uint4 *>(a.q + (w.x.q0 + t) * a.q_stride + (w.h * a.group + g) * DH + c * 8);
    if constexpr (!FP8) {
      *reinterpret_cast<uint4 *>(sq + (n / 8) * (kChunks * 128) + c * 128 + (n % 8) * 16) = u;
    } else {
      // scaled by a power of two into (224, 448], then hi = rn(x), lo = rn(x - hi)
      const uint32_t m2 = max_mag(u, 0);
      uint32_t m = max(m2 & 0xffffu, m2 >> 16);
#pragma unroll
      for (int o = kChunks / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      const int byte = scale_byte(m);
      float x[8];
      unpack8(u, x);
      const float f = __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float p = x[2 * e] * f, q = x[2 * e + 1] * f;
        const uint16_t hh = f32_to_e4m3x2(p, q);
        const float2 b = e4m3x2_to_f32(hh);
        hi[e] = hh;
        lo[e] = f32_to_e4m3x2(p - b.x, q - b.y);
      }
      uint8_t *d = sq + (n / 8) * (DH / 16 * 128) + (c / 2) * 128 + (n % 8) * 16 + (c & 1) * 8;
      *reinterpret_cast<uint2 *>(d) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
      *reinterpret_cast<uint2 *>(d + N * DH) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
      if (c == 0) info.scale[n] = scale_of(m < 0x7f80u ? byte : 255);   // a row with an infinity or NaN scores NaN
    }
    if (c == 0) {
      int lo = 0, hi = 0x7fffffff;   // a column that is no row masks nothing; its results go nowhere
      if (live) visible(a, static_cast<long long>(w.x.pos) + t, w.x.L, lo, hi);
      info.lo[n] = lo;
      info.hi[n] = hi;
      info.out[n] = live ? (w.x.q0 + t) * a.Hq + w.h * a.group + g : -1;
    }
  }
}

template <int DH, bool FP8, int N>
__global__ void __launch_bounds__(Cfg<DH, FP8, N>::kThreads, 1)
paged_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const PagedArgs a,
                  const int min_tiles) {
  using C = Cfg<DH, FP8, N>;
  constexpr int kSt = C::kStages, kCols = C::kCols, kSBuf = C::kSBuf;
  constexpr bool kByTile = C::kByTile;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *misc = smem + C::kOffMisc;
  RowInfo<N> *info = reinterpret_cast<RowInfo<N> *>(misc);                // [2]: this piece's and the next one's
  float *m_s = reinterpret_cast<float *>(info + 2);                       // [group][kCols] reference maxima
  float *corr_s = m_s + 2 * kCols;                                        // [group][kCols]
  float *red_s = corr_s + 2 * kCols;                                      // [quarter][group][kCols]
  uint8_t *scales = reinterpret_cast<uint8_t *>(red_s + 8 * kCols);           // [kScaleSlots][K, V][kTile]
  uint32_t *pages_of = reinterpret_cast<uint32_t *>(scales + C::kScaleSlots * 2 * kTile);   // [kScaleSlots]: pages the tile has
  uint64_t *bars = reinterpret_cast<uint64_t *>(pages_of + ((C::kScaleSlots + 1) & ~1));
  uint64_t *full = bars;                    // [kSt] stage loaded
  uint64_t *empty = full + kSt;             // [kSt] stage read by its MMAs (or converted)
  uint64_t *s_full = empty + kSt;           // [kSBuf]
  uint64_t *s_free = s_full + kSBuf;        // [kSBuf]
  uint64_t *p_full = s_free + kSBuf;        // [kPBuf]
  uint64_t *p_free = p_full + kPBuf;        // [kPBuf] O^T MMAs of the tile done
  uint64_t *c_full = p_free + kPBuf;        // [kCBuf] V piece converted
  uint64_t *c_free = c_full + kCBuf;        // [kCBuf] its O^T MMAs done
  uint64_t *sc_full = c_free + kCBuf;       // [kScaleSlots]
  uint64_t *q_full = sc_full + C::kScaleSlots;
  uint64_t *o_full = q_full + 1;
  uint64_t *o_free = o_full + 1;
  long long *s_scan = reinterpret_cast<long long *>(o_free + 1);          // [32]
  Start *start = reinterpret_cast<Start *>(s_scan + 32);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(start + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  static_assert(2 * sizeof(RowInfo<N>) + 12 * kCols * 4 + (2 * kSt + 2 * kSBuf + 2 * kPBuf + 2 * kCBuf + 3) * 8 + 256 + 64 +
                        C::kScaleSlots * (2 * kTile + 8 + 4) + 4 <= C::kMisc - 1024,
                "row tables and barriers");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  if (threadIdx.x == 0) {
    constexpr int kTileWarps = C::kByTile ? 4 : 8;   // softmax warps of one tile
    for (int s = 0; s < kSt; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], FP8 && (s & 1) ? 4 : 1);
    }
    for (int b = 0; b < kSBuf; ++b) { mbar_init(&s_full[b], 1); mbar_init(&s_free[b], kTileWarps); }
    for (int b = 0; b < kPBuf; ++b) { mbar_init(&p_full[b], kTileWarps); mbar_init(&p_free[b], 1); }
    for (int b = 0; b < kCBuf; ++b) { mbar_init(&c_full[b], 4); mbar_init(&c_free[b], 1); }
    for (int b = 0; b < C::kScaleSlots; ++b) mbar_init(&sc_full[b], 1);
    mbar_init(q_full, 8);
    mbar_init(o_full, 1);
    mbar_init(o_free, 8);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t t_o = tmem + kSBuf * N;

  pdl_wait();   // the batch's metadata, the pages and the queries may come from the previous kernel
  find_start(a, N, min_tiles, s_scan, start);
  Walk w(a, N);
  w.left = start->left;
  if (w.left > 0) {
    w.i = start->i;
    w.load();
    w.item = static_cast<int>(start->residual / w.n);
    w.j = static_cast<int>(start->residual - static_cast<long long>(w.item) * w.n);
  }

  if (warp < 4) {
  reg_dealloc<C::kRegsIssue>();
  if (warp == 0) {
    // ------------------------------------------------------------- producer
    const int per_tile = kTile >> a.c.page_shift;
    const int page_rows = 1 << a.c.page_shift;
    const int none = static_cast<int>((static_cast<long long>(a.c.num_pages) * a.c.heads << a.c.page_shift) / 8);
    bool bad = false, ok = true;
    uint32_t n = 0, issued = 0;
    while (ok && w.next()) {
      const int nT = w.tiles();
      const int32_t *row = a.c.table + static_cast<size_t>(w.i) * a.c.max_pages;
      // 8-row group of lane's page of tile j; pages without cached rows read as zeros
      auto group_of = [&](int j) {
        if (lane >= per_tile || j >= w.j0 + nT) return none;
        const long long u = static_cast<long long>(w.t.tile(j)) * kTile + lane * page_rows;
        if (u >= w.x.L) return none;
        const int page = __ldg(row + (u >> a.c.page_shift));
        if (page < 0 || page >= a.c.num_pages) { bad = true; return none; }
        return ((page * a.c.heads + w.h) << a.c.page_shift) / 8;
      };
      int g = group_of(w.j0);
      for (int j = w.j0; j < w.j0 + nT; ++j, ++n) {
        const int g_next = group_of(j + 1);     // its latency passes behind this tile's waits
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const uint32_t pos = 2 * n + kv, st = pos % kSt, round = pos / kSt;
          if (round > 0) ok = mbar_wait(&empty[st], (round - 1) & 1, abort_flag);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          if (lane == 0) mbar_arrive_expect_tx(&full[st], C::kRaw);
          __syncwarp();
          if (lane < per_tile)
            tma_load_4d(smem + st * C::kRaw + lane * page_rows * (C::kGroup8 / 8), kv ? &tm_v : &tm_k, &full[st], g);
          issued = pos + 1;
          if constexpr (FP8) {
            if (kv == 0) {   // the tile's scales, page_rows bytes of each page
              const bool live = g < none;
              const uint32_t slot = n % C::kScaleSlots, pages = __ballot_sync(0xffffffffu, live);
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
          }
        }
        if (!ok) break;
        g = g_next;
      }
    }
    if (bad) atomicOr(a.status, DLLM_DEV_PAGE);
    // after an abort: the loads in flight land before the CTA's memory is given up
    if (!ok && lane < kSt && lane < issued) mbar_drain(&full[lane], ((issued - 1 - lane) / kSt) & 1);
    if constexpr (FP8) {
      const uint32_t tiles = (issued + 1) / 2;
      if (!ok && lane < C::kScaleSlots && lane < tiles)
        mbar_drain(&sc_full[lane], ((tiles - 1 - lane) / C::kScaleSlots) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- S^T MMAs
    uint32_t n = 0, seg = 0;
    bool ok = true;
    const uint32_t sq = smem_u32(smem + C::kOffQ);
    while (ok && w.next()) {
      const int nT = w.tiles();
      if (nT == 0) continue;
      ok = warp_wait(q_full, seg++ & 1, abort_flag);
      for (int j = 0; ok && j < nT; ++j, ++n) {
        const uint32_t pos = 2 * n, st = pos % kSt, b = n % kSBuf;
        ok = warp_wait(&full[st], (pos / kSt) & 1, abort_flag);
        if (ok && n >= kSBuf) ok = warp_wait(&s_free[b], (n / kSBuf - 1) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sk = smem_u32(smem + st * C::kRaw);
        if (elect_one()) {
          if constexpr (!FP8) {
            const uint64_t dk = sw128_desc(sk, 16, C::kGroup8), dq = plain_desc(sq, 128, DH / 8 * 128);
#pragma unroll
            for (int kk = 0; kk < DH / 16; ++kk)
              umma_bf16(tmem + b * N, dk + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), dq + ((kk * 256) >> 4),
                        idesc_bf16(128, N, 0, 0), kk > 0);
          } else {
            const uint64_t dk = DH == 128 ? sw128_desc(sk, 16, C::kGroup8) : sw64_desc(sk, 16, C::kGroup8);
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              const uint64_t dq = plain_desc(sq + part * N * DH, 128, DH / 16 * 128);
#pragma unroll
              for (int kk = 0; kk < DH / 32; ++kk)
                umma_f8(tmem + b * N, dk + ((kk * 32) >> 4), dq + ((kk * 256) >> 4), idesc_e4m3(128, N), part + kk > 0);
            }
          }
          umma_commit(&s_full[b]);
          umma_commit(&empty[st]);
        }
        __syncwarp();
      }
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------- O^T MMAs
    uint32_t n = 0, seg = 0;
    bool ok = true;
    while (ok && w.next()) {
      const int nT = w.tiles();
      if (nT == 0) continue;
      for (int j = 0; ok && j < nT; ++j, ++n) {
        const uint32_t pos = 2 * n + 1, st = pos % kSt, b = n % kPBuf;
        ok = warp_wait(&p_full[b], (n / kPBuf) & 1, abort_flag);
        if (ok && j == 0 && seg > 0) ok = warp_wait(o_free, (seg - 1) & 1, abort_flag);
        if (ok && !FP8) ok = warp_wait(&full[st], (pos / kSt) & 1, abort_flag);
        const uint32_t t_d = kByTile ? t_o + (n & 1) * N : t_o;
        const bool first = j == 0 || (kByTile && j == 1);   // of its accumulator
        const uint64_t dp = plain_desc(smem_u32(smem + C::kOffP + b * C::kP), 128, 2048);
        // bf16: the tile as one piece; e4m3: its converted pieces
        constexpr int kPieces = FP8 ? kTile / kConvKeys : 1, kSteps = 8 / kPieces;
#pragma unroll
        for (int piece = 0; piece < kPieces; ++piece) {
          const uint32_t cn = n * kPieces + piece, cb = cn % kCBuf;
          if (FP8 && ok) ok = warp_wait(&c_full[cb], (cn / kCBuf) & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sv = smem_u32(FP8 ? smem + C::kOffConv + cb * (kConvKeys * DH * 2) : smem + st * C::kRaw);
          if (elect_one()) {
            const uint64_t dv = sw128_desc(sv, 1024, C::kVGroup8);
#pragma unroll
            for (int kk = 0; kk < kSteps; ++kk)
              umma_bf16(t_d, dv + ((kk * 2 * C::kVGroup8) >> 4), dp + (((piece * kSteps + kk) * 256) >> 4),
                        idesc_bf16(DH, N, 1, 1), !first || piece + kk > 0);
            umma_commit(FP8 ? &c_free[cb] : &empty[st]);
            if (piece + 1 == kPieces) {
              umma_commit(&p_free[b]);
              if (j + 1 == nT) umma_commit(o_full);
            }
          }
          __syncwarp();
        }
      }
      ++seg;
    }
  }
  } else if (FP8 && warp >= C::kConvWarp0) {
    // ------------------------------------------------------------- V codes -> bf16
    if constexpr (FP8) {
      reg_dealloc<C::kRegsConv>();
      // a thread takes half of a key's row
      constexpr int kChunks = DH / 32;   // 16-byte pieces of codes
      const int t = (warp - C::kConvWarp0) * 32 + lane, k64 = t % kConvKeys, ch = t / kConvKeys * kChunks;
      uint32_t n = 0;
      while (w.next()) {
        const int nT = w.tiles();
        for (int j = 0; j < nT; ++j, ++n) {
          const uint32_t pos = 2 * n + 1, st = pos % kSt;
          mbar_wait(&full[st], (pos / kSt) & 1, abort_flag);
#pragma unroll 1
          for (int half = 0; half < kTile / kConvKeys; ++half) {
            const uint32_t cn = n * (kTile / kConvKeys) + half, cb = cn % kCBuf;
            const int key = half * kConvKeys + k64, u = w.t.tile(w.j0 + j) * kTile + key;
            const bool seen = u < w.t.hi && (u >= w.t.lo || u < a.sinks);
            const uint8_t *src = smem + st * C::kRaw + key * DH;
            uint8_t *dst = smem + C::kOffConv + cb * (kConvKeys * DH * 2) + (k64 / 8) * C::kVGroup8 + (k64 % 8) * 128;
            uint4 q[kChunks];
#pragma unroll
            for (int c = 0; c < kChunks; ++c)   // under the load's swizzle (rows of 128 or 64 bytes)
              q[c] = *reinterpret_cast<const uint4 *>(src + (DH == 128 ? (ch + c) ^ (key & 7) : (ch + c) ^ ((key >> 1) & 3)) * 16);
            if (cn >= kCBuf) mbar_wait(&c_free[cb], (cn / kCBuf - 1) & 1, abort_flag);
            if (!seen) {   // whatever lies there: 0 * NaN would not be 0
#pragma unroll
              for (int c = 0; c < kChunks; ++c) q[c] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              const uint2 a0 = e4m3x4_to_bf16_0213(q[c].x), a1 = e4m3x4_to_bf16_0213(q[c].y);
              const uint2 b0 = e4m3x4_to_bf16_0213(q[c].z), b1 = e4m3x4_to_bf16_0213(q[c].w);
              const int o = 2 * (ch + c);       // bf16 pieces o and o + 1 of the row, eight to a 128-byte column piece
              uint8_t *d = dst + (o / 8) * 1024;
              *reinterpret_cast<uint4 *>(d + ((o & 7) ^ (key & 7)) * 16) = make_uint4(a0.x, a0.y, a1.x, a1.y);
              *reinterpret_cast<uint4 *>(d + (((o + 1) & 7) ^ (key & 7)) * 16) = make_uint4(b0.x, b0.y, b1.x, b1.y);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c_full[cb]);
          }
          if (lane == 0) mbar_arrive(&empty[st]);
        }
      }
    }
  } else {
    // ------------------------------------------------------------- softmax
    reg_alloc<C::kRegsSoft>();
    const int wg = (warp - 4) >> 2, quarter = warp & 3, tid = threadIdx.x & 127;
    const int key = quarter * 32 + lane;
    const int c0 = kByTile ? 0 : wg * kCols;   // first column of the group's tiles
    const int g0 = wg * kCols;                 // its part of the groups' arrays
    constexpr int kOut = N / 2;                // rows that a group stages and writes
    const int out0 = wg * kOut;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    constexpr float kLazy = 8.f;
    constexpr float kNone = -3.0e38f;   // reference of a row that has seen no key: finite, so that x is not NaN
    const auto maxop = [](float p, float q) { return fmaxf(p, q); };
    const auto addop = [](float p, float q) { return p + q; };
    uint32_t n = 0, seg = 0, o_seg = 0;
    bool more = w.next();
    bool joined = false;       // this CTA's last piece began an item that others finish
    if (more) {
      stage_queries<DH, FP8, N, kOut>(a, w, smem + C::kOffQ, info[0], out0, tid);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && w.tiles() > 0) mbar_arrive(q_full);
    }
    while (more) {
      const RowInfo<N> &ri = info[seg & 1];
      const int nT = w.tiles();
      float l[kCols];
#pragma unroll
      for (int e = 0; e < kCols; ++e) l[e] = 0.f;
      named_bar_sync(3, 256);               // the rows' info is written, the last piece's maxima are read
      if (tid < kCols) m_s[g0 + tid] = kNone;
      named_bar_sync(1 + wg, 128);
      bool first = true;                    // of the group's tiles
      for (int j = 0; j < nT; ++j, ++n) {
        if (kByTile && (n & 1) != wg) continue;
        const uint32_t b = n % kSBuf, pb = n % kPBuf;
        const int key0 = w.t.tile(w.j0 + j) * kTile, u = key0 + key;
        // every row of the tile sees every key of it?
        const bool all_seen = key0 + kTile <= w.t.hi_first && (key0 >= w.t.lo_last || key0 + kTile <= a.sinks);
        const bool seen = u < w.t.hi && (u >= w.t.lo || u < a.sinks);   // this key, by any row
        float c = a.scale_log2, vs = 1.f;
        if constexpr (FP8) {
          const uint32_t slot = n % C::kScaleSlots;
          mbar_wait(&sc_full[slot], (n / C::kScaleSlots) & 1, abort_flag);
          // a key without a page is a row of zeros, one that no row sees may have any scale
          if ((pages_of[slot] >> (key >> a.c.page_shift) & 1) && seen) {
            const uint8_t *sc = scales + slot * (2 * kTile) + key;
            c *= scale_of(sc[0]);
            vs = scale_of(sc[kTile]);
          }
        }
        mbar_wait(&s_full[b], (n / kSBuf) & 1, abort_flag);
        tc_fence_after();
        uint32_t s[kCols];
        const uint32_t t_s = tmem + lane_base + b * N + c0;
        tmem_load<kCols>(t_s, s);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[b]);
        // x = score - reference in log2 units, two columns at a time; nobody
        // past the reference by more than 2^8 is the common case
        float x[kCols];
        auto score2 = [&](int e) {
          float2 f = make_float2(c, c);
          if constexpr (FP8) f = __fmul2_rn(f, *reinterpret_cast<const float2 *>(&ri.scale[c0 + e]));
          return f;
        };
#pragma unroll
        for (int e = 0; e < kCols; e += 2) {
          const float2 m2 = *reinterpret_cast<const float2 *>(&m_s[g0 + e]);
          const float2 y = __ffma2_rn(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), score2(e),
                                      make_float2(-m2.x, -m2.y));
          x[e] = y.x;
          x[e + 1] = y.y;
        }
        if (!all_seen) mask_columns<kCols>(x, ri.lo + c0, ri.hi + c0, u, a.sinks);
        float top = -INFINITY;
#pragma unroll
        for (int e = 0; e < kCols; e += 2) top = fmaxf(top, fmaxf(x[e], x[e + 1]));
        if (bar_any(1 + wg, 128, top > kLazy)) {
          // new references: the columns' maxima over the tile
          float v[kCols];
#pragma unroll
          for (int e = 0; e < kCols; e += 2) {
            const float2 y = __fmul2_rn(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), score2(e));
            v[e] = y.x;
            v[e + 1] = y.y;
          }
          if (!all_seen) mask_columns<kCols>(v, ri.lo + c0, ri.hi + c0, u, a.sinks);
#pragma unroll
          for (int e = 0; e < kCols; ++e) x[e] = v[e];
          const float most = reduce_columns<kCols>(v, lane, maxop);
          if (lane < kCols) red_s[quarter * (2 * kCols) + g0 + lane] = most;
          named_bar_sync(1 + wg, 128);
          if (tid < kCols) {
            const int e = g0 + tid;
            const float mx = fmaxf(fmaxf(red_s[e], red_s[2 * kCols + e]), fmaxf(red_s[4 * kCols + e], red_s[6 * kCols + e]));
            const float old = m_s[e], now = mx > old + kLazy ? mx : old;
            corr_s[e] = now == old ? 1.f : ex2_approx(old - now);
            m_s[e] = now;
          }
          named_bar_sync(1 + wg, 128);
#pragma unroll
          for (int e = 0; e < kCols; ++e) {
            l[e] *= corr_s[g0 + e];
            x[e] -= m_s[g0 + e];
          }
          if (!first) {
            // O holds exactly the group's tiles before this one once the MMAs of the last are done
            const uint32_t last = n - (kByTile ? 2 : 1), t_d = t_o + lane_base + (kByTile ? wg * N : c0);
            mbar_wait(&p_free[last % kPBuf], (last / kPBuf) & 1, abort_flag);
            tc_fence_after();
            uint32_t o[kCols];
            tmem_load<kCols>(t_d, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < kCols; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr_s[g0 + e]);
            tmem_store<kCols>(t_d, o);
            tmem_st_wait();
            tc_fence_before();
          }
        }
        // P = 2^x, its column sums per key, and P * v scale as bf16
        uint32_t pk[kCols / 2];
#pragma unroll
        for (int e = 0; e < kCols; e += 2) {
          float2 p = make_float2(ex2_approx(x[e]), ex2_approx(x[e + 1]));
          const float2 sum = __fadd2_rn(make_float2(l[e], l[e + 1]), p);
          l[e] = sum.x;
          l[e + 1] = sum.y;
          if constexpr (FP8) p = __fmul2_rn(p, make_float2(vs, vs));
          pk[e / 2] = pack_bf16x2(p.x, p.y);
        }
        if (n >= kPBuf) mbar_wait(&p_free[pb], (n / kPBuf - 1) & 1, abort_flag);
        uint8_t *sp = smem + C::kOffP + pb * C::kP + (c0 / 8) * 2048 + (key / 8) * 128 + (key % 8) * 16;
#pragma unroll
        for (int e = 0; e < kCols / 8; ++e)
          *reinterpret_cast<uint4 *>(sp + e * 2048) = make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
        if constexpr (!FP8) {
          // rows of V that no query row sees may hold anything, and 0 * NaN is not 0
          if ((kByTile || wg == 0) && !seen) {
            const uint32_t pos = 2 * n + 1, st = pos % kSt;
            mbar_wait(&full[st], (pos / kSt) & 1, abort_flag);
            uint8_t *sv = smem + st * C::kRaw + (key / 8) * C::kGroup8 + (key % 8) * 128;
#pragma unroll
            for (int e = 0; e < DH / 8; ++e)
              *reinterpret_cast<uint4 *>(sv + (e / 8) * 1024 + (e % 8) * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[pb]);
        first = false;
      }
      // the next piece's queries are staged before this one's results are
      // written, so that its scores run meanwhile: once every S^T of this
      // piece is done, the last of which may be the other group's
      if (kByTile && nT > 0 && ((n - 1) & 1) != wg) mbar_wait(&s_full[(n - 1) % kSBuf], ((n - 1) / kSBuf) & 1, abort_flag);
      const Walk done = w;
      more = w.next();
      ++seg;
      if (more) {
        stage_queries<DH, FP8, N, kOut>(a, w, smem + C::kOffQ, info[seg & 1], out0, tid);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && w.tiles() > 0) mbar_arrive(q_full);
      }
      const float part = reduce_columns<kCols>(l, lane, addop);
      if (lane < kCols) red_s[quarter * (2 * kCols) + g0 + lane] = part;
      named_bar_sync(1 + wg, 128);
      if (tid < kCols) {
        const int e = g0 + tid;
        corr_s[e] = (red_s[e] + red_s[2 * kCols + e]) + (red_s[4 * kCols + e] + red_s[6 * kCols + e]);
      }
      if (nT > 0) {
        mbar_wait(o_full, o_seg & 1, abort_flag);
        ++o_seg;
        tc_fence_after();
      }
      named_bar_sync(3, 256);
      // rows [out0, out0 + kOut): maximum, sum, and what the groups' O count for
      uint32_t o[kOut];
      if constexpr (kByTile) {
        uint32_t o1[kOut];
        // a single tile leaves the other group without an O
        const bool has0 = nT > 1 || (nT == 1 && ((n - 1) & 1) == 0), has1 = nT > 1 || (nT == 1 && ((n - 1) & 1) == 1);
        if (nT > 0) {
          tmem_load<kOut>(t_o + lane_base + out0, o);
          tmem_load<kOut>(t_o + lane_base + N + out0, o1);
          tmem_ld_wait();
        }
#pragma unroll
        for (int e = 0; e < kOut; ++e) {
          const float m0 = m_s[out0 + e], m1 = m_s[kCols + out0 + e], m = fmaxf(m0, m1);
          const float y0 = has0 ? __uint_as_float(o[e]) * ex2_approx(m0 - m) : 0.f;
          const float y1 = has1 ? __uint_as_float(o1[e]) * ex2_approx(m1 - m) : 0.f;
          o[e] = __float_as_uint(y0 + y1);
        }
      } else {
        if (nT > 0) {
          tmem_load<kOut>(t_o + lane_base + out0, o);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < kOut; ++e) o[e] = 0;
        }
      }
      if (nT > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_free);
      }
      auto merged = [&](int e) {   // {maximum, sum} of row e
        if constexpr (!kByTile) return make_float2(m_s[e], corr_s[e]);
        const float m = fmaxf(m_s[e], m_s[kCols + e]);
        return make_float2(m, corr_s[e] * ex2_approx(m_s[e] - m) + corr_s[kCols + e] * ex2_approx(m_s[kCols + e] - m));
      };
      // M = 64: rows 16 q .. 16 q + 15 lie in the first 16 lanes of quarter q
      // converted V rows hold every four elements in the order 0, 2, 1, 3
      const int dm = DH == 128 ? key : quarter * 16 + lane;
      const int dc = FP8 ? (dm & ~3) | ((dm & 1) << 1) | ((dm >> 1) & 1) : dm;
      const bool dlive = DH == 128 || lane < 16;
      if (done.whole()) {
#pragma unroll
        for (int e = 0; e < kOut; ++e) {
          const int row = ri.out[out0 + e];
          if (row < 0) break;
          const float sum = merged(out0 + e).y;
          const float y = sum != 0.f ? __uint_as_float(o[e]) / sum : 0.f;
          if (dlive) {
            if (a.out_fp32) static_cast<float *>(a.out)[static_cast<size_t>(row) * DH + dc] = y;
            else static_cast<uint16_t *>(a.out)[static_cast<size_t>(row) * DH + dc] = f32_to_bf16(y);
          }
        }
        if (a.lse && tid < kOut && ri.out[out0 + tid] >= 0) {
          const float2 ml = merged(out0 + tid);
          a.lse[ri.out[out0 + tid]] = ml.y != 0.f ? (ml.x + log2f(ml.y)) * 0.69314718055994531f : -INFINITY;
        }
      } else {
        // the first piece of a CTA goes to its first slot, a later one (its last) to the second
        const size_t slot = static_cast<size_t>(blockIdx.x) * 2 + (seg > 1 ? 1 : 0);
        float *po = a.part_o + (slot * N + out0) * DH + dc;
        if (dlive)
#pragma unroll
          for (int e = 0; e < kOut; ++e) po[e * DH] = __uint_as_float(o[e]);
        if (tid < kOut) a.part_ml[slot * N + out0 + tid] = merged(out0 + tid);
        if (done.j0 == 0) {
          joined = true;
          if (tid == 0 && wg == 0) {
            // the item's other pieces are the first slots of the next CTAs
            const int parts = 1 + static_cast<int>((done.n - done.j1 + start->per - 1) / start->per);
            a.join[blockIdx.x] = make_int4(done.i, done.h * done.row_tiles + done.rt, static_cast<int>(slot), parts);
          }
        }
      }
    }
    if (a.join && !joined && tid == 0 && wg == 0) a.join[blockIdx.x] = make_int4(0, 0, 0, 0);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  if (threadIdx.x == 0 && *abort_flag) atomicOr(a.status, DLLM_DEV_WAIT_TIMEOUT);
}

// Joins the partial results of the item that CTA blockIdx.x began and others
// finished: block y takes the item's rows y, y + gridDim.y, ...
constexpr int kJoinThreads = 256;

template <int DH>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const PagedArgs a, const int n_rows) {
  constexpr int kGroups = kJoinThreads / DH;      // threads of one column: each takes every kGroups-th piece
  __shared__ float weight[2 * kMaxCtas];
  __shared__ float acc[kJoinThreads];
  __shared__ float sum_s;
  pdl_trigger();
  pdl_wait();
  const int4 job = a.join[blockIdx.x];
  const int parts = job.w;
  if (parts == 0) return;
  const Extent x = paged_extent(a, job.x, false);
  const int row_tiles = (x.W * a.group + n_rows - 1) / n_rows;
  const int h = job.y / row_tiles, rt = job.y - h * row_tiles;
  const int tid = threadIdx.x, c = tid % DH, grp = tid / DH;
  auto slot_of = [&](int p) { return static_cast<size_t>(p == 0 ? job.z : 2 * (blockIdx.x + p)); };
  for (int n = blockIdx.y; n < n_rows; n += gridDim.y) {
    const int r = rt * n_rows + n, t = r / a.group;
    if (t >= x.W) break;
    const int row = (x.q0 + t) * a.Hq + h * a.group + (r - t * a.group);
    if (tid < 32) {
      float m = -INFINITY, l = 0.f;   // a piece without keys: m = -3e38, l = 0
      for (int p = tid; p < parts; p += 32) m = fmaxf(m, a.part_ml[slot_of(p) * n_rows + n].x);
      m = warp_max(m);
      for (int p = tid; p < parts; p += 32) {
        const float2 ml = a.part_ml[slot_of(p) * n_rows + n];
        const float wgt = ex2_approx(ml.x - m);
        weight[p] = wgt;
        l += wgt * ml.y;
      }
      l = warp_sum(l);
      if (tid == 0) {
        sum_s = l;
        if (a.lse) a.lse[row] = l != 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
      }
    }
    __syncthreads();
    float y = 0.f;
#pragma unroll 4
    for (int p = grp; p < parts; p += kGroups) {
      const float wgt = weight[p];
      if (wgt != 0.f) y += wgt * a.part_o[(slot_of(p) * n_rows + n) * DH + c];
    }
    acc[tid] = y;
    __syncthreads();
    if (grp == 0) {
#pragma unroll
      for (int g = 1; g < kGroups; ++g) y += acc[g * DH + c];
      y = sum_s != 0.f ? y / sum_s : 0.f;
      if (a.out_fp32) static_cast<float *>(a.out)[static_cast<size_t>(row) * DH + c] = y;
      else static_cast<uint16_t *>(a.out)[static_cast<size_t>(row) * DH + c] = f32_to_bf16(y);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
dllm_status check_shape(const dllm_kv_pages *pages, const dllm_paged_attn_args *a) {
  const dllm_status st = check_pages(pages);
  if (st != DLLM_OK) return st;
  if (!a || a->B < 0 || a->Hq < 1 || a->max_q < 0 || a->max_kv < 0 || a->q_rows < 0 || a->max_pages < 0 || a->sinks < 0)
    return DLLM_ERR_INVALID_ARG;
  if (a->Hq % pages->heads || a->Hq / pages->heads > 64 || a->B > 4096) return DLLM_ERR_UNSUPPORTED;
  if (a->left >= (1 << 30) || a->right >= (1 << 30) || a->sinks >= (1 << 30)) return DLLM_ERR_UNSUPPORTED;
  if (a->max_kv >= (1 << 30)) return DLLM_ERR_UNSUPPORTED;
  if (static_cast<long long>(a->q_rows) * a->Hq >= (1ll << 31) || static_cast<long long>(a->max_q) * a->Hq >= (1ll << 31))
    return DLLM_ERR_UNSUPPORTED;
  return DLLM_OK;
}

// Columns of a row tile: the least of 16, 32 and 64 that holds a request's
// rows of one cached head, 64 where none does.
int row_tile(const dllm_kv_pages *pages, const dllm_paged_attn_args *a) {
  const long long rows = static_cast<long long>(a->max_q) * (a->Hq / pages->heads);
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

// A CTA's piece is at least kMinTiles tiles: items of no more are never cut.
bool may_split(const dllm_paged_attn_args *a) { return a->max_kv > kMinTiles * kTile; }

struct Ws {
  size_t part_ml, join, total;   // part_o at 0
};

Ws ws_layout(const dllm_kv_pages *pages, const dllm_paged_attn_args *a) {
  Ws w{};
  if (a->B == 0 || a->max_q == 0 || !may_split(a)) return w;
  const size_t rows = static_cast<size_t>(2 * kMaxCtas) * row_tile(pages, a);
  w.part_ml = align256(rows * pages->dh * 4);
  w.join = w.part_ml + align256(rows * 8);
  w.total = w.join + align256(kMaxCtas * 16);
  return w;
}

template <int DH, bool FP8, int N>
dllm_status launch(const dllm_kv_pages *pages, const dllm_paged_attn_args *a, PagedArgs &g, cudaStream_t s) {
  using C = Cfg<DH, FP8, N>;
  CUtensorMap tk, tv;
  const uint64_t rows = static_cast<uint64_t>(pages->num_pages) * pages->heads * pages->page_size;
  if (!make_tmap_page_rows(&tk, pages->k, rows, DH, FP8 ? 1 : 2, pages->page_size) ||
      !make_tmap_page_rows(&tv, pages->v, rows, DH, FP8 ? 1 : 2, pages->page_size))
    return DLLM_ERR_CUDA;
  auto kern = paged_attn_kernel<DH, FP8, N>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  if (e != cudaSuccess) return cuda_error(e);
  // most tiles that the bounds allow, and so most CTAs with work
  const long long row_tiles = (static_cast<long long>(a->max_q) * g.group + N - 1) / N;
  const long long per_item = g.max_kv > 0 ? (g.max_kv + kTile - 1) / kTile : 1;
  const bool split = may_split(a);
  const int min_tiles = split ? kMinTiles : static_cast<int>(per_item);
  g.uniform = split ? 0 : min_tiles;
  const double most = static_cast<double>(a->B) * pages->heads * row_tiles * per_item;
  int ctas = sm_budget() < kMaxCtas ? sm_budget() : kMaxCtas;
  if (most / min_tiles < ctas) ctas = static_cast<int>(most / min_tiles) + 1;
  e = launch_pdl(kern, dim3(ctas), dim3(C::kThreads), C::kBytes, s, tk, tv, g, min_tiles);
  if (e != cudaSuccess) return cuda_error(e);
  unsigned launches = 1;
  if (split) {
    e = launch_pdl(paged_join_kernel<DH>, dim3(ctas, N < 16 ? N : 16), dim3(kJoinThreads), 0, s, g, N);
    if (e != cudaSuccess) return cuda_error(e);
    launches = 2;
  }
  return launch_status(launches);
}

template <int DH, bool FP8>
dllm_status launch_n(const dllm_kv_pages *pages, const dllm_paged_attn_args *a, PagedArgs &g, cudaStream_t s) {
  switch (row_tile(pages, a)) {
    case 16: return launch<DH, FP8, 16>(pages, a, g, s);
    case 32: return launch<DH, FP8, 32>(pages, a, g, s);
    default: return launch<DH, FP8, 64>(pages, a, g, s);
  }
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" size_t dllm_paged_attn_workspace(const dllm_kv_pages *pages, const dllm_paged_attn_args *a) {
  if (check_shape(pages, a) != DLLM_OK) return 0;
  return ws_layout(pages, a).total;
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
  const Ws layout = ws_layout(pages, a);
  if (layout.total > 0 && (!ws || ws_bytes < layout.total || (reinterpret_cast<uintptr_t>(ws) & 255)))
    return DLLM_ERR_WORKSPACE;
  PagedArgs g{};
  g.c = device_pages(pages, a->page_table, a->max_pages);
  g.q = a->q; g.q_stride = a->q_stride; g.out = a->out; g.out_fp32 = a->out_fp32; g.lse = a->lse;
  g.q_off = a->q_off; g.kv_len = a->kv_len; g.q_pos = a->q_pos;
  g.B = a->B; g.Hq = a->Hq; g.group = a->Hq / pages->heads; g.max_q = a->max_q; g.q_rows = a->q_rows;
  // keys beyond the table are not there
  const long long table = static_cast<long long>(a->max_pages) * pages->page_size;
  g.max_kv = static_cast<int>(table < a->max_kv ? table : a->max_kv);
  g.scale_log2 = a->scale * 1.4426950408889634f;
  g.left = a->left; g.right = a->right; g.sinks = a->left >= 0 ? a->sinks : 0;
  cudaError_t e = cudaGetSymbolAddress(reinterpret_cast<void **>(&g.status), g_status_paged);
  if (e != cudaSuccess) return cuda_error(e);
  if (layout.total > 0) {
    char *base = static_cast<char *>(ws);
    g.part_o = reinterpret_cast<float *>(base);
    g.part_ml = reinterpret_cast<float2 *>(base + layout.part_ml);
    g.join = reinterpret_cast<int4 *>(base + layout.join);
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool fp8 = pages->type == DLLM_KV_E4M3;
  if (pages->dh == 64) return fp8 ? launch_n<64, true>(pages, a, g, s) : launch_n<64, false>(pages, a, g, s);
  return fp8 ? launch_n<128, true>(pages, a, g, s) : launch_n<128, false>(pages, a, g, s);
}
