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
#include <type_traits>

#include "paged.cuh"

namespace dllm {

DLLM_DEFINE_STATUS(paged)

namespace {

constexpr int kPBuf = 2, kCBuf = 2;

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
  static constexpr int kRegsIssue = FP8 ? 96 : 104, kRegsSoft = FP8 ? 160 : 200, kRegsConv = 96;
  static_assert(FP8 ? kRegsIssue + 2 * kRegsSoft + kRegsConv <= 4 * 128 : kRegsIssue + 2 * kRegsSoft <= 3 * 168, "registers");
  static constexpr int kRaw = kTile * DH * (FP8 ? 1 : 2);       // one K or V tile as it is cached
  static constexpr int kGroup8 = 8 * DH * (FP8 ? 1 : 2);        // eight cached rows
  static constexpr int kVGroup8 = 8 * DH * 2;                   // eight bf16 rows of V
  static constexpr int kP = kTile * N * 2;
  static constexpr int kQ = N * DH * 2;                         // bf16, or two e4m3 parts
  static constexpr int kConv = FP8 ? kCBuf * kConvKeys * DH * 2 : 0;
  static constexpr int kMisc = FP8 ? 12288 : 8192;              // row tables, scales, barriers, alignment
  static constexpr int kFixed = kConv + kPBuf * kP + 2 * kQ + kMisc;
  static constexpr int kMaxStages = (232448 - kFixed) / kRaw;
  // even, so that K tiles have the even stages; 192 KB in flight are enough
  static constexpr int kStages = (kMaxStages * kRaw > 196608 ? 196608 / kRaw : kMaxStages) & ~1;
  static constexpr int kOffConv = kStages * kRaw;
  static constexpr int kOffP = kOffConv + kConv;
  static constexpr int kOffQ = kOffP + kPBuf * kP;
  static constexpr int kOffMisc = kOffQ + 2 * kQ;               // this piece's query rows and the next one's
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

// A piece of an item as the warps that work on it need it.
template <int N>
struct alignas(16) Piece {
  RowInfo<N> rows;
  TileList t;
  int j0, tiles;           // first tile of the piece, tiles of it that hold visible keys
  int more;                // 0: there is no such piece, the CTA is done
  int whole;               // the whole item: its results are final
  int slot;                // else where its partial results go
};

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

// The query rows of a row tile into shared memory as the B operand of S^T
// (core matrices along K, row groups of 8), by one warp, with what the
// softmax needs to know of each row.
template <int DH, bool FP8, int N>
__device__ __forceinline__ void stage_queries(const PagedArgs &a, const Walk &w, uint8_t *sq, RowInfo<N> &info, int lane) {
  const int rows = w.x.W * a.group, r0 = w.rt * N;
#pragma unroll
  for (int n = lane; n < N; n += 32) {
    const int r = r0 + n, t = r / a.group;
    int lo = 0, hi = 0x7fffffff;   // a column that is no row masks nothing; its results go nowhere
    if (r < rows) visible(a, w.x.pos + t, w.x.L, lo, hi);
    info.lo[n] = lo;
    info.hi[n] = hi;
    info.out[n] = r < rows ? (w.x.q0 + t) * a.Hq + w.h * a.group + (r - t * a.group) : -1;
  }
  constexpr int kChunks = DH / 8;                  // 16-byte chunks of a bf16 row
  constexpr int kRows = 32 / kChunks;              // rows of one round of the warp
  constexpr int kRounds = N / kRows, kAtOnce = kRounds < 8 ? kRounds : 8;   // loads on their way before the first store
  const int c = lane % kChunks;
#pragma unroll 1
  for (int n0 = lane / kChunks; n0 < N; n0 += kRows * kAtOnce) {
    uint4 u[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int r = r0 + n0 + i * kRows, t = r / a.group, g = r - t * a.group;
      u[i] = make_uint4(0, 0, 0, 0);
      if (r < rows)
        u[i] = __ldg(reinterpret_cast<const uint4 *>(a.q + (w.x.q0 + t) * a.q_stride + (w.h * a.group + g) * DH + c * 8));
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int n = n0 + i * kRows;
      if constexpr (!FP8) {
        *reinterpret_cast<uint4 *>(sq + (n / 8) * (kChunks * 128) + c * 128 + (n % 8) * 16) = u[i];
      } else {
        const uint32_t m2 = max_mag(u[i], 0);
        uint32_t m = max(m2 & 0xffffu, m2 >> 16);
#pragma unroll
        for (int o = kChunks / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        uint2 hi, lo;
        const int byte = split_e4m3(u[i], m, hi, lo);
        uint8_t *d = sq + (n / 8) * (DH / 16 * 128) + (c / 2) * 128 + (n % 8) * 16 + (c & 1) * 8;
        *reinterpret_cast<uint2 *>(d) = hi;
        *reinterpret_cast<uint2 *>(d + N * DH) = lo;
        if (c == 0) info.scale[n] = scale_of(m < 0x7f80u ? byte : 255);   // a row with an infinity or NaN scores NaN
      }
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
  Piece<N> *pieces = reinterpret_cast<Piece<N> *>(misc);                  // [2]: this one and the next one
  float *m_s = reinterpret_cast<float *>(pieces + 2);                       // [group][kCols] reference maxima
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
  uint64_t *q_full = sc_full + C::kScaleSlots;   // [2] piece prepared
  uint64_t *q_free = q_full + 2;            // [2] its last use over
  uint64_t *o_full = q_free + 2;
  uint64_t *o_free = o_full + 1;
  long long *s_scan = reinterpret_cast<long long *>(o_free + 1);          // [32]
  Start *start = reinterpret_cast<Start *>(s_scan + 32);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(start + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  static_assert(2 * sizeof(Piece<N>) + 12 * kCols * 4 + (2 * kSt + 2 * kSBuf + 2 * kPBuf + 2 * kCBuf + 6) * 8 + 256 + 64 +
                        C::kScaleSlots * (2 * kTile + 8 + 4) + 4 <= C::kMisc - 1024,
                "row tables and barriers");
  static_assert(sizeof(Piece<N>) % 16 == 0 && kCols % 16 == 0, "scales, 16-byte aligned for the bulk loads");

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
    for (int b = 0; b < 2; ++b) {
      mbar_init(&q_full[b], 1);
      mbar_init(&q_free[b], 8 + 2 + (FP8 ? 4 : 0));   // the warps that read the piece
    }
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
  if (warp < 4) {
  reg_dealloc<C::kRegsIssue>();
  if (warp == 0) {
    // ------------------------------------------------------------- producer
    load_tiles<DH, FP8 ? 1 : 2, kSt, C::kScaleSlots>(a, *start, N, &tm_k, &tm_v, smem, full, empty, scales, pages_of, sc_full,
                                                     abort_flag, lane);
  } else if (warp == 1) {
    // ------------------------------------------------------------- S^T MMAs
    if (elect_one()) {
    uint32_t n = 0;
    bool ok = true;
    for (uint32_t seg = 0; ok; ++seg) {
      const uint32_t pi = seg & 1;
      ok = mbar_wait(&q_full[pi], (seg >> 1) & 1, abort_flag);
      if (!ok || !pieces[pi].more) break;
      const int nT = pieces[pi].tiles;
      const uint32_t sq = smem_u32(smem + C::kOffQ + pi * C::kQ);
      for (int j = 0; j < nT; ++j, ++n) {
        const uint32_t pos = 2 * n, st = pos % kSt, b = n % kSBuf;
        ok = mbar_wait(&full[st], (pos / kSt) & 1, abort_flag);
        if (ok && n >= kSBuf) ok = mbar_wait(&s_free[b], (n / kSBuf - 1) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sk = smem_u32(smem + st * C::kRaw);
        {
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
      }
      mbar_arrive(&q_free[pi]);
    }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------- O^T MMAs
    if (elect_one()) {
    uint32_t n = 0, o_seg = 0;
    bool ok = true;
    for (uint32_t seg = 0; ok; ++seg) {
      const uint32_t pi = seg & 1;
      ok = mbar_wait(&q_full[pi], (seg >> 1) & 1, abort_flag);
      if (!ok || !pieces[pi].more) break;
      const int nT = pieces[pi].tiles;
      for (int j = 0; ok && j < nT; ++j, ++n) {
        const uint32_t pos = 2 * n + 1, st = pos % kSt, b = n % kPBuf;
        ok = mbar_wait(&p_full[b], (n / kPBuf) & 1, abort_flag);
        if (ok && j == 0 && o_seg > 0) ok = mbar_wait(o_free, (o_seg - 1) & 1, abort_flag);
        if (ok && !FP8) ok = mbar_wait(&full[st], (pos / kSt) & 1, abort_flag);
        const uint32_t t_d = kByTile ? t_o + (n & 1) * N : t_o;
        const bool first = j == 0 || (kByTile && j == 1);   // of its accumulator
        const uint64_t dp = plain_desc(smem_u32(smem + C::kOffP + b * C::kP), 128, 2048);
        // bf16: the tile as one piece; e4m3: its converted pieces
        constexpr int kPieces = FP8 ? kTile / kConvKeys : 1, kSteps = 8 / kPieces;
#pragma unroll
        for (int piece = 0; piece < kPieces; ++piece) {
          const uint32_t cn = n * kPieces + piece, cb = cn % kCBuf;
          if (FP8 && ok) ok = mbar_wait(&c_full[cb], (cn / kCBuf) & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sv = smem_u32(FP8 ? smem + C::kOffConv + cb * (kConvKeys * DH * 2) : smem + st * C::kRaw);
          {
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
        }
      }
      o_seg += nT > 0;
      mbar_arrive(&q_free[pi]);
    }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- pieces and their query rows
    // One piece ahead of the others, so that its metadata and its rows are
    // there when the scores of the last one are.
    Walk w(a, N, *start);
    bool more = true, began = false;
    for (uint32_t seg = 0; more; ++seg) {
      const uint32_t pi = seg & 1;
      if (seg >= 2 && !warp_wait(&q_free[pi], ((seg >> 1) - 1) & 1, abort_flag)) break;
      Piece<N> &pc = pieces[pi];
      more = w.next();
      if (lane == 0) {
        pc.more = more;
        if (more) {
          pc.t = w.t;
          pc.j0 = w.j0;
          pc.tiles = w.tiles();
          pc.whole = w.whole();
          // a CTA's first piece has its first slot, its last one the second
          pc.slot = 2 * blockIdx.x + (seg > 0);
          began |= begin_join(a, w, *start, pc.slot);
        }
      }
      if (more) stage_queries<DH, FP8, N>(a, w, smem + C::kOffQ + pi * C::kQ, pc.rows, lane);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[pi]);
    }
    if (a.join && lane == 0 && !began) a.join[blockIdx.x].parts = 0;
  }
  } else if (FP8 && warp >= C::kConvWarp0) {
    // ------------------------------------------------------------- V codes -> bf16
    if constexpr (FP8) {
      reg_dealloc<C::kRegsConv>();
      const int t = (warp - C::kConvWarp0) * 32 + lane;
      uint32_t n = 0;
      for (uint32_t seg = 0;; ++seg) {
        const uint32_t pi = seg & 1;
        if (!warp_wait(&q_full[pi], (seg >> 1) & 1, abort_flag) || !pieces[pi].more) break;
        const TileList tl = pieces[pi].t;
        const int j0 = pieces[pi].j0, nT = pieces[pi].tiles;
        for (int j = 0; j < nT; ++j, ++n) {
          const uint32_t pos = 2 * n + 1, st = pos % kSt;
          mbar_wait(&full[st], (pos / kSt) & 1, abort_flag);
#pragma unroll 1
          for (int half = 0; half < kTile / kConvKeys; ++half) {
            const uint32_t cn = n * (kTile / kConvKeys) + half, cb = cn % kCBuf;
            const int u = tl.tile(j0 + j) * kTile + half * kConvKeys + t % kConvKeys;
            convert_v<DH>(smem + st * C::kRaw, smem + C::kOffConv + cb * (kConvKeys * DH * 2), half, t,
                          u < tl.hi && (u >= tl.lo || u < a.sinks),
                          [&] { if (cn >= kCBuf) mbar_wait(&c_free[cb], (cn / kCBuf - 1) & 1, abort_flag); },
                          [](uint2 v) { return v; });
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c_full[cb]);
          }
          if (lane == 0) mbar_arrive(&empty[st]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_free[pi]);
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
    const auto maxop = [](float p, float q) { return fmaxf(p, q); };
    const auto addop = [](float p, float q) { return p + q; };
    uint32_t n = 0, o_seg = 0;
    for (uint32_t seg = 0;; ++seg) {
      const uint32_t pi = seg & 1;
      // all of both groups go on or none does (the last piece's maxima are read, too)
      if (bar_any(3, 256, !mbar_wait(&q_full[pi], (seg >> 1) & 1, abort_flag))) break;
      const Piece<N> &pc = pieces[pi];
      if (!pc.more) break;
      const RowInfo<N> &ri = pc.rows;
      const TileList tl = pc.t;
      const int nT = pc.tiles, j0 = pc.j0;
      float l[kCols];
#pragma unroll
      for (int e = 0; e < kCols; ++e) l[e] = 0.f;
      if (tid < kCols) m_s[g0 + tid] = kNone;
      named_bar_sync(1 + wg, 128);
      bool first = true;                    // of the group's tiles
      for (int j = 0; j < nT; ++j, ++n) {
        if (kByTile && (n & 1) != wg) continue;
        const uint32_t b = n % kSBuf, pb = n % kPBuf;
        const int key0 = tl.tile(j0 + j) * kTile, u = key0 + key;
        // every row of the tile sees every key of it?
        const bool all_seen = key0 + kTile <= tl.hi_first && (key0 >= tl.lo_last || key0 + kTile <= a.sinks);
        const bool seen = u < tl.hi && (u >= tl.lo || u < a.sinks);   // this key, by any row
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
      if (pc.whole) {
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
          a.lse[ri.out[out0 + tid]] = ml.y != 0.f ? (ml.x + log2f(ml.y)) * kLn2 : -INFINITY;
        }
      } else {
        const size_t slot = pc.slot;
        float *po = a.part_o + (slot * N + out0) * DH + dc;
        if (dlive)
#pragma unroll
          for (int e = 0; e < kOut; ++e) po[e * DH] = __uint_as_float(o[e]);
        if (tid < kOut) a.part_ml[slot * N + out0 + tid] = merged(out0 + tid);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_free[pi]);
    }
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
// finished: one warp per row, the pieces in their order with a running
// maximum, four of them on the way at a time.
constexpr int kJoinThreads = 256;

template <int DH>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const PagedArgs a, const int n_rows) {
  using Vec = typename std::conditional<DH == 128, float4, float2>::type;   // a lane's columns
  constexpr int kVec = DH / 32, kAhead = 4;
  pdl_trigger();
  pdl_wait();
  const JoinJob job = a.join[blockIdx.x];
  const int n = blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (job.parts == 0 || n >= n_rows || job.r0 + n >= job.rows) return;
  const int c = lane * kVec;
  float m = -INFINITY, l = 0.f, o[kVec] = {};
  for (int p0 = 0; p0 < job.parts; p0 += kAhead) {
    float2 ml[kAhead];
    Vec y[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int p = p0 + k;
      const size_t slot = static_cast<size_t>(p == 0 ? job.slot : 2 * (blockIdx.x + p)) * n_rows;
      if (p < job.parts) {
        ml[k] = a.part_ml[slot + n];
        // [slot][row][DH], and of many rows [slot][DH / 4][row][4]
        y[k] = *reinterpret_cast<const Vec *>(a.part_o + slot * DH + (n_rows <= 32 ? n * DH + c : (c / 4 * n_rows + n) * 4 + c % 4));
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (p0 + k >= job.parts) break;
      const float mn = fmaxf(m, ml[k].x), f = ex2_approx(m - mn), g = ex2_approx(ml[k].x - mn);
      l = l * f + ml[k].y * g;
      const float *v = reinterpret_cast<const float *>(&y[k]);
#pragma unroll
      for (int e = 0; e < kVec; ++e) o[e] = o[e] * f + v[e] * g;
      m = mn;
    }
  }
  const int r = job.r0 + n, t = r / a.group;
  const size_t row = static_cast<size_t>(job.q0 + t) * a.Hq + job.h * a.group + (r - t * a.group);
#pragma unroll
  for (int e = 0; e < kVec; ++e) o[e] = l != 0.f ? o[e] / l : 0.f;
  if (a.out_fp32) {
    float *d = static_cast<float *>(a.out) + row * DH + lane * kVec;
#pragma unroll
    for (int e = 0; e < kVec; ++e) d[e] = o[e];
  } else {
    uint32_t *d = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + row * DH + lane * kVec);
#pragma unroll
    for (int e = 0; e < kVec; e += 2) d[e / 2] = pack_bf16x2(o[e], o[e + 1]);
  }
  if (a.lse && lane == 0) a.lse[row] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
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
  if (static_cast<long long>(a->q_rows) * a->Hq >= (1ll << 30) || static_cast<long long>(a->max_q) * a->Hq >= (1ll << 30))
    return DLLM_ERR_UNSUPPORTED;
  return DLLM_OK;
}

// Rows of a row tile: the least of 16, 32 and 128 that holds a request's rows
// of one cached head, 256 where none does. Up to 32 they are the N of the
// MMAs here, from there on the M of those in paged_rows.cu.
int row_tile(const dllm_kv_pages *pages, const dllm_paged_attn_args *a) {
  const long long rows = static_cast<long long>(a->max_q) * (a->Hq / pages->heads);
  return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 128 ? 128 : 256;
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
  w.total = w.join + align256(kMaxCtas * sizeof(JoinJob));
  return w;
}

template <int DH, bool FP8, int N>
dllm_status launch(const CUtensorMap &tk, const CUtensorMap &tv, const PagedArgs &g, int min_tiles, int ctas, cudaStream_t s) {
  using C = Cfg<DH, FP8, N>;
  auto kern = paged_attn_kernel<DH, FP8, N>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  if (e == cudaSuccess) e = launch_pdl(kern, dim3(ctas), dim3(C::kThreads), C::kBytes, s, tk, tv, g, min_tiles);
  return e == cudaSuccess ? DLLM_OK : cuda_error(e);
}

template <int DH, bool FP8>
dllm_status launch_attn(const dllm_kv_pages *pages, const dllm_paged_attn_args *a, PagedArgs &g, cudaStream_t s) {
  CUtensorMap tk, tv;
  const uint64_t rows = static_cast<uint64_t>(pages->num_pages) * pages->heads * pages->page_size;
  if (!make_tmap_page_rows(&tk, pages->k, rows, DH, FP8 ? 1 : 2, pages->page_size) ||
      !make_tmap_page_rows(&tv, pages->v, rows, DH, FP8 ? 1 : 2, pages->page_size))
    return DLLM_ERR_CUDA;
  // most tiles that the bounds allow, and so most CTAs with work
  const int n = row_tile(pages, a);
  const long long row_tiles = (static_cast<long long>(a->max_q) * g.group + n - 1) / n;
  const long long per_item = g.max_kv > 0 ? (g.max_kv + kTile - 1) / kTile : 1;
  const bool split = may_split(a);
  const int min_tiles = split ? kMinTiles : static_cast<int>(per_item);
  g.uniform = split ? 0 : min_tiles;
  const double most = static_cast<double>(a->B) * pages->heads * row_tiles * per_item;
  int ctas = sm_budget() < kMaxCtas ? sm_budget() : kMaxCtas;
  if (most / min_tiles < ctas) ctas = static_cast<int>(most / min_tiles) + 1;
  const dllm_status st = n == 16   ? launch<DH, FP8, 16>(tk, tv, g, min_tiles, ctas, s)
                         : n == 32 ? launch<DH, FP8, 32>(tk, tv, g, min_tiles, ctas, s)
                                   : launch_paged_rows(DH, FP8, n, tk, tv, g, min_tiles, ctas, s);
  if (st != DLLM_OK) return st;
  unsigned launches = 1;
  if (split) {
    const cudaError_t e = launch_pdl(paged_join_kernel<DH>, dim3(ctas, (n * 32 + kJoinThreads - 1) / kJoinThreads),
                                     dim3(kJoinThreads), 0, s, g, n);
    if (e != cudaSuccess) return cuda_error(e);
    launches = 2;
  }
  return launch_status(launches);
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
    g.join = reinterpret_cast<JoinJob *>(base + layout.join);
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool fp8 = pages->type == DLLM_KV_E4M3;
  if (pages->dh == 64) return fp8 ? launch_attn<64, true>(pages, a, g, s) : launch_attn<64, false>(pages, a, g, s);
  return fp8 ? launch_attn<128, true>(pages, a, g, s) : launch_attn<128, false>(pages, a, g, s);
}
