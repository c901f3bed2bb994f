// Attention over the paged cache where a request has many query rows per
// cached head (blocks of a denoising step, pieces of prompts): the rows are
// the M = 128 of the tensor-core tile, one per thread of the softmax, so
// row maxima and sums need no exchange, and P goes back to TMEM as the A
// operand of P V.
//
// Two streams share a CTA's tensor core: while one stream's softmax works on
// its scores, the other's MMAs run. With more than 128 rows (tiles of 256)
// each stream has 128 of them and both read every K and V tile; with up to
// 128 the streams take every other key tile of the same rows and their
// results are merged at the end.
//
// Warp roles:
//   warp 0      TMA (load_tiles)
//   warp 1      MMAs, alternating streams: P V of a tile, then the scores of
//               the stream's next tile over the same TMEM (MMAs of one thread
//               run in order)
//   warp 3      walks the CTA's pieces one ahead of the others
//   warps 4..11 two softmax warpgroups, one per stream, one row per thread;
//               they also stage the query rows
//   last four   (e4m3 pages) V codes -> bf16 with the scale folded in (a
//               power of two: exact), and the K scales of the scores' columns
// TMEM (512 columns): S / P of stream s at 128 s, O at 256 + 128 s.
// P is taken against a reference maximum of the row in one pass over the
// scores. P is bf16 and has the range of fp32, so the reference need not be
// the maximum: it follows, from the next tile on, when scores passed it by
// more than 2^8 (the row's O is then rescaled in TMEM), and at once when they
// did by more than 2^32, as on a row's first keys. P V of a tile's first 64
// keys starts while the exponentials of the other 64 run.
// e4m3 pages: K codes and the query rows as in paged_attn.cu (two e4m3 parts
// of the rows); the scores' columns are multiplied by scale * K scale.
// Trees of drafted tokens (TREE): a row's visible keys of a tile are four words,
// cut from its bits of the tokens at the tile's place among them, fetched before
// the wait for the scores, and only by tiles from the first token's key on.
//
// Drafts of 32 requests of 20 to 64 tokens over up to 8192 keys (8 x 4 heads, dh
// 128): e4m3 170 us, bf16 128; two thirds of the 256 rows are tokens'.
// Pieces of two prompts of 1200 to 1536 tokens over 9 to 12 thousand keys (bf16,
// 8 x 4 heads, dh 128, causal) take 331 us with the join: 1.34 PFLOP/s, 72 % of a plain
// matrix product's rate. Bound by the tensor cores: a tile of 256 x 128 costs
// 3.1 k cycles where its MMAs alone take 2.75 k; some 10 us pass until the first
// scores. Four prompts' pieces of 300 to 512 tokens over 1500 to 8000 keys
// (e4m3) take 230 us, 0.86 PFLOP/s: the softmax warps and the converters share
// the issue slots (of 253 us at an earlier stage, 27 went without the K scales' products
// and their loads, 18 without the conversion; a second group of converters
// leaves the softmax too few registers: 28 longer). 16 denoising blocks of 64 to 96 rows over 352 to
// 1120 keys (32 heads, bf16): 54 us, 57 % of the bytes' time; an item has five
// tiles, and its rows, first scores and results cost about as much as six.
#include "paged.cuh"

namespace dllm {

namespace {

// Largest of 64 values, as four chains of three-input maxima.
__device__ __forceinline__ float greatest(const uint32_t (&a)[32], const uint32_t (&b)[32]) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      m[i] = fmaxf(m[i], fmaxf(__uint_as_float(a[e + 2 * i]), __uint_as_float(a[e + 2 * i + 1])));
      m[2 + i] = fmaxf(m[2 + i], fmaxf(__uint_as_float(b[e + 2 * i]), __uint_as_float(b[e + 2 * i + 1])));
    }
  }
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

constexpr uint32_t kColO = 256;
constexpr int kAhead = 4;        // pieces prepared, this one included
constexpr float kJump = 32.f;    // a reference moves at once when a score passes it by more than 2^32

template <int DH, bool FP8, bool TWO>
struct RowsCfg {
  static constexpr int kRows = TWO ? 256 : 128;               // rows of an item
  static constexpr int kConvWarp0 = 12;
  static constexpr int kThreads = 32 * (kConvWarp0 + (FP8 ? 4 : 0));
  // registers a thread: what the TMA and MMA warps and the converters do not
  // need goes to the softmax groups (the sum is the launch's). e4m3 with
  // 72 / 184 / 72, 64 / 192 / 64 or 80 / 176 / 80: 2 to 4 % longer
  static constexpr int kRegsIssue = FP8 ? 96 : 120, kRegsSoft = FP8 ? 160 : 192, kRegsConv = 96;
  static_assert(FP8 ? kRegsIssue + 2 * kRegsSoft + kRegsConv <= 4 * 128 : kRegsIssue + 2 * kRegsSoft <= 3 * 168, "registers");
  static constexpr int kRaw = kTile * DH * (FP8 ? 1 : 2);
  static constexpr int kGroup8 = 8 * DH * (FP8 ? 1 : 2);
  static constexpr int kVGroup8 = 8 * DH * 2;
  static constexpr int kQ = 128 * DH * 2;                     // 128 rows: bf16, or two e4m3 parts
  static constexpr int kQs = 2;                               // one per stream, or this piece's and the next one's
  static constexpr int kCBuf = FP8 ? 4 : 0;                   // converted V pieces: two tiles
  static constexpr int kConv = kCBuf * kConvKeys * DH * 2;
  static constexpr int kScaleBytes = FP8 ? 8192 : 0;          // scale bytes, column factors, row factors
  static constexpr int kMisc = 1984 + kScaleBytes;            // + 1024 of alignment
  static constexpr int kMax = (232448 - 1024 - kQs * kQ - kConv - kMisc) / kRaw;
  static constexpr int kCap = 196608 / kRaw < 12 ? 196608 / kRaw : 12;   // 192 KB in flight are enough
  static constexpr int kStages = kMax < kCap ? kMax : kCap;
  static constexpr int kKSt = kStages / 2, kVSt = kStages - kKSt;
  static constexpr int kLead = FP8 ? 1 : 0;   // (the other way round: bf16 2 to 6 % longer, e4m3 2 to 3 %)
  // a slot is written again once the scores of the tile kKSt before it are
  // done: the factors of every tile up to two before that one are computed
  static constexpr int kScaleSlots = FP8 ? kKSt + 3 : 0;
  static constexpr int kOffConv = kStages * kRaw;
  static constexpr int kOffQ = kOffConv + kConv;
  static constexpr int kOffMisc = kOffQ + kQs * kQ;
  static constexpr int kBytes = kOffMisc + kMisc + 1024;
  static_assert(kConvKeys * 2 == kTile && kStages >= 4 && kBytes <= 232448, "shared memory");
};

struct alignas(16) RowsPiece {
  Extent x;
  TileList t;
  int h, r0;               // head, first flat row
  int two;                 // each stream has rows of its own
  int j0, tiles, more, whole, slot;
};

// Query rows [n0, n0 + CNT) of the 128 in `sq`, flat rows r0 + n, as the A
// operand of the scores (rows of 128 bytes under the 128-byte swizzle, column
// pieces 16 KB apart; e4m3 parts: DH-byte rows, parts 128 DH apart), by 128
// threads. bf16 rows are copied asynchronously: they are there after
// copies_wait. The powers of two of rows in e4m3 parts go to qs.
template <int DH, bool FP8, int CNT>
__device__ __forceinline__ void stage_rows(const PagedArgs &a, const RowsPiece &pc, int r0, int n0, uint8_t *sq, float *qs,
                                           int tid) {
  constexpr int kChunks = DH / 8, kEach = CNT * kChunks / 128, kStep = 128 / kChunks;   // chunks of a thread, rows from one to the next
  constexpr int kAtOnce = kEach < 8 ? kEach : 8;   // loads on their way before the first store
  static_assert(kEach % kAtOnce == 0, "whole rounds");
  // row r = t * group + g, and the step from a thread's row to its next one
  const int rows = pc.x.W * a.group, c = tid % kChunks, step_t = kStep / a.group, step_g = kStep - step_t * a.group;
  int n = n0 + tid / kChunks, r = r0 + n, t = r / a.group, g = r - t * a.group;
  const uint16_t *q = a.q + pc.x.q0 * a.q_stride + pc.h * a.group * DH + c * 8;
  auto source = [&] { return reinterpret_cast<const uint4 *>(r < rows ? q + t * a.q_stride + g * DH : q); };
  auto advance = [&] {
    r += kStep;
    t += step_t;
    g += step_g;
    if (g >= a.group) { g -= a.group; ++t; }
  };
  if constexpr (!FP8) {
    uint8_t *d = sq + (c / 8) * 16384 + (n / 8) * 1024 + (n % 8) * 128 + ((c % 8) ^ (n % 8)) * 16;   // (kStep: whole eights)
    static_assert(kStep % 8 == 0, "the swizzle of a thread's rows");
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      copy16(d + i * (kStep / 8 * 1024), source(), r < rows);
      advance();
    }
  } else {
#pragma unroll 1
    for (int i0 = 0; i0 < kEach; i0 += kAtOnce) {
      uint4 u[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        u[i] = r < rows ? __ldg(source()) : make_uint4(0, 0, 0, 0);
        advance();
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i, n += kStep) {
        const uint32_t m2 = max_mag(u[i], 0);
        uint32_t m = max(m2 & 0xffffu, m2 >> 16);
#pragma unroll
        for (int o = kChunks / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        uint2 hi, lo;
        const int byte = split_e4m3(u[i], m, hi, lo);
        const int sc = DH == 128 ? (c / 2) ^ (n % 8) : (c / 2) ^ ((n / 2) % 4);
        uint8_t *d = sq + n * DH + sc * 16 + (c % 2) * 8;
        *reinterpret_cast<uint2 *>(d) = hi;
        *reinterpret_cast<uint2 *>(d + 128 * DH) = lo;
        if (c == 0) qs[n] = scale_of(m < 0x7f80u ? byte : 255);   // a row with an infinity or NaN scores NaN
      }
    }
  }
}

template <int DH, bool FP8, bool TWO, bool TREE>
__global__ void __launch_bounds__(RowsCfg<DH, FP8, TWO>::kThreads, 1)
paged_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const PagedArgs a) {
  using C = RowsCfg<DH, FP8, TWO>;
  constexpr int kSt = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *misc = smem + C::kOffMisc;
  RowsPiece *pieces = reinterpret_cast<RowsPiece *>(misc);                // [kAhead]
  float2 *ml_s = reinterpret_cast<float2 *>(pieces + kAhead);                  // [128] maxima and sums to merge
  uint64_t *full = reinterpret_cast<uint64_t *>(ml_s + 128);              // [kSt] stage loaded
  uint64_t *empty = full + kSt;             // [kSt] stage read by its MMAs (or converted)
  uint64_t *s_full = empty + kSt;           // [stream]
  uint64_t *p_full = s_full + 2;            // [stream][half]
  uint64_t *h_done = p_full + 4;            // [stream] P V of the first half done
  uint64_t *piece_full = h_done + 2;        // [kAhead]
  uint64_t *piece_free = piece_full + kAhead;   // [kAhead]
  uint64_t *q_full = piece_free + kAhead;   // [kAhead] query rows staged
  uint64_t *o_full = q_full + kAhead;
  uint64_t *o_free = o_full + 1;
  Scan *s_scan = reinterpret_cast<Scan *>(ml_s);                          // before there are any
  Start *start = reinterpret_cast<Start *>(o_free + 1);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(start + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  static_assert(kAhead * sizeof(RowsPiece) + 1024 + (2 * kSt + 10 + 3 * kAhead) * 8 + sizeof(Start) + 8 <= 1984, "piece and barriers");
  // e4m3 pages
  uint8_t *scales = misc + 1984;                                          // [kScaleSlots][K, V][kTile]
  float *col_s = reinterpret_cast<float *>(scales + C::kScaleSlots * 2 * kTile);   // [4][kTile] score factors of a tile's keys
  float *qs_s = col_s + (FP8 ? 4 * kTile : 0);                            // [piece parity][256] powers of two of the rows
  uint64_t *c_full = reinterpret_cast<uint64_t *>(qs_s + (FP8 ? 512 : 0));   // [kCBuf] V piece converted
  uint64_t *c_free = c_full + C::kCBuf;     // [kCBuf] its MMAs done
  uint64_t *sc_full = c_free + C::kCBuf;    // [kScaleSlots] scale bytes loaded
  uint64_t *col_full = sc_full + C::kScaleSlots;   // [4] factors written
  uint32_t *pages_of = reinterpret_cast<uint32_t *>(col_full + 4);        // [kScaleSlots]
  static_assert(!FP8 || C::kScaleSlots * (2 * kTile + 12) + 4 * kTile * 4 + 2048 + (2 * C::kCBuf + 4) * 8 <= C::kScaleBytes,
                "scales");
  static_assert(sizeof(Scan) <= 1024 && 1984 % 16 == 0 && sizeof(RowsPiece) % 16 == 0, "scales, 16-byte aligned for the bulk loads");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kSt; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], FP8 && s >= C::kKSt ? 4 : 1);
    }
    for (int b = 0; b < 2; ++b) { mbar_init(&s_full[b], 1); mbar_init(&h_done[b], 1); }
    for (int b = 0; b < 4; ++b) mbar_init(&p_full[b], 4);
    for (int b = 0; b < kAhead; ++b) {
      mbar_init(&piece_full[b], 1);
      mbar_init(&piece_free[b], 8 + 1 + (FP8 ? 4 : 0));   // the warps that read it
      mbar_init(&q_full[b], 8);
    }
    mbar_init(o_full, 1);
    mbar_init(o_free, 8);
    if constexpr (FP8) {
      for (int b = 0; b < C::kCBuf; ++b) { mbar_init(&c_full[b], 4); mbar_init(&c_free[b], 1); }
      for (int b = 0; b < C::kScaleSlots; ++b) mbar_init(&sc_full[b], 1);
      for (int b = 0; b < 4; ++b) mbar_init(&col_full[b], 4);
    }
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  pdl_wait();   // the batch's metadata, the pages and the queries may come from the previous kernel
  find_start(a, C::kRows, s_scan, start);

  if (warp < 4) {
    reg_dealloc<C::kRegsIssue>();
    if (warp == 0) {
      load_tiles<DH, FP8 ? 1 : 2, C::kKSt, C::kVSt, C::kLead, C::kScaleSlots>(a, *start, C::kRows, &tm_k, &tm_v, smem, full, empty,
                                                                              scales, pages_of, sc_full, abort_flag, lane);
    } else if (warp == 1) {
      // ----------------------------------------------------------- MMAs
      // (one elected thread through the whole loop: a warp that stays
      // together and elects around each group of MMAs took 12 % longer)
      if (elect_one()) {
        uint32_t n0 = 0, o_seg = 0, cnt[2] = {0, 0};   // tiles and streams' tiles before this piece
        bool ok = true;
        for (uint32_t seg = 0; ok; ++seg) {
          const uint32_t pi = seg % kAhead;
          ok = mbar_wait(&piece_full[pi], (seg / kAhead) & 1, abort_flag);
          if (!ok || !pieces[pi].more) break;
          const int nT = pieces[pi].tiles;
          const bool two = TWO && pieces[pi].two;
          const int n_s[2] = {two ? nT : (nT + 1) / 2, two ? nT : nT / 2};
          ok = mbar_wait(&q_full[pi], (seg / kAhead) & 1, abort_flag);
          // scores of stream s's k-th tile
          auto scores = [&](int s, int k) {
            const uint32_t n = n0 + (two ? k : 2 * k + s), st = n % C::kKSt;
            ok = ok && mbar_wait(&full[st], (n / C::kKSt) & 1, abort_flag);
            tc_fence_after();
            if (ok) {
              const uint32_t sk = smem_u32(smem + st * C::kRaw), t_s = tmem + s * 128;
              const uint32_t sq = smem_u32(smem + C::kOffQ + (TWO ? (two ? s : 0) : seg & 1) * C::kQ);
              if constexpr (!FP8) {
                const uint64_t dq = sw128_desc(sq, 16, 1024), dk = sw128_desc(sk, 16, C::kGroup8);
  #pragma unroll
                for (int kk = 0; kk < DH / 16; ++kk)
                  umma_bf16(t_s, dq + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4), dk + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4),
                            idesc_bf16(128, 128, 0, 0), kk > 0);
              } else {
                const uint64_t dk = DH == 128 ? sw128_desc(sk, 16, C::kGroup8) : sw64_desc(sk, 16, C::kGroup8);
  #pragma unroll
                for (int part = 0; part < 2; ++part) {
                  const uint32_t sp = sq + part * 128 * DH;
                  const uint64_t dq = DH == 128 ? sw128_desc(sp, 16, 8 * DH) : sw64_desc(sp, 16, 8 * DH);
  #pragma unroll
                  for (int kk = 0; kk < DH / 32; ++kk)
                    umma_f8(t_s, dq + ((kk * 32) >> 4), dk + ((kk * 32) >> 4), idesc_f8(128, 128, kE4M3, kE4M3, 0, 0), part + kk > 0);
                }
              }
              umma_commit(&s_full[s]);
              if (!two || s == 1) umma_commit(&empty[st]);
            }
          };
          // O of stream s += P V of its k-th tile
          auto values = [&](int s, int k) {
            const uint32_t n = n0 + (two ? k : 2 * k + s), st = C::kKSt + n % C::kVSt;
            const uint32_t ns = cnt[s] + k;
            if (k == 0 && s == 0 && o_seg > 0) ok = ok && mbar_wait(o_free, (o_seg - 1) & 1, abort_flag);
            if constexpr (!FP8) ok = ok && mbar_wait(&full[st], (n / C::kVSt) & 1, abort_flag);
  #pragma unroll
            for (int half = 0; half < 2; ++half) {
              ok = ok && mbar_wait(&p_full[s * 2 + half], ns & 1, abort_flag);
              const uint32_t cn = 2 * n + half, cb = FP8 ? cn % (C::kCBuf + !FP8) : 0;
              if constexpr (FP8) ok = ok && mbar_wait(&c_full[cb], (cn / C::kCBuf) & 1, abort_flag);
              tc_fence_after();
              if (ok) {
                const uint32_t sv = smem_u32(FP8 ? smem + C::kOffConv + cb * (kConvKeys * DH * 2)
                                                 : smem + st * C::kRaw + half * 8 * C::kVGroup8);
                const uint64_t dv = sw128_desc(sv, 1024, C::kVGroup8);
  #pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  umma_bf16_tmem_a(tmem + kColO + s * 128, tmem + s * 128 + (half * 4 + kk) * 8,
                                   dv + ((kk * 2 * C::kVGroup8) >> 4), idesc_bf16(128, DH, 0, 1), k > 0 || half + kk > 0);
                if (half == 0) umma_commit(&h_done[s]);
                if (FP8 && (!two || s == 1)) umma_commit(&c_free[cb]);
                if (!FP8 && half == 1 && (!two || s == 1)) umma_commit(&empty[st]);
              }
            }
          };
          if (nT > 0) {
            scores(0, 0);
            if (n_s[1] > 0) scores(1, 0);
            for (int k = 0; ok && k < n_s[0]; ++k) {
              values(0, k);
              if (k + 1 < n_s[0]) scores(0, k + 1);
              if (k < n_s[1]) values(1, k);
              if (k + 1 < n_s[1]) scores(1, k + 1);
            }
            if (ok) umma_commit(o_full);
            ++o_seg;
          }
          n0 += nT;
          cnt[0] += n_s[0];
          cnt[1] += n_s[1];
          mbar_arrive(&piece_free[pi]);
        }
      }
      __syncwarp();
    } else if (warp == 3) {
      // ----------------------------------------------------------- pieces
      Walk w(a, C::kRows, *start);
      bool more = true, began = false;
      for (uint32_t seg = 0; more; ++seg) {
        const uint32_t pi = seg % kAhead;
        if (seg >= kAhead && !warp_wait(&piece_free[pi], (seg / kAhead - 1) & 1, abort_flag)) break;
        more = w.next();
        if (lane == 0) {
          RowsPiece &pc = pieces[pi];
          pc.more = more;
          if (more) {
            pc.x = w.x;
            pc.t = w.t;
            pc.h = w.h;
            pc.r0 = w.rt * C::kRows;
            pc.two = w.x.W * a.group - pc.r0 > 128;
            pc.j0 = w.j0;
            pc.tiles = w.tiles();
            pc.whole = w.whole();
            // a CTA's first piece has its first slot, its last one the second
            pc.slot = 2 * blockIdx.x + (seg > 0);
            began |= begin_join(a, w, *start, pc.slot);
          }
          mbar_arrive(&piece_full[pi]);
        }
        __syncwarp();
        if (more) prefetch_rows(a, w, C::kRows, DH, lane);
      }
      if (a.join && lane == 0 && !began) a.join[blockIdx.x].parts = 0;
    }
  } else if (FP8 && warp >= C::kConvWarp0) {
    // ------------------------------------------------------------- V codes -> bf16, K scales
    if constexpr (FP8) {
      reg_dealloc<C::kRegsConv>();
      const int t = (warp - C::kConvWarp0) * 32 + lane;
      uint32_t n = 0;
      for (uint32_t seg = 0;; ++seg) {
        const uint32_t pi = seg % kAhead;
        if (!warp_wait(&piece_full[pi], (seg / kAhead) & 1, abort_flag) || !pieces[pi].more) break;
        const TileList tl = pieces[pi].t;
        const int j0 = pieces[pi].j0, nT = pieces[pi].tiles;
        for (int j = 0; j < nT; ++j, ++n) {
          const uint32_t st = C::kKSt + n % C::kVSt, slot = n % C::kScaleSlots;
          const int key0 = tl.tile(j0 + j) * kTile;
          auto seen = [&](int key) { return key0 + key < tl.hi && (key0 + key >= tl.lo || key0 + key < a.sinks); };
          // a key without a page is a row of zeros, one that no row sees may have any scale
          auto byte_of = [&](int key, int kv) {
            const bool has = (pages_of[slot] >> (key >> a.c.page_shift) & 1) && seen(key);
            return has ? static_cast<uint32_t>(scales[slot * (2 * kTile) + kv * kTile + key]) : 127u;
          };
          mbar_wait(&sc_full[slot], (n / C::kScaleSlots) & 1, abort_flag);
          col_s[(n % 4) * kTile + t] = a.scale_log2 * scale_of(byte_of(t, 0));
          __syncwarp();
          if (lane == 0) mbar_arrive(&col_full[n % 4]);
          mbar_wait(&full[st], (n / C::kVSt) & 1, abort_flag);
#pragma unroll 1
          for (int half = 0; half < kTile / kConvKeys; ++half) {
            const uint32_t cn = n * (kTile / kConvKeys) + half, cb = cn % C::kCBuf;
            const int key = half * kConvKeys + t % kConvKeys;
            const uint32_t f = bf16x2_of(scale_of(byte_of(key, 1)));
            convert_v<DH>(smem + st * C::kRaw, smem + C::kOffConv + cb * (kConvKeys * DH * 2), half, t, seen(key),
                          [&] { if (cn >= C::kCBuf) mbar_wait(&c_free[cb], (cn / C::kCBuf - 1) & 1, abort_flag); },
                          [&](uint2 v) { return make_uint2(mul_bf16x2(v.x, f), mul_bf16x2(v.y, f)); });
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c_full[cb]);
          }
          if (lane == 0) mbar_arrive(&empty[st]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&piece_free[pi]);
      }
    }
  } else {
    // ------------------------------------------------------------- softmax
    reg_alloc<C::kRegsSoft>();
    const int s = (warp - 4) >> 2, quarter = warp & 3, tid = threadIdx.x & 127;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + lane_base + s * 128, t_o = tmem + lane_base + kColO + s * 128;
    uint32_t n0 = 0, ns = 0, o_seg = 0;
    // This group's part of piece `seg`'s query rows: begun, and there. When
    // its wait gave up the piece is not read: what lies there may be anything.
    // (Then the abort flag is up for good, and both groups leave before the
    // next piece.)
    auto stage = [&](uint32_t seg) {
      const uint32_t pi = seg % kAhead;
      if (!warp_wait(&piece_full[pi], (seg / kAhead) & 1, abort_flag)) return;
      const RowsPiece &pc = pieces[pi];
      if (!pc.more) return;
      float *qs = qs_s + (seg & 1) * 256;
      if (TWO && pc.two)
        stage_rows<DH, FP8, 128>(a, pc, pc.r0 + s * 128, 0, smem + C::kOffQ + s * C::kQ, qs + s * 128, tid);
      else
        stage_rows<DH, FP8, 64>(a, pc, pc.r0, s * 64, smem + C::kOffQ + (TWO ? 0 : seg & 1) * C::kQ, qs, tid);
    };
    auto staged = [&](uint32_t seg) {
      if constexpr (!FP8) copies_wait();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[seg % kAhead]);
    };
    for (uint32_t seg = 0;; ++seg) {
      const uint32_t pi = seg % kAhead;
      // all of both groups go on or none does
      if (bar_any(3, 256, *abort_flag || !mbar_wait(&piece_full[pi], (seg / kAhead) & 1, abort_flag))) break;
      const RowsPiece &pc = pieces[pi];
      if (!pc.more) break;
      if (seg == 0) {
        stage(0);
        staged(0);
        if constexpr (FP8) named_bar_sync(3, 256);   // the rows' powers of two
      }
      const TileList tl = pc.t;
      const int nT = pc.tiles, j0 = pc.j0, rows = pc.x.W * a.group;
      const bool two = TWO && pc.two;
      const int r = pc.r0 + (two ? s * 128 : 0) + tid, t = r / a.group;
      int lo = 0, hi = 0x7fffffff;   // a row that is none masks nothing; its results go nowhere
      if (r < rows) visible(a, pc.x.pos, t, pc.x.L, lo, hi);
      const int every = TREE ? tree_prefix(pc.x) : tl.hi_first;   // keys before it are behind no row
      const float qs = FP8 ? qs_s[(seg & 1) * 256 + (two ? s * 128 : 0) + tid] : 1.f;
      const int cnt = two ? nT : s == 0 ? (nT + 1) / 2 : nT / 2;
      // Streams with rows of their own, in this piece and the next: a stream's
      // space is free as soon as its last scores are done, and bf16 rows are
      // copied while its last weights are computed.
      bool early = false;
      if constexpr (TWO && !FP8) {
        const uint32_t next = (seg + 1) % kAhead;
        if (bar_any(3, 256, !mbar_wait(&piece_full[next], ((seg + 1) / kAhead) & 1, abort_flag))) break;
        early = two && nT > 0 && pieces[next].more && pieces[next].two;
      }
      // every row's O times its factor, by the whole warp (tcgen05.ld / st)
      auto rescale = [&](float corr) {
#pragma unroll 1
        for (int c0 = 0; c0 < DH; c0 += 32) {
          uint32_t o[32];
          tmem_ld32(t_o + c0, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
          tmem_st32(t_o + c0, o);
        }
        tmem_st_wait();
      };
      // m: the row's reference, l: its sum, top: how far scores have passed the reference
      float m = kNone, l = 0.f, top = -INFINITY;
      for (int k = 0; k < cnt; ++k, ++ns) {
        const uint32_t n = n0 + (two ? k : 2 * k + s);
        const int key0 = tl.tile(j0 + (two ? k : 2 * k + s)) * kTile;
        const bool masked = !(key0 + kTile <= every && (key0 >= tl.lo_last || key0 + kTile <= a.sinks));
        // trees: the keys of a masked tile that this row sees, fetched before the wait for the scores
        uint32_t tree[4] = {0, 0, 0, 0};
        if (TREE && masked) {
          const uint32_t *bits = a.mask + static_cast<size_t>(pc.x.q0 + t) * a.mask_stride;
          auto word = [&](long long i) {
            return r < rows && i >= 0 && i < a.mask_words ? __ldg(bits + i) & below(a.max_q - static_cast<int>(i) * 32) : 0u;
          };
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            // the first of these 32 keys is new token c: words floor(c / 32) and the next one, moved into place;
            // every row sees the tokens before the first, and itself
            const long long c = static_cast<long long>(key0) + w * 32 - pc.x.pos, own = t - c;
            const long long i = c >> 5;
            tree[w] = __funnelshift_r(word(i), word(i + 1), static_cast<uint32_t>(c) & 31);
            if (c < 0) tree[w] |= below(c <= -32 ? 32 : static_cast<int>(-c));
            if (own >= 0 && own < 32) tree[w] |= 1u << own;
            tree[w] &= below(pc.x.L - key0 - w * 32);
          }
        }
        const float c = FP8 ? qs : a.scale_log2;
        if constexpr (FP8) mbar_wait(&col_full[n % 4], (n / 4) & 1, abort_flag);
        if constexpr (!FP8) {
          // rows of V that no query row sees may hold anything, and 0 * NaN is not 0
          const int u = key0 + tid;
          if ((!two || s == 0) && !(u < tl.hi && (u >= tl.lo || u < a.sinks))) {
            const uint32_t st = C::kKSt + n % C::kVSt;
            mbar_wait(&full[st], (n / C::kVSt) & 1, abort_flag);
            uint8_t *sv = smem + st * C::kRaw + (tid / 8) * C::kGroup8 + (tid % 8) * 128;
#pragma unroll
            for (int e = 0; e < DH / 8; ++e)
              *reinterpret_cast<uint4 *>(sv + (e / 8) * 1024 + (e % 8) * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
          }
          __syncwarp();
        }
        mbar_wait(&s_full[s], ns & 1, abort_flag);
        tc_fence_after();
        // (without TWO: into the space of the last piece's rows)
        const bool ahead = TWO ? early && k == cnt - 1 : k == 0;
        if (!FP8 && ahead) stage(seg + 1);
        if (__any_sync(0xffffffffu, top > kLazy)) {
          // O holds exactly the stream's tiles before this one: their MMAs
          // were issued before this tile's scores, which are done
          const float corr = top > kLazy ? ex2_approx(-top) : 1.f;
          if (top > kLazy) m += top;
          l *= corr;
          rescale(corr);
        }
        top = -INFINITY;
        const float4 *col = FP8 ? reinterpret_cast<const float4 *>(col_s + (n % 4) * kTile) : nullptr;
        // scores of keys 32 w .. to score * factor - ref in log2 units, -inf
        // where the row does not see the key
        auto relative = [&](uint32_t (&x)[32], int w, float ref) {
          const float2 cv = make_float2(c, c), rv = make_float2(-ref, -ref);
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float2 y0 = make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1]));
            float2 y1 = make_float2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
            float2 c0 = cv, c1 = cv;
            if constexpr (FP8) {
              // The keys' K scales times the row's factor first: exact, and no
              // product on the way overflows unless the score does. (The score
              // times the K scale first: 238 us for four prompts' pieces, dh 64
              // 205; this way 230 and 196, but 237 and 209 where the compiler
              // places the loads.)
              const float4 f = load_shared4(col + w * 8 + e / 4);
              c0 = __fmul2_rn(cv, make_float2(f.x, f.y));
              c1 = __fmul2_rn(cv, make_float2(f.z, f.w));
            }
            y0 = __ffma2_rn(y0, c0, rv);
            y1 = __ffma2_rn(y1, c1, rv);
            x[e] = __float_as_uint(y0.x); x[e + 1] = __float_as_uint(y0.y);
            x[e + 2] = __float_as_uint(y1.x); x[e + 3] = __float_as_uint(y1.y);
          }
          if (masked) {
            const uint32_t mask = TREE ? (w < 2 ? (w == 0 ? tree[0] : tree[1]) : w == 2 ? tree[2] : tree[3])
                                       : below(hi - key0 - w * 32) & (~below(lo - key0 - w * 32) | below(a.sinks - key0 - w * 32));
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(mask >> e & 1)) x[e] = 0xff800000u;
          }
        };
        // 64 keys at a time: enough independent work to fill the pipes
        // between the steps that depend on each other
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const uint32_t t_h = t_s + half * 64;
          uint32_t xa[32], xb[32];
          tmem_ld32(t_h, xa);
          tmem_ld32(t_h + 32, xb);
          tmem_ld_wait();
          relative(xa, half * 2, m);
          relative(xb, half * 2 + 1, m);
          float past = greatest(xa, xb);
          if (__any_sync(0xffffffffu, past > kJump)) {
            // new references for the rows that are far off, from these scores
            // (they are still in TMEM); O is rescaled once it is final for
            // what came before: P V of the first half is done
            tmem_ld32(t_h, xa);
            tmem_ld32(t_h + 32, xb);
            tmem_ld_wait();
            relative(xa, half * 2, 0.f);
            relative(xb, half * 2 + 1, 0.f);
            const float now = past > kJump ? greatest(xa, xb) : m;
            const float corr = now == m ? 1.f : ex2_approx(m - now);
            l *= corr;
            top -= now - m;
            m = now;
            if (half == 1) {
              mbar_wait(&h_done[s], ns & 1, abort_flag);
              tc_fence_after();
            }
            if (half == 1 || k > 0) rescale(corr);
            tmem_ld32(t_h, xa);
            tmem_ld32(t_h + 32, xb);
            tmem_ld_wait();
            relative(xa, half * 2, m);
            relative(xb, half * 2 + 1, m);
            past = greatest(xa, xb);
          }
          top = fmaxf(top, past);
          // P as bf16 pairs, over scores that have been read
          float2 acc = make_float2(0.f, 0.f);
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const uint32_t *x = e < 16 ? xa + 2 * e : xb + 2 * e - 32;
            const float2 p = make_float2(ex2_approx(__uint_as_float(x[0])), ex2_approx(__uint_as_float(x[1])));
            acc = __fadd2_rn(acc, p);
            pk[e] = pack_bf16x2(p.x, p.y);
          }
          l += acc.x + acc.y;
          tmem_st32(t_s + half * 32, pk);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[s * 2 + half]);
        }
        if (ahead) {
          if (FP8) stage(seg + 1);
          staged(seg + 1);
        }
      }
      n0 += nT;
      if (TWO ? !early : cnt == 0) {
        if (TWO) named_bar_sync(3, 256);   // both streams' scores are done, the query rows' space is free
        stage(seg + 1);
        staged(seg + 1);
      }
      if (nT > 0) {
        mbar_wait(o_full, o_seg & 1, abort_flag);
        ++o_seg;
        tc_fence_after();
      }
      // What the streams' O count for: f[0] this one's, f[1] the other's
      // (streams with rows of their own: 1 and 0). Each group writes half of
      // the columns of the shared rows, all columns of its own.
      float f0 = 1.f, f1 = 0.f;
      if (!two) {
        if (s == 1) ml_s[tid] = make_float2(m, l);
        named_bar_sync(3, 256);
        if (s == 0) {
          const float2 other = ml_s[tid];
          const float mm = fmaxf(m, other.x);
          f0 = cnt > 0 ? ex2_approx(m - mm) : 0.f;
          f1 = nT > 1 ? ex2_approx(other.x - mm) : 0.f;
          l = l * f0 + other.y * f1;
          m = mm;
        }
        named_bar_sync(3, 256);
        if (s == 0) ml_s[tid] = make_float2(f0, f1);
        named_bar_sync(3, 256);
        if (s == 1) {
          const float2 f = ml_s[tid];
          f0 = f.y;
          f1 = f.x;
        }
      }
      // final results are divided by the row's sum, which the first group has
      const bool whole = pc.whole;
      if (whole) {
        float inv = l != 0.f ? 1.f / l : 0.f;
        if (!two) {
          named_bar_sync(3, 256);
          if (s == 0) ml_s[tid] = make_float2(inv, 0.f);
          named_bar_sync(3, 256);
          inv = ml_s[tid].x;
        }
        f0 *= inv;
        f1 *= inv;
      }
      const uint32_t t_other = tmem + lane_base + kColO + (s ^ 1) * 128;
      const int c_begin = two ? 0 : s * (DH / 2), c_end = two ? DH : c_begin + DH / 2;
      const size_t row = static_cast<size_t>(pc.x.q0 + t) * a.Hq + pc.h * a.group + (r - t * a.group);
      const int rs = (two ? s * 128 : 0) + tid;   // row of the slot
#pragma unroll 1
      for (int c0 = c_begin; c0 < c_end; c0 += 16) {
        uint32_t o[16], o1[16];
        float y[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = o1[e] = 0;
        if (nT > 0) {   // an O that no tile was added to holds anything
          tmem_ld16(t_o + c0, o);
          if (!two) tmem_ld16(t_other + c0, o1);
          tmem_ld_wait();
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          // converted V rows hold every four elements in the order 0, 2, 1, 3
          const int i = FP8 ? (e & ~3) | ((e & 1) << 1) | ((e >> 1) & 1) : e;
          y[i] = f0 != 0.f ? __uint_as_float(o[e]) * f0 : 0.f;
          if (f1 != 0.f) y[i] += __uint_as_float(o1[e]) * f1;
        }
        if (!whole) {
          // [slot][DH / 4][row][4]: a warp's rows side by side
          float4 *d = reinterpret_cast<float4 *>(a.part_o) + (static_cast<size_t>(pc.slot) * (DH / 4) + c0 / 4) * C::kRows + rs;
#pragma unroll
          for (int e = 0; e < 16; e += 4) d[e / 4 * C::kRows] = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
        } else if (r < rows) {
          if (a.out_fp32) {
            float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + row * DH + c0);
#pragma unroll
            for (int e = 0; e < 16; e += 4) d[e / 4] = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
          } else {
            uint4 *d = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + row * DH + c0);
            d[0] = pack8(y);
            d[1] = pack8(y + 8);
          }
        }
      }
      if (two || s == 0) {
        if (!whole) a.part_ml[static_cast<size_t>(pc.slot) * C::kRows + rs] = make_float2(m, l);
        else if (r < rows && a.lse) a.lse[row] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (nT > 0) mbar_arrive(o_free);
        mbar_arrive(&piece_free[pi]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort_flag) atomicOr(a.status, DLLM_DEV_WAIT_TIMEOUT);
}

template <int DH, bool FP8, bool TWO>
dllm_status launch(const CUtensorMap &tk, const CUtensorMap &tv, const PagedArgs &a, int ctas, cudaStream_t s) {
  using C = RowsCfg<DH, FP8, TWO>;
  auto kern = a.mask ? paged_rows_kernel<DH, FP8, TWO, true> : paged_rows_kernel<DH, FP8, TWO, false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  if (e == cudaSuccess) e = launch_pdl(kern, dim3(ctas), dim3(C::kThreads), C::kBytes, s, tk, tv, a);
  return e == cudaSuccess ? DLLM_OK : cuda_error(e);
}

}  // namespace

dllm_status launch_paged_rows(int dh, bool fp8, int n_rows, const CUtensorMap &tk, const CUtensorMap &tv,
                              const PagedArgs &a, int ctas, cudaStream_t s) {
  const bool two = n_rows == 256;
  if (dh == 64) {
    if (fp8) return two ? launch<64, true, true>(tk, tv, a, ctas, s) : launch<64, true, false>(tk, tv, a, ctas, s);
    return two ? launch<64, false, true>(tk, tv, a, ctas, s) : launch<64, false, false>(tk, tv, a, ctas, s);
  }
  if (fp8) return two ? launch<128, true, true>(tk, tv, a, ctas, s) : launch<128, true, false>(tk, tv, a, ctas, s);
  return two ? launch<128, false, true>(tk, tv, a, ctas, s) : launch<128, false, false>(tk, tv, a, ctas, s);
}

}  // namespace dllm
