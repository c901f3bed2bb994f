// Attention of new tokens over the paged K/V cache (bf16 or e4m3 pages):
// grouped query heads, causal or bidirectional, sliding window with the
// first tokens visible. This kernel takes up to 32 query rows per request and
// cached head (paged_rows.cu takes more), and joins divided items of both.
//
// The work of one (request, cached head) is S^T = K Q^T over the head's
// cached rows, with the query rows that share the head (W rows x group heads)
// as N. Keys are the M = 128 rows of the tensor-core tile, so N is as small
// as the rows are (16 or 32): a single token costs a tile of 16, not of 128,
// the exponentials of one key tile spread over 128 threads (one key each,
// whatever N is), and a key's scales and visibility are one thread's scalars.
// O^T = V^T P^T accumulates in TMEM.
//
// The key tiles of all (request, head, row tile) items form one line that is
// cut into equal pieces, one per CTA: long and short requests balance, and a
// single long one spreads over the whole GPU. An item that a cut divides
// leaves partial (m, l, O) of its pieces in the workspace, and a second
// kernel joins them.
//
// Warp roles:
//   warp 0      TMA: one box per page and tile (load_tiles)
//   warp 1      S^T MMAs: K tile (A) x query rows (B) into an S buffer
//   warp 2      O^T MMAs: V tile (A, transposed by its descriptor) x P (B)
//   warp 3      walks the CTA's pieces ahead of the others
//   warps 4..11 two softmax warpgroups, one key per thread, taking the key
//               tiles in turn, each with references, sums and an O of its own
//               that are merged at the end: the steps of one tile depend on
//               each other, and two tiles under way hide that. They also
//               stage the rows.
// A reference maximum per row moves only when a score passes it by more than
// 2^kLazy, so most tiles need no maximum at all, only the vote that nobody
// passed it.
//
// e4m3 pages: K and V codes go to the tensor cores as they are.
//   Scores: the query rows are split into two e4m3 parts and the key's scale
//   is a factor of its thread's scores. The rows are scaled so that their
//   largest lies in (224, 448]. High + low is exact for elements from 1/4 on
//   (eight significant bits, the last of them no less than the least e4m3 step
//   2^-9), and 2^-10 off below: exact within 2^-9 of the row's largest, else up
//   to 2^-10 / 224 = 2^-17.8 of that off.
//   Weights: P times the V scale, relative to the largest V scale so far, is
//   split into three e5m2 parts (three bits each: half a step of the ninth, and
//   half of fp16's before: 2^-8.8 off). e5m2 spans 2^32; weights below 2^-10
//   go, 2^12 times larger, to accumulator columns of their own, so that this
//   holds down to 2^-32 of the largest; below, half of e5m2's least step and of
//   fp16's step there remain, (2^-17 + 2^-19) / 2^25 = 2^-41.6 of it. (Codes
//   converted to bf16 by four more warps, with P in bf16: the conversion took
//   1.9 k cycles a tile, the loads of a tile 1.4 k.)
//
// Bound by memory where the keys are long: 4 requests of 20 to 40 thousand
// keys (bf16, 8 x 4 heads, dh 128) take 95 us, 5.7 TB/s and 85 % of a copy's
// rate; 64 requests of 1 to 8192 keys (e4m3) 125 us, 4.7 TB/s and 69 %; 32
// requests that see 4096 keys each (e4m3, 4 x 8 heads) 42 us, 47 %: there some
// 5 us until the first scores, 3 us of joining and the steps of one tile, of
// which an e4m3 tile's load hides less, remain. One token over 257 keys
// (16 heads of 64): 9 us, all of it such latencies.
#include <type_traits>

#include "paged.cuh"

namespace dllm {

DLLM_DEFINE_STATUS(paged)

namespace {

constexpr int kAhead = 4;        // pieces prepared, the current one included

template <int DH, bool FP8, int N>
struct Cfg {
  static constexpr int kGroups = 2;                             // softmax warpgroups (three: no gain)
  static constexpr int kSBuf = 2 * kGroups, kPBuf = kGroups;
  static constexpr int kThreads = 128 * (1 + kGroups);
  // registers a thread: what the TMA and MMA warps do not need goes to the
  // softmax groups (the sum is the launch's)
  static constexpr int kRegsIssue = 104, kRegsSoft = 200;
  static_assert(kRegsIssue + kGroups * kRegsSoft <= 3 * 168, "registers");
  static constexpr int kRaw = kTile * DH * (FP8 ? 1 : 2);       // one K or V tile
  static constexpr int kGroup8 = 8 * DH * (FP8 ? 1 : 2);        // eight cached rows
  static constexpr int kO = FP8 ? 2 * N : N;                    // columns of a group's O, and of a part of P
  static constexpr int kPart = kTile * kO * (FP8 ? 1 : 2);
  static constexpr int kP = kPart * (FP8 ? 3 : 1);
  static constexpr int kQ = N * DH * 2;                         // bf16, or two e4m3 parts
  static constexpr int kMisc = FP8 ? 12288 : 8192;              // row tables, scales, barriers, alignment
  static constexpr int kFixed = kPBuf * kP + kQ + kMisc;
  static constexpr int kMaxStages = (232448 - kFixed) / kRaw;
  static constexpr int kStages = kMaxStages * kRaw > 196608 ? 196608 / kRaw : kMaxStages;   // 192 KB in flight are enough
  static constexpr int kKSt = kStages / 2, kVSt = kStages - kKSt, kLead = 2;   // (1 or 3: the same time)
  static constexpr int kOffP = kStages * kRaw;
  static constexpr int kOffQ = kOffP + kPBuf * kP;
  static constexpr int kOffMisc = kOffQ + kQ;
  static constexpr int kBytes = kOffMisc + kMisc;
  // Scales of a tile's keys. A slot is written again once the K stage of the
  // tile kKSt before it is free: that tile's S^T is done, so the scores and
  // scales of every tile up to kSBuf before that one are read.
  static constexpr int kScaleSlots = FP8 ? kKSt + kSBuf + 1 : 0;
  static constexpr int kUsedCols = kSBuf * N + kGroups * kO;    // S buffers and O
  static constexpr uint32_t kTmemCols = kUsedCols <= 128 ? 128 : 256;
  static_assert(kStages >= 4 && kBytes <= 232448, "shared memory");
  static_assert(kUsedCols <= kTmemCols, "tensor memory");
};

// What the softmax needs to know of the row tile's rows.
template <int N>
struct alignas(16) RowInfo {
  int lo[N], hi[N];   // the keys the row sees, apart from the sinks
  int out[N];         // row of out [q_rows * Hq], or -1: not a query row
  float scale[N];     // e4m3 parts: what the query row was divided by
};

// A piece of an item as the warps that work on it need it.
struct alignas(16) Piece {
  Extent x;
  TileList t;
  int h, r0;               // head, first flat row
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

// The N query rows of a piece into shared memory as the B operand of S^T
// (core matrices along K, row groups of 8), by 256 threads, with what the
// softmax needs to know of each row.
template <int DH, bool FP8, int N>
__device__ __forceinline__ void stage_queries(const PagedArgs &a, const Piece &pc, uint8_t *sq, RowInfo<N> &info, int tid) {
  const int rows = pc.x.W * a.group;
  constexpr int kChunks = DH / 8;                  // 16-byte chunks of a bf16 row
  constexpr int kEach = (N * kChunks + 255) / 256;
  uint4 u[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {                // every load on its way before the first store
    const int idx = tid + i * 256, r = pc.r0 + idx / kChunks, t = r / a.group, g = r - t * a.group;
    u[i] = make_uint4(0, 0, 0, 0);
    if (idx < N * kChunks && r < rows)
      u[i] = __ldg(reinterpret_cast<const uint4 *>(a.q + (pc.x.q0 + t) * a.q_stride + (pc.h * a.group + g) * DH + idx % kChunks * 8));
  }
  if (tid < N) {
    const int r = pc.r0 + tid, t = r / a.group;
    int lo = 0, hi = 0x7fffffff;   // a column that is no row masks nothing; its results go nowhere
    if (r < rows) visible(a, pc.x.pos, t, pc.x.L, lo, hi);
    info.lo[tid] = lo;
    info.hi[tid] = hi;
    info.out[tid] = r < rows ? (pc.x.q0 + t) * a.Hq + pc.h * a.group + (r - t * a.group) : -1;
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int idx = tid + i * 256, n = idx / kChunks, c = idx % kChunks;
    if (idx >= N * kChunks) break;                 // whole warps
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

// Weights of four rows (w >= 0) into three e5m2 parts, [part][0: as they are
// times 2^13, 1: the small ones times 2^25, zero in the other].
__device__ __forceinline__ void split_e5m2(const float (&w)[4], uint32_t (&out)[3][2]) {
  constexpr float kSmall = 1.f / 1024.f;
  float t[4], y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t[i] = w[i] - kSmall;                                 // its sign: small
    y[i] = w[i] * (t[i] < 0.f ? 33554432.f : 8192.f);
  }
  uint32_t h[2], part[3];
  uint16_t lo[2];
  uint32_t r[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    // e5m2 is the upper byte of f16: two parts are cut off, the third rounds the rest
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h[i]) : "f"(y[2 * i + 1]), "f"(y[2 * i]));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r[i]) : "r"(h[i]), "r"(h[i] & 0xff00ff00u));
    uint32_t r2;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r2) : "r"(r[i]), "r"(r[i] & 0xff00ff00u));
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(lo[i]) : "r"(r2));
  }
  part[0] = __byte_perm(h[0], h[1], 0x7531);
  part[1] = __byte_perm(r[0], r[1], 0x7531);
  part[2] = lo[0] | (static_cast<uint32_t>(lo[1]) << 16);
  // 0xff in the bytes of the small ones: sign bytes replicated
  uint32_t s01, s23;
  asm("prmt.b32 %0, %1, %2, 0xfbfb;" : "=r"(s01) : "r"(__float_as_uint(t[0])), "r"(__float_as_uint(t[1])));
  asm("prmt.b32 %0, %1, %2, 0xfbfb;" : "=r"(s23) : "r"(__float_as_uint(t[2])), "r"(__float_as_uint(t[3])));
  const uint32_t small = __byte_perm(s01, s23, 0x5410);
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    out[p][0] = part[p] & ~small;
    out[p][1] = part[p] & small;
  }
}

template <int DH, bool FP8, int N>
__global__ void __launch_bounds__(Cfg<DH, FP8, N>::kThreads, 1)
paged_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const PagedArgs a) {
  using C = Cfg<DH, FP8, N>;
  constexpr int kSt = C::kStages, kO = C::kO, kG = C::kGroups, kSBuf = C::kSBuf, kPBuf = C::kPBuf;
  // FP8: the V scale enters the weights, so they must not pass 2^2
  constexpr float kPass = FP8 ? 2.f : kLazy;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *misc = smem + C::kOffMisc;
  RowInfo<N> *info = reinterpret_cast<RowInfo<N> *>(misc);                // [piece parity]
  Piece *pieces = reinterpret_cast<Piece *>(info + 2);                    // [kAhead]
  float *m_s = reinterpret_cast<float *>(pieces + kAhead);                // [group][N] reference maxima
  float *corr_s = m_s + kG * N;                                           // [group][N]
  float *red_s = corr_s + kG * N;                                         // [quarter][group][N]
  int *eref_s = reinterpret_cast<int *>(red_s + 4 * kG * N);              // [group], [quarter][group] exponents of V scales
  uint8_t *scales = reinterpret_cast<uint8_t *>(eref_s + 16);             // [kScaleSlots][K, V][kTile]
  uint32_t *pages_of = reinterpret_cast<uint32_t *>(scales + C::kScaleSlots * 2 * kTile);   // [kScaleSlots]: pages the tile has
  uint64_t *full = reinterpret_cast<uint64_t *>(pages_of + ((C::kScaleSlots + 1) & ~1));    // [kSt] stage loaded
  uint64_t *empty = full + kSt;             // [kSt] stage read by its MMAs
  uint64_t *s_full = empty + kSt;           // [kSBuf]
  uint64_t *s_free = s_full + kSBuf;        // [kSBuf]
  uint64_t *p_full = s_free + kSBuf;        // [kPBuf]
  uint64_t *p_free = p_full + kPBuf;        // [kPBuf] O^T MMAs of the tile done
  uint64_t *sc_full = p_free + kPBuf;       // [kScaleSlots]
  uint64_t *piece_full = sc_full + C::kScaleSlots;   // [kAhead]
  uint64_t *piece_free = piece_full + kAhead;        // [kAhead] its last use over
  uint64_t *q_full = piece_free + kAhead;   // [kAhead] its rows staged
  uint64_t *o_full = q_full + kAhead;
  uint64_t *o_free = o_full + 1;
  Scan *s_scan = reinterpret_cast<Scan *>(o_free + 1);
  Start *start = reinterpret_cast<Start *>(s_scan + 1);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(start + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  static_assert(2 * sizeof(RowInfo<N>) + kAhead * sizeof(Piece) + 6 * kG * N * 4 + 64 + C::kScaleSlots * (2 * kTile + 12) + 4 +
                        (2 * kSt + 2 * kSBuf + 2 * kPBuf + 3 * kAhead + 2) * 8 + sizeof(Scan) + sizeof(Start) + 8 <=
                    C::kMisc - 1024,
                "row tables and barriers");
  static_assert(sizeof(Piece) % 16 == 0 && (6 * kG * N * 4 + 64) % 16 == 0 && 5 * kG <= 16, "scales, 16-byte aligned for the bulk loads");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kSt; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int b = 0; b < kSBuf; ++b) { mbar_init(&s_full[b], 1); mbar_init(&s_free[b], 4); }
    for (int b = 0; b < kPBuf; ++b) { mbar_init(&p_full[b], 4); mbar_init(&p_free[b], 1); }
    for (int b = 0; b < C::kScaleSlots; ++b) mbar_init(&sc_full[b], 1);
    for (int b = 0; b < kAhead; ++b) {
      mbar_init(&piece_full[b], 1);
      mbar_init(&piece_free[b], 4 * kG + 2);   // the warps that read the piece
      mbar_init(&q_full[b], 8);
    }
    mbar_init(o_full, 1);
    mbar_init(o_free, 8);             // the groups that read O
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
  const uint32_t t_o = tmem + kSBuf * N;    // O of group g at kO g

  pdl_wait();   // the batch's metadata, the pages and the queries may come from the previous kernel
  find_start(a, N, s_scan, start);

  if (warp < 4) {
    reg_dealloc<C::kRegsIssue>();
    if (warp == 0) {
      load_tiles<DH, FP8 ? 1 : 2, C::kKSt, C::kVSt, C::kLead, C::kScaleSlots>(a, *start, N, &tm_k, &tm_v, smem, full, empty, scales,
                                                                              pages_of, sc_full, abort_flag, lane);
    } else if (warp == 1) {
      // ----------------------------------------------------------- S^T MMAs
      // (one elected thread through the whole loop: see paged_rows.cu)
      if (elect_one()) {
        uint32_t n = 0;
        bool ok = true;
        for (uint32_t seg = 0; ok; ++seg) {
          const uint32_t pi = seg % kAhead;
          ok = mbar_wait(&piece_full[pi], (seg / kAhead) & 1, abort_flag);
          if (!ok || !pieces[pi].more) break;
          ok = mbar_wait(&q_full[pi], (seg / kAhead) & 1, abort_flag);
          const int nT = pieces[pi].tiles;
          const uint32_t sq = smem_u32(smem + C::kOffQ);
          for (int j = 0; ok && j < nT; ++j, ++n) {
            const uint32_t st = n % C::kKSt, b = n % kSBuf;
            ok = mbar_wait(&full[st], (n / C::kKSt) & 1, abort_flag);
            if (ok && n >= kSBuf) ok = mbar_wait(&s_free[b], (n / kSBuf - 1) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const uint32_t sk = smem_u32(smem + st * C::kRaw);
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
                  umma_f8(tmem + b * N, dk + ((kk * 32) >> 4), dq + ((kk * 256) >> 4), idesc_f8(128, N, kE4M3, kE4M3, 0, 0),
                          part + kk > 0);
              }
            }
            umma_commit(&s_full[b]);
            umma_commit(&empty[st]);
          }
          mbar_arrive(&piece_free[pi]);
        }
      }
      __syncwarp();
    } else if (warp == 2) {
      // ----------------------------------------------------------- O^T MMAs
      if (elect_one()) {
        uint32_t n = 0, o_seg = 0;
        bool ok = true;
        for (uint32_t seg = 0; ok; ++seg) {
          const uint32_t pi = seg % kAhead;
          ok = mbar_wait(&piece_full[pi], (seg / kAhead) & 1, abort_flag);
          if (!ok || !pieces[pi].more) break;
          const int nT = pieces[pi].tiles;
          for (int j = 0; ok && j < nT; ++j, ++n) {
            const uint32_t st = C::kKSt + n % C::kVSt, b = n % kPBuf;
            if (j == 0 && o_seg > 0) ok = mbar_wait(o_free, (o_seg - 1) & 1, abort_flag);
            ok = ok && mbar_wait(&full[st], (n / C::kVSt) & 1, abort_flag);
            ok = ok && mbar_wait(&p_full[b], (n / kPBuf) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const uint32_t t_d = t_o + n % kG * kO;
            const uint32_t add = j >= kG;   // the first tile of each group's accumulator
            const uint32_t sv = smem_u32(smem + st * C::kRaw), sp = smem_u32(smem + C::kOffP + b * C::kP);
            if constexpr (!FP8) {
              const uint64_t dv = sw128_desc(sv, 1024, C::kGroup8), dp = plain_desc(sp, 128, 2048);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                umma_bf16(t_d, dv + ((kk * 2 * C::kGroup8) >> 4), dp + ((kk * 256) >> 4), idesc_bf16(DH, N, 1, 1),
                          kk > 0 ? 1u : add);
            } else {
              const uint64_t dv = DH == 128 ? sw128_desc(sv, 1024, C::kGroup8) : sw64_desc(sv, 1024, C::kGroup8);
#pragma unroll
              for (int part = 0; part < 3; ++part) {
                const uint64_t dp = plain_desc(sp + part * C::kPart, 128, 2048);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  umma_f8(t_d, dv + ((kk * 4 * C::kGroup8) >> 4), dp + ((kk * 512) >> 4), idesc_f8(DH, kO, kE4M3, kE5M2, 1, 1),
                          part + kk > 0 ? 1u : add);
              }
            }
            umma_commit(&empty[st]);
            umma_commit(&p_free[b]);
            if (j + 1 == nT) umma_commit(o_full);
          }
          o_seg += nT > 0;
          mbar_arrive(&piece_free[pi]);
        }
      }
      __syncwarp();
    } else {
      // ----------------------------------------------------------- pieces
      Walk w(a, N, *start);
      bool more = true, began = false;
      for (uint32_t seg = 0; more; ++seg) {
        const uint32_t pi = seg % kAhead;
        if (seg >= kAhead && !warp_wait(&piece_free[pi], (seg / kAhead - 1) & 1, abort_flag)) break;
        more = w.next();
        if (lane == 0) {
          Piece &pc = pieces[pi];
          pc.more = more;
          if (more) {
            pc.x = w.x;
            pc.t = w.t;
            pc.h = w.h;
            pc.r0 = w.rt * N;
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
        if (more) prefetch_rows(a, w, N, DH, lane);
      }
      if (a.join && lane == 0 && !began) a.join[blockIdx.x].parts = 0;
    }
  } else {
    // ------------------------------------------------------------- softmax
    reg_alloc<C::kRegsSoft>();
    const int wg = (warp - 4) >> 2, quarter = warp & 3, tid = threadIdx.x & 127;
    const int key = quarter * 32 + lane;
    const int g0 = wg * N;                     // the group's part of the groups' arrays
    constexpr int kOut = N / 2;                // rows that a group writes
    const int out0 = wg * kOut;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_d = t_o + lane_base + wg * kO;
    const auto maxop = [](float p, float q) { return fmaxf(p, q); };
    const auto addop = [](float p, float q) { return p + q; };
    uint32_t n = 0, o_seg = 0;
    // Piece seg's query rows. When its wait gave up the piece is not read:
    // what lies there may be anything. (Then the abort flag is up for good,
    // and both groups leave before the rows would be used.)
    auto stage = [&](uint32_t seg) {
      const uint32_t pi = seg % kAhead;
      if (!warp_wait(&piece_full[pi], (seg / kAhead) & 1, abort_flag)) return;
      if (!pieces[pi].more) return;
      stage_queries<DH, FP8, N>(a, pieces[pi], smem + C::kOffQ, info[seg & 1], threadIdx.x - 128);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[pi]);
    };
    stage(0);
    for (uint32_t seg = 0;; ++seg) {
      const uint32_t pi = seg % kAhead;
      // all of both groups go on or none does; the rows' info is written, the last piece's maxima are read
      if (bar_any(4, 128 * kG, *abort_flag || !mbar_wait(&piece_full[pi], (seg / kAhead) & 1, abort_flag))) break;
      const Piece &pc = pieces[pi];
      if (!pc.more) break;
      const RowInfo<N> &ri = info[seg & 1];
      const TileList tl = pc.t;
      const int nT = pc.tiles, j0 = pc.j0;
      float l[N];
#pragma unroll
      for (int e = 0; e < N; ++e) l[e] = 0.f;
      if (tid < N) m_s[g0 + tid] = kNone;
      int eref = -128;                      // V scales are relative to 2^eref
      named_bar_sync(1 + wg, 128);
      bool first = true;                    // of the group's tiles
      for (int j = 0; j < nT; ++j, ++n) {
        if (n % kG != wg) continue;
        const uint32_t b = n % kSBuf, pb = n % kPBuf;
        const int key0 = tl.tile(j0 + j) * kTile, u = key0 + key;
        // every row of the tile sees every key of it?
        const bool all_seen = key0 + kTile <= tl.hi_first && (key0 >= tl.lo_last || key0 + kTile <= a.sinks);
        const bool seen = u < tl.hi && (u >= tl.lo || u < a.sinks);   // this key, by any row
        float c = a.scale_log2;
        int vexp = -128;                    // exponent of the key's V scale
        bool vnan = false;
        if constexpr (FP8) {
          const uint32_t slot = n % C::kScaleSlots;
          mbar_wait(&sc_full[slot], (n / C::kScaleSlots) & 1, abort_flag);
          // a key without a page is a row of zeros, one that no row sees may have any scale
          if ((pages_of[slot] >> (key >> a.c.page_shift) & 1) && seen) {
            const uint8_t *sc = scales + slot * (2 * kTile) + key;
            c *= scale_of(sc[0]);
            vnan = sc[kTile] == 255;
            vexp = vnan ? -128 : static_cast<int>(sc[kTile]) - 127;
          }
        }
        mbar_wait(&s_full[b], (n / kSBuf) & 1, abort_flag);
        tc_fence_after();
        uint32_t s[N];
        tmem_load<N>(tmem + lane_base + b * N, s);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[b]);
        // x = score - reference in log2 units, two columns at a time, -inf
        // where the column's row does not see the key
        float x[N];
        auto relative = [&](const float *ref) {
#pragma unroll
          for (int e = 0; e < N; e += 2) {
            float2 f = make_float2(c, c), r = make_float2(0.f, 0.f);
            if constexpr (FP8) f = __fmul2_rn(f, *reinterpret_cast<const float2 *>(&ri.scale[e]));
            if (ref) r = *reinterpret_cast<const float2 *>(ref + e);
            const float2 y = __ffma2_rn(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), f, make_float2(-r.x, -r.y));
            x[e] = y.x;
            x[e + 1] = y.y;
          }
          if (!all_seen) {
#pragma unroll
            for (int e = 0; e < N; ++e)
              if (!(u < ri.hi[e] && (u >= ri.lo[e] || u < a.sinks))) x[e] = -INFINITY;
          }
        };
        relative(m_s + g0);
        float top = -INFINITY;
#pragma unroll
        for (int e = 0; e < N; e += 2) top = fmaxf(top, fmaxf(x[e], x[e + 1]));
        // nobody past its reference is the common case
        if (bar_any(1 + wg, 128, top > kPass || (FP8 && vexp > eref))) {
          // new references: the columns' maxima over the tile, the largest V scale
          relative(nullptr);
          float v[N];
#pragma unroll
          for (int e = 0; e < N; ++e) v[e] = x[e];
          const float most = reduce_columns<N>(v, lane, maxop);
          if (lane < N) red_s[quarter * (kG * N) + g0 + lane] = most;
          if constexpr (FP8) {
            const int e = __reduce_max_sync(0xffffffffu, vexp);
            if (lane == 0) eref_s[kG + quarter * kG + wg] = e;
          }
          named_bar_sync(1 + wg, 128);
          int e_new = eref;
          if constexpr (FP8)
            e_new = max(max(max(eref_s[kG + wg], eref_s[2 * kG + wg]), max(eref_s[3 * kG + wg], eref_s[4 * kG + wg])), eref);
          if (tid < N) {
            const int e = g0 + tid;
            const float mx = fmaxf(fmaxf(red_s[e], red_s[kG * N + e]), fmaxf(red_s[2 * kG * N + e], red_s[3 * kG * N + e]));
            const float old = m_s[e], now = mx > old + kPass ? mx : old;
            corr_s[e] = now == old ? 1.f : ex2_approx(old - now);
            m_s[e] = now;
          }
          named_bar_sync(1 + wg, 128);
#pragma unroll
          for (int e = 0; e < N; ++e) {
            l[e] *= corr_s[g0 + e];
            x[e] -= m_s[g0 + e];
          }
          if (!first) {
            // O holds exactly the group's tiles before this one once the MMAs of the last are done
            mbar_wait(&p_free[pb], (n / kPBuf - 1) & 1, abort_flag);
            tc_fence_after();
            const float ev = FP8 ? ex2_approx(static_cast<float>(eref - e_new)) : 1.f;
#pragma unroll
            for (int q = 0; q < kO; q += N) {
              uint32_t o[N];
              tmem_load<N>(t_d + q, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < N; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * (corr_s[g0 + e] * ev));
              tmem_store<N>(t_d + q, o);
            }
            tmem_st_wait();
            tc_fence_before();
          }
          eref = e_new;
        }
        // P = 2^x and its column sums per key
        if (n >= kPBuf) mbar_wait(&p_free[pb], (n / kPBuf - 1) & 1, abort_flag);
        uint8_t *sp = smem + C::kOffP + pb * C::kP + (key / 8) * 128 + (key % 8) * 16;
        if constexpr (!FP8) {
#pragma unroll
          for (int e = 0; e < N; e += 8) {
            uint32_t pk[4];
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const float2 p = make_float2(ex2_approx(x[e + i]), ex2_approx(x[e + i + 1]));
              const float2 sum = __fadd2_rn(make_float2(l[e + i], l[e + i + 1]), p);
              l[e + i] = sum.x;
              l[e + i + 1] = sum.y;
              pk[i / 2] = pack_bf16x2(p.x, p.y);
            }
            *reinterpret_cast<uint4 *>(sp + e / 8 * 2048) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
        } else {
          // (no page: a weight of 0 for a row of zeros)
          const float vs = vnan ? NAN : ex2_approx(static_cast<float>(vexp - eref));
#pragma unroll
          for (int e = 0; e < N; e += 16) {
            uint32_t pk[3][2][4];
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              float w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float p = ex2_approx(x[e + i + k]);
                l[e + i + k] += p;
                w[k] = p * vs;
              }
              uint32_t q[3][2];
              split_e5m2(w, q);
#pragma unroll
              for (int p = 0; p < 3; ++p) { pk[p][0][i / 4] = q[p][0]; pk[p][1][i / 4] = q[p][1]; }
            }
#pragma unroll
            for (int p = 0; p < 3; ++p)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                *reinterpret_cast<uint4 *>(sp + p * C::kPart + (h * (N / 16) + e / 16) * 2048) =
                    make_uint4(pk[p][h][0], pk[p][h][1], pk[p][h][2], pk[p][h][3]);
          }
        }
        // rows of V that no query row sees may hold anything, and 0 * NaN is not 0
        if (!seen) {
          const uint32_t st = C::kKSt + n % C::kVSt;
          mbar_wait(&full[st], (n / C::kVSt) & 1, abort_flag);
          // (the swizzles permute 16-byte pieces within a row)
          if constexpr (FP8) {
            uint8_t *sv = smem + st * C::kRaw + key * DH;
#pragma unroll
            for (int e = 0; e < DH / 16; ++e) *reinterpret_cast<uint4 *>(sv + e * 16) = make_uint4(0, 0, 0, 0);
          } else {
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
      // the next piece's rows are staged before this one's results are
      // written, so that its scores run meanwhile: every S^T of this piece
      // is done
      named_bar_sync(4, 128 * kG);
      stage(seg + 1);
      const float part = reduce_columns<N>(l, lane, addop);
      if (lane < N) red_s[quarter * (kG * N) + g0 + lane] = part;
      if (FP8 && tid == 0) eref_s[wg] = eref;
      named_bar_sync(1 + wg, 128);
      if (tid < N) {
        const int e = g0 + tid;
        corr_s[e] = (red_s[e] + red_s[kG * N + e]) + (red_s[2 * kG * N + e] + red_s[3 * kG * N + e]);
      }
      if (nT > 0) {
        mbar_wait(o_full, o_seg & 1, abort_flag);
        ++o_seg;
        tc_fence_after();
      }
      named_bar_sync(4, 128 * kG);
      // rows [out0, out0 + kOut): maximum, sum, and what the groups' O count for
      auto highest = [&](int e) {
        float m = m_s[e];
#pragma unroll
        for (int g = 1; g < kG; ++g) m = fmaxf(m, m_s[g * N + e]);
        return m;
      };
      uint32_t o[kOut];
#pragma unroll
      for (int e = 0; e < kOut; ++e) o[e] = 0;
#pragma unroll
      for (int g = 0; g < kG; ++g) {
        // few tiles leave groups without an O
        if ((g + kG - (n - nT) % kG) % kG >= static_cast<uint32_t>(nT)) continue;
        uint32_t y[kOut], z[kOut];
        tmem_load<kOut>(t_o + lane_base + g * kO + out0, y);
        if constexpr (FP8) tmem_load<kOut>(t_o + lane_base + g * kO + N + out0, z);
        tmem_ld_wait();
        const float ev = FP8 ? scale_of(max(eref_s[g] + 127, 0)) : 1.f;
#pragma unroll
        for (int e = 0; e < kOut; ++e) {
          const float f = ex2_approx(m_s[g * N + out0 + e] - highest(out0 + e));
          float w = __uint_as_float(y[e]);
          if constexpr (FP8) w = (w * 0x1p-13f + __uint_as_float(z[e]) * 0x1p-25f) * ev;
          o[e] = __float_as_uint(__uint_as_float(o[e]) + w * f);
        }
      }
      if (nT > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_free);
      }
      auto merged = [&](int e) {   // {maximum, sum} of row e
        const float m = highest(e);
        float sum = 0.f;
#pragma unroll
        for (int g = 0; g < kG; ++g) sum += corr_s[g * N + e] * ex2_approx(m_s[g * N + e] - m);
        return make_float2(m, sum);
      };
      // M = 64: rows 16 q .. 16 q + 15 lie in the first 16 lanes of quarter q
      const int dc = DH == 128 ? key : quarter * 16 + lane;
      const bool dlive = DH == 128 || lane < 16;
      if (pc.whole) {
#pragma unroll
        for (int e = 0; e < kOut; ++e) {
          const int row = ri.out[out0 + e];
          if (row < 0) break;
          const float sum = merged(out0 + e).y;
          const float y = sum != 0.f ? __fdividef(__uint_as_float(o[e]), sum) : 0.f;
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
      if (lane == 0) mbar_arrive(&piece_free[pi]);
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
// finished, of up to 32 rows: one warp per row, the pieces in their order with a running
// maximum, four of them on the way at a time. About 3 us after single tokens:
// the partial results are still in L2, so it is latency.
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
        y[k] = *reinterpret_cast<const Vec *>(a.part_o + slot * DH + n * DH + c);   // [slot][row][DH]
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

// The same for row tiles of paged_rows.cu, whose partial results lie as
// [slot][DH / 4][row][4]: a block joins 32 rows, one per lane, each warp DH / 8
// of their columns, so that a load has a warp's rows side by side (a warp per
// row read half of each 32-byte sector: 5 to 8 us longer after prompts' pieces).
template <int DH>
__global__ void __launch_bounds__(kJoinThreads) paged_join_rows_kernel(const PagedArgs a, const int n_rows) {
  constexpr int kQuads = DH / 4 / (kJoinThreads / 32), kCols = 4 * kQuads;   // of a warp
  pdl_trigger();
  pdl_wait();
  const JoinJob job = a.join[blockIdx.x];
  const int n = blockIdx.y * 32 + (threadIdx.x & 31), quad0 = (threadIdx.x >> 5) * kQuads;
  if (job.parts == 0 || job.r0 + n >= job.rows) return;   // (n < n_rows: whole blocks)
  float m = -INFINITY, l = 0.f, o[kCols] = {};
  auto load = [&](int p, float2 &ml, float4 (&y)[kQuads]) {
    const size_t slot = static_cast<size_t>(p == 0 ? job.slot : 2 * (blockIdx.x + p)) * n_rows;
    ml = a.part_ml[slot + n];
    const float4 *src = reinterpret_cast<const float4 *>(a.part_o + slot * DH) + n;
#pragma unroll
    for (int i = 0; i < kQuads; ++i) y[i] = src[(quad0 + i) * n_rows];
  };
  float2 ml;
  float4 y[kQuads];
  load(0, ml, y);
  for (int p = 0; p < job.parts; ++p) {
    float2 ml_next = ml;
    float4 next[kQuads];
    if (p + 1 < job.parts) load(p + 1, ml_next, next);   // on its way meanwhile
    const float mn = fmaxf(m, ml.x), f = ex2_approx(m - mn), g = ex2_approx(ml.x - mn);
    l = l * f + ml.y * g;
    m = mn;
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      o[4 * i] = o[4 * i] * f + y[i].x * g;
      o[4 * i + 1] = o[4 * i + 1] * f + y[i].y * g;
      o[4 * i + 2] = o[4 * i + 2] * f + y[i].z * g;
      o[4 * i + 3] = o[4 * i + 3] * f + y[i].w * g;
      y[i] = next[i];
    }
    ml = ml_next;
  }
  const int r = job.r0 + n, t = r / a.group;
  const size_t row = static_cast<size_t>(job.q0 + t) * a.Hq + job.h * a.group + (r - t * a.group);
#pragma unroll
  for (int e = 0; e < kCols; ++e) o[e] = l != 0.f ? o[e] / l : 0.f;
  if (a.out_fp32) {
    float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + row * DH) + quad0;
#pragma unroll
    for (int i = 0; i < kQuads; ++i) d[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
  } else {
    uint4 *d = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + row * DH + quad0 * 4);
#pragma unroll
    for (int i = 0; i < kCols / 8; ++i) d[i] = pack8(o + 8 * i);
  }
  if (a.lse && quad0 == 0) a.lse[row] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
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

// Rows of a row tile. Up to 32 rows of a request and cached head are the N of
// the MMAs here, more are the M of those in paged_rows.cu. Measured (us; cached
// heads x group, dh 128, keys of a request):
//   4 rows, 32 requests, 8 x 4, 4000 keys:  tiles of 16: 87 (e4m3: 61), 32: 89 (74), 128: 93 (107)
//   32 rows, else the same:                 32: 90 (86), 128: 95 (108)
//   128 rows, 16 requests, else the same:   128: 50 (61), 256: 52 (61); 64 as N: half as long again as 128
// Tiles of 256 read each K and V tile once for twice the rows, but leave
// partial results of twice the size where items are divided, which weighs more
// in small calls. Measured by key tiles of all 256-row items together:
//   400 rows, 2000 keys, 2 x 8, dh 64 (512):           128: 19 (26), 256: 22 (27)
//   512 rows, 4000 keys, 4 requests x 8 heads (2048):  128: 38 (58), 256: 46 (59)
//   1200 rows, 4000 keys, 2 x 8 (2560):                128: 48 (71), 256: 52 (68)
//   2048 rows, 1000 keys, 4 x 8 (2048):                128: 53 (81), 256: 48 (64)
//   512 rows, 4000 keys, 8 x 8 (4096):                 128: 82 (109), 256: 66 (91)
//   512 rows, 4000 keys, 24 x 8 (12288):               128: 255 (279), 256: 176 (240)
// (the fourth line's call stays with 128 in bf16, 10 % longer). max_kv tiles are
// counted under a window too, which sees fewer: 2000 rows and 16 x 1 heads over
// 16000 keys have 128 items of 256 rows then, one per CTA, and 256 of 128 rows.
//   dh 64, window 256:                                 128: 26 (34), 256: 23 (28)
//   dh 64, window 1024:                                128: 35 (46), 256: 33 (40)
//   dh 64, window 4096:                                128: 68 (103), 256: 70 (86)
//   dh 128, window 1024:                               128: 44 (60), 256: 40 (47)
// (never more with a larger B, max_q or max_kv: the workspace grows with it)
constexpr double kFewTiles = 3000, kFewTilesE4m3 = 1500;

int row_tile(const dllm_kv_pages *pages, const dllm_paged_attn_args *a) {
  const long long rows = static_cast<long long>(a->max_q) * (a->Hq / pages->heads);
  if (rows <= 128) return rows <= 16 ? 16 : rows <= 32 ? 32 : 128;
  const double tiles = static_cast<double>(a->B) * pages->heads * ((rows + 255) / 256) * ((a->max_kv + kTile - 1) / kTile);
  return tiles <= (pages->type == DLLM_KV_E4M3 ? kFewTilesE4m3 : kFewTiles) ? 128 : 256;
}

// Whether items may be divided: those of up to kWholeTiles tiles are not, and
// the call has one launch and no workspace. Measured (one request, one token,
// 8 x 4 heads, dh 128, bf16): 500 keys whole 10.0 us, divided 11.3; 1000 keys
// whole 12.8, divided 11.5.
bool may_split(const dllm_paged_attn_args *a) { return a->max_kv > kWholeTiles * kTile; }

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
dllm_status launch(const CUtensorMap &tk, const CUtensorMap &tv, const PagedArgs &g, int ctas, cudaStream_t s) {
  using C = Cfg<DH, FP8, N>;
  auto kern = paged_attn_kernel<DH, FP8, N>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  if (e == cudaSuccess) e = launch_pdl(kern, dim3(ctas), dim3(C::kThreads), C::kBytes, s, tk, tv, g);
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
  g.whole = !split;
  const double most = static_cast<double>(a->B) * pages->heads * row_tiles * per_item;
  int ctas = sm_budget() < kMaxCtas ? sm_budget() : kMaxCtas;
  // (a whole item per CTA, or at least kMinTiles tiles)
  const double useful = split ? most / kMinTiles : most / per_item;
  if (useful < ctas) ctas = static_cast<int>(useful) + 1;
  const dllm_status st = n == 16   ? launch<DH, FP8, 16>(tk, tv, g, ctas, s)
                         : n == 32 ? launch<DH, FP8, 32>(tk, tv, g, ctas, s)
                                   : launch_paged_rows(DH, FP8, n, tk, tv, g, ctas, s);
  if (st != DLLM_OK) return st;
  unsigned launches = 1;
  if (split) {
    const cudaError_t e =
        n <= 32 ? launch_pdl(paged_join_kernel<DH>, dim3(ctas, (n * 32 + kJoinThreads - 1) / kJoinThreads), dim3(kJoinThreads), 0, s, g, n)
                : launch_pdl(paged_join_rows_kernel<DH>, dim3(ctas, n / 32), dim3(kJoinThreads), 0, s, g, n);
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
  if (!a->q || !a->out || !a->q_off || !a->kv_len || (!a->page_table && a->max_pages > 0)) return DLLM_ERR_INVALID_ARG;
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
