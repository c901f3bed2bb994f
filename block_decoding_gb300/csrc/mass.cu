// The weight that attention gave to every cached row: for each position of a
// request and cached head, the sum over query rows (and the query heads that
// share the cached head) of exp(scale <q, k> - lse), added to what the row's
// slot holds from earlier steps, times a decay.
//
// lse is known, so there is no maximum to follow and no second pass: S^T = K Q^T
// with the cached rows as the M = 128 of the tensor-core tile and query rows as
// its N puts all scores of one cached row into one thread's TMEM lane, and the
// sum over query rows is that thread's alone. No exchange, no atomics, an order
// that the shapes decide. The key's scale, slot and visibility are scalars of
// its thread. What depends on the query row is read by every thread of the CTA,
// 4 bytes a score: with bf16 pages lse is therefore part of the product, as three
// more columns of the query rows (-lse / scale in bf16 parts) against ones. (As
// factors and terms from shared memory, 16 warps' reads of 16 bytes for all
// lanes took 2 k cycles of a unit's 3.3 k.)
//
// Query rows pass by in chunks of up to 128, each read once for all tiles of an
// item. An item is 512 keys of one request and cached head, 128 of them for each
// of four epilogue warpgroups. Over e4m3 pages, chunks of up to 64 rows (decode
// steps) take 1024 keys, two a thread: a tile is half as long on its way, and
// what an item costs by itself is spread over more of them. Neighbouring items of
// a head whose rows are one chunk share it. The items form one line, each as long
// as its chunks and what every item costs, cut into equal stretches, one per CTA.
//
// Warp roles:
//   warp 0        K tiles by TMA, one box per page, two tiles to a stage, and the
//                 slots' old values (and scales), whole items ahead
//   warps 1, 2    MMAs, of every other tile (one thread for all is short of time
//                 with few query rows: some 900 cycles a tile; four: no gain)
//   warp 3        walks the CTA's items ahead of the others
//   warps 4..7    a chunk's query rows, their lse and bounds. bf16 pages: the rows
//                 by TMA. e4m3 pages and few rows: in two e4m3 parts as
//                 paged_attn.cu has them, for K codes go to the tensor cores as
//                 they are (converted to bf16 by four warps: 2.1 k cycles a tile,
//                 the loads of a tile 0.7 k). With more rows the rows cost more
//                 than the codes, and are needed once a chunk and item.
//   warps 8..23   four groups: (e4m3 pages and many rows) codes to bf16,
//                 exponentials and sums
//
// 64 single tokens over 1 to 8192 keys (8 x 4 heads, dh 128): e4m3 55 us, 4.9
// TB/s and 73 % of a copy's rate; bf16 87 us, 89 %. e4m3 is bound by the roles'
// steps for an item, one after the other (without any loads and sums 39 us). The
// last 50 to 64 tokens of four prompts over 9 to 12 thousand keys, bf16: 30.5 us,
// of which 5 pass until the first scores; the last 1000 to 1200: 343 us, 1.02
// PFLOP/s, 53 % of a plain matrix product's rate (e4m3 369 us): a chunk's MMAs on
// four tiles take some 2.3 k cycles, their exponentials 2 k, the unit 3.8 k.
#include <math.h>

#include <type_traits>

#include "paged.cuh"

namespace dllm {

DLLM_DEFINE_STATUS(mass)

namespace {

struct MassArgs : PagedArgs {
  float *mass;
  const int32_t *fresh;
  float decay;
  int tokens;       // query tokens of a chunk: tokens * group rows
  int columns;      // ... rounded up to the N of the MMA
  int item_keys;    // keys of an item
  int k_stages;     // stages of two tiles, and where the chunks lie
  int off_q, q_bytes;
  float lse_scale;  // - 1 / scale
};

constexpr int kGroups = 4;       // epilogue warpgroups
constexpr int kNarrow = 64;      // rows of a chunk that two keys a thread go with (they are all of a request's: had it more,
                                 // its chunks would have 65 or more; so a stage is free again as soon as it is read)
constexpr int kChunkRows = 128;
constexpr int kAhead = 8;        // items prepared, the current one included
constexpr int kInfo = 3;         // chunks whose rows' numbers are prepared
constexpr int kItemLength = 2;   // what an item costs beside its chunks, in chunks (0 to 4: the same time where requests are alike)

template <int DH, bool FP8, bool NARROW, bool FOLD>
struct MassCfg {
  static constexpr int kPer = NARROW ? 2 : 1;                  // keys of a thread
  static constexpr int kTiles = kGroups * kPer, kItemKeys = kTiles * kTile;
  // e4m3 pages and few rows: the codes are the MMA's operand; else converted
  static_assert(FP8 || !NARROW, "two keys a thread: codes");
  static constexpr bool kCodes = NARROW;
  static constexpr int kLoad = kTile * DH * (FP8 ? 1 : 2);     // a K tile as it is loaded, to the end of its space
  static constexpr int kRaw = kTile * DH * (kCodes ? 1 : 2);   // ... as the MMAs read it
  static constexpr int kStage = 2 * kRaw;
  static constexpr int kGroup8 = 8 * DH * (kCodes ? 1 : 2);
  static constexpr int kQSt = 2;
  static constexpr int kMaxKSt = 6;
  static constexpr int kTables = 16128;                        // numbers, pieces and slots, before the barriers
  static constexpr int kSlotBytes = kItemKeys * 5 + kItemKeys / 16 * 4;
  static constexpr int kSlots = NARROW ? 2 : 4;                // items whose slots are loaded
  static constexpr int kOffOnes = 17408;                       // FOLD: a key's ones, and lse's parts of kInfo chunks
  static constexpr int kFold = FOLD ? kTile * 32 : 0;
  static constexpr int kOffK = kOffOnes + (1 + kInfo) * kFold; // stages, then chunks of query rows
  static constexpr int kMost = 232448 - 1024;
  static constexpr int kThreads = 32 * (8 + 4 * kGroups);
  // Bytes of a chunk (bf16, or two e4m3 parts), and the stages that fit beside kQSt chunks.
  static int chunk_bytes(int columns) { return columns * DH * 2; }
  static int stages(int columns) {
    const int fit = (kMost - kOffK - kQSt * chunk_bytes(columns)) / kStage;
    return fit < kMaxKSt ? fit : kMaxKSt;
  }
  static_assert(kOffK % 1024 == 0 && (kMost - kOffK - kQSt * (NARROW ? kNarrow : kChunkRows) * DH * 2) / kStage >= 2, "shared memory");
};

// A place in a ring of n and the parity of its round: `full` barriers complete
// phase `round`, `empty` ones (waited for with the other parity) the one before.
struct Ring {
  uint32_t at = 0, round = 0;
  __device__ __forceinline__ void next(uint32_t n) {
    if (++at == n) {
      at = 0;
      round ^= 1;
    }
  }
};

struct MassPiece {
  Extent x;
  int i, h, key0;          // request, head, first key
  int fresh;               // positions from here on start from 0
  int first, chunks;       // chunks [first, chunks) hold rows that see a key of the item
  int again, keep;         // the chunk is the last item's, is the next one's too
  int tiles;               // key tiles, 1 to kTiles (4, or 8 with two keys a thread)
  int more;
};

struct alignas(16) Numbers {   // of a chunk's query rows
  float neg_lse[kChunkRows];   // - lse in log2 units
  float scale[kChunkRows];     // e4m3 parts: what the row was divided by
  int hi[kChunkRows];          // keys before it are seen; 0: not a row, or one that saw nothing
  int every[kChunkRows / 16];  // keys before it are seen by all of 16
};

template <int KEYS>
struct alignas(16) Slots { // of an item's keys
  float old[KEYS];
  uint8_t scale[KEYS];
  int page[KEYS / 16];     // cache row of the head's first slot of each page, -1: no page
};

struct MassStart {
  long long left;          // length of the CTA's stretch from its first item on
  int i, item;
  Extent x;
};

__device__ __forceinline__ void mass_request(const MassArgs &a, const Extent &x, int &items, int &length) {
  items = x.W > 0 ? (x.L + a.item_keys - 1) / a.item_keys * a.c.heads : 0;
  length = (x.W + a.tokens - 1) / a.tokens + kItemLength;
}

// The CTA's first item, by all threads: the first that begins in its stretch.
__device__ __forceinline__ void mass_start(const MassArgs &a, long long *s_sum, MassStart *s_start) {
  const int nt = blockDim.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int chunk = (a.B + nt - 1) / nt, i0 = tid * chunk, i1 = min(a.B, i0 + chunk);
  long long mine = 0;
  int items, length;
  for (int i = i0; i < i1; ++i) {
    mass_request(a, paged_extent(a, i, blockIdx.x == 0), items, length);
    mine += static_cast<long long>(items) * length;
  }
  long long up = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += y;
  }
  if (lane == 31) s_sum[warp] = up;
  if (tid == 0) s_start->left = 0;
  __syncthreads();
  // the sums of all warps, and of those before this one
  long long total = lane < nt / 32 ? s_sum[lane] : 0, before = lane < warp ? total : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  before += up - mine;
  const long long per = quotient(total + gridDim.x - 1, gridDim.x), begin = per * blockIdx.x;
  if (begin >= before && begin < before + mine) {
    long long at = before;
    for (int i = i0; i < i1; ++i) {
      const Extent x = paged_extent(a, i, false);
      mass_request(a, x, items, length);
      const long long m = static_cast<long long>(items) * length;
      if (begin < at + m) {
        const int item = static_cast<int>(quotient(begin - at + length - 1, length));
        s_start->i = i;
        s_start->item = item;
        s_start->x = x;
        s_start->left = begin + per - (at + static_cast<long long>(item) * length);
        break;
      }
      at += m;
    }
  }
  __syncthreads();
}

// The 3-D box of a chunk's query rows: elements from x on of heads from h on of tokens from t on.
__device__ __forceinline__ void tma_load_rows(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int h, int t) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(h), "r"(t), "r"(smem_u32(bar))
      : "memory");
}

// Rows of chunk c, rounded up to the N of an MMA.
__device__ __forceinline__ int chunk_columns(const MassArgs &a, int W, int c) {
  return (min(a.tokens, W - c * a.tokens) * a.group + 15) & ~15;
}

// The query rows of chunk c in two e4m3 parts (DH-byte rows as K's are loaded,
// the parts a.columns rows apart) and the powers of two that they were divided
// by, by 128 threads.
template <int DH>
__device__ __forceinline__ void stage_chunk(const MassArgs &a, const Extent &x, int h, int c, uint8_t *rows, float *scale, int tid) {
  constexpr int kChunks = DH / 8, kStep = 128 / kChunks, kAtOnce = 4;   // 16-byte pieces of a row, rows of a step
  const int count = min(a.tokens, x.W - c * a.tokens) * a.group, piece = tid % kChunks;
  const uint16_t *q = a.q + (x.q0 + static_cast<long long>(c) * a.tokens) * a.q_stride + h * a.group * DH + piece * 8;
  for (int n0 = tid / kChunks; n0 - tid / kChunks < count; n0 += kAtOnce * kStep) {    // whole warps
    uint4 u[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int n = n0 + i * kStep, t = n / a.group;
      u[i] = n < count ? __ldg(reinterpret_cast<const uint4 *>(q + t * a.q_stride + (n - t * a.group) * DH)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int n = n0 + i * kStep;
      const uint32_t m2 = max_mag(u[i], 0);
      uint32_t m = max(m2 & 0xffffu, m2 >> 16);
#pragma unroll
      for (int o = kChunks / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (n >= count) continue;
      uint2 hi, lo;
      const int byte = split_e4m3(u[i], m, hi, lo);
      const int at = DH == 128 ? (piece / 2) ^ (n % 8) : (piece / 2) ^ ((n / 2) % 4);
      uint8_t *d = rows + n * DH + at * 16 + (piece % 2) * 8;
      *reinterpret_cast<uint2 *>(d) = hi;
      *reinterpret_cast<uint2 *>(d + a.columns * DH) = lo;
      if (piece == 0) scale[n] = scale_of(m < 0x7f80u ? byte : 255);   // a row with an infinity or NaN scores NaN
    }
  }
}

// lse, bound and the share in `every` of row n of chunk c, by whole warps of
// neighbouring rows.
__device__ __forceinline__ void numbers_of(const MassArgs &a, const Extent &x, int h, int c, int n, float &lse, int &hi, int &every) {
  const int at = n / a.group, t = c * a.tokens + at;
  hi = 0;
  lse = 0.f;
  if (at < a.tokens && t < x.W) {
    int lo;
    lse = __ldg(&a.lse[static_cast<size_t>(x.q0 + t) * a.Hq + h * a.group + (n - at * a.group)]);
    visible(a, x.pos, t, x.L, lo, hi);
    if (lse == -INFINITY) {
      hi = 0;
      lse = 0.f;
    }
  }
  every = hi;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) every = min(every, __shfl_xor_sync(0xffffffffu, every, o));
}

// A tile of e4m3 codes, which the loads put into the upper half of its space
// (DH-byte rows under their swizzle), to the bf16 rows that the codes and scales
// stand for, exactly, in the layout of a bf16 tile. By 128 threads, of row `key`
// each; all of them have read their codes before any writes (c_read). Returns
// whether the wait for that went well.
template <int DH>
__device__ __forceinline__ bool convert_codes(uint8_t *tile, int key, uint32_t scale2, uint64_t *c_read, uint32_t parity,
                                              volatile int *abort) {
  constexpr int kChunks = DH / 16;
  const uint8_t *src = tile + kTile * DH + key * DH;
  uint4 w[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c)
    w[c] = *reinterpret_cast<const uint4 *>(src + (DH == 128 ? c ^ (key & 7) : c ^ ((key >> 1) & 3)) * 16);
  __syncwarp();
  if (threadIdx.x % 32 == 0) mbar_arrive(c_read);
  if (!warp_wait(c_read, parity, abort)) return false;
  uint8_t *dst = tile + (key / 8) * (8 * DH * 2) + (key % 8) * 128;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const uint32_t in[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
    uint32_t out[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint2 v = e4m3x4_to_bf16_0213(in[e]);
      const uint32_t even = mul_bf16x2(v.x, scale2), odd = mul_bf16x2(v.y, scale2);
      out[2 * e] = __byte_perm(even, odd, 0x5410);
      out[2 * e + 1] = __byte_perm(even, odd, 0x7632);
    }
    uint8_t *d = dst + (c / 4) * 1024;   // 64 columns: eight 16-byte pieces
    *reinterpret_cast<uint4 *>(d + (((2 * c) & 7) ^ (key & 7)) * 16) = make_uint4(out[0], out[1], out[2], out[3]);
    *reinterpret_cast<uint4 *>(d + (((2 * c + 1) & 7) ^ (key & 7)) * 16) = make_uint4(out[4], out[5], out[6], out[7]);
  }
  return true;
}

// y as three bf16 parts that add up to it within 2^-24 (an infinity: itself and zeros).
__device__ __forceinline__ uint4 three_parts(float y) {
  const uint32_t hi = f32_to_bf16(y);
  const bool whole = (hi & 0x7fffu) == 0x7f80u;
  const float r = whole ? 0.f : y - bf16_to_f32(static_cast<uint16_t>(hi));
  const uint32_t mid = f32_to_bf16(r), lo = f32_to_bf16(r - bf16_to_f32(static_cast<uint16_t>(mid)));
  return make_uint4(hi | (mid << 16), lo, 0u, 0u);
}

template <int DH, bool FP8, bool NARROW, bool FOLD>
__global__ void __launch_bounds__(MassCfg<DH, FP8, NARROW, FOLD>::kThreads, 1)
mass_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ MassArgs a) {
  using C = MassCfg<DH, FP8, NARROW, FOLD>;
  using SlotsOf = Slots<C::kItemKeys>;
  static_assert(sizeof(SlotsOf) == C::kSlotBytes && !(C::kCodes && FOLD), "slots");
  constexpr int kQSt = C::kQSt, kTables = C::kTables, kSlots = C::kSlots;
  constexpr bool kCodes = C::kCodes, kConvert = FP8 && !kCodes;
  constexpr int kWidth = NARROW ? kNarrow : kChunkRows;        // columns of a tile's scores
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Numbers *numbers = reinterpret_cast<Numbers *>(smem);                      // [kInfo]
  SlotsOf *slots = reinterpret_cast<SlotsOf *>(numbers + kInfo);             // [kSlots]
  MassPiece *pieces = reinterpret_cast<MassPiece *>(slots + kSlots);         // [kAhead]
  uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + kTables);           // [k_stages]
  uint64_t *k_empty = k_full + C::kMaxKSt;
  uint64_t *q_full = k_empty + C::kMaxKSt; // [kQSt]
  uint64_t *q_empty = q_full + kQSt;
  uint64_t *n_full = q_empty + kQSt;       // [kInfo]
  uint64_t *n_empty = n_full + kInfo;
  uint64_t *slot_full = n_empty + kInfo;   // [kSlots]
  uint64_t *slot_empty = slot_full + kSlots;
  uint64_t *s_full = slot_empty + kSlots;  // [kTiles] scores of a tile
  uint64_t *s_empty = s_full + C::kTiles;
  uint64_t *c_full = s_empty + C::kTiles;         // [kGroups] codes of a group's tile are bf16
  uint64_t *c_read = c_full + kGroups;            // [kGroups] ... are read
  uint64_t *piece_full = c_read + kGroups;        // [kAhead]
  uint64_t *piece_empty = piece_full + kAhead;
  long long *s_sum = reinterpret_cast<long long *>(piece_empty + kAhead);    // [24]
  MassStart *start = reinterpret_cast<MassStart *>(s_sum + 24);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(start + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  static_assert(kInfo * sizeof(Numbers) + kSlots * sizeof(SlotsOf) + kAhead * sizeof(MassPiece) <= kTables && kTables % 16 == 0, "tables");
  static_assert(kTables + (2 * C::kMaxKSt + 2 * kQSt + 2 * kInfo + 2 * kSlots + 2 * C::kTiles + 2 * kGroups + 2 * kAhead + 24) * 8 + sizeof(MassStart) + 8 <=
                    C::kOffOnes, "barriers");
  uint8_t *const tiles_at = smem + C::kOffK, *const rows_at = smem + a.off_q;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.k_stages; ++s) { mbar_init(&k_full[s], 1); mbar_init(&k_empty[s], kConvert ? 2 + 4 * kGroups : 2); }
    for (int s = 0; s < kQSt; ++s) { mbar_init(&q_full[s], kCodes ? 4 : 5); mbar_init(&q_empty[s], 2); }
    for (int s = 0; s < kInfo; ++s) { mbar_init(&n_full[s], 4); mbar_init(&n_empty[s], 4 * kGroups); }
    for (int s = 0; s < kSlots; ++s) { mbar_init(&slot_full[s], 33); mbar_init(&slot_empty[s], 4 * kGroups); }
    for (int s = 0; s < kGroups; ++s) { mbar_init(&c_full[s], 4); mbar_init(&c_read[s], 4); }
    for (int s = 0; s < C::kTiles; ++s) { mbar_init(&s_full[s], 1); mbar_init(&s_empty[s], 4); }
    for (int s = 0; s < kAhead; ++s) {
      mbar_init(&piece_full[s], 1);
      mbar_init(&piece_empty[s], 1 + 2 + 4 + 4 * kGroups);   // the warps that read it
    }
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_k);
    if (!kCodes) tma_prefetch_desc(&tm_q);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if constexpr (FOLD) {
    // ones, and the second half of each of lse's rows, which stays 0
    for (int n = threadIdx.x; n < kTile * 2; n += C::kThreads)
      *reinterpret_cast<uint4 *>(smem + C::kOffOnes + n * 16) = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    for (int n = threadIdx.x; n < kInfo * kChunkRows; n += C::kThreads)
      *reinterpret_cast<uint4 *>(smem + C::kOffOnes + C::kFold + n / 8 * 256 + 128 + n % 8 * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  pdl_wait();   // everything that is read may come from the previous kernel
  mass_start(a, s_sum, start);

  // The item of number `seg`, or null when there is none (or a wait gave up:
  // then the slot is not read). By a whole warp.
  auto piece = [&](uint32_t seg) -> const MassPiece * {
    const MassPiece *p = &pieces[seg % kAhead];
    if (!warp_wait(&piece_full[seg % kAhead], (seg / kAhead) & 1, abort_flag)) return nullptr;
    return p->more ? p : nullptr;
  };
  auto piece_done = [&](uint32_t seg) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&piece_empty[seg % kAhead]);
  };

  if (warp == 0) {
    // --------------------------------------------------------------- K tiles, slots
    constexpr int kPages = C::kItemKeys / 16 / 32;      // pages of a lane, at most: lane + 32 q
    const int page_rows = 1 << a.c.page_shift, item_pages = C::kItemKeys >> a.c.page_shift;
    const int none = static_cast<int>((static_cast<long long>(a.c.num_pages) * a.c.heads << a.c.page_shift) / 8);
    // this lane's pages of an item, looked up while the item before it waits for room
    auto look_up = [&](const MassPiece *p, int (&page)[kPages]) {
#pragma unroll
      for (int q = 0; q < kPages; ++q) {
        const int n = lane + 32 * q, u = p->key0 + n * page_rows;
        page[q] = 0;
        if (n < item_pages && u < p->x.L)
          page[q] = __ldg(a.c.table + static_cast<size_t>(p->i) * a.c.max_pages + (u >> a.c.page_shift));
      }
    };
    bool ok = true;
    Ring k, sl;
    uint32_t n = 0;
    int page[kPages], page_next[kPages] = {};
    const MassPiece *p = piece(0);
    if (p) look_up(p, page);
    for (uint32_t seg = 0; ok && p; ++seg) {
      const int tiles = p->first < p->chunks ? p->tiles : 0;
      int row[kPages];             // cache row of the head's first slot of the page, -1: none
#pragma unroll
      for (int q = 0; q < kPages; ++q) {
        const int at = lane + 32 * q;
        const bool held = at < item_pages && p->key0 + at * page_rows < p->x.L, bad = held && (page[q] < 0 || page[q] >= a.c.num_pages);
        if (bad) atomicOr(a.status, DLLM_DEV_PAGE);
        row[q] = held && !bad ? (page[q] * a.c.heads + p->h) << a.c.page_shift : -1;
      }
      const MassPiece *p_next = piece(seg + 1);
      if (p_next) look_up(p_next, page_next);
      ok = warp_wait(&slot_empty[sl.at], sl.round ^ 1, abort_flag);
      if (!ok) break;
      SlotsOf &s = slots[sl.at];
#pragma unroll
      for (int q = 0; q < kPages; ++q)
        if (lane + 32 * q < item_pages) s.page[lane + 32 * q] = row[q];
      __syncwarp();
      // the slots 16 bytes a lane (bulk copies, one per page: some 100 cycles each)
#pragma unroll 4
      for (int at = lane * 4; at < C::kItemKeys; at += 128) {
        const int page = s.page[at >> a.c.page_shift];
        if (page >= 0) copy16(s.old + at, a.mass + page + (at & (page_rows - 1)), true);
      }
      if constexpr (FP8) {
#pragma unroll
        for (int at = lane * 16; at < C::kItemKeys; at += 512) {
          const int page = s.page[at >> a.c.page_shift];
          if (page >= 0) copy16(s.scale + at, a.c.k_scale + page + (at & (page_rows - 1)), true);
        }
      }
      copies_arrive(&slot_full[sl.at]);
      if (lane == 0) mbar_arrive(&slot_full[sl.at]);      // (the pages' rows are written)
      sl.next(kSlots);
      for (int j = 0; ok && j < tiles; j += 2) {
        ok = warp_wait(&k_empty[k.at], k.round ^ 1, abort_flag);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&k_full[k.at], 2 * C::kLoad);
        __syncwarp();
#pragma unroll
        for (int q = 0; q < kPages; ++q) {
          const int at = (lane + 32 * q) * page_rows - j * kTile;   // row of the stage
          if (at >= 0 && at < 2 * kTile)      // (what there is none of reads as zeros)
            tma_load_4d(tiles_at + k.at * C::kStage + (at / kTile + 1) * C::kRaw - C::kLoad + at % kTile * (C::kLoad / kTile), &tm_k,
                        &k_full[k.at], row[q] >= 0 ? row[q] / 8 : none);
        }
        k.next(a.k_stages);
        ++n;
      }
      piece_done(seg);
      p = p_next;
#pragma unroll
      for (int q = 0; q < kPages; ++q) page[q] = page_next[q];
    }
    // after an abort the loads in flight land before the CTA's memory is given up
    if (!ok || *abort_flag) {
      if (lane < a.k_stages && lane < n) mbar_drain(&k_full[lane], ((n - 1 - lane) / a.k_stages) & 1);
      copies_wait();
    }
    __syncwarp();
  } else if (warp <= 2) {
    // --------------------------------------------------------------- MMAs
    // (one elected thread through the whole loop: see paged_rows.cu)
    const int j = warp - 1;         // tiles j, j + 2, ..: one of a stage's two
    if (elect_one()) {
      bool ok = true;
      Ring t, q, in;                // stages, chunks, lse
      uint32_t ns[C::kTiles / 2] = {};   // units of the tiles
      uint32_t nc[C::kTiles / 2] = {};   // tiles converted
      for (uint32_t seg = 0; ok; ++seg) {
        const uint32_t pi = seg % kAhead;
        ok = mbar_wait(&piece_full[pi], (seg / kAhead) & 1, abort_flag);
        if (!ok || !pieces[pi].more) break;
        const MassPiece &p = pieces[pi];
        const int first = p.first, chunks = p.chunks, W = p.x.W, tiles = p.tiles;
        const bool again = p.again, keep = p.keep;
        Ring stage = t;
        for (int c = first; ok && c < chunks; ++c) {
          if (!again) ok = mbar_wait(&q_full[q.at], q.round, abort_flag);
          const uint32_t sq = smem_u32(rows_at + q.at * a.q_bytes);
          const int columns = chunk_columns(a, W, c);
          stage = t;
#pragma unroll
          for (int s = 0; s < C::kTiles / 2; ++s) {
            if (2 * s >= tiles || !ok) break;
            const int tile = 2 * s + j;
            if (c == first) ok = mbar_wait(&k_full[stage.at], stage.round, abort_flag);
            if (ok && tile < tiles) {
              const uint32_t t_s = tmem + tile * kWidth;
              if (kConvert && c == first) ok = mbar_wait(&c_full[tile], nc[s]++ & 1, abort_flag);
              ok = ok && mbar_wait(&s_empty[tile], (ns[s] & 1) ^ 1, abort_flag);
              if (!ok) break;
              tc_fence_after();
              const uint32_t sk = smem_u32(tiles_at + stage.at * C::kStage + j * C::kRaw);
              if constexpr (!kCodes) {
                const uint32_t idesc = idesc_bf16(128, columns, 0, 0);
                const uint64_t dk = sw128_desc(sk, 16, C::kGroup8), dq = sw128_desc(sq, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < DH / 16; ++kk)
                  umma_bf16(t_s, dk + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4),
                            dq + (((kk >> 2) * (a.columns * 128) + (kk & 3) * 32) >> 4), idesc, kk > 0);
                if constexpr (FOLD) {     // (last: sums are cut off at their size, and now they get small; first, 3 times the error)
                  const uint32_t ones = smem_u32(smem + C::kOffOnes);
                  umma_bf16(t_s, plain_desc(ones, 128, 256), plain_desc(ones + (1 + in.at) * C::kFold, 128, 256), idesc, 1);
                }
              } else {
                const uint32_t idesc = idesc_f8(128, columns, kE4M3, kE4M3, 0, 0);
                const uint64_t dk = DH == 128 ? sw128_desc(sk, 16, C::kGroup8) : sw64_desc(sk, 16, C::kGroup8);
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                  const uint32_t sp = sq + part * a.columns * DH;
                  const uint64_t dq = DH == 128 ? sw128_desc(sp, 16, 8 * DH) : sw64_desc(sp, 16, 8 * DH);
#pragma unroll
                  for (int kk = 0; kk < DH / 32; ++kk) umma_f8(t_s, dk + ((kk * 32) >> 4), dq + ((kk * 32) >> 4), idesc, part + kk > 0);
                }
              }
              umma_commit(&s_full[tile]);
              ++ns[s];
            }
            if (ok && c + 1 == chunks) umma_commit(&k_empty[stage.at]);
            stage.next(a.k_stages);
          }
          if (!keep) {
            if (ok) umma_commit(&q_empty[q.at]);
            q.next(kQSt);
            in.next(kInfo);
          }
        }
        t = stage;                  // behind the item's stages
        mbar_arrive(&piece_empty[pi]);
      }
    }
    __syncwarp();
  } else if (warp == 3) {
    // --------------------------------------------------------------- items
    long long left = start->left;
    int i = start->i, item = start->item, items = 0, length = 1;
    Extent x{};
    auto fresh_of = [&] { return a.fresh ? a.fresh[i] : 0x7fffffff; };
    int fresh = 0;
    if (left > 0) {
      x = start->x;
      mass_request(a, x, items, length);
      fresh = fresh_of();
    }
    bool more = true, again = false;
    int per_head = 1, h = 0, at = 0;       // items of a head, and where the item is
    auto divide = [&] {
      if (items == 0) return;
      per_head = items / a.c.heads;
      h = item / per_head;
      at = item - h * per_head;
    };
    divide();
    for (uint32_t seg = 0; more; ++seg) {
      const uint32_t pi = seg % kAhead;
      if (seg >= kAhead && !warp_wait(&piece_empty[pi], (seg / kAhead - 1) & 1, abort_flag)) break;
      more = left > 0;
      while (more && item >= items) {
        item = 0;
        if (++i >= a.B) { more = false; break; }
        x = paged_extent(a, i, false);
        mass_request(a, x, items, length);
        fresh = fresh_of();
        divide();
      }
      const int key0 = at * C::kItemKeys, chunks = length - kItemLength;
      // the chunk of the first row that sees a key
      auto first_of = [&](int key) {
        if (a.right < 0) return 0;
        const long long t = max(static_cast<long long>(key) - x.pos - a.right, 0ll);
        return t == 0 ? 0 : t < x.W ? static_cast<int>(t) / a.tokens : chunks;
      };
      const bool keep = more && chunks == 1 && at + 1 < per_head && left > length && first_of(key0 + C::kItemKeys) < 1;
      if (lane == 0) {
        MassPiece &p = pieces[pi];
        p.more = more;
        if (more) {
          p.x = x;
          p.i = i;
          p.h = h;
          p.key0 = key0;
          p.fresh = fresh;
          p.tiles = min((x.L - key0 + kTile - 1) / kTile, C::kTiles);
          p.chunks = chunks;
          p.first = first_of(key0);
          p.again = again;
          p.keep = keep;
        }
        mbar_arrive(&piece_full[pi]);
      }
      __syncwarp();
      again = keep;
      left -= length;
      ++item;
      if (++at == per_head) {
        at = 0;
        ++h;
      }
    }
  } else if (warp < 8) {
    // --------------------------------------------------------------- query rows and their numbers
    const int n = threadIdx.x - 128;       // row of a chunk
    bool ok = true;
    Ring q, in;
    uint32_t asked = 0;
    for (uint32_t seg = 0; ok; ++seg) {
      const MassPiece *p = piece(seg);
      if (!p) break;
      const Extent x = p->x;
      const int chunks = p->chunks, h = p->h;
      for (int c = p->again ? chunks : p->first; ok && c < chunks; ++c) {
        // (every warp waits: one that arrived twice in a round of q_full would complete it for another)
        ok = warp_wait(&q_empty[q.at], q.round ^ 1, abort_flag);
        if (!ok) break;
        if (!kCodes && warp == 4) {
          if (lane == 0) {
            mbar_arrive_expect_tx(&q_full[q.at], a.tokens * a.group * (DH * 2));
#pragma unroll
            for (int d = 0; d < DH / 64; ++d)
              tma_load_rows(rows_at + q.at * a.q_bytes + d * (a.columns * 128), &tm_q, &q_full[q.at], d * 64, h * a.group,
                            x.q0 + c * a.tokens);
          }
          ++asked;
          __syncwarp();
        }
        float lse;
        int hi, every;
        numbers_of(a, x, h, c, n, lse, hi, every);
        ok = warp_wait(&n_empty[in.at], in.round ^ 1, abort_flag);
        if (!ok) break;
        Numbers &s = numbers[in.at];
        if constexpr (FOLD) {
          *reinterpret_cast<uint4 *>(smem + C::kOffOnes + (1 + in.at) * C::kFold + n / 8 * 256 + n % 8 * 16) = three_parts(lse * a.lse_scale);
          fence_proxy_async_smem();
        } else {
          s.neg_lse[n] = lse * -1.4426950408889634f;
        }
        s.hi[n] = hi;
        if (n % 16 == 0) s.every[n / 16] = every;
        if constexpr (kCodes) {
          stage_chunk<DH>(a, x, h, c, rows_at + q.at * a.q_bytes, s.scale, n);
          fence_proxy_async_smem();
        }
        __syncwarp();
        // (groups with a tile read the numbers when its scores are there, MMAs wait for q_full)
        if (lane == 0) {
          mbar_arrive(&n_full[in.at]);
          mbar_arrive(&q_full[q.at]);
        }
        q.next(kQSt);
        in.next(kInfo);
      }
      piece_done(seg);
    }
    if (!kCodes && (!ok || *abort_flag))
      if (lane < kQSt && lane < asked) mbar_drain(&q_full[lane], ((asked - 1 - lane) / kQSt) & 1);
    __syncwarp();
  } else {
    // --------------------------------------------------------------- exponentials and sums
    constexpr int kPer = C::kPer;
    const int g = (warp - 8) >> 2, quarter = warp & 3;
    const int key = g * kTile + quarter * 32 + lane;      // of the item, and key + kGroups * kTile
    const uint32_t t_s = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + g * kWidth;
    bool ok = true;
    Ring in, sl;
    [[maybe_unused]] Ring t;
    uint32_t ns[kPer] = {};
    [[maybe_unused]] uint32_t nc = 0;
    for (uint32_t seg = 0; ok; ++seg) {
      const MassPiece *p = piece(seg);
      if (!p) break;
      ok = warp_wait(&slot_full[sl.at], sl.round, abort_flag);
      if (!ok) break;
      const int key0 = p->key0, L = p->x.L, W = p->x.W, chunks = p->chunks, tiles = p->tiles;
      const bool again = p->again, keep = p->keep;
      const SlotsOf &slot = slots[sl.at];
      float c[kPer], sum[kPer] = {};
      int page[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int k = key + i * kGroups * kTile;
        page[i] = key0 + k < L ? slot.page[k >> a.c.page_shift] : -1;
        c[i] = kCodes && page[i] >= 0 ? a.scale_log2 * scale_of(slot.scale[k]) : a.scale_log2;
      }
      const int end = key0 + (g + 1 + (kPer - 1) * kGroups) * kTile;   // behind the last of its keys
      if constexpr (kConvert) {
        // Every warp waits for every stage of the item, with a tile in it or not, and a stage is not loaded again before all
        // have: a wait tells a phase from the next one only, so none may go by unseen and nobody may be two behind.
#pragma unroll 1
        for (int s = 0; ok && p->first < chunks && 2 * s < tiles; ++s) {
          ok = warp_wait(&k_full[t.at], t.round, abort_flag);
          if (!ok) break;
          if (lane == 0) mbar_arrive(&k_empty[t.at]);
          if (s == g / 2 && g < tiles) {
            const uint32_t byte = page[0] >= 0 ? slot.scale[key] : 127u;      // (codes of no page are 0)
            ok = convert_codes<DH>(tiles_at + t.at * C::kStage + (g & 1) * C::kRaw, key % kTile, bf16x2_of(scale_of(byte)),
                                   &c_read[g], nc & 1, abort_flag);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c_full[g]);
            ++nc;
          }
          t.next(a.k_stages);
        }
      }
      for (int k = p->first; ok && k < chunks; ++k) {
        if (g >= tiles) {
          // no tile, no scores to wait for: but not ahead of the chunk
          if (!again) ok = warp_wait(&n_full[in.at], in.round, abort_flag);
        } else {
          bool there[kPer];
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            there[i] = g + i * kGroups < tiles;
            if (there[i]) ok = ok && warp_wait(&s_full[g + i * kGroups], ns[i]++ & 1, abort_flag);
          }
          if (ok) {
            tc_fence_after();
            // (written before the arrival that the MMAs waited for, at q_full, and so before their scores)
            const Numbers &s = numbers[in.at];
            const int columns = chunk_columns(a, W, k);
            float2 acc[kPer][2] = {};
            auto add_some = [&](auto &x, int c0, auto masked) {
#pragma unroll
              for (int e = 0; e < static_cast<int>(sizeof(x[0]) / 4); e += 4) {
                float4 z{};
                [[maybe_unused]] float4 f{};
                int4 hi{};
                if constexpr (!FOLD) z = *reinterpret_cast<const float4 *>(&s.neg_lse[c0 + e]);
                if constexpr (kCodes) f = *reinterpret_cast<const float4 *>(&s.scale[c0 + e]);
                if constexpr (decltype(masked)::value) hi = *reinterpret_cast<const int4 *>(&s.hi[c0 + e]);
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                  float2 f0 = make_float2(c[i], c[i]), f1 = f0;
                  if constexpr (kCodes) {  // the row's factor and the key's first: no product on the way overflows
                    f0 = __fmul2_rn(f0, make_float2(f.x, f.y));
                    f1 = __fmul2_rn(f1, make_float2(f.z, f.w));
                  }
                  float2 y0 = make_float2(__uint_as_float(x[i][e]), __uint_as_float(x[i][e + 1]));
                  float2 y1 = make_float2(__uint_as_float(x[i][e + 2]), __uint_as_float(x[i][e + 3]));
                  y0 = FOLD ? __fmul2_rn(y0, f0) : __ffma2_rn(y0, f0, make_float2(z.x, z.y));
                  y1 = FOLD ? __fmul2_rn(y1, f1) : __ffma2_rn(y1, f1, make_float2(z.z, z.w));
                  if constexpr (decltype(masked)::value) {
                    const int u = key0 + key + i * kGroups * kTile;
                    if (u >= hi.x) y0.x = -INFINITY;
                    if (u >= hi.y) y0.y = -INFINITY;
                    if (u >= hi.z) y1.x = -INFINITY;
                    if (u >= hi.w) y1.y = -INFINITY;
                  }
                  acc[i][0] = __fadd2_rn(acc[i][0], make_float2(ex2_approx(y0.x), ex2_approx(y0.y)));
                  acc[i][1] = __fadd2_rn(acc[i][1], make_float2(ex2_approx(y1.x), ex2_approx(y1.y)));
                }
              }
            };
            // (a branch: as selects under a condition the comparisons are all computed)
            auto add = [&](auto &x, int c0, int every) {
              if (end > every) add_some(x, c0, std::true_type{});
              else add_some(x, c0, std::false_type{});
            };
            int c0 = 0;
            if constexpr (!NARROW) {
              for (; c0 + 32 <= columns; c0 += 32) {
                uint32_t x[1][32];
                tmem_ld32(t_s + c0, x[0]);
                tmem_ld_wait();
                add(x, c0, min(s.every[c0 / 16], s.every[c0 / 16 + 1]));
              }
            }
            for (; c0 < columns; c0 += 16) {
              uint32_t x[kPer][16];
              tmem_ld16(t_s + c0, x[0]);
              if constexpr (kPer > 1) tmem_ld16(t_s + kGroups * kWidth + c0, x[kPer - 1]);   // (anything where there is no tile)
              tmem_ld_wait();
              add(x, c0, s.every[c0 / 16]);
            }
            tc_fence_before();
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
              if (there[i] && lane == 0) mbar_arrive(&s_empty[g + i * kGroups]);
              sum[i] += (acc[i][0].x + acc[i][0].y) + (acc[i][1].x + acc[i][1].y);
            }
          }
        }
        if (!keep) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&n_empty[in.at]);
          in.next(kInfo);
        }
      }
      if (ok) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int k = key + i * kGroups * kTile;
          if (page[i] >= 0)
            a.mass[static_cast<size_t>(page[i]) + (k & ((1 << a.c.page_shift) - 1))] =
                (key0 + k < p->fresh ? slot.old[k] * a.decay : 0.f) + sum[i];
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&slot_empty[sl.at]);
      sl.next(kSlots);
      piece_done(seg);
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

template <int DH, bool FP8, bool NARROW, bool FOLD>
dllm_status launch_mass(const dllm_kv_pages *pages, MassArgs &g, cudaStream_t s) {
  using C = MassCfg<DH, FP8, NARROW, FOLD>;
  CUtensorMap tk, tq;
  const uint64_t rows = static_cast<uint64_t>(pages->num_pages) * pages->heads * pages->page_size;
  if (!make_tmap_page_rows(&tk, pages->k, rows, DH, FP8 ? 1 : 2, pages->page_size) ||
      !make_tmap_query_rows(&tq, g.q, g.q_rows, g.Hq, DH, g.q_stride, g.group, g.tokens))
    return DLLM_ERR_CUDA;
  g.item_keys = C::kItemKeys;
  g.k_stages = C::stages(g.columns);
  g.off_q = C::kOffK + g.k_stages * C::kStage;
  g.q_bytes = C::chunk_bytes(g.columns);
  const int smem = g.off_q + C::kQSt * g.q_bytes + 1024;
  auto kern = mass_kernel<DH, FP8, NARROW, FOLD>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kMost + 1024);
  const long long items = static_cast<long long>(g.B) * pages->heads * ((g.max_kv + C::kItemKeys - 1) / C::kItemKeys);
  const int ctas = items < sm_budget() ? static_cast<int>(items) : sm_budget();
  if (e == cudaSuccess) e = launch_pdl(kern, dim3(ctas), dim3(C::kThreads), smem, s, tk, tq, g);
  return e == cudaSuccess ? launch_status() : cuda_error(e);
}

template <int DH>
dllm_status launch_mass(const dllm_kv_pages *pages, float scale, MassArgs &g, cudaStream_t s) {
  const bool fp8 = pages->type == DLLM_KV_E4M3;
  // e4m3 pages and few rows: codes as they are. 16 requests, 9 to 12 thousand
  // keys, 8 x 4 heads: 4 rows a head 39 us, converted 68; 64 rows 47 and 73. (The
  // most rows that eight tiles' scores leave room for. Two keys a thread over bf16
  // pages: 61 to 63 us, one 60 to 61.)
  if (fp8 && g.columns <= kNarrow) return launch_mass<DH, true, true, false>(pages, g, s);
  // lse / scale has to be a number
  const float size = fabsf(scale);
  if (size >= 0x1p-40f && size <= 0x1p40f) {
    g.lse_scale = -1.f / scale;
    return fp8 ? launch_mass<DH, true, false, true>(pages, g, s) : launch_mass<DH, false, false, true>(pages, g, s);
  }
  return fp8 ? launch_mass<DH, true, false, false>(pages, g, s) : launch_mass<DH, false, false, false>(pages, g, s);
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
  if (!aligned16(a->q) || !aligned16(a->mass) || a->q_stride < static_cast<long long>(a->Hq) * pages->dh || a->q_stride % 8) return DLLM_ERR_INVALID_ARG;
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
  g.tokens = kChunkRows / g.group < a->max_q ? kChunkRows / g.group : a->max_q;
  g.columns = (g.tokens * g.group + 15) / 16 * 16;
  cudaError_t e = cudaGetSymbolAddress(reinterpret_cast<void **>(&g.status), g_status_mass);
  if (e != cudaSuccess) return cuda_error(e);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return pages->dh == 64 ? launch_mass<64>(pages, a->scale, g, s) : launch_mass<128>(pages, a->scale, g, s);
}
