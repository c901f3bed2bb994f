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
// its thread; lse and the bound of every query row come from shared memory.
//
// An item is two key tiles (256 rows) of one request and cached head, one for
// each of two epilogue warpgroups; query rows pass by in chunks of up to 128,
// each read once for both tiles. The items form one line, each as long as its
// chunks and what every item costs, cut into equal stretches, one per CTA.
//
// Warp roles:
//   warp 0      K tiles by TMA, one box per page
//   warp 1      MMAs
//   warp 2      query rows by TMA, lse and bounds of each chunk's rows
//   warp 3      walks the CTA's items ahead of the others
//   warps 4..11 two groups, one key per thread: exponentials and sums
//   last four   (e4m3 pages) K codes to bf16, exactly; the scale is a factor of
//               the scores
#include <math.h>

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
};

constexpr int kItemKeys = 2 * kTile;
constexpr int kChunkRows = 128;
constexpr int kAhead = 4;        // items prepared, the current one included
constexpr int kInfo = 4;         // chunks whose rows' numbers are prepared
constexpr int kItemLength = 2;   // what an item costs beside its chunks, in chunks

template <int DH, bool FP8>
struct MassCfg {
  static constexpr int kRaw = kTile * DH * (FP8 ? 1 : 2);      // a K tile as it is loaded
  static constexpr int kTileBytes = kTile * DH * 2;            // ... as the MMAs read it
  static constexpr int kGroup8 = 8 * DH * 2;
  static constexpr int kQ = kChunkRows * DH * 2;
  static constexpr int kQSt = 2;
  static constexpr int kCSt = FP8 ? 2 : 0;                     // converted tiles
  static constexpr int kKSt = FP8 ? (DH == 128 ? 5 : 8) : (DH == 128 ? 4 : 8);
  static constexpr int kOffConv = kKSt * kRaw;
  static constexpr int kOffQ = kOffConv + kCSt * kTileBytes;
  static constexpr int kOffMisc = kOffQ + kQSt * kQ;
  static constexpr int kMisc = 8192;
  static constexpr int kBytes = kOffMisc + kMisc + 1024;
  static constexpr int kThreads = 32 * (12 + (FP8 ? 4 : 0));
  static_assert(kBytes <= 232448 && kOffConv % 1024 == 0, "shared memory");
};

struct MassPiece {
  Extent x;
  int i, h, key0;          // request, head, first key
  int first, chunks;       // chunks [first, chunks) hold rows that see a key of the item
  int tiles;               // key tiles (1 or 2)
  int more;
};

struct alignas(16) Numbers {   // of a chunk's query rows
  float neg_lse[kChunkRows];   // - lse in log2 units
  int hi[kChunkRows];          // keys before it are seen; 0: not a row, or one that saw nothing
  int every;                   // keys before it are seen by all of them
};

struct MassStart {
  long long left;          // length of the CTA's stretch from its first item on
  int i, item;
};

__device__ __forceinline__ void mass_request(const MassArgs &a, const Extent &x, int &items, int &length) {
  items = x.W > 0 ? (x.L + kItemKeys - 1) / kItemKeys * a.c.heads : 0;
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
  long long total = 0, before = up - mine;
  for (int w = 0; w < nt / 32; ++w) {
    if (w < warp) before += s_sum[w];
    total += s_sum[w];
  }
  const long long per = quotient(total + gridDim.x - 1, gridDim.x), begin = per * blockIdx.x;
  if (begin >= before && begin < before + mine) {
    long long at = before;
    for (int i = i0; i < i1; ++i) {
      mass_request(a, paged_extent(a, i, false), items, length);
      const long long m = static_cast<long long>(items) * length;
      if (begin < at + m) {
        const int item = static_cast<int>(quotient(begin - at + length - 1, length));
        s_start->i = i;
        s_start->item = item;
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

template <int DH, bool FP8>
__global__ void __launch_bounds__(MassCfg<DH, FP8>::kThreads, 1)
mass_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ MassArgs a) {
  using C = MassCfg<DH, FP8>;
  constexpr int kKSt = C::kKSt, kQSt = C::kQSt, kCSt = C::kCSt;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *misc = smem + C::kOffMisc;
  Numbers *numbers = reinterpret_cast<Numbers *>(misc);                      // [kInfo]
  MassPiece *pieces = reinterpret_cast<MassPiece *>(numbers + kInfo);        // [kAhead]
  uint64_t *k_full = reinterpret_cast<uint64_t *>(misc + 5120);              // [kKSt]
  uint64_t *k_empty = k_full + kKSt;
  uint64_t *c_full = k_empty + kKSt;       // [kCSt] converted
  uint64_t *c_empty = c_full + kCSt;
  uint64_t *q_full = c_empty + kCSt;       // [kQSt]
  uint64_t *q_empty = q_full + kQSt;
  uint64_t *n_full = q_empty + kQSt;       // [kInfo]
  uint64_t *n_empty = n_full + kInfo;
  uint64_t *s_full = n_empty + kInfo;      // [group][2]
  uint64_t *s_empty = s_full + 4;
  uint64_t *piece_full = s_empty + 4;      // [kAhead]
  uint64_t *piece_empty = piece_full + kAhead;
  long long *s_sum = reinterpret_cast<long long *>(piece_empty + kAhead);    // [16]
  MassStart *start = reinterpret_cast<MassStart *>(s_sum + 16);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(start + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  static_assert(kInfo * sizeof(Numbers) + kAhead * sizeof(MassPiece) <= 5120, "tables");
  static_assert(5120 + (2 * kKSt + 2 * kCSt + 2 * kQSt + 2 * kInfo + 8 + 2 * kAhead + 16) * 8 + sizeof(MassStart) + 8 <= C::kMisc,
                "barriers");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kKSt; ++s) { mbar_init(&k_full[s], 1); mbar_init(&k_empty[s], FP8 ? 4 : 1); }
    for (int s = 0; s < kCSt; ++s) { mbar_init(&c_full[s], 4); mbar_init(&c_empty[s], 1); }
    for (int s = 0; s < kQSt; ++s) { mbar_init(&q_full[s], 1); mbar_init(&q_empty[s], 1); }
    for (int s = 0; s < kInfo; ++s) { mbar_init(&n_full[s], 1); mbar_init(&n_empty[s], 8); }
    for (int s = 0; s < 4; ++s) { mbar_init(&s_full[s], 1); mbar_init(&s_empty[s], 4); }
    for (int s = 0; s < kAhead; ++s) {
      mbar_init(&piece_full[s], 1);
      mbar_init(&piece_empty[s], 3 + 8 + (FP8 ? 4 : 0));   // the warps that read it
    }
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_q);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
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
    // --------------------------------------------------------------- K tiles
    const int per_tile = kTile >> a.c.page_shift, page_rows = 1 << a.c.page_shift;
    const int none = static_cast<int>((static_cast<long long>(a.c.num_pages) * a.c.heads << a.c.page_shift) / 8);
    bool ok = true;
    uint32_t n = 0;
    for (uint32_t seg = 0; ok; ++seg) {
      const MassPiece *p = piece(seg);
      if (!p) break;
      const int32_t *row = a.c.table + static_cast<size_t>(p->i) * a.c.max_pages;
      const int tiles = p->first < p->chunks ? p->tiles : 0;
      for (int j = 0; ok && j < tiles; ++j, ++n) {
        const uint32_t st = n % kKSt;
        int g = none;              // 8-row group of this lane's page; what there is none of reads as zeros
        const int u = p->key0 + j * kTile + lane * page_rows;
        if (lane < per_tile && u < p->x.L) {
          const int page = __ldg(row + (u >> a.c.page_shift));
          if (page >= 0 && page < a.c.num_pages) g = ((page * a.c.heads + p->h) << a.c.page_shift) / 8;
        }
        if (n >= kKSt) ok = warp_wait(&k_empty[st], (n / kKSt - 1) & 1, abort_flag);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&k_full[st], C::kRaw);
        __syncwarp();
        if (lane < per_tile) tma_load_4d(smem + st * C::kRaw + lane * page_rows * (C::kRaw / kTile), &tm_k, &k_full[st], g);
      }
      piece_done(seg);
    }
    // after an abort the loads in flight land before the CTA's memory is given up
    if (!ok || *abort_flag)
      if (lane < kKSt && lane < n) mbar_drain(&k_full[lane], ((n - 1 - lane) / kKSt) & 1);
    __syncwarp();
  } else if (warp == 1) {
    // --------------------------------------------------------------- MMAs
    if (elect_one()) {
      const uint32_t idesc = idesc_bf16(128, a.columns, 0, 0);
      bool ok = true;
      uint32_t n = 0, nq = 0, ns[2] = {0, 0};     // key tiles, chunks, units of the groups before this item
      for (uint32_t seg = 0; ok; ++seg) {
        const uint32_t pi = seg % kAhead;
        ok = mbar_wait(&piece_full[pi], (seg / kAhead) & 1, abort_flag);
        if (!ok || !pieces[pi].more) break;
        const int chunks = pieces[pi].chunks - pieces[pi].first, tiles = pieces[pi].tiles;
        for (int c = 0; ok && c < chunks; ++c, ++nq) {
          const uint32_t qs = nq % kQSt;
          ok = mbar_wait(&q_full[qs], (nq / kQSt) & 1, abort_flag);
          const uint64_t dq = sw128_desc(smem_u32(smem + C::kOffQ + qs * C::kQ), 16, 1024);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (j >= tiles || !ok) break;
            const uint32_t t = n + j, b = ns[j] & 1, st = FP8 ? t % (kCSt + !FP8) : t % kKSt;
            if (c == 0) ok = FP8 ? mbar_wait(&c_full[st], (t / (kCSt + !FP8)) & 1, abort_flag)
                                 : mbar_wait(&k_full[st], (t / kKSt) & 1, abort_flag);
            if (ok && ns[j] >= 2) ok = mbar_wait(&s_empty[j * 2 + b], (ns[j] / 2 - 1) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const uint64_t dk = sw128_desc(smem_u32(FP8 ? smem + C::kOffConv + st * C::kTileBytes : smem + st * C::kRaw), 16, C::kGroup8);
#pragma unroll
            for (int kk = 0; kk < DH / 16; ++kk)
              umma_bf16(tmem + (j * 2 + b) * 128, dk + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4),
                        dq + (((kk >> 2) * (kChunkRows * 128) + (kk & 3) * 32) >> 4), idesc, kk > 0);
            umma_commit(&s_full[j * 2 + b]);
            ++ns[j];
            if (c + 1 == chunks) umma_commit(FP8 ? &c_empty[st] : &k_empty[st]);
          }
          if (ok) umma_commit(&q_empty[qs]);
        }
        if (chunks > 0) n += tiles;
        mbar_arrive(&piece_empty[pi]);
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // --------------------------------------------------------------- query rows and their numbers
    const uint32_t bytes = static_cast<uint32_t>(a.tokens * a.group) * DH * 2;
    bool ok = true;
    uint32_t nq = 0, asked = 0;
    for (uint32_t seg = 0; ok; ++seg) {
      const MassPiece *p = piece(seg);
      if (!p) break;
      const Extent x = p->x;
      const int chunks = p->chunks, h = p->h;
      for (int c = p->first; ok && c < chunks; ++c, ++nq) {
        const uint32_t qs = nq % kQSt, in = nq % kInfo;
        if (nq >= kQSt) ok = warp_wait(&q_empty[qs], (nq / kQSt - 1) & 1, abort_flag);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&q_full[qs], bytes);
#pragma unroll
          for (int d = 0; d < DH / 64; ++d)
            tma_load_rows(smem + C::kOffQ + qs * C::kQ + d * (kChunkRows * 128), &tm_q, &q_full[qs], d * 64, h * a.group,
                          x.q0 + c * a.tokens);
        }
        ++asked;
        __syncwarp();
        float lse[kChunkRows / 32];
        int hi[kChunkRows / 32], every = 0x7fffffff;
#pragma unroll
        for (int e = 0; e < kChunkRows / 32; ++e) {
          const int r = e * 32 + lane, t = c * a.tokens + r / a.group;
          hi[e] = 0;
          lse[e] = 0.f;
          if (r < a.tokens * a.group && t < x.W) {
            int lo;
            lse[e] = a.lse[static_cast<size_t>(x.q0 + t) * a.Hq + h * a.group + r % a.group];
            visible(a, x.pos, t, x.L, lo, hi[e]);
          }
        }
#pragma unroll
        for (int e = 0; e < kChunkRows / 32; ++e) {
          if (lse[e] == -INFINITY) hi[e] = 0;
          if (e * 32 + lane < a.columns) every = min(every, hi[e]);
        }
        every = __reduce_min_sync(0xffffffffu, every);
        if (nq >= kInfo) ok = warp_wait(&n_empty[in], (nq / kInfo - 1) & 1, abort_flag);
        if (!ok) break;
        Numbers &s = numbers[in];
#pragma unroll
        for (int e = 0; e < kChunkRows / 32; ++e) {
          s.neg_lse[e * 32 + lane] = lse[e] * -1.4426950408889634f;
          s.hi[e * 32 + lane] = hi[e];
        }
        if (lane == 0) s.every = every;
        __syncwarp();
        if (lane == 0) mbar_arrive(&n_full[in]);
      }
      piece_done(seg);
    }
    if (!ok || *abort_flag)
      if (lane < kQSt && lane < asked) mbar_drain(&q_full[lane], ((asked - 1 - lane) / kQSt) & 1);
    __syncwarp();
  } else if (warp == 3) {
    // --------------------------------------------------------------- items
    long long left = start->left;
    int i = start->i, item = start->item, items = 0, length = 1;
    Extent x{};
    if (left > 0) {
      x = paged_extent(a, i, false);
      mass_request(a, x, items, length);
    }
    bool more = true;
    for (uint32_t seg = 0; more; ++seg) {
      const uint32_t pi = seg % kAhead;
      if (seg >= kAhead && !warp_wait(&piece_empty[pi], (seg / kAhead - 1) & 1, abort_flag)) break;
      more = left > 0;
      while (more && item >= items) {
        item = 0;
        if (++i >= a.B) { more = false; break; }
        x = paged_extent(a, i, false);
        mass_request(a, x, items, length);
      }
      if (lane == 0) {
        MassPiece &p = pieces[pi];
        p.more = more;
        if (more) {
          const int per_head = items / a.c.heads, h = item / per_head;
          const int key0 = (item - h * per_head) * kItemKeys;
          p.x = x;
          p.i = i;
          p.h = h;
          p.key0 = key0;
          p.tiles = x.L - key0 > kTile ? 2 : 1;
          p.chunks = length - kItemLength;
          // the first row that sees the item's first key
          long long t = a.right < 0 ? 0 : static_cast<long long>(key0) - x.pos - a.right;
          t = max(t, 0ll);
          p.first = t < x.W ? static_cast<int>(t) / a.tokens : p.chunks;
        }
        mbar_arrive(&piece_full[pi]);
      }
      __syncwarp();
      left -= length;
      ++item;
    }
  } else if (FP8 && warp >= 12) {
    // --------------------------------------------------------------- K codes -> bf16
    if constexpr (FP8) {
      const int key = (warp - 12) * 32 + lane;
      bool ok = true;
      uint32_t n = 0;
      for (uint32_t seg = 0; ok; ++seg) {
        const MassPiece *p = piece(seg);
        if (!p) break;
        const int tiles = p->first < p->chunks ? p->tiles : 0;
        for (int j = 0; ok && j < tiles; ++j, ++n) {
          const uint32_t st = n % kKSt, cs = n % kCSt;
          ok = warp_wait(&k_full[st], (n / kKSt) & 1, abort_flag);
          if (ok && n >= kCSt) ok = warp_wait(&c_empty[cs], (n / kCSt - 1) & 1, abort_flag);
          if (!ok) break;
          const uint8_t *src = smem + st * C::kRaw + key * DH;
          uint8_t *dst = smem + C::kOffConv + cs * C::kTileBytes + (key / 8) * C::kGroup8 + (key % 8) * 128;
#pragma unroll
          for (int c = 0; c < DH / 16; ++c) {   // under the load's swizzle (rows of 128 or 64 bytes)
            const uint4 w = *reinterpret_cast<const uint4 *>(src + (DH == 128 ? c ^ (key & 7) : c ^ ((key >> 1) & 3)) * 16);
            const uint32_t in[4] = {w.x, w.y, w.z, w.w};
            uint32_t out[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint2 v = e4m3x4_to_bf16_0213(in[e]);
              out[2 * e] = __byte_perm(v.x, v.y, 0x5410);
              out[2 * e + 1] = __byte_perm(v.x, v.y, 0x7632);
            }
            uint8_t *d = dst + (c / 4) * 1024;   // 64 columns: eight 16-byte pieces
            *reinterpret_cast<uint4 *>(d + (((2 * c) & 7) ^ (key & 7)) * 16) = make_uint4(out[0], out[1], out[2], out[3]);
            *reinterpret_cast<uint4 *>(d + (((2 * c + 1) & 7) ^ (key & 7)) * 16) = make_uint4(out[4], out[5], out[6], out[7]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&c_full[cs]);
            mbar_arrive(&k_empty[st]);
          }
        }
        piece_done(seg);
      }
    }
  } else {
    // --------------------------------------------------------------- exponentials and sums
    const int g = (warp - 4) >> 2, quarter = warp & 3;
    const int key = quarter * 32 + lane;
    const uint32_t t_s = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + g * 256;
    bool ok = true;
    uint32_t nq = 0, ns = 0;
    for (uint32_t seg = 0; ok; ++seg) {
      const MassPiece *p = piece(seg);
      if (!p) break;
      const int u = p->key0 + g * kTile + key, chunks = p->chunks - p->first;
      const bool there = g < p->tiles;            // this group's tile
      float c = a.scale_log2, old = 0.f;
      int row = -1;
      size_t at = 0;
      if (u < p->x.L) {
        row = page_row(a.c, p->i, u);
        if (row < 0) {
          atomicOr(a.status, DLLM_DEV_PAGE);
        } else {
          at = row + (static_cast<size_t>(p->h) << a.c.page_shift);
          if (!(a.fresh && u >= a.fresh[p->i])) old = a.mass[at] * a.decay;
          if constexpr (FP8) c *= scale_of(a.c.k_scale[at]);
        }
      }
      float sum = 0.f;
      for (int k = 0; ok && k < chunks; ++k, ++nq) {
        const uint32_t in = nq % kInfo;
        ok = warp_wait(&n_full[in], (nq / kInfo) & 1, abort_flag);
        if (ok && there) {
          const uint32_t b = ns & 1;
          ok = warp_wait(&s_full[g * 2 + b], (ns / 2) & 1, abort_flag);
          if (ok) {
            tc_fence_after();
            const Numbers &s = numbers[in];
            const bool masked = p->key0 + (g + 1) * kTile > s.every;
            float2 acc = make_float2(0.f, 0.f);
            for (int c0 = 0; c0 < a.columns; c0 += 16) {
              uint32_t x[16];
              tmem_ld16(t_s + b * 128 + c0, x);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; e += 4) {
                const float4 z = *reinterpret_cast<const float4 *>(&s.neg_lse[c0 + e]);
                float2 y0 = __ffma2_rn(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), make_float2(c, c), make_float2(z.x, z.y));
                float2 y1 = __ffma2_rn(make_float2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), make_float2(c, c), make_float2(z.z, z.w));
                if (masked) {
                  const int4 hi = *reinterpret_cast<const int4 *>(&s.hi[c0 + e]);
                  if (u >= hi.x) y0.x = -INFINITY;
                  if (u >= hi.y) y0.y = -INFINITY;
                  if (u >= hi.z) y1.x = -INFINITY;
                  if (u >= hi.w) y1.y = -INFINITY;
                }
                acc = __fadd2_rn(acc, make_float2(ex2_approx(y0.x), ex2_approx(y0.y)));
                acc = __fadd2_rn(acc, make_float2(ex2_approx(y1.x), ex2_approx(y1.y)));
              }
            }
            sum += acc.x + acc.y;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[g * 2 + b]);
            ++ns;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&n_empty[in]);
      }
      if (ok && row >= 0) a.mass[at] = old + sum;
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

template <int DH, bool FP8>
dllm_status launch_mass(const dllm_kv_pages *pages, MassArgs &g, cudaStream_t s) {
  using C = MassCfg<DH, FP8>;
  CUtensorMap tk, tq;
  const uint64_t rows = static_cast<uint64_t>(pages->num_pages) * pages->heads * pages->page_size;
  if (!make_tmap_page_rows(&tk, pages->k, rows, DH, FP8 ? 1 : 2, pages->page_size) ||
      !make_tmap_query_rows(&tq, g.q, g.q_rows, g.Hq, DH, g.q_stride, g.group, g.tokens))
    return DLLM_ERR_CUDA;
  auto kern = mass_kernel<DH, FP8>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  const long long items = static_cast<long long>(g.B) * pages->heads * ((g.max_kv + kItemKeys - 1) / kItemKeys);
  const int ctas = items < sm_budget() ? static_cast<int>(items) : sm_budget();
  if (e == cudaSuccess) e = launch_pdl(kern, dim3(ctas), dim3(C::kThreads), C::kBytes, s, tk, tq, g);
  return e == cudaSuccess ? launch_status() : cuda_error(e);
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
  if (!aligned16(a->q) || a->q_stride < static_cast<long long>(a->Hq) * pages->dh || a->q_stride % 8) return DLLM_ERR_INVALID_ARG;
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
  const bool fp8 = pages->type == DLLM_KV_E4M3;
  if (pages->dh == 64) return fp8 ? launch_mass<64, true>(pages, g, s) : launch_mass<64, false>(pages, g, s);
  return fp8 ? launch_mass<128, true>(pages, g, s) : launch_mass<128, false>(pages, g, s);
}
