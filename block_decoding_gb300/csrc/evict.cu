// Moving rows within the paged cache, and choosing the rows that stay when a
// cache is cut down to a budget.
//
// Choosing is bound by latency (a head's weights are some 40 KB): 9.4 us for
// 8242 weights, of which 3 until they are in shared memory, 4 for three passes
// with their scans, 2.5 for the positions in their order. Moving is bound by
// memory: 262 k rows of 128 bytes, a third of those read past, to other pages in
// 30 us, 4.5 TB/s, beside as many sectors for scales and weights of single rows;
// 192 k rows in place, 64 lists of 2 to 4 thousand, in 27 us. One request's 701
// rows cut down to 512 in place: 8.9 us, both in one launch.
#include "pages.cuh"
#include "umma_pages.cuh"

namespace dllm {

DLLM_DEFINE_STATUS(evict)

namespace {

// All threads of the cluster are here; of what they have written nothing is known.
// Reads before it and other CTAs' writes of the same rows behind it are in order all
// the same: by then each value that was read, scales and weights by plain loads
// too, is in the reader's shared memory or registers, so its load is over.
// (As release and acquire: lists per head in place 28.9 us for 26.8, one request's 9.2
// for 8.8.)
__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// ---------------------------------------------------------------------------
// selection
// ---------------------------------------------------------------------------
struct SelectArgs {
  KvPages c;
  const float *mass;
  const int32_t *kv_len;
  int32_t *keep;               // [B][heads][budget]
  int budget, max_kv, sinks, recent;
  unsigned int *status;
  // rows that the same kernel moves, in place
  int ctas, share;             // CTAs of a list, rows of a CTA
  int32_t *new_len;            // [B]
  float *move_mass;            // null: stays
};

constexpr int kMaxSelWarps = 32;
constexpr int kBins = 2048;      // 11 bits at a time
constexpr int kBatch = 8;        // loads of a thread on their way
constexpr int kCached = 49152;   // weights that shared memory holds (192 KB)
constexpr int kSelectBytes = 4 * kCached + 16384;      // dynamic shared memory, at most (10 KB beside it)

// Order of weights as unsigned numbers: -0 is 0, NaN is above everything.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Chosen rows of ROW bytes on their way to their places, through shared memory.
__host__ __device__ constexpr long long few_bytes(int row, long long budget) {
  return row > 0 ? (budget * (2 * row + 14) + 15) / 16 * 16 : 0;
}

template <int ROW>
struct Few {
  static constexpr int kChunks = ROW / 16;
  uint4 *k, *v;                // [share][kChunks]
  int *from, *dest;            // [share]: positions that stay, then cache rows for head 0; -1: nothing moves
  float *mass;
  uint8_t *k_scale, *v_scale;
  __device__ Few(void *smem, int share) {
    k = reinterpret_cast<uint4 *>(smem);
    v = k + share * kChunks;
    from = reinterpret_cast<int *>(v + share * kChunks);
    dest = from + share;
    mass = reinterpret_cast<float *>(dest + share);
    k_scale = reinterpret_cast<uint8_t *>(mass + share);
    v_scale = k_scale + share;
  }

  // The kept rows rank, rank + ctas, .. of k, in `from`.
  __device__ __forceinline__ void move(const SelectArgs &a, int i, int h, int rank, int kept) const {
    const int tid = threadIdx.x, nt = blockDim.x, count = (kept - rank + a.ctas - 1) / a.ctas;
    const size_t head = static_cast<size_t>(h) << a.c.page_shift;
    __syncthreads();
    for (int j = tid; j < count; j += nt) {
      const int u = from[j], at = j * a.ctas + rank;
      int f = -1, d = -1;
      if (u != at) {
        f = page_row(a.c, i, u);
        d = page_row(a.c, i, at);
        if (f < 0 || d < 0) {
          atomicOr(a.status, DLLM_DEV_PAGE);
          f = d = -1;
        }
      }
      from[j] = f;
      dest[j] = d;
      if (f < 0) continue;
      if (a.c.k_scale) { k_scale[j] = a.c.k_scale[f + head]; v_scale[j] = a.c.v_scale[f + head]; }
      if (a.move_mass) mass[j] = a.move_mass[f + head];
    }
    __syncthreads();
    for (int p = tid; p < count * kChunks; p += nt) {
      const int f = from[p / kChunks];
      if (f < 0) continue;
      copy16(k + p, a.c.k + (f + head) * ROW + p % kChunks * 16, true);
      copy16(v + p, a.c.v + (f + head) * ROW + p % kChunks * 16, true);
    }
    copies_wait();
    cluster_barrier();
    for (int p = tid; p < count * kChunks; p += nt) {
      const int d = dest[p / kChunks];
      if (d < 0) continue;
      *reinterpret_cast<uint4 *>(a.c.k + (d + head) * ROW + p % kChunks * 16) = k[p];
      *reinterpret_cast<uint4 *>(a.c.v + (d + head) * ROW + p % kChunks * 16) = v[p];
    }
    for (int j = tid; j < count; j += nt) {
      const int d = dest[j];
      if (d < 0) continue;
      if (a.c.k_scale) { a.c.k_scale[d + head] = k_scale[j]; a.c.v_scale[d + head] = v_scale[j]; }
      if (a.move_mass) a.move_mass[d + head] = mass[j];
    }
  }
};

// One CTA per cached head and request. The weights that are chosen from are
// read once into shared memory (CACHED; more than fit are read again by every
// pass, from L2). Radix selection finds the least weight that stays, 11 bits at a
// time: a histogram, and the bin in which the count from above passes the number
// of rows that stay, by one scan over all bins. Then every warp counts its own
// run of positions and, behind the sum over the warps before it, writes those
// that stay in their order.
//
// ROW > 0: a.ctas CTAs of a cluster, which all choose the same rows, then move
// them, of ROW bytes, in place, in turn: all through shared memory, every one
// read before any is written (a cluster barrier between the two).
template <bool CACHED, int ROW>
__global__ void __launch_bounds__(1024) select_kernel(const __grid_constant__ SelectArgs a) {
  extern __shared__ uint4 smem_select[];         // ROW > 0: what moves; CACHED: keys [max_kv]
  uint32_t *const s_key = reinterpret_cast<uint32_t *>(reinterpret_cast<uint8_t *>(smem_select) + few_bytes(ROW, a.share));
  __shared__ uint32_t s_hist[kBins];
  __shared__ int s_sum[kMaxSelWarps], s_tie[kMaxSelWarps];
  __shared__ uint32_t s_bin;
  __shared__ int s_left, s_of_bin;
  pdl_trigger();
  pdl_wait();
  const int rank = ROW > 0 ? static_cast<int>(blockIdx.x) % a.ctas : 0, h = ROW > 0 ? static_cast<int>(blockIdx.x) / a.ctas : blockIdx.x;
  const int i = blockIdx.y, tid = threadIdx.x, nt = blockDim.x, warp = tid / 32, lane = tid % 32, warps = nt / 32;
  int n = a.kv_len[i];
  if (n < 0 || n > a.max_kv) {
    if (tid + blockIdx.x == 0) atomicOr(a.status, DLLM_DEV_OFFSETS);
    n = min(max(n, 0), a.max_kv);
  }
  int32_t *keep = a.keep + (static_cast<size_t>(i) * a.c.heads + h) * a.budget;
  const int k = min(n, a.budget);
  if (rank == 0) {
    for (int j = tid + k; j < a.budget; j += nt) keep[j] = -1;
    if constexpr (ROW > 0) {
      if (h == 0 && tid == 0) a.new_len[i] = k;
    }
  }
  if (n <= a.budget) {
    if (rank == 0)
      for (int j = tid; j < k; j += nt) keep[j] = j;
    if constexpr (ROW > 0) cluster_barrier();    // (every CTA comes to one)
    return;
  }
  const int32_t *table = a.c.table + static_cast<size_t>(i) * a.c.max_pages;
  const int s = a.sinks, e = n - a.recent;       // [s, e) is chosen from: at least n - budget rows
  // The weights of positions u, u + nt, .. below e: pages first, so that the
  // loads of a batch wait together.
  auto fetch = [&](int u, uint32_t (&x)[kBatch]) {
    int page[kBatch];
    float w[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) page[q] = u + q * nt < e ? __ldg(table + ((u + q * nt) >> a.c.page_shift)) : 0;
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const bool held = u + q * nt < e, bad = page[q] < 0 || page[q] >= a.c.num_pages;
      w[q] = 0.f;
      if (held && !bad)
        w[q] = a.mass[(static_cast<size_t>(page[q] * a.c.heads + h) << a.c.page_shift) + ((u + q * nt) & ((1 << a.c.page_shift) - 1))];
      if (held && bad) {       // (without a weight: the least of all)
        atomicOr(a.status, DLLM_DEV_PAGE);
        w[q] = -INFINITY;
      }
    }
#pragma unroll
    for (int q = 0; q < kBatch; ++q) x[q] = order_of(w[q]);
  };
  auto key = [&](int u) {                        // (of [s, e))
    if (CACHED) return s_key[u];
    const int row = page_row(a.c, i, u);
    return order_of(row < 0 ? -INFINITY : a.mass[row + (static_cast<size_t>(h) << a.c.page_shift)]);
  };
  int left = k - s - a.recent;                   // how many of them stay
  uint32_t least = 0;                            // the bits of the least that stays, found so far
  int shift = 32;                                // ... from this bit on
  for (int bits = 0; left > 0 && shift > 0; ) {
    const bool filled = shift < 32;              // the weights are in shared memory
    bits = shift == 32 || shift == 21 ? 11 : 10;
    for (int b = tid; b < kBins; b += nt) s_hist[b] = 0;
    __syncthreads();
    const int low = shift - bits;
    const uint32_t mask = (1u << bits) - 1;
    if (CACHED && filled) {
      for (int u = s + tid; u < e; u += nt) {
        const uint32_t x = s_key[u];
        if (x >> shift == least >> shift) atomicAdd(&s_hist[x >> low & mask], 1u);
      }
    } else {
      for (int u0 = s + tid; u0 < e; u0 += kBatch * nt) {
        uint32_t x[kBatch];
        fetch(u0, x);
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          const int u = u0 + q * nt;
          if (u >= e) break;
          if (CACHED) s_key[u] = x[q];
          if (!filled || x[q] >> shift == least >> shift) atomicAdd(&s_hist[x[q] >> low & mask], 1u);
        }
      }
    }
    __syncthreads();
    // counts from the highest bin down: thread t has kBins / nt bins, the highest first
    const int per = kBins / nt, top = kBins - 1 - tid * per;
    int mine = 0;
    for (int b = 0; b < per; ++b) mine += s_hist[top - b];
    int up = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += y;
    }
    if (lane == 31) s_sum[warp] = up;
    __syncthreads();
    int before = up - mine;
    {
      const int y = lane < warp ? s_sum[lane] : 0;
      before += __reduce_add_sync(0xffffffffu, y);
    }
    if (before < left && left <= before + mine) {     // one thread
      int b = 0;
      while (before + static_cast<int>(s_hist[top - b]) < left) before += s_hist[top - b++];
      s_bin = top - b;
      s_left = left - before;
      s_of_bin = s_hist[top - b];
    }
    __syncthreads();
    least |= s_bin << low;
    left = s_left;
    shift = low;
    if (s_of_bin == left) break;                 // all of the bin stay
  }
  // Rows whose bits from `shift` on are those of `least` are ties: the first
  // `left` of them stay, and all above. (With left <= 0 no row of [s, e) stays,
  // and `shift` may be 32.) A warp has a run of positions, 32 x 32 at a time:
  // lane l keeps the votes of the l-th 32.
  const int run = ((n + warps - 1) / warps + 31) / 32 * 32, u0 = warp * run, u1 = min(n, u0 + run);
  const bool some = left > 0;
  auto votes = [&](int from, uint32_t &in_votes, uint32_t &tie_votes) {
    in_votes = tie_votes = 0;
    const int rounds = min((u1 - from + 31) / 32, 32);
    for (int l = 0; l < rounds; ++l) {
      const int u = from + l * 32 + lane;
      bool in = false, tie = false;
      if (u < u1) {
        if (u < s || u >= e) {
          in = true;
        } else if (some) {
          const uint32_t x = key(u) >> shift, y = least >> shift;
          in = x > y;
          tie = x == y;
        }
      }
      const uint32_t iv = __ballot_sync(0xffffffffu, in), tv = __ballot_sync(0xffffffffu, tie);
      if (lane == l) {
        in_votes = iv;
        tie_votes = tv;
      }
    }
  };
  uint32_t in_votes = 0, tie_votes = 0;
  int count = 0, ties = 0;
  for (int from = u0; from < u1; from += 1024) {
    votes(from, in_votes, tie_votes);
    count += __popc(in_votes);
    ties += __popc(tie_votes);
  }
  count = __reduce_add_sync(0xffffffffu, count);
  ties = __reduce_add_sync(0xffffffffu, ties);
  __syncthreads();                               // s_sum is read by all
  if (lane == 0) {
    s_sum[warp] = count;
    s_tie[warp] = ties;
  }
  __syncthreads();
  // ties before this warp, and rows that stay before it
  const int c = lane < warp ? s_sum[lane] : 0, t = lane < warp ? s_tie[lane] : 0;
  int tie_at = __reduce_add_sync(0xffffffffu, t);
  int at = __reduce_add_sync(0xffffffffu, c) + min(tie_at, max(left, 0));
  auto before = [&](int x) {                     // sum over the lanes before this one
    int up = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += y;
    }
    return up - x;
  };
  for (int from = u0; from < u1; from += 1024) {
    if (run > 1024) votes(from, in_votes, tie_votes);      // (else they are the first pass's)
    // the lane's ties that stay: the lowest
    const int room = left - tie_at - before(__popc(tie_votes));
    uint32_t stay = tie_votes;
    while (__popc(stay) > max(room, 0)) stay ^= 0x80000000u >> __clz(stay);
    tie_at += __reduce_add_sync(0xffffffffu, __popc(tie_votes));
    stay |= in_votes;
    const int mine = at + before(__popc(stay));
    at += __reduce_add_sync(0xffffffffu, __popc(stay));
    const int rounds = min((u1 - from + 31) / 32, 32);
    for (int l = 0; l < rounds; ++l) {
      const uint32_t m = __shfl_sync(0xffffffffu, stay, l);
      const int to = __shfl_sync(0xffffffffu, mine, l) + __popc(m & ((1u << lane) - 1));
      if (m >> lane & 1) {
        if (rank == 0) keep[to] = from + l * 32 + lane;
        if constexpr (ROW > 0) {
          if (to % a.ctas == rank) Few<ROW>(smem_select, a.share).from[to / a.ctas] = from + l * 32 + lane;
        }
      }
    }
  }
  if constexpr (ROW > 0) Few<ROW>(smem_select, a.share).move(a, i, h, rank, k);
}

template <int ROW>
cudaError_t launch_select(const SelectArgs &g, int B, cudaStream_t s) {
  // (16 x 8 heads of 1000 rows and half of them kept: 256 threads 15.4 us, 1024 14.5; one request's 16 of 701: 9.6 and 10.2)
  const int threads = g.max_kv <= 768 ? 256 : 1024;
  if (g.max_kv > kCached) return launch_pdl(select_kernel<false, 0>, dim3(g.c.heads, B), dim3(threads), 0, s, g);
  const int smem = static_cast<int>(few_bytes(ROW, g.share)) + g.max_kv * 4;
  cudaError_t e = cudaFuncSetAttribute(select_kernel<true, ROW>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelectBytes);
  if (e != cudaSuccess) return e;
  if (ROW == 0) return launch_pdl(select_kernel<true, ROW>, dim3(g.c.heads, B), dim3(threads), smem, s, g);
  return launch_pdl_clusters(select_kernel<true, ROW>, g.ctas, dim3(g.c.heads * g.ctas, B), dim3(threads), smem, s, g);
}

// CTAs of a list that move the rows that they chose, or 0: short requests in place,
// where the rows fit into the CTAs' shared memory and there is an SM for each. (Both
// in one launch, and in two: one request's 16 heads of 701 rows, 512 kept, 8.9 and 9.7
// us, of 1400 10.8 and 12.0, of 4000 12.2 and 12.3, of 8000 13.3 and 13.0; eight
// requests of 1000 13.8 and 16.1, of 4000 16.2 and 18.3. To other pages 10.4 and
// 9.8, 14.3 and 14.5.)
int moving_ctas(const SelectArgs &g, int row, int B) {
  if (g.max_kv > 4096 || g.new_len == g.kv_len) return 0;      // (the other heads' CTAs read the length)
  // (16 clusters of 8 CTAs, an SM each, do not run at a time: 17.5 us for the 1000 rows' 10.8)
  const long long lists = static_cast<long long>(B) * g.c.heads;
  const int n = 12 * lists <= num_sms() ? 8 : 4 * lists <= num_sms() ? 4 : 2 * lists <= num_sms() ? 2 : 1;
  return n * lists <= num_sms() && few_bytes(row, (g.budget + n - 1) / n) + 4ll * g.max_kv <= kSelectBytes ? n : 0;
}

// ---------------------------------------------------------------------------
// moves
// ---------------------------------------------------------------------------
struct ShiftArgs {
  KvPages c;
  const int32_t *dst_table;
  int dst_pages;
  const int32_t *src;          // [B][src_heads][max_n]
  int src_heads, max_n;
  const int32_t *count, *first;   // [B]; first may be null: 0
  int most;                    // rows of a list, at most
  int32_t *new_len;            // null, or where the rows of a list are written: then more than `most` is no mistake
  float *mass;
  unsigned int *status;
};

constexpr int kMoveThreads = 256;

// Rows of a thread, 16 bytes of K and of V each: elsewhere all that a block
// has (four instead of two: 33 us for 30), in place what it has at a time. (192 k
// rows of 128 and of 256 bytes in place: two rows 29 and 64 us, four 27 and 56, six
// 33 and 67, eight 38 and 68; 262 k rows of 16 requests, with the choice: 40, 44,
// 57, 58. In registers, two at a time, the next two on their way: 35 and 75, 55.
// In shared memory, the next round on its way: one row 30 and 63, 41; two 29 and 63, 47.)
constexpr int kEachAway = 2, kEachInPlace = 4;
constexpr int kAtOnce = 4;       // ... whose places are looked up together

// Rows of ROW bytes that a CTA moves at a time.
constexpr int round_rows(int row_bytes, bool in_place) {
  return kMoveThreads * (in_place ? kEachInPlace : kEachAway) * 16 / row_bytes;
}

template <int ROW, bool IN_PLACE>
struct Mover {
  static constexpr int kChunks = ROW / 16, kStep = kMoveThreads / kChunks;   // rows of a CTA that lie side by side
  const ShiftArgs &a;
  const int i, n, first, c;      // request, rows of its list, first position, the thread's 16 bytes of a row
  const int32_t *src;
  const size_t head;

  // The cache rows, for head 0, that COUNT of the thread's entries from entry j
  // on, `step` apart, come from and go to: -1 where nothing moves.
  template <int COUNT>
  __device__ __forceinline__ void find(int j, int step, int (&from)[COUNT], int (&dest)[COUNT]) const {
    KvPages to = a.c;
    to.table = a.dst_table;
    to.max_pages = a.dst_pages;
#pragma unroll
    for (int q = 0; q < COUNT; ++q, j += step) {
      from[q] = dest[q] = -1;
      if (j >= n) continue;
      const int u = src[j];
      const long long d = static_cast<long long>(first) + j;
      bool bad = d < 0 || d > 0x7fffffffll;
      if constexpr (IN_PLACE) {
        bad |= u < d || (j > 0 && src[j - 1] >= u);
        if (u == d && !bad) continue;                 // stays
      }
      if (!bad) {
        from[q] = page_row(a.c, i, u);
        dest[q] = page_row(to, i, static_cast<int>(d));
      }
      if (from[q] < 0 || dest[q] < 0) {
        atomicOr(a.status, DLLM_DEV_PAGE);
        from[q] = dest[q] = -1;
      }
    }
  }
  __device__ __forceinline__ uint8_t *k_at(int row) const { return a.c.k + (row + head) * ROW + c * 16; }
  __device__ __forceinline__ uint8_t *v_at(int row) const { return a.c.v + (row + head) * ROW + c * 16; }
};

template <int ROW, bool IN_PLACE>
__device__ __forceinline__ Mover<ROW, IN_PLACE> mover(const ShiftArgs &a) {
  const int h = blockIdx.y, i = blockIdx.z;
  int n = a.count[i];
  const int first = a.first ? a.first[i] : 0;
  if (n < 0 || n > a.most) {
    if (threadIdx.x == 0 && !a.new_len) atomicOr(a.status, DLLM_DEV_OFFSETS);
    n = min(max(n, 0), a.most);
  }
  // (new_len may be count: whoever reads the number after this finds the same n)
  if (a.new_len && blockIdx.x + h + threadIdx.x == 0) a.new_len[i] = n;
  return Mover<ROW, IN_PLACE>{a, i, n, first, static_cast<int>(threadIdx.x) % (ROW / 16),
                              a.src + (static_cast<size_t>(i) * a.src_heads + (a.src_heads > 1 ? h : 0)) * a.max_n,
                              static_cast<size_t>(h) << a.c.page_shift};
}

// One request and cached head, K and V, to other pages: a CTA of the grid's x
// takes round_rows of the list.
template <int ROW>
__global__ void __launch_bounds__(kMoveThreads) shift_kernel(const __grid_constant__ ShiftArgs a) {
  pdl_trigger();
  pdl_wait();
  const Mover<ROW, false> m = mover<ROW, false>(a);
  const int j0 = blockIdx.x * round_rows(ROW, false);       // (n < 2^30)
  if (j0 >= m.n) return;
  int from[kEachAway], dest[kEachAway];
  uint4 k[kEachAway], v[kEachAway];
  float mass[kEachAway];
  uint8_t k_scale[kEachAway], v_scale[kEachAway];
  m.find(j0 + threadIdx.x / m.kChunks, m.kStep, from, dest);
#pragma unroll
  for (int q = 0; q < kEachAway; ++q) {
    if (from[q] < 0) continue;
    const size_t s = from[q] + m.head;
    k[q] = *reinterpret_cast<const uint4 *>(m.k_at(from[q]));
    v[q] = *reinterpret_cast<const uint4 *>(m.v_at(from[q]));
    if (m.c == 0) {
      if (a.c.k_scale) { k_scale[q] = a.c.k_scale[s]; v_scale[q] = a.c.v_scale[s]; }
      if (a.mass) mass[q] = a.mass[s];
    }
  }
#pragma unroll
  for (int q = 0; q < kEachAway; ++q) {
    if (from[q] < 0) continue;
    const size_t s = dest[q] + m.head;
    *reinterpret_cast<uint4 *>(m.k_at(dest[q])) = k[q];
    *reinterpret_cast<uint4 *>(m.v_at(dest[q])) = v[q];
    if (m.c == 0) {
      if (a.c.k_scale) { a.c.k_scale[s] = k_scale[q]; a.c.v_scale[s] = v_scale[q]; }
      if (a.mass) a.mass[s] = mass[q];
    }
  }
}

// What a thread of shift_in_place_kernel holds between reading and writing:
// shared memory of its own, so that many rows fit and loads need no registers.
struct Held {
  uint4 k[kEachInPlace][kMoveThreads], v[kEachInPlace][kMoveThreads];
  float mass[kEachInPlace][kMoveThreads];
  int dest[kEachInPlace][kMoveThreads];
  uint8_t k_scale[kEachInPlace][kMoveThreads], v_scale[kEachInPlace][kMoveThreads];
};

// In place the CTAs of x are a cluster that walks the list from its start, round
// by round: every row of a round is read before any is written (a cluster barrier
// between the two), and since lists ascend and no row moves to a later position,
// a place is written in no earlier round than it is read: position first + j is
// row src[j'] of the list with j' <= j if it is any. The next round's rows lie
// behind all places written so far, so its loads wait for nobody.
template <int ROW>
__global__ void __launch_bounds__(kMoveThreads) shift_in_place_kernel(const __grid_constant__ ShiftArgs a) {
  extern __shared__ uint4 smem_held[];
  Held &held = *reinterpret_cast<Held *>(smem_held);
  pdl_trigger();
  pdl_wait();
  const Mover<ROW, true> m = mover<ROW, true>(a);
  const int tid = threadIdx.x, rows = round_rows(ROW, true);
  for (int base = 0; base < m.n; base += gridDim.x * rows) {
#pragma unroll 1
    for (int q0 = 0; q0 < kEachInPlace; q0 += kAtOnce) {
      int from[kAtOnce], dest[kAtOnce];
      // (kStep rows to a CTA in turn: short lists have all of the cluster's loads)
      m.find(base + (q0 * gridDim.x + blockIdx.x) * m.kStep + tid / m.kChunks, gridDim.x * m.kStep, from, dest);
      float mass[kAtOnce];
      uint8_t k_scale[kAtOnce], v_scale[kAtOnce];
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q) {
        held.dest[q0 + q][tid] = dest[q];
        if (from[q] < 0) continue;
        copy16(&held.k[q0 + q][tid], m.k_at(from[q]), true);
        copy16(&held.v[q0 + q][tid], m.v_at(from[q]), true);
        const size_t s = from[q] + m.head;
        if (m.c == 0) {
          if (a.c.k_scale) { k_scale[q] = a.c.k_scale[s]; v_scale[q] = a.c.v_scale[s]; }
          if (a.mass) mass[q] = a.mass[s];
        }
      }
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q) {
        if (from[q] < 0 || m.c != 0) continue;
        if (a.c.k_scale) { held.k_scale[q0 + q][tid] = k_scale[q]; held.v_scale[q0 + q][tid] = v_scale[q]; }
        if (a.mass) held.mass[q0 + q][tid] = mass[q];
      }
    }
    copies_wait();
    // The round's reads are over (each value is in shared memory); of writes
    // before nothing has to be known. Every CTA reaches the barrier.
    cluster_barrier();
#pragma unroll
    for (int q = 0; q < kEachInPlace; ++q) {
      const int dest = held.dest[q][tid];
      if (dest < 0) continue;
      *reinterpret_cast<uint4 *>(m.k_at(dest)) = held.k[q][tid];
      *reinterpret_cast<uint4 *>(m.v_at(dest)) = held.v[q][tid];
      if (m.c == 0) {
        const size_t s = dest + m.head;
        if (a.c.k_scale) { a.c.k_scale[s] = held.k_scale[q][tid]; a.c.v_scale[s] = held.v_scale[q][tid]; }
        if (a.mass) a.mass[s] = held.mass[q][tid];
      }
    }
  }
}

template <int ROW>
cudaError_t launch_shift_rows(const ShiftArgs &g, bool in_place, int heads, int B, cudaStream_t s) {
  if (!in_place)
    return launch_pdl(shift_kernel<ROW>, dim3((g.max_n - 1) / round_rows(ROW, false) + 1, heads, B), dim3(kMoveThreads), 0, s, g);
  const int parts = (g.max_n - 1) / Mover<ROW, true>::kStep + 1;
  // As many CTAs as there are parts, up to the most that every cluster may have.
  // (One request, 800 rows that move: 8 CTAs 12 us with
  // the choice, one 40.)
  const unsigned cluster = parts > 4 ? 8 : parts > 2 ? 4 : parts;
  const cudaError_t e = cudaFuncSetAttribute(shift_in_place_kernel<ROW>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Held));
  if (e != cudaSuccess) return e;
  return launch_pdl_clusters(shift_in_place_kernel<ROW>, cluster, dim3(cluster, heads, B), dim3(kMoveThreads), sizeof(Held), s, g);
}

dllm_status launch_shift(const dllm_kv_pages *pages, const ShiftArgs &g, bool in_place, int B, cudaStream_t s) {
  const int row = pages->dh * (pages->type == DLLM_KV_E4M3 ? 1 : 2);
  const cudaError_t e = row == 64    ? launch_shift_rows<64>(g, in_place, pages->heads, B, s)
                        : row == 128 ? launch_shift_rows<128>(g, in_place, pages->heads, B, s)
                                     : launch_shift_rows<256>(g, in_place, pages->heads, B, s);
  return e == cudaSuccess ? DLLM_OK : cuda_error(e);
}

// Rows go to another table, or stay in theirs: no table at all has no pages.
bool tables_agree(const int32_t *table, int pages, const int32_t *dst, int dst_pages) {
  return dst ? dst != table || dst_pages == pages : dst_pages == 0;
}

}  // namespace
}  // namespace dllm

using namespace dllm;

extern "C" dllm_status dllm_kv_move(const dllm_kv_pages *pages, const dllm_kv_move_args *a, dllm_stream stream) {
  const dllm_status st = check_pages(pages);
  if (st != DLLM_OK) return st;
  if (!a || a->B < 0 || a->max_n < 0 || a->max_pages < 0 || a->dst_pages < 0) return DLLM_ERR_INVALID_ARG;
  if (a->src_heads != 1 && a->src_heads != pages->heads) return DLLM_ERR_INVALID_ARG;
  if (a->B > 4096 || a->max_n >= (1 << 30)) return DLLM_ERR_UNSUPPORTED;
  if (a->B == 0 || a->max_n == 0) return DLLM_OK;
  const dllm_status sp = check_page_pointers(pages);
  if (sp != DLLM_OK) return sp;
  if (!a->src || !a->count || (!a->page_table && a->max_pages > 0) || !tables_agree(a->page_table, a->max_pages, a->dst_table, a->dst_pages))
    return DLLM_ERR_INVALID_ARG;
  ShiftArgs g{};
  g.c = device_pages(pages, a->page_table, a->max_pages);
  const bool in_place = !a->dst_table || a->dst_table == a->page_table;
  g.dst_table = in_place ? a->page_table : a->dst_table;
  g.dst_pages = in_place ? a->max_pages : a->dst_pages;
  g.src = a->src; g.src_heads = a->src_heads; g.max_n = a->max_n; g.count = a->count; g.first = a->first; g.mass = a->mass;
  g.most = a->max_n;
  cudaError_t e = cudaGetSymbolAddress(reinterpret_cast<void **>(&g.status), g_status_evict);
  if (e != cudaSuccess) return cuda_error(e);
  const dllm_status sl = launch_shift(pages, g, in_place, a->B, static_cast<cudaStream_t>(stream));
  return sl == DLLM_OK ? launch_status() : sl;
}

extern "C" dllm_status dllm_kv_evict(const dllm_kv_pages *pages, const dllm_kv_evict_args *a, dllm_stream stream) {
  const dllm_status st = check_pages(pages);
  if (st != DLLM_OK) return st;
  if (!a || a->B < 0 || a->max_pages < 0 || a->dst_pages < 0 || a->budget < 1 || a->max_kv < 0 || a->sinks < 0 || a->recent < 0)
    return DLLM_ERR_INVALID_ARG;
  if (a->B > 4096 || a->max_kv >= (1 << 30) || a->budget >= (1 << 30)) return DLLM_ERR_UNSUPPORTED;
  if (static_cast<long long>(a->sinks) + a->recent > a->budget) return DLLM_ERR_INVALID_ARG;
  if (a->B == 0) return DLLM_OK;
  const dllm_status sp = check_page_pointers(pages);
  if (sp != DLLM_OK) return sp;
  if (!a->mass || !a->kv_len || (!a->page_table && a->max_pages > 0) || !a->new_len || !a->keep ||
      !tables_agree(a->page_table, a->max_pages, a->dst_table, a->dst_pages))
    return DLLM_ERR_INVALID_ARG;
  SelectArgs g{};
  g.c = device_pages(pages, a->page_table, a->max_pages);
  const long long table = static_cast<long long>(a->max_pages) * pages->page_size;   // rows beyond the table are not there
  g.mass = a->mass; g.kv_len = a->kv_len; g.keep = a->keep;
  g.budget = a->budget; g.max_kv = static_cast<int>(table < a->max_kv ? table : a->max_kv);
  g.sinks = a->sinks; g.recent = a->recent;
  cudaError_t e = cudaGetSymbolAddress(reinterpret_cast<void **>(&g.status), g_status_evict);
  if (e != cudaSuccess) return cuda_error(e);
  ShiftArgs m{};
  m.c = g.c;
  const bool in_place = !a->dst_table || a->dst_table == a->page_table;
  m.dst_table = in_place ? a->page_table : a->dst_table;
  m.dst_pages = in_place ? a->max_pages : a->dst_pages;
  m.src = a->keep; m.src_heads = pages->heads; m.max_n = a->budget; m.count = a->kv_len;
  m.most = g.max_kv < a->budget ? g.max_kv : a->budget;
  m.new_len = a->new_len;
  m.mass = a->move_mass ? a->mass : nullptr;
  m.status = g.status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int row = pages->dh * (pages->type == DLLM_KV_E4M3 ? 1 : 2);
  g.new_len = a->new_len; g.move_mass = m.mass;
  g.ctas = in_place ? moving_ctas(g, row, a->B) : 0;
  if (g.ctas > 0) {
    g.share = (g.budget + g.ctas - 1) / g.ctas;
    e = row == 64 ? launch_select<64>(g, a->B, s) : row == 128 ? launch_select<128>(g, a->B, s) : launch_select<256>(g, a->B, s);
    return e == cudaSuccess ? launch_status() : cuda_error(e);
  }
  e = launch_select<0>(g, a->B, s);
  if (e != cudaSuccess) return cuda_error(e);
  const dllm_status sl = launch_shift(pages, m, in_place, a->B, s);
  return sl == DLLM_OK ? launch_status(2) : sl;
}
