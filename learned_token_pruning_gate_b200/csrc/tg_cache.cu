// The pages of a paged cache: the tables of a decoding step (fork, free, growth),
// compaction, page copies and appended rows.
//
// The table kernels are integer work on a few hundred kilobytes that later steps
// depend on, so what bounds them is the chain of dependent accesses and barriers:
// one launch does all phases of a call, in one CTA or in a cluster of eight with
// cluster barriers between the phases, and every CTA computes the scans over the
// (at most 1024) sequences for itself.  Counts are integers, so the atomic updates
// give the same result in any order.  Reference counts and tables that other CTAs
// of the cluster write are read through L2 (__ldcg).  A beam search's step of 32
// sequences of 70 pages in a pool of 2048 (fork, growth, page copies of 4 layers)
// takes 11.7 us on the device.
//
// The data kernels (page copies, appended rows) are 16-byte streams bound by HBM:
// 343 MB of a compaction move at the copy rate (49.5 us, 6.9 TB/s).
#include "tg_internal.cuh"

namespace tg {
namespace {

constexpr int kMaxTabCtas = 8;
constexpr int kTabThreads = 1024;
constexpr int kTabWarps = kTabThreads / 32;
constexpr int kPiece = 128;  // table entries a warp has in flight
static_assert(kTabThreads >= kMaxSeqs, "a thread per sequence");

// Inclusive scan over the block's threads; `warp_sums` holds 32 words and may be
// reused after the next __syncthreads().
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int s = warp_sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  *total = __shfl_sync(0xffffffffu, s, 31);
  const int before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
  return warp > 0 ? x + before : x;
}

// The largest x of the block; `warp_max` holds 32 words.
__device__ __forceinline__ int block_max(int x, int* warp_max) {
  x = __reduce_max_sync(0xffffffffu, x);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = x;
  __syncthreads();
  x = __reduce_max_sync(0xffffffffu, warp_max[threadIdx.x & 31]);
  __syncthreads();
  return x;
}

// The CTAs of a table call: a cluster, or one CTA alone, whose barriers are an order cheaper.
template <int kCtas>
struct Team {
  static __device__ __forceinline__ int rank() { return kCtas == 1 ? 0 : static_cast<int>(cluster_ctarank()); }
  // all threads of the team; global and shared memory written before is seen after it
  static __device__ __forceinline__ void sync() {
    if constexpr (kCtas == 1) __syncthreads();
    else cluster_sync_all();
  }
  // All CTAs of the team run: their shared memory may be written after started(), which waits for
  // every CTA's starting().
  static __device__ __forceinline__ void starting() {
    if constexpr (kCtas > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }
  static __device__ __forceinline__ void started() {
    if constexpr (kCtas > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  // writes v into word `slot` of the array at the same place in every CTA, once all of them run
  static __device__ __forceinline__ void publish(int* array, int slot, int v) {
    if constexpr (kCtas == 1) {
      array[slot] = v;
    } else {
      const uint32_t at = smem_u32(array + slot);
      for (uint32_t r = 0; r < kCtas; ++r)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(at, r)), "r"(v) : "memory");
    }
  }
};

__device__ __forceinline__ int pages_of(int64_t tokens, int shift) {
  return static_cast<int>((tokens + (int64_t{1} << shift) - 1) >> shift);
}

// A length as the table can hold it.
__device__ __forceinline__ int checked_len(int len, int max_pages, int shift, bool* bad) {
  const int64_t most = static_cast<int64_t>(max_pages) << shift;
  if (len < 0) {
    *bad = true;
    return 0;
  }
  if (len > most) {
    *bad = true;
    return static_cast<int>(most);
  }
  return len;
}

// ---- fork, free and growth ---------------------------------------------------------------------
template <int kTabCtas>
__global__ void __launch_bounds__(kTabThreads) cache_update_kernel(const __grid_constant__ CacheUpdateArgs a) {
  using Team = Team<kTabCtas>;
  __shared__ int kids[kMaxSeqs];    // output sequences per input sequence
  __shared__ int in_pages[kMaxSeqs];  // pages of every input sequence
  __shared__ int from_seq[kMaxSeqs];  // the input sequence of every output sequence, or -1
  __shared__ __align__(16) int shared_page[kMaxSeqs];  // the partly filled page a growing sequence shares, or -1
  __shared__ int ends[kMaxSeqs];    // inclusive scan of the pages that sequences need
  __shared__ int firsts[kMaxSeqs];  // 2 x the table slot of the first page a sequence gets, + 1 for a copy
  __shared__ int sums[32], sums2[32], free_count[kTabCtas];
  const int tid = threadIdx.x, lane = tid & 31;
  const int rank = Team::rank();
  const int gwarp = rank * kTabWarps + (tid >> 5);
  constexpr int kWarps = kTabCtas * kTabWarps;
  const int page = 1 << a.page_shift;
  bool bad = false;
  grid_dep_wait();
  grid_dep_launch();

  // children per input sequence; the output sequence of this thread
  kids[tid] = a.parent ? 0 : 1;
  __syncthreads();
  int from = tid < a.batch_out ? tid : -1;
  if (tid < a.batch_out && a.parent) {
    from = a.parent[tid];
    if (from < -1 || from >= a.batch_in) {
      bad = true;
      from = -1;
    }
    if (from >= 0) atomicAdd(&kids[from], 1);
  }
  from_seq[tid] = from;
  const int mine_in =
      tid < a.batch_in ? pages_of(checked_len(a.lens_in[tid], a.max_pages, a.page_shift, &bad), a.page_shift) : 0;
  in_pages[tid] = mine_in;
  const int longest = block_max(mine_in, sums);
  // tokens of output sequence tid
  const int held = from >= 0 ? checked_len(a.lens_in[from], a.max_pages, a.page_shift, &bad) : 0;
  if (a.refs_out != a.refs_in)
    for (int p = rank * kTabThreads + tid; p < a.n_pages; p += kTabCtas * kTabThreads)
      a.refs_out[p] = a.refs_in[p];
  Team::sync();

  // The counts follow the children; the tables follow the parents.  A warp takes kPiece entries of
  // a row at a time, the longest row setting how many pieces there are.
  const int pieces = (longest + kPiece - 1) / kPiece;
  if (a.parent) {
    for (int64_t w = gwarp; w < static_cast<int64_t>(a.batch_in) * pieces; w += kWarps) {
      const int b = static_cast<int>(w / pieces), j0 = static_cast<int>(w - static_cast<int64_t>(b) * pieces) * kPiece;
      const int change = kids[b] - 1, used = in_pages[b];
      if (change == 0) continue;
      const int32_t* row = a.table_in + static_cast<int64_t>(b) * a.max_pages;
#pragma unroll
      for (int u = 0; u < kPiece; u += 32) {
        const int j = j0 + u + lane;
        if (j >= used) continue;
        const int p = row[j];
        if (p >= 0 && p < a.n_pages) atomicAdd(a.refs_out + p, change);
        else bad = true;
      }
    }
  }
  if (a.table_out != a.table_in) {
    for (int64_t w = gwarp; w < static_cast<int64_t>(a.batch_out) * pieces; w += kWarps) {
      const int i = static_cast<int>(w / pieces), j0 = static_cast<int>(w - static_cast<int64_t>(i) * pieces) * kPiece;
      const int source = from_seq[i];
      if (source < 0) continue;
      const int used = in_pages[source];
      const int32_t* row = a.table_in + static_cast<int64_t>(source) * a.max_pages + j0 + lane;
      int32_t* dst = a.table_out + static_cast<int64_t>(i) * a.max_pages + j0 + lane;
      int32_t x[kPiece / 32];
#pragma unroll
      for (int u = 0; u < kPiece / 32; ++u)
        if (j0 + lane + 32 * u < used) x[u] = row[32 * u];
#pragma unroll
      for (int u = 0; u < kPiece / 32; ++u)
        if (j0 + lane + 32 * u < used) dst[32 * u] = x[u];
    }
  }
  Team::sync();

  // what each sequence needs
  int n = 0, used = 0, grown = 0, last = -1, count = 0;
  bool fits = false, shares = false;
  if (tid < a.batch_out) {
    if (a.cu_new) {
      const int64_t d = static_cast<int64_t>(a.cu_new[tid + 1]) - a.cu_new[tid];
      if (d < 0) bad = true;
      else n = static_cast<int>(d > INT32_MAX ? INT32_MAX : d);
    }
    used = pages_of(held, a.page_shift);
    const int64_t want = static_cast<int64_t>(held) + n;
    fits = want <= (static_cast<int64_t>(a.max_pages) << a.page_shift) && want <= INT32_MAX;
    grown = fits ? pages_of(want, a.page_shift) : used;
    if (n > 0 && fits && (held & (page - 1)) != 0) {
      last = __ldcg(a.table_out + static_cast<int64_t>(tid) * a.max_pages + used - 1);
      if (last < 0 || last >= a.n_pages) {
        bad = true;
        fits = false;  // nothing can be written there
        grown = used;
      } else {
        count = __ldcg(a.refs_out + last);
        shares = count > 1;
      }
    }
  }
  shared_page[tid] = shares ? last : -1;
  // free pages of this CTA's part of the pool, a contiguous run per thread
  const int per_cta = (a.n_pages + kTabCtas - 1) / kTabCtas;
  const int per_thread = (per_cta + kTabThreads - 1) / kTabThreads;
  const int cta_end = min(a.n_pages, (rank + 1) * per_cta);
  const int p0 = min(cta_end, rank * per_cta + tid * per_thread), p1 = min(cta_end, p0 + per_thread);
  int mine = 0;
  if (a.cu_new)
    for (int p = p0; p < p1; ++p) mine += __ldcg(a.refs_out + p) <= 0;
  int cta_free = 0;
  const int free_end = block_scan(mine, sums, &cta_free);  // (its barrier publishes shared_page too)
  if (tid == 0) Team::publish(free_count, rank, cta_free);
  // of the holders of a shared page that grow, the last one in order keeps it if nobody else holds it
  bool copies = false;
  if (shares) {
    int before = 0;
    for (int j = 0; j < tid >> 2; ++j) {
      const int4 p = reinterpret_cast<const int4*>(shared_page)[j];
      before += (p.x == last) + (p.y == last) + (p.z == last) + (p.w == last);
    }
    for (int j = tid & ~3; j < tid; ++j) before += shared_page[j] == last;
    copies = count - before > 1;
  }
  // (no more than n_pages + 1, which is never served, so that 1024 of them add up within 32 bits)
  const int need = fits ? min(grown - used + (copies ? 1 : 0), a.n_pages + 1) : 0;
  int total_need = 0;
  const int end = block_scan(need, sums2, &total_need);
  ends[tid] = end;
  firsts[tid] = copies ? 2 * (used - 1) + 1 : 2 * used;
  Team::sync();

  int total_free = 0, free_before = 0;
#pragma unroll
  for (int r = 0; r < kTabCtas; ++r) {
    if (r < rank) free_before += free_count[r];
    total_free += free_count[r];
  }
  const bool served = tid < a.batch_out && fits && (end <= total_free || (need == 0 && !shares));
  if (rank == 0 && tid < a.batch_out) {
    const bool copied = served && copies;
    a.start[tid] = served ? held : -1;
    a.lens_out[tid] = served ? held + n : held;
    a.copy_src[tid] = copied ? last : -1;
    if (copied) atomicSub(a.refs_out + last, 1);
    else a.copy_dst[tid] = -1;
  }
  // hand the free pages out: the j-th goes to the sequence whose needs reach past j
  if (a.batch_out > 0) {
    int limit = min(total_need, total_free);
    int j = free_before + free_end - mine;
    for (int p = p0; p < p1 && j < limit; ++p) {
      if (__ldcg(a.refs_out + p) > 0) continue;
      int lo = 0, hi = a.batch_out - 1;  // the first sequence with ends > j
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] > j) hi = mid;
        else lo = mid + 1;
      }
      if (ends[lo] > total_free) break;  // that sequence and all after it go without
      const int begin = lo > 0 ? ends[lo - 1] : 0;
      a.table_out[static_cast<int64_t>(lo) * a.max_pages + (firsts[lo] >> 1) + (j - begin)] = p;
      a.refs_out[p] = 1;
      if (j == begin && (firsts[lo] & 1)) a.copy_dst[lo] = p;
      ++j;
    }
  }
  if (bad) atomicOr(a.status, kDevPageIndex);
}

// ---- compaction --------------------------------------------------------------------------------
template <int kTabCtas>
__global__ void __launch_bounds__(kTabThreads) cache_compact_kernel(const __grid_constant__ CacheCompactArgs a) {
  using Team = Team<kTabCtas>;
  __shared__ int row_pages[kMaxSeqs];  // pages of every sequence
  __shared__ int sums[32], sums2[32], live_count[kTabCtas], move_count[kTabCtas];
  const int tid = threadIdx.x, lane = tid & 31;
  const int rank = Team::rank();
  constexpr int kThreads = kTabCtas * kTabThreads;
  bool bad = false;
  Team::starting();
  grid_dep_wait();
  grid_dep_launch();

  const int mine_in =
      tid < a.batch ? pages_of(checked_len(a.lens[tid], a.max_pages, a.page_shift, &bad), a.page_shift) : 0;
  row_pages[tid] = mine_in;
  const int longest = block_max(mine_in, sums2);

  // live pages, counted in a contiguous run per thread
  const int per_cta = (a.n_pages + kTabCtas - 1) / kTabCtas;
  const int per_thread = (per_cta + kTabThreads - 1) / kTabThreads;
  const int cta_end = min(a.n_pages, (rank + 1) * per_cta);
  const int p0 = min(cta_end, rank * per_cta + tid * per_thread), p1 = min(cta_end, p0 + per_thread);
  int mine = 0;
  for (int p = p0; p < p1; ++p) mine += a.refs_in[p] > 0;
  int cta_live = 0;
  block_scan(mine, sums, &cta_live);
  Team::started();  // (no barrier of the team came before)
  if (tid == 0) Team::publish(live_count, rank, cta_live);
  Team::sync();
  int n = 0;
#pragma unroll
  for (int r = 0; r < kTabCtas; ++r) n += live_count[r];

  // Movers: live at n or above.  Holes: free below n.  There are as many of one as of the other
  // (n live pages, n places).
  int holes = 0, moves = 0;
  for (int p = p0; p < p1; ++p) {
    const bool live = a.refs_in[p] > 0;
    holes += !live && p < n;
    moves += live && p >= n;
  }
  int cta_holes = 0, cta_moves = 0;
  const int hole_end = block_scan(holes, sums2, &cta_holes);
  __syncthreads();
  const int move_end = block_scan(moves, sums, &cta_moves);
  __shared__ int hole_count[kTabCtas];
  if (tid == 0) {
    Team::publish(hole_count, rank, cta_holes);
    Team::publish(move_count, rank, cta_moves);
  }
  Team::sync();
  int hole_at = hole_end - holes, move_at = move_end - moves, total = 0;
#pragma unroll
  for (int r = 0; r < kTabCtas; ++r) {
    if (r < rank) {
      hole_at += hole_count[r];
      move_at += move_count[r];
    }
    total += move_count[r];
  }
  for (int p = p0; p < p1; ++p) {
    const int refs = a.refs_in[p];
    const bool live = refs > 0;
    if (live && p >= n) a.copy_src[move_at++] = p;
    if (!live && p < n) a.copy_dst[hole_at++] = p;
    a.page_map[p] = live && p < n ? p : -1;
    if (a.refs_out != a.refs_in) a.refs_out[p] = live && p < n ? refs : 0;
  }
  for (int i = total + rank * kTabThreads + tid; i < a.n_pages; i += kThreads) a.copy_src[i] = a.copy_dst[i] = -1;
  if (rank == 0 && tid == 0) {
    a.counts[0] = n;
    a.counts[1] = total;
  }
  Team::sync();

  for (int i = rank * kTabThreads + tid; i < total; i += kThreads) {
    const int src = __ldcg(a.copy_src + i), dst = __ldcg(a.copy_dst + i);
    a.page_map[src] = dst;
    const int refs = __ldcg(a.refs_in + src);
    a.refs_out[dst] = refs;
    if (a.refs_out == a.refs_in) a.refs_out[src] = 0;
  }
  Team::sync();

  const int pieces = (longest + kPiece - 1) / kPiece;
  for (int64_t w = rank * kTabWarps + (tid >> 5); w < static_cast<int64_t>(a.batch) * pieces; w += kTabCtas * kTabWarps) {
    const int b = static_cast<int>(w / pieces), j0 = static_cast<int>(w - static_cast<int64_t>(b) * pieces) * kPiece;
    const int32_t* row = a.table_in + static_cast<int64_t>(b) * a.max_pages + j0 + lane;
    int32_t* dst = a.table_out + static_cast<int64_t>(b) * a.max_pages + j0 + lane;
    int32_t x[kPiece / 32];
#pragma unroll
    for (int u = 0; u < kPiece / 32; ++u) {
      x[u] = -1;
      if (j0 + lane + 32 * u >= row_pages[b]) continue;
      const int p = row[32 * u];
      if (p >= 0 && p < a.n_pages) x[u] = __ldcg(a.page_map + p);
      else bad = true;
    }
#pragma unroll
    for (int u = 0; u < kPiece / 32; ++u)
      if (x[u] >= 0) dst[32 * u] = x[u];
  }
  if (bad) atomicOr(a.status, kDevPageIndex);
}

// ---- page copies -------------------------------------------------------------------------------
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;
constexpr int kCopyVecs = kCopyThreads * kCopyUnroll;  // 16-byte pieces per work item (32 KB)

struct CopyParams {
  char* base[TG_MAX_GATHER_TENSORS];
  int64_t page_vecs[TG_MAX_GATHER_TENSORS];
  int64_t layer_vecs[TG_MAX_GATHER_TENSORS];
  int32_t parts[TG_MAX_GATHER_TENSORS];       // work items per page
  int32_t item_end[TG_MAX_GATHER_TENSORS];    // inclusive scan of layers x parts
  int32_t n_pools;
};

// A work item is up to 32 KB of one page of one layer; a persistent grid strides over
// (pair, item), so pairs that are not there (-1) cost one look at the list.
__global__ void __launch_bounds__(kCopyThreads)
    cache_copy_kernel(const __grid_constant__ CopyParams p, int n_pages, const int32_t* __restrict__ src,
                      const int32_t* __restrict__ dst, int n_copies, const int32_t* __restrict__ count,
                      uint32_t* status) {
  grid_dep_wait();
  grid_dep_launch();
  const int n = count ? min(n_copies, *count) : n_copies;
  const int items = p.item_end[p.n_pools - 1];
  const int64_t total = static_cast<int64_t>(n) * items;
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const int pair = static_cast<int>(w / items);
    int item = static_cast<int>(w - static_cast<int64_t>(pair) * items);
    const int from = src[pair], to = dst[pair];
    if (from < 0 || to < 0 || from == to) continue;
    if (from >= n_pages || to >= n_pages) {
      if (threadIdx.x == 0) atomicOr(status, kDevPageIndex);
      continue;
    }
    int t = 0;
    while (item >= p.item_end[t]) ++t;
    if (t > 0) item -= p.item_end[t - 1];
    const int layer = item / p.parts[t], part = item - layer * p.parts[t];
    const int64_t vecs = p.page_vecs[t];
    uint4* base = reinterpret_cast<uint4*>(p.base[t]) + layer * p.layer_vecs[t];
    const uint4* s = base + from * vecs;
    uint4* d = base + to * vecs;
    const int64_t v0 = static_cast<int64_t>(part) * kCopyVecs + threadIdx.x;
    uint4 x[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
      if (v0 + u * kCopyThreads < vecs) x[u] = s[v0 + u * kCopyThreads];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
      if (v0 + u * kCopyThreads < vecs) d[v0 + u * kCopyThreads] = x[u];
  }
}

// ---- appended rows -----------------------------------------------------------------------------
// A warp per row: where it goes, then its k and v of all heads, eight 16-byte pieces a lane in
// flight.  12700 rows of 8 x 128 bf16 take 20.5 us (floor 16.2; the lookups and the launch are the
// rest).  A CTA that looks up 64 rows at once and streams them with all threads took 22.0.
constexpr int kAppendUnroll = 8;
__global__ void __launch_bounds__(256, 4) cache_append_kernel(const __grid_constant__ CacheAppendArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  const int page = 1 << a.page_shift;
  const int hv = a.head_bytes >> 4;  // 16-byte pieces per head
  const int row_vecs = a.hkv * hv;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); r < a.rows; r += warps) {
    int lo = 0, hi = a.batch - 1;  // the sequence: the first b with cu_new[b + 1] > r
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (a.cu_new[mid + 1] > r) hi = mid;
      else lo = mid + 1;
    }
    const int64_t first = a.cu_new[lo], end = a.cu_new[lo + 1];
    if (r < first || r >= end) continue;  // a row behind the last sequence
    const int begin = a.start[lo];
    if (begin < 0) continue;
    const int64_t pos = begin + (r - first);
    const int64_t slot = pos >> a.page_shift;
    const int at = slot < a.max_pages ? a.table[static_cast<int64_t>(lo) * a.max_pages + slot] : -1;
    if (at < 0 || at >= a.n_pages) {
      if (lane == 0) atomicOr(a.status, kDevPageIndex);
      continue;
    }
    const int off = static_cast<int>(pos & (page - 1));
    const int64_t base = (static_cast<int64_t>(at) * a.hkv * page + off) * hv;
    const uint4* ks = static_cast<const uint4*>(a.k) + r * row_vecs;
    const uint4* vs = static_cast<const uint4*>(a.v) + r * row_vecs;
    for (int i0 = lane; i0 < 2 * row_vecs; i0 += 32 * kAppendUnroll) {
      uint4 x[kAppendUnroll];
#pragma unroll
      for (int u = 0; u < kAppendUnroll; ++u) {
        const int i = i0 + 32 * u;
        if (i < 2 * row_vecs) x[u] = i < row_vecs ? ks[i] : vs[i - row_vecs];
      }
#pragma unroll
      for (int u = 0; u < kAppendUnroll; ++u) {
        const int i = i0 + 32 * u;
        if (i >= 2 * row_vecs) break;
        const int j = i < row_vecs ? i : i - row_vecs;
        const int head = j / hv;
        static_cast<uint4*>(i < row_vecs ? a.k_pages : a.v_pages)[base + static_cast<int64_t>(head) * page * hv + (j - head * hv)] = x[u];
      }
    }
    if (lane == 0 && a.logsig_pages)
      a.logsig_pages[static_cast<int64_t>(at) * page + off] = a.logsig ? a.logsig[r] : 0.0f;
  }
}

}  // namespace

namespace {

// A table call's launch: one CTA, or a cluster of eight when there is enough to share.
template <typename Args>
cudaError_t launch_tables(void (*one)(Args), void (*eight)(Args), bool small, const Args& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(small ? 1 : kMaxTabCtas);
  cfg.blockDim = dim3(kTabThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kMaxTabCtas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = small ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, small ? one : eight, a);
}

// One CTA up to 4096 pages and 64 sequences, the cluster beyond: on the device an update of 32
// sequences of 64 pages takes 7.9 us in one CTA and 9.1 in the cluster, of 256 sequences of 8 pages
// 16.7 and 11.4, of one sequence in a pool of 16384 pages 11.0 and 6.7.  A compaction takes 5.3 us in
// one CTA (32 sequences, 2048 pages) and 8.9 in the cluster (32 sequences, 8192 pages).
bool small_tables(int n_pages, int batch) { return n_pages <= 4096 && batch <= 64; }

}  // namespace

tg_status launch_cache_update(const CacheUpdateArgs& a, cudaStream_t st) {
  return cuda_check(launch_tables(cache_update_kernel<1>, cache_update_kernel<kMaxTabCtas>,
                                  small_tables(a.n_pages, a.batch_in > a.batch_out ? a.batch_in : a.batch_out), a, st),
                    "cache update launch");
}

tg_status launch_cache_compact(const CacheCompactArgs& a, cudaStream_t st) {
  return cuda_check(launch_tables(cache_compact_kernel<1>, cache_compact_kernel<kMaxTabCtas>,
                                  small_tables(a.n_pages, a.batch), a, st),
                    "cache compact launch");
}

tg_status launch_cache_copy(const tg_page_pool* pools, int n_pools, int n_pages, const int32_t* src,
                            const int32_t* dst, int n_copies, const int32_t* count, uint32_t* status,
                            cudaStream_t st) {
  CopyParams p = {};
  p.n_pools = n_pools;
  int end = 0;
  for (int t = 0; t < n_pools; ++t) {
    p.base[t] = static_cast<char*>(pools[t].base);
    p.page_vecs[t] = pools[t].page_bytes / 16;
    p.layer_vecs[t] = p.page_vecs[t] * n_pages;
    p.parts[t] = static_cast<int32_t>((p.page_vecs[t] + kCopyVecs - 1) / kCopyVecs);
    end += pools[t].layers * p.parts[t];
    p.item_end[t] = end;
  }
  const int64_t work = static_cast<int64_t>(n_copies) * end;
  const int64_t cap = static_cast<int64_t>(num_sms()) * 8;
  const dim3 grid(static_cast<unsigned>(work < cap ? work : cap));
  return cuda_check(launch_pdl(cache_copy_kernel, grid, dim3(kCopyThreads), 0, st, p, n_pages, src, dst,
                               n_copies, count, status),
                    "page copy launch");
}

tg_status launch_cache_append(const CacheAppendArgs& a, cudaStream_t st) {
  int64_t blocks = (a.rows + 7) / 8;
  const int64_t cap = static_cast<int64_t>(num_sms()) * 4;
  if (blocks > cap) blocks = cap;
  return cuda_check(launch_pdl(cache_append_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, a),
                    "cache append launch");
}

}  // namespace tg
