// The best continuations of each group of beams: log-softmax over the vocabulary,
// the beam's score added, and the n best of beams x vocabulary in order.
//
// Within a beam the order of the candidates is the order of the logits, so the
// vocabulary is read once: beam_chunk_kernel takes 32 KB of one row into
// registers and leaves the chunk's maximum, its sum of exponentials and its n
// best logits, sorted.  beam_merge_kernel, one CTA per group, joins the sums
// into the rows' log-sums in 64 bits and picks the n best of the lists.
//
// Both pick by a threshold, a lower bound on the n-th best: among the largest of
// disjoint sets (a thread's logits; a sorted list) the n-th largest is one.  Only
// what is not below it is collected (rarely more than 2 n), and a collected key's
// place is the number of larger ones.  Keys are distinct, since the index is part
// of them, so ties go to the lower index and the order of collection does not
// matter.  A chunk finds its threshold by bisection over the threads' maxima, one
// barrier with a count per step; it stops as soon as the count is close to n.
//
// What bounds them: the chunk kernel its instructions (about 900 a thread for 64
// logits; the exponentials alone are 2.8 us of the special-function units for 96
// rows of 131071) and the chain of its barriers, the merge the dependent steps of
// one CTA per group (log-sums in 64 bits 1.5 us, rankings 1.8 us).  96 rows of
// 131071 bf16 logits take 14.9 us on the device (HBM floor 3.9), 4 rows of 32000
// fp32 7.0 us.  With a chunk's threshold found by comparing every thread's maximum
// with every other's the chunks took 48 us instead of 12; with a group joined in
// the CTA that finishes its last chunk, in place of a second launch, the calls
// took 18.9 and 8.3 us.
//
// The scores are compared in 64 bits: beams meet at sums that differ in the last
// places of 32.  A chunk's sum is taken in 32 bits: a term d below the maximum is
// off by 2^-22 (the approximate exponential) and 2.5 d 2^-24 (difference, product and
// log2e rounded) of itself, where d averages to at most the log of the chunk's length,
// 9.7; the additions, 32 and a tree of 14, by 2^-24 each: at most 5e-6 of the sum.  On
// random logits it is off by some 1e-8.
#include <cmath>

#include "tg_internal.cuh"

namespace tg {
namespace {

constexpr int kChunkThreads = 256;
constexpr int kMaxOut = 2 * TG_MAX_BEAMS;
constexpr int kMaxVocab = 1 << 20;  // as the C ABI checks
// Logits per thread and per CTA: 128 bytes a thread.
template <typename T>
constexpr int kPerThread = 128 / static_cast<int>(sizeof(T));
template <typename T>
constexpr int kChunk = kChunkThreads * kPerThread<T>;
constexpr int kChunkKeys = 2048;  // room for a chunk's collected keys
constexpr int kBatch = 8;         // keys a ranking compares at a time (arrays are that much longer than they need be)
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMergeThreads = 512;

// What a chunk leaves: per (row, chunk) n keys, and {m, sum e^(x - m)}, with m the
// largest logit (-inf: none above it, and the sum is 0).
struct BeamWork {
  float2* sums;
  uint64_t* keys;
};

__device__ __forceinline__ uint32_t raw_bits(float x) { return __float_as_uint(x); }
__device__ __forceinline__ uint32_t raw_bits(__nv_bfloat16 x) { return __bfloat16_as_ushort(x); }

// A thread's logits as they come from memory: 16-byte pieces, unpacked where they are used, so
// that bf16 ones take half the registers.
template <typename T>
struct Logits {
  static constexpr int kN = kPerThread<T>;
  uint32_t w[32];
  static constexpr bool kHalf = sizeof(T) == 2;
  __device__ __forceinline__ float get(int e) const {
    if constexpr (kHalf) return __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
    else return __uint_as_float(w[e]);
  }
  __device__ __forceinline__ void set(int e, float x) {  // x is a number of type T
    const uint32_t b = __float_as_uint(x);
    if constexpr (kHalf) w[e >> 1] = e & 1 ? (w[e >> 1] & 0xffffu) | (b & 0xffff0000u) : (w[e >> 1] & 0xffff0000u) | (b >> 16);
    else w[e] = b;
  }
  __device__ __forceinline__ float largest() const {  // (NaN is passed over)
    if constexpr (kHalf) {
      __nv_bfloat162 m, x;
      memcpy(&m, &w[0], 4);
#pragma unroll
      for (int e = 1; e < 32; ++e) {
        memcpy(&x, &w[e], 4);
        m = __hmax2(m, x);
      }
      return fmaxf(__low2float(m), __high2float(m));
    } else {
      float m = get(0);
#pragma unroll
      for (int e = 1; e < 32; ++e) m = fmaxf(m, get(e));
      return m;
    }
  }
  // Which logits are not below `bound`: bits[0] and bits[1] name the elements first(b) and up.
  __device__ __forceinline__ void not_below(float bound, uint32_t (&bits)[2]) const {
    bits[0] = bits[1] = 0;
    if constexpr (kHalf) {
      const __nv_bfloat162 b = __bfloat162bfloat162(__float2bfloat16_ru(bound));
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        __nv_bfloat162 x;
        memcpy(&x, &w[e], 4);
        bits[e >> 4] |= __hge2_mask(x, b) & (0x00010001u << (e & 15));
      }
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (get(e) >= bound) bits[0] |= 1u << e;
    }
  }
  // The element that bit b of bits[half] stands for.
  static __device__ __forceinline__ int element(int half, int b) {
    return kHalf ? half * 32 + (b & 15) * 2 + (b >> 4) : b;
  }
};

// The 16-byte pieces that hold `kLead` elements of what comes before a lane's tokens, turned into its
// tokens: each piece's last words and the first of the next, which the next lane has (lane 31's next
// is lane 0's of the piece after; `behind` for the last).
template <typename T, int kLead>
__device__ __forceinline__ void shift_pieces(Logits<T>& x, const uint32_t (&behind)[4]) {
  constexpr int kBytes = kLead * static_cast<int>(sizeof(T)), kWord = kBytes / 4;
  constexpr bool kSplit = kBytes % 4 != 0;  // tokens straddle words
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t w[8];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      w[n] = x.w[4 * i + n];
      const uint32_t next = i < 7 ? x.w[4 * (i + 1 < 8 ? i + 1 : 7) + n] : behind[n];
      w[4 + n] = n < kWord + kSplit ? __shfl_sync(0xffffffffu, lane == 0 ? next : w[n], (lane + 1) & 31) : 0u;
    }
#pragma unroll
    for (int n = 0; n < 4; ++n)
      x.w[4 * i + n] = kSplit ? __funnelshift_r(w[n + kWord], w[n + kWord + 1 < 8 ? n + kWord + 1 : 7], 16) : w[n + kWord];
  }
}

template <typename T>
__host__ __device__ inline int chunks_of(int vocab) {
  return (vocab + kChunk<T> - 1) / kChunk<T>;
}

// Larger logit first, then the lower token; 0 for what is no candidate.
__device__ __forceinline__ uint64_t logit_key(float x, int token) {
  if (!(x > -INFINITY)) return 0;  // -inf, NaN
  return (static_cast<uint64_t>(order_key(x)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(token));
}
// The number whose order_key is k (k > 0).
__device__ __forceinline__ float from_order_key(uint32_t k) {
  return __uint_as_float((k >> 31) ? (k & 0x7FFFFFFFu) : ~k);
}
constexpr uint32_t kLowestKey = 0x00800000u;  // order_key of the lowest finite number

template <typename T>
__global__ void __launch_bounds__(kChunkThreads, 4)
    beam_chunk_kernel(const T* __restrict__ logits, int rows, int vocab, int n_out, int chunks, BeamWork ws) {
  using L = Logits<T>;
  constexpr int kVec = 16 / static_cast<int>(sizeof(T));
  constexpr int kWarps = kChunkThreads / 32;
  static_assert(kChunkKeys >= (kMaxOut - 1) * 32, "most logits of a chunk in which fewer than n threads have any");
  __shared__ __align__(16) uint64_t found[kChunkKeys + kBatch];
  __shared__ int n_found;
  __shared__ uint32_t red_max[kWarps], red_min[kWarps];
  __shared__ float red_sum[kWarps];
  __shared__ uint64_t red_key[kWarps];
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / chunks;
  const int chunk = static_cast<int>(blockIdx.x - row * chunks);
  // Which tokens a thread has does not depend on where the row starts, so rows of the same logits
  // have the same sums to the last bit.  A row may start anywhere: its 16-byte pieces begin at the
  // boundary at or before a lane's first token, `lead` tokens early, and are then moved by that much.
  // (With tokens counted from the boundary in place of the move, and a CTA's pieces side by side,
  // 96 x 131071 bf16 took 16.3 us for 14.9 and 4 x 32000 fp32 6.8 for 7.0.)
  const T* r = logits + row * vocab;
  const int left = static_cast<int>(min((rows - row) * vocab, int64_t{1} << 30));  // what can be read from here
  const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(r) & 15u) / sizeof(T));
  const int t0 = chunk * kChunk<T> + (warp * 8 * 32 + lane) * kVec;  // the thread's first token
  auto token = [&](int e) { return t0 + (e / kVec) * (32 * kVec) + e % kVec; };
  L x;
  uint32_t behind[4] = {};
  auto load = [&](int t, uint32_t* w) {  // (t < 0 lies in the row before: a first row has no lead)
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    if (t < vocab && t + kVec <= left) u = __ldg(reinterpret_cast<const uint4*>(r + t));
    w[0] = u.x;
    w[1] = u.y;
    w[2] = u.z;
    w[3] = u.w;
  };
  auto load_end = [&](int t, uint32_t* w) {  // a piece that reaches past the last row: its tokens one at a time
    if (t >= vocab || t + kVec <= left) return;
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < kVec / 4; ++e)
        if (t + n * (kVec / 4) + e < vocab) w[n] |= raw_bits(r[t + n * (kVec / 4) + e]) << (16 * e);
  };
#pragma unroll
  for (int i = 0; i < 8; ++i) load(t0 + i * 32 * kVec - lead, &x.w[4 * i]);
  if (lead != 0 && lane == 0) load(t0 + 8 * 32 * kVec - lead, behind);
  if (left < vocab + kVec && (chunk + 1) * kChunk<T> + kVec > vocab && (left + lead) % kVec != 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) load_end(t0 + i * 32 * kVec - lead, &x.w[4 * i]);
    if (lead != 0 && lane == 0) load_end(t0 + 8 * 32 * kVec - lead, behind);
  }
  if (lead != 0) {
    if constexpr (L::kHalf) {
      switch (lead) {
        case 1: shift_pieces<T, 1>(x, behind); break;
        case 2: shift_pieces<T, 2>(x, behind); break;
        case 3: shift_pieces<T, 3>(x, behind); break;
        case 4: shift_pieces<T, 4>(x, behind); break;
        case 5: shift_pieces<T, 5>(x, behind); break;
        case 6: shift_pieces<T, 6>(x, behind); break;
        default: shift_pieces<T, 7>(x, behind);
      }
    } else {
      switch (lead) {
        case 1: shift_pieces<T, 1>(x, behind); break;
        case 2: shift_pieces<T, 2>(x, behind); break;
        default: shift_pieces<T, 3>(x, behind);
      }
    }
  }
  if (t0 + 7 * 32 * kVec + kVec > vocab) {  // what lies behind the row
#pragma unroll
    for (int e = 0; e < L::kN; ++e)
      if (token(e) >= vocab) x.set(e, -INFINITY);
  }

  // the thread's largest logit; the largest and smallest of these in the chunk (the smallest above
  // -inf: a ragged chunk has threads without tokens)
  const uint32_t key = order_key(x.largest());
  const uint32_t warp_max = __reduce_max_sync(0xffffffffu, key);
  const uint32_t warp_min = __reduce_min_sync(0xffffffffu, key >= kLowestKey ? key : 0xffffffffu);
  if (lane == 0) {
    red_max[warp] = warp_max;
    red_min[warp] = warp_min;
  }
  if (tid == 0) n_found = 0;
  __syncthreads();
  const uint32_t top = __reduce_max_sync(0xffffffffu, red_max[lane % kWarps]);
  const uint32_t low = __reduce_min_sync(0xffffffffu, red_min[lane % kWarps]);
  // Sum of exponentials, 2^((x - m) log2e).  The maximum is subtracted first: x log2e - m log2e is
  // off by m's rounding error, in the exponent, and overflows where a mask's value (the lowest of
  // its type, say) is all that a chunk holds.  NaN and +inf make the sum NaN; a chunk without a
  // logit above -inf leaves 0.
  const float largest = top >= kLowestKey ? from_order_key(top) : -INFINITY;
  const float minus_m = largest == -INFINITY ? 0.0f : -largest;
  float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int e = 0; e < L::kN; e += 2) {
    const float2 y = __fmul2_rn(__fadd2_rn(make_float2(x.get(e), x.get(e + 1)), make_float2(minus_m, minus_m)),
                                make_float2(kLog2e, kLog2e));
    s2 = __fadd2_rn(s2, make_float2(exp2_approx(y.x), exp2_approx(y.y)));
  }
  float s = s2.x + s2.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) red_sum[warp] = s;

  // The threshold lo: at least n threads hold a logit not below it (or it is the lowest finite
  // number).  Bisection between the chunk's smallest and largest thread maximum.
  uint32_t lo = max(low, kLowestKey), hi = top + 1;
  if (__syncthreads_count(key >= lo) >= n_out) {
    const int enough = n_out + (n_out >> 1) + 4;
    while (hi - lo > 1) {
      const uint32_t mid = lo + ((hi - lo) >> 1);
      const int above = __syncthreads_count(key >= mid);
      if (above >= n_out) {
        lo = mid;
        if (above <= enough) break;
      } else {
        hi = mid;
      }
    }
  } else {
    lo = kLowestKey;
  }
  if (key >= lo) {
    uint32_t bits[2];
    x.not_below(from_order_key(lo), bits);
#pragma unroll
    for (int half = 0; half < L::kN / 32; ++half)
      for (uint32_t b = bits[half]; b; b &= b - 1) {
        const int at = atomicAdd(&n_found, 1);
        const int t = token(L::element(half, __ffs(b) - 1));
        if (at < kChunkKeys) found[at] = logit_key(static_cast<float>(r[t]), t);
      }
  }
  __syncthreads();
  const int n = n_found;
  uint64_t* out = ws.keys + (row * chunks + chunk) * n_out;
  if (n <= kChunkKeys) {
    for (int i = tid; i < n; i += kChunkThreads) {
      const uint64_t k = found[i];
      int above = 0;
      for (int j = 0; j < n; j += kBatch) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) above += (found[j + u] > k) & (j + u < n);
      }
      if (above < n_out) out[above] = k;
    }
    for (int i = n + tid; i < n_out; i += kChunkThreads) out[i] = 0;
  } else {
    // More logits than there is room for share the threshold (a flat row): one best after another.
    uint64_t last = ~0ull;
    for (int i = 0; i < n_out; ++i) {
      uint64_t k = 0;
#pragma unroll 1
      for (int e = 0; e < L::kN; ++e) {
        const int t = token(e);
        if (t >= vocab) continue;
        const uint64_t one = logit_key(static_cast<float>(r[t]), t);
        if (one < last && one > k) k = one;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint64_t other = __shfl_xor_sync(0xffffffffu, k, o);
        k = other > k ? other : k;
      }
      if (lane == 0) red_key[warp] = k;
      __syncthreads();
      for (int w = 0; w < kWarps; ++w) k = red_key[w] > k ? red_key[w] : k;
      if (tid == 0) out[i] = k;
      last = k;
      __syncthreads();
    }
  }
  if (tid == 0) {
    float total = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += red_sum[w];
    ws.sums[row * chunks + chunk] = make_float2(largest, total);
  }
}

// A candidate of the group: larger score first, then the lower place in beams x vocabulary.
struct Cand {
  uint64_t score;  // order-preserving, 0 for none
  uint32_t place;
};
__device__ __forceinline__ bool before(const Cand& a, const Cand& b) {
  // (no short cut: the branches cost more than both comparisons)
  return (a.score > b.score) | ((a.score == b.score) & (a.place < b.place));
}
__device__ __forceinline__ uint64_t order_key64(double x) {
  if (!(fabs(x) < INFINITY)) return 0;  // not finite: no candidate
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));  // -0 becomes +0
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double from_order_key64(uint64_t k) {
  return __longlong_as_double(static_cast<long long>((k >> 63) ? (k & 0x7FFFFFFFFFFFFFFFull) : ~k));
}
__device__ __forceinline__ float logit_of(uint64_t key) { return from_order_key(static_cast<uint32_t>(key >> 32)); }

__global__ void __launch_bounds__(kMergeThreads)
    beam_merge_kernel(const float* __restrict__ scores, int beams, int vocab, int n_out, int chunks,
                      BeamWork ws, float* __restrict__ scores_out, int32_t* __restrict__ parent_out,
                      int32_t* __restrict__ token_out) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int lists = beams * chunks;
  const int room = n_out * (n_out + 1) / 2;
  uint64_t* const head_score = reinterpret_cast<uint64_t*>(smem);                         // [lists]
  uint64_t* const found_score = head_score + lists + kBatch;                              // [room]
  uint32_t* const head_place = reinterpret_cast<uint32_t*>(found_score + room + kBatch);  // [lists]
  uint32_t* const found_place = head_place + lists + kBatch;                              // [room]
  __shared__ double largest[TG_MAX_BEAMS], log_sum[TG_MAX_BEAMS];  // of a beam's logits, and of their e^(x - largest)
  __shared__ int ranked[kMaxOut];  // the lists by their heads
  __shared__ Cand limit;           // the n-th head
  __shared__ int n_found;
  grid_dep_wait();
  grid_dep_launch();
  constexpr int kWarps = kMergeThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * beams;
  if (tid == 0) {
    limit.score = 1;
    limit.place = 0xFFFFFFFFu;
    n_found = 0;
  }
  if (tid < kMaxOut) ranked[tid] = -1;
  // the heads' keys, on their way while the sums are joined
  const uint64_t* const keys = ws.keys + row0 * chunks * n_out;
  const uint64_t first_head = tid < lists ? keys[static_cast<int64_t>(tid) * n_out] : 0;
  // a warp per beam: log of the row's sum of exponentials
  for (int beam = warp; beam < beams; beam += kWarps) {
    const float2* part = ws.sums + (row0 + beam) * chunks;
    float top = -INFINITY;
    for (int c = lane; c < chunks; c += 32) top = fmaxf(top, part[c].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    double s = 0.0;
    for (int c = lane; c < chunks; c += 32) {
      const float2 p = part[c];
      if (p.y != 0.0f) s += static_cast<double>(p.y) * exp(static_cast<double>(p.x) - top);  // NaN stays NaN
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) {
      largest[beam] = top;
      log_sum[beam] = log(s);
    }
  }
  __syncthreads();
  auto cand = [&](int list, uint64_t key) {
    const int beam = list / chunks;
    Cand c = {0, 0};
    if (key) {
      const uint32_t token = 0xFFFFFFFFu - static_cast<uint32_t>(key);
      // (in this order: log_sum is below the last place of a logit of the type's lowest value)
      c.score = order_key64(static_cast<double>(scores[row0 + beam]) + ((static_cast<double>(logit_of(key)) - largest[beam]) - log_sum[beam]));
      c.place = static_cast<uint32_t>(beam) * static_cast<uint32_t>(vocab) + token;
    }
    return c;
  };
  for (int l = tid; l < lists; l += kMergeThreads) {
    const Cand c = cand(l, l == tid ? first_head : keys[static_cast<int64_t>(l) * n_out]);
    head_score[l] = c.score;
    head_place[l] = c.place;
  }
  __syncthreads();
  // how many of n places come before c
  auto ahead = [](const uint64_t* score, const uint32_t* place, int n, const Cand& c) {
    int above = 0;
    for (int j = 0; j < n; j += kBatch) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) above += before(Cand{score[j + u], place[j + u]}, c) & (j + u < n);
    }
    return above;
  };
  for (int l = tid; l < lists; l += kMergeThreads) {
    const Cand c = {head_score[l], head_place[l]};
    if (!c.score) continue;
    const int above = ahead(head_score, head_place, lists, c);
    if (above < n_out) ranked[above] = l;
    if (above == n_out - 1) limit = c;
  }
  __syncthreads();
  // The list whose head is r-th can add n - r candidates: r heads and its own earlier ones come
  // before the others.  Of these the ones not behind the n-th head count.
  for (int r = warp; r < n_out; r += kWarps) {
    const int l = ranked[r];
    if (l < 0) break;
    for (int i = lane; i < n_out - r; i += 32) {
      const Cand c = cand(l, keys[static_cast<int64_t>(l) * n_out + i]);
      if (!c.score || before(limit, c)) continue;
      const int at = atomicAdd(&n_found, 1);
      found_score[at] = c.score;
      found_place[at] = c.place;
    }
  }
  __syncthreads();
  const int n = n_found;
  const int64_t out = static_cast<int64_t>(blockIdx.x) * n_out;
  for (int i = tid; i < n; i += kMergeThreads) {
    const Cand c = {found_score[i], found_place[i]};
    const int above = ahead(found_score, found_place, n, c);
    if (above >= n_out) continue;
    const uint32_t beam = c.place / static_cast<uint32_t>(vocab);
    scores_out[out + above] = static_cast<float>(from_order_key64(c.score));
    parent_out[out + above] = static_cast<int32_t>(row0 + beam);
    token_out[out + above] = static_cast<int32_t>(c.place - beam * static_cast<uint32_t>(vocab));
  }
  for (int i = n + tid; i < n_out; i += kMergeThreads) {
    scores_out[out + i] = -INFINITY;
    parent_out[out + i] = -1;
    token_out[out + i] = -1;
  }
}

}  // namespace

// Dynamic shared memory of a merge: the heads of the lists and the candidates.
static size_t merge_smem(int lists, int n_out) {
  return (static_cast<size_t>(lists) + n_out * (n_out + 1) / 2 + 2 * kBatch) * (sizeof(uint64_t) + sizeof(uint32_t));
}

size_t beam_select_workspace_bytes(int groups, int beams, int vocab, int n_out) {
  const size_t lists = static_cast<size_t>(groups) * beams * chunks_of<float>(vocab);  // (bf16 takes fewer)
  return (lists * sizeof(float2) + 15) / 16 * 16 + lists * n_out * sizeof(uint64_t);
}

tg_status launch_beam_select(const void* logits, tg_dtype dt, const float* scores, int groups, int beams,
                             int vocab, int n_out, float* scores_out, int32_t* parent_out,
                             int32_t* token_out, void* workspace, cudaStream_t st) {
  const int chunks = dt == TG_BF16 ? chunks_of<__nv_bfloat16>(vocab) : chunks_of<float>(vocab);
  const size_t lists = static_cast<size_t>(groups) * beams * chunks;
  BeamWork ws;
  ws.sums = static_cast<float2*>(workspace);
  ws.keys = reinterpret_cast<uint64_t*>(static_cast<char*>(workspace) + (lists * sizeof(float2) + 15) / 16 * 16);
  const dim3 grid(static_cast<unsigned>(lists));
  cudaError_t e =
      dt == TG_BF16
          ? launch_pdl(beam_chunk_kernel<__nv_bfloat16>, grid, dim3(kChunkThreads), 0, st,
                       static_cast<const __nv_bfloat16*>(logits), groups * beams, vocab, n_out, chunks, ws)
          : launch_pdl(beam_chunk_kernel<float>, grid, dim3(kChunkThreads), 0, st,
                       static_cast<const float*>(logits), groups * beams, vocab, n_out, chunks, ws);
  if (e != cudaSuccess) return cuda_check(e, "beam chunk launch");
  const size_t smem = merge_smem(beams * chunks, n_out);
  if (smem > 40 * 1024) {  // (48 KB without asking, of which the kernel has some for itself)
    // always the most that any call needs, so that calls of several host threads set the same
    e = cudaFuncSetAttribute(beam_merge_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(merge_smem(TG_MAX_BEAMS * chunks_of<float>(kMaxVocab), kMaxOut)));
    if (e != cudaSuccess) return cuda_check(e, "beam merge shared memory");
  }
  return cuda_check(launch_pdl(beam_merge_kernel, dim3(static_cast<unsigned>(groups)), dim3(kMergeThreads), smem,
                               st, scores, beams, vocab, n_out, chunks, ws, scores_out, parent_out, token_out),
                    "beam merge launch");
}

}  // namespace tg
