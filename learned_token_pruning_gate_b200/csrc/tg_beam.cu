// The best continuations of each group of beams: log-softmax over the vocabulary,
// the beam's score added, and the n best of beams x vocabulary in order.
//
// Within a beam the order of the candidates is the order of the logits, so the
// vocabulary is read once: beam_chunk_kernel takes 8192 logits of one row into
// registers and leaves the chunk's maximum, its sum of exponentials and its n
// best logits, sorted.  beam_merge_kernel, one CTA per group, joins the sums
// into the rows' log-sums in 64 bits and picks the n best of the lists.
//
// Both pick by a threshold: among the largest keys of disjoint sets (a thread's
// logits; a sorted list) the n-th largest is a lower bound on the n-th best
// overall, so only keys not below it are collected (rarely more than 2 n), and
// a collected key's place is the number of larger ones.  Keys are distinct,
// since the index is part of them, so ties go to the lower index and the order
// of collection does not matter.
//
// The scores are compared in 64 bits: beams meet at sums that differ in the last
// places of 32, and a chunk's sum in 32 bits (32 terms per thread, then a tree)
// is off by less than 1e-7 of itself.
#include <cmath>

#include "tg_internal.cuh"

namespace tg {
namespace {

constexpr int kChunkThreads = 256;
constexpr int kPerThread = 32;
constexpr int kChunk = kChunkThreads * kPerThread;  // logits per CTA
constexpr int kMaxOut = 2 * TG_MAX_BEAMS;
// Collected keys: fewer than n threads whose largest is above the threshold, with 32 each, and
// the threshold itself; fewer than n threads with any key, when there is no threshold.
constexpr int kChunkKeys = kMaxOut * kPerThread;
constexpr int kMergeThreads = 1024;
// Likewise: at most n lists of n keys each.
constexpr int kMergeKeys = kMaxOut * kMaxOut;

// What a chunk leaves: per (row, chunk) its maximum and sum, and n keys.
struct BeamWork {
  float2* sums;
  uint64_t* keys;
};

__host__ __device__ inline int chunks_of(int vocab, int vec) { return (vocab + vec - 1 + kChunk - 1) / kChunk; }

// Larger logit first, then the lower token; 0 for what is no candidate.
__device__ __forceinline__ uint64_t logit_key(float x, int token) {
  if (!(x > -INFINITY)) return 0;  // -inf, NaN
  return (static_cast<uint64_t>(order_key(x)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(token));
}

template <typename T>
__global__ void __launch_bounds__(kChunkThreads)
    beam_chunk_kernel(const T* __restrict__ logits, int vocab, int n_out, int chunks, BeamWork ws) {
  constexpr int kVec = 16 / static_cast<int>(sizeof(T));
  constexpr int kVecs = kPerThread / kVec;
  __shared__ __align__(16) uint64_t heads[kChunkThreads];
  __shared__ __align__(16) uint64_t found[kChunkKeys];
  __shared__ uint64_t floor_key;
  __shared__ int n_found;
  __shared__ float red[kChunkThreads / 32];
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / chunks;
  const int chunk = static_cast<int>(blockIdx.x - row * chunks);
  // A row may start anywhere: its 16-byte pieces begin at the boundary at or before it, `lead` tokens early.
  const T* r = logits + row * vocab;
  const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(r) & 15u) / sizeof(T));
  float x[kPerThread];
  const int t0 = chunk * kChunk - lead;  // token of the chunk's first element
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int t = t0 + (i * kChunkThreads + tid) * kVec;
    if (t >= 0 && t + kVec <= vocab) {
      const uint4 u = __ldcs(reinterpret_cast<const uint4*>(r + t));
      if constexpr (sizeof(T) == 4) {
        x[i * kVec] = __uint_as_float(u.x);
        x[i * kVec + 1] = __uint_as_float(u.y);
        x[i * kVec + 2] = __uint_as_float(u.z);
        x[i * kVec + 3] = __uint_as_float(u.w);
      } else {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[i * kVec + 2 * e] = __uint_as_float(w[e] << 16);
          x[i * kVec + 2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e)
        x[i * kVec + e] = t + e >= 0 && t + e < vocab ? static_cast<float>(r[t + e]) : -INFINITY;
    }
  }
  auto token = [&](int e) { return t0 + ((e / kVec) * kChunkThreads + tid) * kVec + e % kVec; };

  // the chunk's maximum; the thread's largest key
  float m = x[0];
  int at = 0;
#pragma unroll
  for (int e = 1; e < kPerThread; ++e)
    if (x[e] > m || m != m) {
      m = x[e];
      at = e;
    }
  // (the scan above goes up in e, and the token goes up with e, so equal logits keep the lower one)
  uint64_t best = 0;
#pragma unroll
  for (int e = 0; e < kPerThread; ++e)
    if (e == at) best = logit_key(m, token(e));
  heads[tid] = best;
  float top = m == m ? m : -INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) red[warp] = top;
  if (tid == 0) {
    floor_key = 1;
    n_found = 0;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kChunkThreads / 32; ++w) top = fmaxf(top, red[w]);
  // sum of exponentials; NaN and +inf make it NaN, an empty chunk leaves 0
  float s = 0.0f;
  const float shift = top == -INFINITY ? 0.0f : top;
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) s += exp2_approx((x[e] - shift) * 1.4426950408889634f);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  // the n-th largest of the threads' keys is the floor
  if (best) {
    int above = 0;
#pragma unroll 8
    for (int j = 0; j < kChunkThreads; ++j) above += heads[j] > best;
    if (above == n_out - 1) floor_key = best;
  }
  __syncthreads();
  if (lane == 0) red[warp] = s;
  const uint64_t fl = floor_key;
  if (best >= fl) {
#pragma unroll
    for (int e = 0; e < kPerThread; ++e) {
      const uint64_t key = logit_key(x[e], token(e));
      if (key >= fl) found[atomicAdd(&n_found, 1)] = key;
    }
  }
  __syncthreads();
  const int n = n_found;
  uint64_t* out = ws.keys + (row * chunks + chunk) * n_out;
  for (int i = tid; i < n; i += kChunkThreads) {
    const uint64_t key = found[i];
    int above = 0;
    for (int j = 0; j < n; ++j) above += found[j] > key;
    if (above < n_out) out[above] = key;
  }
  for (int i = n + tid; i < n_out; i += kChunkThreads) out[i] = 0;
  if (tid == 0) {
    float total = 0.0f;
#pragma unroll
    for (int w = 0; w < kChunkThreads / 32; ++w) total += red[w];
    ws.sums[row * chunks + chunk] = make_float2(top, total);
  }
}

// A candidate of the group: larger score first, then the lower place in beams x vocabulary.
struct Cand {
  uint64_t score;  // order-preserving, 0 for none
  uint32_t place;
};
__device__ __forceinline__ bool before(const Cand& a, const Cand& b) {
  return a.score > b.score || (a.score == b.score && a.place < b.place);
}
__device__ __forceinline__ uint64_t order_key64(double x) {
  if (!(fabs(x) < INFINITY)) return 0;  // not finite: no candidate
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));  // -0 becomes +0
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double from_order_key64(uint64_t k) {
  return __longlong_as_double(static_cast<long long>((k >> 63) ? (k & 0x7FFFFFFFFFFFFFFFull) : ~k));
}
__device__ __forceinline__ float logit_of(uint64_t key) {
  const uint32_t k = static_cast<uint32_t>(key >> 32);
  return __uint_as_float((k >> 31) ? (k & 0x7FFFFFFFu) : ~k);
}

__global__ void __launch_bounds__(kMergeThreads)
    beam_merge_kernel(const float* __restrict__ scores, int beams, int vocab, int n_out, int chunks,
                      BeamWork ws, float* __restrict__ scores_out, int32_t* __restrict__ parent_out,
                      int32_t* __restrict__ token_out) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int lists = beams * chunks;
  uint64_t* const head_score = reinterpret_cast<uint64_t*>(smem);          // [lists]
  uint64_t* const found_score = head_score + lists;                        // [kMergeKeys]
  uint32_t* const head_place = reinterpret_cast<uint32_t*>(found_score + kMergeKeys);  // [lists]
  uint32_t* const found_place = head_place + lists;                        // [kMergeKeys]
  __shared__ double log_sum[TG_MAX_BEAMS];
  __shared__ Cand fl;
  __shared__ int n_found;
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * beams;
  if (tid == 0) {
    fl.score = 1;
    fl.place = 0xFFFFFFFFu;
    n_found = 0;
  }
  // a warp per beam: log of the row's sum of exponentials
  if ((tid >> 5) < beams) {
    const float2* part = ws.sums + (row0 + (tid >> 5)) * chunks;
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
    if (lane == 0) log_sum[tid >> 5] = static_cast<double>(top) + log(s);
  }
  __syncthreads();
  auto cand = [&](int list, int i) {
    const int beam = list / chunks;
    const uint64_t key = ws.keys[(row0 * chunks + list) * n_out + i];
    Cand c = {0, 0};
    if (key) {
      const uint32_t token = 0xFFFFFFFFu - static_cast<uint32_t>(key);
      c.score = order_key64(static_cast<double>(scores[row0 + beam]) + (static_cast<double>(logit_of(key)) - log_sum[beam]));
      c.place = static_cast<uint32_t>(beam) * static_cast<uint32_t>(vocab) + token;
    }
    return c;
  };
  for (int l = tid; l < lists; l += kMergeThreads) {
    const Cand c = cand(l, 0);
    head_score[l] = c.score;
    head_place[l] = c.place;
  }
  __syncthreads();
  for (int l = tid; l < lists; l += kMergeThreads) {
    const Cand c = {head_score[l], head_place[l]};
    if (!c.score) continue;
    int above = 0;
    for (int j = 0; j < lists; ++j) above += before(Cand{head_score[j], head_place[j]}, c);
    if (above == n_out - 1) fl = c;
  }
  __syncthreads();
  const Cand limit = fl;
  for (int i = tid; i < lists * n_out; i += kMergeThreads) {
    const int l = i / n_out;
    const Cand h = {head_score[l], head_place[l]};
    if (!h.score || before(limit, h)) continue;  // nothing of this list reaches the floor
    const Cand c = cand(l, i - l * n_out);
    if (!c.score || before(limit, c)) continue;
    const int at = atomicAdd(&n_found, 1);
    found_score[at] = c.score;
    found_place[at] = c.place;
  }
  __syncthreads();
  const int n = n_found;
  const int64_t out = static_cast<int64_t>(blockIdx.x) * n_out;
  for (int i = tid; i < n; i += kMergeThreads) {
    const Cand c = {found_score[i], found_place[i]};
    int above = 0;
    for (int j = 0; j < n; ++j) above += before(Cand{found_score[j], found_place[j]}, c);
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

// The chunks of a row at the wider of the two element counts per 16 bytes, for either dtype.
int max_chunks(int vocab) { return chunks_of(vocab, 8); }

}  // namespace

size_t beam_select_workspace_bytes(int groups, int beams, int vocab, int n_out) {
  const size_t lists = static_cast<size_t>(groups) * beams * max_chunks(vocab);
  return (lists * sizeof(float2) + 15) / 16 * 16 + lists * n_out * sizeof(uint64_t);
}

tg_status launch_beam_select(const void* logits, tg_dtype dt, const float* scores, int groups, int beams,
                             int vocab, int n_out, float* scores_out, int32_t* parent_out,
                             int32_t* token_out, void* workspace, cudaStream_t st) {
  const int chunks = max_chunks(vocab);
  const size_t lists = static_cast<size_t>(groups) * beams * chunks;
  BeamWork ws;
  ws.sums = static_cast<float2*>(workspace);
  ws.keys = reinterpret_cast<uint64_t*>(static_cast<char*>(workspace) + (lists * sizeof(float2) + 15) / 16 * 16);
  const dim3 grid(static_cast<unsigned>(lists));
  cudaError_t e =
      dt == TG_BF16
          ? launch_pdl(beam_chunk_kernel<__nv_bfloat16>, grid, dim3(kChunkThreads), 0, st,
                       static_cast<const __nv_bfloat16*>(logits), vocab, n_out, chunks, ws)
          : launch_pdl(beam_chunk_kernel<float>, grid, dim3(kChunkThreads), 0, st,
                       static_cast<const float*>(logits), vocab, n_out, chunks, ws);
  if (e != cudaSuccess) return cuda_check(e, "beam chunk launch");
  const size_t smem = (static_cast<size_t>(beams) * chunks + kMergeKeys) * (sizeof(uint64_t) + sizeof(uint32_t));
  e = cudaFuncSetAttribute(beam_merge_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return cuda_check(e, "beam merge shared memory");
  return cuda_check(launch_pdl(beam_merge_kernel, dim3(static_cast<unsigned>(groups)), dim3(kMergeThreads), smem,
                               st, scores, beams, vocab, n_out, chunks, ws, scores_out, parent_out, token_out),
                    "beam merge launch");
}

}  // namespace tg
