// Gated attention of one new token per sequence over a paged cache:
//   logit_j = q . k_j / (sqrt(d) tau_h) + g_h l_j,   out = softmax(logit) v
#include <cmath>

#include "tg_internal.cuh"

namespace tg {
namespace {

constexpr int kPagedThreads = 256;
constexpr int kPagedWarps = kPagedThreads / 32;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// One CTA per (sequence, query head), a warp per key.
template <typename T, int D>
__global__ void __launch_bounds__(kPagedThreads) paged_attn_kernel(const PagedAttnArgs a) {
  constexpr int kPer = D / 32;
  __shared__ float part_m[kPagedWarps], part_l[kPagedWarps], part_o[kPagedWarps][D];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.x, b = blockIdx.y;
  const int hk = h / (a.hq / a.hkv);
  const int64_t most = static_cast<int64_t>(a.max_pages) << a.page_shift;
  int len = a.lens[b];
  bool bad = len < 0 || len > most;
  len = len < 0 ? 0 : len > most ? static_cast<int>(most) : len;
  const T* q = static_cast<const T*>(a.q) + (static_cast<int64_t>(b) * a.hq + h) * D + lane * kPer;
  float qx[kPer], o[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    qx[e] = to_f32(q[e]);
    o[e] = 0.0f;
  }
  // Natural units: log2(e) times a gate of the lowest fp32 value would be infinite.
  constexpr float kLog2e = 1.4426950408889634f;
  const float scale = 1.0f / (sqrtf(static_cast<float>(D)) * a.temp[h]);
  const float gain = a.gain[h];
  float m = -INFINITY, l = 0.0f;
  const int page = 1 << a.page_shift;
  for (int j = warp; j < len; j += kPagedWarps) {
    const int p = a.table[static_cast<int64_t>(b) * a.max_pages + (j >> a.page_shift)];
    if (p < 0 || p >= a.n_pages) {
      bad = true;
      continue;
    }
    const float ls = a.logsig_pages ? a.logsig_pages[static_cast<int64_t>(p) * page + (j & (page - 1))] : 0.0f;
    if (ls == -INFINITY) continue;
    const int64_t at = ((static_cast<int64_t>(p) * a.hkv + hk) * page + (j & (page - 1))) * D + lane * kPer;
    const T* k = static_cast<const T*>(a.k_pages) + at;
    const T* v = static_cast<const T*>(a.v_pages) + at;
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) s = fmaf(qx[e], to_f32(k[e]), s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s = fmaf(s, scale, gain * ls);
    if (s == -INFINITY) continue;  // a gain above 1 on such a gate
    const float m2 = fmaxf(m, s), c = exp2f((m - m2) * kLog2e), w = exp2f((s - m2) * kLog2e);
    m = m2;
    l = l * c + w;
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[e] = fmaf(w, to_f32(v[e]), o[e] * c);
  }
  if (lane == 0) {
    part_m[warp] = m;
    part_l[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) part_o[warp][lane * kPer + e] = o[e];
  __syncthreads();
  float top = -INFINITY, total = 0.0f;
  for (int w = 0; w < kPagedWarps; ++w) top = fmaxf(top, part_m[w]);
  const float shift = top == -INFINITY ? 0.0f : top;
  for (int w = 0; w < kPagedWarps; ++w) total += part_l[w] * exp2f((part_m[w] - shift) * 1.4426950408889634f);
  T* out = static_cast<T*>(a.out) + (static_cast<int64_t>(b) * a.hq + h) * D;
  for (int d = threadIdx.x; d < D; d += kPagedThreads) {
    float x = 0.0f;
    for (int w = 0; w < kPagedWarps; ++w) x = fmaf(part_o[w][d], exp2f((part_m[w] - shift) * 1.4426950408889634f), x);
    put(out + d, total != 0.0f ? x / total : 0.0f);
  }
  if (threadIdx.x == 0 && a.lse)
    a.lse[static_cast<int64_t>(h) * a.batch + b] = top + logf(total);
  if (bad && lane == 0) atomicOr(a.status, kDevPageIndex);
}

template <typename T>
cudaError_t launch_paged_t(const PagedAttnArgs& a, int head_dim, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.hq), static_cast<unsigned>(a.batch));
  return head_dim == 128 ? launch_pdl(paged_attn_kernel<T, 128>, grid, dim3(kPagedThreads), 0, st, a)
                         : launch_pdl(paged_attn_kernel<T, 64>, grid, dim3(kPagedThreads), 0, st, a);
}

}  // namespace

size_t paged_attention_workspace_bytes(tg_dtype, int, int, int, int) { return 0; }

tg_status launch_paged_attention(const PagedAttnArgs& a, tg_dtype dt, int head_dim, void*, cudaStream_t st) {
  return cuda_check(dt == TG_BF16 ? launch_paged_t<__nv_bfloat16>(a, head_dim, st)
                                  : launch_paged_t<float>(a, head_dim, st),
                    "paged attention launch");
}

}  // namespace tg
