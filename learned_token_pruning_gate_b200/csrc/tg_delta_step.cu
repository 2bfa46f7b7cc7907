// One token of the gated delta rule per sequence (see tg_delta.cu for the rule):
//   S' = alpha S + beta (v - alpha S k^) k^^T,   o = S' q^
// Rows of S are independent: row i needs only (S k)_i, (S q)_i and v_i.  With
//   c_i = beta (v_i - alpha (S k^)_i),   o_i = alpha (S q^)_i + c_i (k^ . q^)
// both products are taken of the old row, so a row is read once, kept in
// registers, and written once.
//
// Memory bound: 8 d^2 bytes of state per head against 7 d^2 flop.  Eight lanes
// share a row (d / 8 columns each, in 16-byte pieces 128 bytes apart), a warp
// holds four rows at a time, and the five dot products of a row (S k, S q,
// |k|^2, |q|^2, k . q) end in three shuffles each; there is no shared memory and
// no barrier.  A CTA takes 32 rows of one head, so that a single sequence of
// 16 heads already spreads over 64 CTAs at head_dim 128.  48 sequences of 32 heads
// of 128 (203 MB) take 31.4 us, the copy rate; one sequence of 16 heads 2.1 us.
#include <cmath>

#include "tg_internal.cuh"

namespace tg {
namespace {

constexpr int kStepThreads = 256;
constexpr int kStepRows = kStepThreads / 8;  // state rows per CTA

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ float dot4(float4 a, float4 b, float s) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, s))));
}
// sum over the eight lanes of a row
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <typename T, int D>
__global__ void __launch_bounds__(kStepThreads)
    delta_step_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                      const float* __restrict__ log_alpha, const float* __restrict__ beta, int heads,
                      float eps, float q_scale, const float* state_in, int n_states,
                      const int32_t* __restrict__ parent, float* state_out, T* __restrict__ out,
                      uint32_t* status) {
  constexpr int kSlices = D / kStepRows;
  constexpr int kVec = D / 32;  // 16-byte pieces of a row per lane
  grid_dep_wait();
  grid_dep_launch();
  const int slice = blockIdx.x % kSlices;
  const int64_t bh = blockIdx.x / kSlices;
  const int b = static_cast<int>(bh / heads), h = static_cast<int>(bh - static_cast<int64_t>(b) * heads);
  const int sub = threadIdx.x & 7;
  const int row = slice * kStepRows + (threadIdx.x >> 3);
  int from = parent ? parent[b] : b;
  if (from < -1 || from >= n_states) {
    if (threadIdx.x == 0) atomicOr(status, kDevPageIndex);
    from = -1;
  }
  float4 s[kVec], kx[kVec], qx[kVec];
  const int64_t at = (static_cast<int64_t>(from) * heads + h) * D * D + row * D + sub * 4;
#pragma unroll
  for (int i = 0; i < kVec; ++i)
    s[i] = from >= 0 ? load4(state_in + at + i * 32) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    kx[i] = load4(k + bh * D + sub * 4 + i * 32);
    qx[i] = load4(q + bh * D + sub * 4 + i * 32);
  }
  const float alpha = expf(log_alpha[bh]), be = beta[bh];
  const float vx = static_cast<float>(v[bh * D + row]);
  float sk = 0.0f, sq = 0.0f, kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    kk = dot4(kx[i], kx[i], kk);
    qq = dot4(qx[i], qx[i], qq);
    kq = dot4(kx[i], qx[i], kq);
    sk = dot4(s[i], kx[i], sk);
    sq = dot4(s[i], qx[i], sq);
  }
  kk = row_sum(kk);
  qq = row_sum(qq);
  kq = row_sum(kq);
  sk = row_sum(sk);
  sq = row_sum(sq);
  const float ik = 1.0f / sqrtf(kk + eps), iq = q_scale / sqrtf(qq + eps);
  const float c = be * (vx - alpha * (sk * ik));
  const float ck = c * ik;
  float* dst = state_out + (bh * D + row) * D + sub * 4;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const float4 n = make_float4(fmaf(ck, kx[i].x, alpha * s[i].x), fmaf(ck, kx[i].y, alpha * s[i].y),
                                 fmaf(ck, kx[i].z, alpha * s[i].z), fmaf(ck, kx[i].w, alpha * s[i].w));
    *reinterpret_cast<float4*>(dst + i * 32) = n;
  }
  if (sub == 0) store1(out + bh * D + row, fmaf(ck, kq, alpha * sq) * iq);
}

template <typename T, int D>
tg_status launch_step_t(const void* q, const void* k, const void* v, const float* log_alpha,
                        const float* beta, int batch, int heads, float eps, const float* state_in,
                        int n_states, const int32_t* parent, float* state_out, void* out,
                        uint32_t* status, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(batch) * heads * (D / kStepRows)));
  return cuda_check(launch_pdl(delta_step_kernel<T, D>, grid, dim3(kStepThreads), 0, st,
                               static_cast<const T*>(q), static_cast<const T*>(k),
                               static_cast<const T*>(v), log_alpha, beta, heads, eps,
                               1.0f / std::sqrt(static_cast<float>(D)), state_in, n_states, parent,
                               state_out, static_cast<T*>(out), status),
                    "delta step launch");
}

}  // namespace

tg_status launch_delta_step(const void* q, const void* k, const void* v, tg_dtype dt,
                            const float* log_alpha, const float* beta, int batch, int heads,
                            int head_dim, float eps, const float* state_in, int n_states,
                            const int32_t* parent, float* state_out, void* out, uint32_t* status,
                            cudaStream_t st) {
  if (dt == TG_BF16)
    return head_dim == 128
               ? launch_step_t<__nv_bfloat16, 128>(q, k, v, log_alpha, beta, batch, heads, eps, state_in,
                                                   n_states, parent, state_out, out, status, st)
               : launch_step_t<__nv_bfloat16, 64>(q, k, v, log_alpha, beta, batch, heads, eps, state_in,
                                                  n_states, parent, state_out, out, status, st);
  return head_dim == 128 ? launch_step_t<float, 128>(q, k, v, log_alpha, beta, batch, heads, eps, state_in,
                                                     n_states, parent, state_out, out, status, st)
                         : launch_step_t<float, 64>(q, k, v, log_alpha, beta, batch, heads, eps, state_in,
                                                    n_states, parent, state_out, out, status, st);
}

}  // namespace tg
