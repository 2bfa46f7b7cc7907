// Gated attention of one new token per sequence over a paged cache:
//   logit_j = q . k_j / (sqrt(d) tau_h) + g_h l_j,   out = softmax(logit) v
//
// Every cached row is read once and used by the few query heads that share it, so
// the call is bound by HBM (2 flop per byte and query head of a group), and what
// matters is that all SMs read all the time, whatever the lengths.
//
// Work: a unit is (sequence, kv head, block of its query heads), cut into tiles of
// 64 keys.  The tiles of all units form one list, and every CTA takes an equal run
// of it, computed from the lengths on the device.  A CTA that holds a unit whole
// writes its output; a unit that several CTAs share is joined from their partial
// sums (running maximum, sum, weighted v) by the last of them to arrive, in the
// order of the list, so the result does not depend on the schedule.
//
// Within a tile a warp takes 16 keys, which lie in one page.  There is no shared
// memory on the way: rows go from HBM to registers in 16-byte pieces, the next
// 16 keys' K is requested as soon as this one's products are issued, and V
// likewise, so a warp has 4 to 8 KB in flight at all times.
//
// bf16: the legacy m16n8k16 tensor instruction with keys as its 16 rows and query
// heads as its 8 columns: S^T = K Q^T, O^T = V^T P.  Its fragments can be had
// without any exchange: the contraction over d may run in any order, so the 8
// consecutive elements a lane loads of a row serve two k-steps as they are (Q is
// loaded the same way); for V^T a lane loads the same 8 columns of the four keys
// it needs and interleaves them with byte permutes; S^T becomes the B operand of
// the second product by one transpose instruction per 8 keys.  tcgen05 would need
// the tiles in shared memory and 128 rows of query heads; at 8 columns its rate
// is not what bounds this call.
// fp32: the same schedule on the CUDA cores, eight lanes to a key.
//
// Maxima move lazily: a warp keeps its reference maximum until a logit exceeds it
// by more than 8, so that weights stay below e^8 and the accumulators are rarely
// rescaled.  Logits are held in natural units: log2(e) times a gate of the lowest
// fp32 value would be infinite.
#include <cmath>

#include "tg_internal.cuh"

namespace tg {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 16 * kWarps;  // keys of a tile, 16 per warp
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.0f;  // how far a logit may exceed the reference maximum

// Heads of a unit: at most 16 (two column tiles) in bf16, 4 in fp32.
__host__ __device__ constexpr int heads_per_unit(bool bf16, int group) {
  return bf16 ? (group <= 8 ? 8 : 16) : (group <= 1 ? 1 : group <= 2 ? 2 : 4);
}

// CTAs per SM, as many as the accumulators and the rows in flight leave registers for.
__host__ __device__ constexpr int ctas_per_sm(bool bf16, int heads, int head_dim) {
  return bf16 ? (heads == 8 ? 3 : 2) : (heads == 1 || (heads == 2 && head_dim == 64) ? 3 : 2);
}

struct Plan {
  PagedAttnArgs a;
  int32_t group;       // query heads per kv head
  int32_t blocks;      // blocks of query heads per kv head
  int32_t units;       // units per sequence: hkv * blocks
  int32_t* counters;   // [batch * units], or null: no unit is shared
  float* partial;      // [2 * grid][heads][d + 2]
};

// 16 bytes of a row, not kept in L1 (each is used once).
__device__ __forceinline__ uint4 load_row16(const void* p) {
  uint4 x;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "l"(p));
  return x;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit elements held as a fragment.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// exp(x - m) for a reference m that may still be -inf (then only x = -inf comes here).
__device__ __forceinline__ float weight(float x, float m) {
  return exp2_approx((x - (m == -INFINITY ? 0.0f : m)) * kLog2e);
}

// A warp's 16 keys of one page: where they are, how many count, their log-gates.
struct Keys {
  int64_t row;   // first row: (page * hkv + kv head) * page size + offset
  int32_t n;     // keys below the length; 0 when the page is not to be read
  int64_t gate;  // first log-gate
};

__device__ __forceinline__ Keys locate(const Plan& p, int b, int hk, int len, int key, bool* bad) {
  Keys k = {0, 0, 0};
  if (key >= len) return k;
  const int page = p.a.table[static_cast<int64_t>(b) * p.a.max_pages + (key >> p.a.page_shift)];
  if (page < 0 || page >= p.a.n_pages) {
    *bad = true;
    return k;
  }
  const int off = key & ((1 << p.a.page_shift) - 1);
  k.row = ((static_cast<int64_t>(page) * p.a.hkv + hk) << p.a.page_shift) + off;
  k.gate = (static_cast<int64_t>(page) << p.a.page_shift) + off;
  k.n = min(16, len - key);
  return k;
}

// ---- bf16: a warp's share of a segment -----------------------------------------------------------
// Columns of the instruction are query heads.  The weights enter the second product as the sum
// of two bf16 numbers (the weight rounded, and what that cut off), so that the output is off by
// little more than its own rounding; the extra products cost no memory time.
template <int D, int NT>
struct CoreBf16 {
  static constexpr int kHeads = 8 * NT;
  static constexpr int kKv = D / 32;  // 16-byte pieces per lane and row half, for K and for Q
  static constexpr int kVv = D / 64;  // 16-byte pieces per lane and key, for V
  static constexpr int kMinCtas = ctas_per_sm(true, kHeads, D);

  static __device__ __forceinline__ void run(const Plan& p, int b, int hk, int h0, int nh, int key0, int key_end,
                                             int len, float* part_m, float* part_l, float* part_o, bool* bad) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(p.a.k_pages);
    const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(p.a.v_pages);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);

    Keys at = locate(p, b, hk, min(len, key_end), key0 + warp * 16, bad);
    uint4 k[2][kKv], v[4][kVv];
    float gate[2];
    auto load_k = [&](const Keys& s) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const bool in = g + 8 * r < s.n;
        const __nv_bfloat16* src = kp + (s.row + g + 8 * r) * D + t * 8;
#pragma unroll
        for (int c = 0; c < kKv; ++c) k[r][c] = in ? load_row16(src + c * 32) : zero;
        gate[r] = !in ? -INFINITY : p.a.logsig_pages ? p.a.logsig_pages[s.gate + g + 8 * r] : 0.0f;
      }
    };
    auto load_v = [&](const Keys& s) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = 2 * t + (i & 1) + 8 * (i >> 1);
        const __nv_bfloat16* src = vp + (s.row + key) * D + g * 8;
#pragma unroll
        for (int c = 0; c < kVv; ++c) v[i][c] = key < s.n ? load_row16(src + c * 64) : zero;
      }
    };
    load_k(at);
    load_v(at);

    // the query rows as B fragments: column g of tile n is head h0 + 8 n + g
    uint4 q[NT][kKv];
    float scale[NT][2], gain[NT][2];
    const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(p.a.q) + static_cast<int64_t>(b) * p.a.hq * D;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int col = 8 * n + g;
#pragma unroll
      for (int c = 0; c < kKv; ++c)
        q[n][c] = col < nh ? load_row16(qp + static_cast<int64_t>(h0 + col) * D + t * 8 + c * 32) : zero;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = 8 * n + 2 * t + e;
        scale[n][e] = h < nh ? 1.0f / (sqrtf(static_cast<float>(D)) * p.a.temp[h0 + h]) : 0.0f;
        gain[n][e] = h < nh ? p.a.gain[h0 + h] : 0.0f;
      }
    }
    float m[NT][2], l[NT][2], o[NT][D / 16][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[n][e] = -INFINITY;
        l[n][e] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][i][e] = 0.0f;
    }

    for (int key = key0 + warp * 16; key < key_end; key += kTile) {
      const Keys next = locate(p, b, hk, min(len, key_end), key + kTile, bad);
      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
#pragma unroll
        for (int c = 0; c < kKv; ++c) {
          mma16816(s[n], k[0][c].x, k[1][c].x, k[0][c].y, k[1][c].y, q[n][c].x, q[n][c].y);
          mma16816(s[n], k[0][c].z, k[1][c].z, k[0][c].w, k[1][c].w, q[n][c].z, q[n][c].w);
        }
      }
      const float gate0 = gate[0], gate1 = gate[1];
      load_k(next);
      // a token whose log-gate is -inf has no weight whatever its v holds: 0 x NaN must not reach the sums
      const bool out0 = gate0 == -INFINITY, out1 = gate1 == -INFINITY;
      const uint32_t gone0 = __ballot_sync(0xffffffffu, out0), gone1 = __ballot_sync(0xffffffffu, out1);
      if (gone0 | gone1) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (((i >> 1 ? gone1 : gone0) >> (4 * (2 * t + (i & 1)))) & 1u)
#pragma unroll
            for (int c = 0; c < kVv; ++c) v[i][c] = zero;
      }
      bool over = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s[n][e] = out0 ? -INFINITY : fmaf(s[n][e], scale[n][e], gain[n][e] * gate0);
          s[n][2 + e] = out1 ? -INFINITY : fmaf(s[n][2 + e], scale[n][e], gain[n][e] * gate1);
          over |= fmaxf(s[n][e], s[n][2 + e]) > m[n][e] + kSlack;
        }
      if (__any_sync(0xffffffffu, over)) {  // (a reference of -inf is exceeded by any logit)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(m[n][e], fmaxf(s[n][e], s[n][2 + e]));
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
            const float c = weight(m[n][e], x);
            m[n][e] = x;
            l[n][e] *= c;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              o[n][i][e] *= c;
              o[n][i][2 + e] *= c;
            }
          }
      }
      uint32_t pb[NT][2], pc[NT][2];  // the rounded weights, what they lack
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float w0 = weight(s[n][2 * r], m[n][0]), w1 = weight(s[n][2 * r + 1], m[n][1]);
          const __nv_bfloat162 hi = __floats2bfloat162_rn(w0, w1);
          const float2 f = __bfloat1622float2(hi);
          const __nv_bfloat162 lo = __floats2bfloat162_rn(w0 - f.x, w1 - f.y);
          l[n][0] += w0;
          l[n][1] += w1;
          uint32_t bits;
          memcpy(&bits, &hi, 4);
          pb[n][r] = transpose8x8(bits);
          memcpy(&bits, &lo, 4);
          pc[n][r] = transpose8x8(bits);
        }
      }
#pragma unroll
      for (int c = 0; c < kVv; ++c) {
        const uint32_t* v0 = &v[0][c].x;
        const uint32_t* v1 = &v[1][c].x;
        const uint32_t* v2 = &v[2][c].x;
        const uint32_t* v3 = &v[3][c].x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // rows g and g + 8 of the instruction are columns c * 64 + g * 8 + 2 i and the next
          const uint32_t a0 = __byte_perm(v0[i], v1[i], 0x5410), a1 = __byte_perm(v0[i], v1[i], 0x7632);
          const uint32_t a2 = __byte_perm(v2[i], v3[i], 0x5410), a3 = __byte_perm(v2[i], v3[i], 0x7632);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma16816(o[n][c * 4 + i], a0, a1, a2, a3, pb[n][0], pb[n][1]);
            mma16816(o[n][c * 4 + i], a0, a1, a2, a3, pc[n][0], pc[n][1]);
          }
        }
      }
      load_v(next);
    }

    // the warp's sums, over the eight lanes of a column
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], w);
        const int h = 8 * n + 2 * t + e;
        if (h >= nh) continue;
        if (g == 0) {
          part_m[warp * kHeads + h] = m[n][e];
          part_l[warp * kHeads + h] = l[n][e];
        }
        float* dst = part_o + (warp * kHeads + h) * D + g * 8;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          dst[(i >> 2) * 64 + 2 * (i & 3)] = o[n][i][e];
          dst[(i >> 2) * 64 + 2 * (i & 3) + 1] = o[n][i][2 + e];
        }
      }
  }
};

// ---- fp32: eight lanes to a key, each with D / 8 of its columns ----------------------------------
template <int D, int NH>
struct CoreFp32 {
  static constexpr int kHeads = NH;
  static constexpr int kVec = D / 32;  // 16-byte pieces per lane and row
  static constexpr int kMinCtas = ctas_per_sm(false, NH, D);

  static __device__ __forceinline__ float4 load4(const float* p) {
    const uint4 x = load_row16(p);
    return make_float4(__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w));
  }

  static __device__ __forceinline__ void run(const Plan& p, int b, int hk, int h0, int nh, int key0, int key_end,
                                             int len, float* part_m, float* part_l, float* part_o, bool* bad) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane & 7, kg = lane >> 3;  // the lane's columns; its key of four
    const float* kp = static_cast<const float*>(p.a.k_pages);
    const float* vp = static_cast<const float*>(p.a.v_pages);
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float4 k[2][kVec], v[2][kVec];
    float gate[2];
    // a step is 8 keys: half of the warp's 16, keys kg and kg + 4 of it on this lane
    auto load_k = [&](const Keys& s, int half) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int key = half * 8 + r * 4 + kg;
        const bool in = key < s.n;
#pragma unroll
        for (int c = 0; c < kVec; ++c) k[r][c] = in ? load4(kp + (s.row + key) * D + sub * 4 + c * 32) : zero;
        gate[r] = !in ? -INFINITY : p.a.logsig_pages ? p.a.logsig_pages[s.gate + key] : 0.0f;
      }
    };
    auto load_v = [&](const Keys& s, int half) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int key = half * 8 + r * 4 + kg;
#pragma unroll
        for (int c = 0; c < kVec; ++c)
          v[r][c] = key < s.n ? load4(vp + (s.row + key) * D + sub * 4 + c * 32) : zero;
      }
    };
    Keys at = locate(p, b, hk, min(len, key_end), key0 + warp * 16, bad);
    load_k(at, 0);
    load_v(at, 0);
    float4 q[NH][kVec], o[NH][kVec];
    float scale[NH], gain[NH], m[NH], l[NH];
    const float* qp = static_cast<const float*>(p.a.q) + (static_cast<int64_t>(b) * p.a.hq + h0) * D;
#pragma unroll
    for (int h = 0; h < NH; ++h) {
#pragma unroll
      for (int c = 0; c < kVec; ++c) {
        q[h][c] = h < nh ? load4(qp + h * D + sub * 4 + c * 32) : zero;
        o[h][c] = zero;
      }
      scale[h] = h < nh ? 1.0f / (sqrtf(static_cast<float>(D)) * p.a.temp[h0 + h]) : 0.0f;
      gain[h] = h < nh ? p.a.gain[h0 + h] : 0.0f;
      m[h] = -INFINITY;
      l[h] = 0.0f;
    }
    for (int key = key0 + warp * 16; key < key_end; key += kTile) {
      const Keys next = locate(p, b, hk, min(len, key_end), key + kTile, bad);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float s[NH][2];
        bool over = false;
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float x = 0.0f;
#pragma unroll
            for (int c = 0; c < kVec; ++c)
              x = fmaf(q[h][c].x, k[r][c].x, fmaf(q[h][c].y, k[r][c].y, fmaf(q[h][c].z, k[r][c].z, fmaf(q[h][c].w, k[r][c].w, x))));
#pragma unroll
            for (int w = 1; w < 8; w <<= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
            s[h][r] = gate[r] == -INFINITY ? -INFINITY : fmaf(x, scale[h], gain[h] * gate[r]);
            over |= s[h][r] > m[h] + kSlack;
          }
        const bool out[2] = {gate[0] == -INFINITY, gate[1] == -INFINITY};
        load_k(half == 0 ? at : next, half ^ 1);
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            const float x = fmaxf(m[h], fmaxf(s[h][0], s[h][1]));
            const float c = weight(m[h], x);
            m[h] = x;
            l[h] *= c;
#pragma unroll
            for (int i = 0; i < kVec; ++i)
              o[h][i] = make_float4(o[h][i].x * c, o[h][i].y * c, o[h][i].z * c, o[h][i].w * c);
          }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (out[r])
#pragma unroll
            for (int c = 0; c < kVec; ++c) v[r][c] = zero;  // 0 x NaN must not reach the sums
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            const float w = weight(s[h][r], m[h]);
            l[h] += w;
#pragma unroll
            for (int c = 0; c < kVec; ++c) {
              o[h][c].x = fmaf(w, v[r][c].x, o[h][c].x);
              o[h][c].y = fmaf(w, v[r][c].y, o[h][c].y);
              o[h][c].z = fmaf(w, v[r][c].z, o[h][c].z);
              o[h][c].w = fmaf(w, v[r][c].w, o[h][c].w);
            }
          }
        }
        load_v(half == 0 ? at : next, half ^ 1);
      }
      at = next;
    }
    // join the four keys' sums of the warp
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      float x = m[h];
#pragma unroll
      for (int w = 8; w < 32; w <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
      const float c = weight(m[h], x);
      float sum = l[h] * c;
#pragma unroll
      for (int w = 8; w < 32; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        float4 y = make_float4(o[h][i].x * c, o[h][i].y * c, o[h][i].z * c, o[h][i].w * c);
#pragma unroll
        for (int w = 8; w < 32; w <<= 1) {
          y.x += __shfl_xor_sync(0xffffffffu, y.x, w);
          y.y += __shfl_xor_sync(0xffffffffu, y.y, w);
          y.z += __shfl_xor_sync(0xffffffffu, y.z, w);
          y.w += __shfl_xor_sync(0xffffffffu, y.w, w);
        }
        if (h < nh && kg == 0) *reinterpret_cast<float4*>(part_o + (warp * NH + h) * D + sub * 4 + i * 32) = y;
      }
      if (h < nh && lane == 0) {
        part_m[warp * NH + h] = x;
        part_l[warp * NH + h] = sum;
      }
    }
  }
};

__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ int checked_length(const Plan& p, int b, bool* bad) {
  const int64_t most = static_cast<int64_t>(p.a.max_pages) << p.a.page_shift;
  const int len = p.a.lens[b];
  if (len >= 0 && len <= most) return len;
  *bad = true;
  return len < 0 ? 0 : static_cast<int>(most);
}

template <typename T, int D, typename Core>
__global__ void __launch_bounds__(kThreads, Core::kMinCtas) paged_attn_kernel(const __grid_constant__ Plan p) {
  constexpr int H = Core::kHeads;
  constexpr int kSlot = H * (D + 2);  // floats of a partial sum: [H][D], then the maxima and the sums
  __shared__ int ends[kMaxSeqs];      // inclusive scan of the sequences' tiles (per unit)
  __shared__ int warp_sums[kWarps];
  __shared__ float part_m[kWarps * H], part_l[kWarps * H];
  __shared__ __align__(16) float part_o[kWarps * H * D];
  __shared__ bool last_to_arrive;
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad = false;

  // tiles of every sequence, scanned: a run of sequences per thread
  const int batch = p.a.batch;
  const int run = (batch + kThreads - 1) / kThreads;
  int sum = 0;
  for (int i = 0; i < run; ++i) {
    const int b = tid * run + i;
    if (b >= batch) break;
    sum += (checked_length(p, b, &bad) + kTile - 1) / kTile;
    ends[b] = sum;
  }
  int scan = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += y;
  }
  if (lane == 31) warp_sums[warp] = scan;
  __syncthreads();
  int before = scan - sum;
  for (int w = 0; w < warp; ++w) before += warp_sums[w];
  for (int i = 0; i < run; ++i) {
    const int b = tid * run + i;
    if (b >= batch) break;
    ends[b] += before;
  }
  __syncthreads();
  const int64_t total = static_cast<int64_t>(ends[batch - 1]) * p.units;
  const int64_t per = p.counters ? (total + gridDim.x - 1) / gridDim.x : 0;

  // the join of kWarps partial sums in shared memory into `out`, or into a slot for the unit's last CTA
  auto finish = [&](int b, int h0, int nh, float* slot) {
    __syncthreads();
    for (int i = tid; i < nh * D; i += kThreads) {
      const int h = i / D, d = i - h * D;
      float top = -INFINITY, l = 0.0f, x = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part_m[w * H + h]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float c = weight(part_m[w * H + h], top);
        l = fmaf(part_l[w * H + h], c, l);
        x = fmaf(part_o[(w * H + h) * D + d], c, x);
      }
      if (slot) {
        slot[i] = x;
        if (d == 0) {
          slot[H * D + h] = top;
          slot[H * D + H + h] = l;
        }
      } else {
        // nothing left of the sequence: 0 and -inf (a sum of nothing is 0, any other holds its reference's weight 1)
        put(static_cast<T*>(p.a.out) + (static_cast<int64_t>(b) * p.a.hq + h0 + h) * D + d, l == 0.0f ? 0.0f : x / l);
        if (d == 0 && p.a.lse) p.a.lse[static_cast<int64_t>(h0 + h) * batch + b] = l == 0.0f ? -INFINITY : top + logf(l);
      }
    }
  };
  auto heads_of = [&](int u, int* hk, int* h0, int* nh) {
    *hk = u / p.blocks;
    const int block = u - *hk * p.blocks;
    *h0 = *hk * p.group + block * H;
    *nh = min(H, p.group - block * H);
  };

  int64_t at = per * blockIdx.x;
  const int64_t end = min(total, at + per);
  int b = 0;
  if (at < end) {
    int hi = batch - 1;  // the first sequence whose tiles reach past `at`
    while (b < hi) {
      const int mid = (b + hi) >> 1;
      if (static_cast<int64_t>(ends[mid]) * p.units > at) hi = mid;
      else b = mid + 1;
    }
  }
  while (at < end) {
    const int first = b > 0 ? ends[b - 1] : 0, tiles = ends[b] - first;
    if (tiles == 0) {
      ++b;
      continue;
    }
    const int64_t in_seq = at - static_cast<int64_t>(first) * p.units;
    const int u = static_cast<int>(in_seq / tiles), j0 = static_cast<int>(in_seq - static_cast<int64_t>(u) * tiles);
    const int n = static_cast<int>(min(static_cast<int64_t>(tiles - j0), end - at));
    int hk, h0, nh;
    heads_of(u, &hk, &h0, &nh);
    const int len = checked_length(p, b, &bad);
    Core::run(p, b, hk, h0, nh, j0 * kTile, (j0 + n) * kTile, len, part_m, part_l, part_o, &bad);
    if (n == tiles) {
      finish(b, h0, nh, nullptr);
    } else {
      // slot 2c + 1: the unit begins in CTA c; slot 2c: it began before
      const int64_t begin = at - j0;
      const int c0 = static_cast<int>(begin / per), c1 = static_cast<int>((begin + tiles - 1) / per);
      finish(b, h0, nh, p.partial + static_cast<int64_t>(2 * blockIdx.x + (j0 == 0)) * kSlot);
      __threadfence();
      __syncthreads();
      int* counter = p.counters + static_cast<int64_t>(b) * p.units + u;
      if (tid == 0) last_to_arrive = atomicAdd(counter, 1) == c1 - c0;
      __syncthreads();
      if (last_to_arrive) {
        __threadfence();
        if (tid == 0) *counter = 0;  // for the next call
        // a warp joins every kWarps-th part, four at a time
        for (int h = 0; h < nh; ++h) {
          constexpr int kPer = D / 32;
          float m = -INFINITY, l = 0.0f, o[kPer] = {};
          for (int c = c0 + warp; c <= c1; c += 4 * kWarps) {
            float pm[4], pl[4], po[4][kPer];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int cc = c + x * kWarps;
              const float* s = p.partial + static_cast<int64_t>(2 * cc + (cc == c0)) * kSlot;
              pm[x] = cc <= c1 ? __ldcg(s + H * D + h) : -INFINITY;
              pl[x] = cc <= c1 ? __ldcg(s + H * D + H + h) : 0.0f;
#pragma unroll
              for (int e = 0; e < kPer; ++e) po[x][e] = cc <= c1 ? __ldcg(s + h * D + lane + 32 * e) : 0.0f;
            }
            const float top = fmaxf(fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])), m);
            const float c_old = weight(m, top);
            m = top;
            l *= c_old;
#pragma unroll
            for (int e = 0; e < kPer; ++e) o[e] *= c_old;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const float w = weight(pm[x], top);
              l = fmaf(pl[x], w, l);
#pragma unroll
              for (int e = 0; e < kPer; ++e) o[e] = fmaf(po[x][e], w, o[e]);
            }
          }
          if (lane == 0) {
            part_m[warp * H + h] = m;
            part_l[warp * H + h] = l;
          }
#pragma unroll
          for (int e = 0; e < kPer; ++e) part_o[(warp * H + h) * D + lane + 32 * e] = o[e];
        }
        finish(b, h0, nh, nullptr);
      }
    }
    __syncthreads();  // the next segment writes the partial sums in shared memory
    at += n;
    if (j0 + n == tiles && u == p.units - 1) ++b;
  }

  // without a workspace: whole units, one after another
  if (!p.counters) {
    const int64_t units = static_cast<int64_t>(batch) * p.units;
    for (int64_t i = blockIdx.x; i < units; i += gridDim.x) {
      const int bb = static_cast<int>(i / p.units);
      int hk, h0, nh;
      heads_of(static_cast<int>(i - static_cast<int64_t>(bb) * p.units), &hk, &h0, &nh);
      const int len = checked_length(p, bb, &bad);
      if (len == 0) continue;
      Core::run(p, bb, hk, h0, nh, 0, (len + kTile - 1) / kTile * kTile, len, part_m, part_l, part_o, &bad);
      finish(bb, h0, nh, nullptr);
      __syncthreads();
    }
  }
  // sequences without tokens are in no run
  for (int i = blockIdx.x; i < batch; i += gridDim.x) {
    if (checked_length(p, i, &bad) != 0) continue;
    for (int x = tid; x < p.a.hq * D; x += kThreads)
      put(static_cast<T*>(p.a.out) + static_cast<int64_t>(i) * p.a.hq * D + x, 0.0f);
    if (p.a.lse)
      for (int h = tid; h < p.a.hq; h += kThreads) p.a.lse[static_cast<int64_t>(h) * batch + i] = -INFINITY;
  }
  if (bad) atomicOr(p.a.status, kDevPageIndex);
}

template <typename T, int D, typename Core>
cudaError_t launch_core(const Plan& p, int grid, cudaStream_t st) {
  return launch_pdl(paged_attn_kernel<T, D, Core>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, st, p);
}

template <int D>
cudaError_t launch_dim(const Plan& p, bool bf16, int heads, int grid, cudaStream_t st) {
  if (bf16)
    return heads == 8 ? launch_core<__nv_bfloat16, D, CoreBf16<D, 1>>(p, grid, st)
                      : launch_core<__nv_bfloat16, D, CoreBf16<D, 2>>(p, grid, st);
  return heads == 1   ? launch_core<float, D, CoreFp32<D, 1>>(p, grid, st)
         : heads == 2 ? launch_core<float, D, CoreFp32<D, 2>>(p, grid, st)
                      : launch_core<float, D, CoreFp32<D, 4>>(p, grid, st);
}

struct Shape {
  int group, heads, blocks, units, grid;
  size_t counter_bytes, slot_bytes;
};

Shape shape_of(bool bf16, int batch, int hq, int hkv, int head_dim) {
  Shape s;
  s.group = hq / hkv;
  s.heads = heads_per_unit(bf16, s.group);
  s.blocks = (s.group + s.heads - 1) / s.heads;
  s.units = hkv * s.blocks;
  s.grid = num_sms() * ctas_per_sm(bf16, s.heads, head_dim);
  s.counter_bytes = (static_cast<size_t>(batch) * s.units * sizeof(int32_t) + 255) / 256 * 256;
  s.slot_bytes = sizeof(float) * s.heads * (head_dim + 2);
  return s;
}

}  // namespace

size_t paged_attention_workspace_bytes(tg_dtype dt, int batch, int hq, int hkv, int head_dim) {
  const Shape s = shape_of(dt == TG_BF16, batch, hq, hkv, head_dim);
  return s.counter_bytes + 2 * s.grid * s.slot_bytes;
}

tg_status launch_paged_attention(const PagedAttnArgs& a, tg_dtype dt, int head_dim, void* workspace,
                                 cudaStream_t st) {
  const bool bf16 = dt == TG_BF16;
  const Shape s = shape_of(bf16, a.batch, a.hq, a.hkv, head_dim);
  Plan p;
  p.a = a;
  p.group = s.group;
  p.blocks = s.blocks;
  p.units = s.units;
  p.counters = static_cast<int32_t*>(workspace);
  p.partial = workspace ? reinterpret_cast<float*>(static_cast<char*>(workspace) + s.counter_bytes) : nullptr;
  return cuda_check(head_dim == 128 ? launch_dim<128>(p, bf16, s.heads, s.grid, st)
                                    : launch_dim<64>(p, bf16, s.heads, s.grid, st),
                    "paged attention launch");
}

}  // namespace tg
