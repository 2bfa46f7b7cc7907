// Gated attention of one new token per sequence over a paged cache:
//   logit_j = q . k_j / (sqrt(d) tau_h) + g_h l_j,   out = softmax(logit) v
//
// Every cached row is read once for the query heads that share it, up to 16 of them
// in bf16 and 4 in fp32 (more read it once per 16 or 4), so the call is bound by HBM
// (2 flop per byte and query head of a group), and what matters is that all SMs read
// all the time, whatever the lengths.
//
// Work: a unit is (sequence, kv head, block of its query heads), cut into tiles of
// 64 keys (128 of bf16 rows of 64 columns).  The tiles of all units form one list,
// and every CTA takes an equal run of it, computed from the lengths on the device.
// A CTA that holds a unit whole writes its output; the partial sums (reference
// maximum, sum, weighted v) of a unit that several CTAs share are joined by a
// second kernel in the order of the list, so the result does not depend on the
// schedule.  Calls of few, short tables need neither list nor second launch: a
// cluster of CTAs takes a unit and joins it through distributed shared memory (see
// cluster_size).  (Joined by the last CTA to arrive instead, one sequence of 256 tokens
// took 8.6 us for 6.9, and one of 4096 with 8 heads to a kv head 23.4 for 8.6: the
// fence, the counter and one SM reading all parts are slower than a dependent
// launch.)
//
// Within a tile a warp takes 16 keys of one page at a time (two such groups where
// rows are short, so that as much is in flight).  There is no shared memory on the
// way: rows go from HBM to registers in 16-byte pieces, the next keys' K is
// requested as soon as this one's products are issued, and V likewise, across unit
// boundaries too, so a warp has 4 to 8 KB in flight at all times.
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
// Measured on the device, bf16, 16 query heads over 8 kv heads of 128: 7 sequences
// of 1151 to 131073 tokens, 227488 in all, 145 us (99% of the copy rate), 16 of 2304
// to 2817 33.6 us (77%).  About 5 us of a call on the list are latency: lengths, table and first
// rows one after another (2.5 us), the last sums and the join; 3 us of one on
// clusters.  32 query heads over 4 of 64, 61 sequences of up to 4353 tokens, 131423 in
// all: 30.6 us (68%).  32 sequences of 2500 tokens with one kv head of 128: 15.8 us for
// 16 query heads (40%: 32 units on clusters of eight, two CTAs an SM of 255 registers),
// 29.7 for 32, which read the rows twice.  fp32, 18 sequences of 2002 tokens, 4 kv heads
// of 128: 27.6 us for 4 or 8 query heads (83%), 32.0 for 16, 49 for 32.
//
// Maxima move lazily: a warp keeps its reference maximum until a logit exceeds it
// by more than 8, so that weights stay below e^8 and the accumulators are rarely
// rescaled.  Logits are held in natural units: log2(e) times a gate of the lowest
// fp32 value would be infinite.
#include <cfloat>
#include <cmath>

#include "tg_internal.cuh"

namespace tg {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxHeads = 512;  // query heads, as the C ABI checks
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kClusterMax = 8;
constexpr float kSlack = 8.0f;  // how far a logit may exceed the reference maximum

// Heads of a unit: at most 16 (two column tiles) in bf16, 4 in fp32.
__host__ __device__ constexpr int heads_per_unit(bool bf16, int group) {
  return bf16 ? (group <= 8 ? 8 : 16) : (group <= 1 ? 1 : group <= 2 ? 2 : 4);
}

// CTAs per SM, as many as the accumulators and the rows in flight leave registers for.
__host__ __device__ constexpr int ctas_per_sm(bool bf16, int heads, int head_dim) {
  return bf16 ? (heads == 8 ? 3 : 2) : (heads == 1 || (heads == 2 && head_dim == 64) ? 3 : 2);
}

// A partial sum: [heads][d], then the heads' maxima and their sums; a multiple of 16 bytes.
__host__ __device__ constexpr int slot_floats(int heads, int head_dim) {
  return heads * head_dim + (2 * heads + 3) / 4 * 4;
}

struct Plan {
  PagedAttnArgs a;
  int32_t group;       // query heads per kv head
  int32_t blocks;      // blocks of query heads per kv head
  int32_t units;       // units per sequence: hkv * blocks
  int2* shares;        // [batch * units] the first and last CTA of a shared unit, {0, -1} otherwise; or null:
                       // every unit is whole
  float* partial;      // [2 * grid] slots
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

// A gate's bias.  Gain times a mask's lowest value may be beyond fp32 where the softmax of the formula
// is not: such tokens among themselves share their weight evenly.  (fminf and fmaxf would drop NaN.  The
// two instructions cost nothing in bf16 and 4% of fp32 with four heads to a kv head; a look at the gates,
// and logits put right only where one is as low, cost 1 to 4% in both.)
__device__ __forceinline__ float bias(float gain, float gate) {
  float x = gain * gate;
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(-FLT_MAX));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(FLT_MAX));
  return x;
}

// A warp's 16 keys of one page: where they are, and how many of them count.
struct Keys {
  int64_t row;   // first row: (page * hkv + kv head) * page size + offset
  int64_t gate;  // first log-gate
  int32_t n;     // keys below the length; 0 when the page is not to be read
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

// ---- bf16: 16 R keys of a warp ---------------------------------------------------------------------
// Columns of the instruction are query heads.  The weights enter the second product as the sum
// of three bf16 numbers (the weight rounded, what that cut off, and what is left of it), which hold
// all 24 bits of a weight, so that the output is a 32-bit evaluation's, rounded once.  With two of
// them 0.2% of the outputs of 16 x 2500 tokens were rounded to the other neighbour, in place of
// 0.05%; the third costs 1% of the time there, 2 to 4% of 61 sequences of 32/4 heads of 64 and up
// to 6% with 16 heads to a kv head.
template <int D, int NT>
struct CoreBf16 {
  static constexpr int kHeads = 8 * NT;
  static constexpr int R = 128 / D;   // groups of 16 keys
  static constexpr int kKeys = 16 * R;
  static constexpr int kSteps = 1;
  static constexpr int kKv = D / 32;  // 16-byte pieces per lane and row half, for K and for Q
  static constexpr int kVv = D / 64;  // 16-byte pieces per lane and key, for V

  uint4 q[NT][kKv], k[R][2][kKv], v[R][4][kVv];
  float gate[R][2], scale[NT][2], gain[NT][2], m[NT][2], l[NT][2], o[NT][D / 16][4];
  float s[R][NT][4];

  static __device__ __forceinline__ int g() { return (threadIdx.x & 31) >> 2; }
  static __device__ __forceinline__ int t() { return threadIdx.x & 3; }

  // the query rows as B fragments: column g of tile n is head h0 + 8 n + g
  __device__ __forceinline__ void load_q(const Plan& p, int b, int h0, int nh) {
    const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(p.a.q) + (static_cast<int64_t>(b) * p.a.hq + h0) * D;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < kKv; ++c)
        q[n][c] = 8 * n + g() < nh ? load_row16(qp + (8 * n + g()) * D + t() * 8 + c * 32) : make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void begin(const float2* heads, int nh) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = 8 * n + 2 * t() + e;
        const float2 x = h < nh ? heads[h] : make_float2(0.0f, 0.0f);
        scale[n][e] = x.x;
        gain[n][e] = x.y;
        m[n][e] = -INFINITY;
        l[n][e] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][i][e] = 0.0f;
    }
  }
  __device__ __forceinline__ void load_k(const Plan& p, const Keys (&keys)[R], int) {
#pragma unroll
    for (int x = 0; x < R; ++x) {
      const Keys& at = keys[x];
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.a.k_pages) + (at.row + g()) * D + t() * 8;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const bool in = g() + 8 * r < at.n;
#pragma unroll
        for (int c = 0; c < kKv; ++c) k[x][r][c] = in ? load_row16(src + 8 * r * D + c * 32) : make_uint4(0u, 0u, 0u, 0u);
        gate[x][r] = !in ? -INFINITY : p.a.logsig_pages ? p.a.logsig_pages[at.gate + g() + 8 * r] : 0.0f;
      }
    }
  }
  __device__ __forceinline__ void load_v(const Plan& p, const Keys (&keys)[R], int) {
#pragma unroll
    for (int x = 0; x < R; ++x) {
      const Keys& at = keys[x];
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.a.v_pages) + (at.row + 2 * t()) * D + g() * 8;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = (i & 1) + 8 * (i >> 1);
#pragma unroll
        for (int c = 0; c < kVv; ++c)
          v[x][i][c] = 2 * t() + key < at.n ? load_row16(src + key * D + c * 64) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
  __device__ __forceinline__ void scores() {
    bool over = false;
#pragma unroll
    for (int x = 0; x < R; ++x) {
      // a token whose log-gate is -inf has no weight whatever its k holds
      const bool out0 = gate[x][0] == -INFINITY, out1 = gate[x][1] == -INFINITY;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float a[4] = {}, b[4] = {};  // two chains of products
#pragma unroll
        for (int c = 0; c < kKv; ++c) {
          mma16816(a, k[x][0][c].x, k[x][1][c].x, k[x][0][c].y, k[x][1][c].y, q[n][c].x, q[n][c].y);
          mma16816(b, k[x][0][c].z, k[x][1][c].z, k[x][0][c].w, k[x][1][c].w, q[n][c].z, q[n][c].w);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s[x][n][e] = out0 ? -INFINITY : fmaf(a[e] + b[e], scale[n][e], bias(gain[n][e], gate[x][0]));
          s[x][n][2 + e] = out1 ? -INFINITY : fmaf(a[2 + e] + b[2 + e], scale[n][e], bias(gain[n][e], gate[x][1]));
          over |= fmaxf(s[x][n][e], s[x][n][2 + e]) > m[n][e] + kSlack;
        }
      }
      // nor whatever its v holds: 0 x NaN must not reach the sums
      const uint32_t gone0 = __ballot_sync(0xffffffffu, out0), gone1 = __ballot_sync(0xffffffffu, out1);
      if (gone0 | gone1) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (((i >> 1 ? gone1 : gone0) >> (4 * (2 * t() + (i & 1)))) & 1u)
#pragma unroll
            for (int c = 0; c < kVv; ++c) v[x][i][c] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    if (__any_sync(0xffffffffu, over)) {  // (a reference of -inf is exceeded by any logit)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y = m[n][e];
#pragma unroll
          for (int x = 0; x < R; ++x) y = fmaxf(y, fmaxf(s[x][n][e], s[x][n][2 + e]));
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, w));
          const float c = weight(m[n][e], y);
          m[n][e] = y;
          l[n][e] *= c;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            o[n][i][e] *= c;
            o[n][i][2 + e] *= c;
          }
        }
    }
  }
  __device__ __forceinline__ void accumulate() {
#pragma unroll
    for (int x = 0; x < R; ++x) {
      uint32_t hi[NT][2], mid[NT][2], lo[NT][2];  // the rounded weights, what they lack, what that lacks
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float w0 = weight(s[x][n][2 * r], m[n][0]), w1 = weight(s[x][n][2 * r + 1], m[n][1]);
          const __nv_bfloat162 h = __floats2bfloat162_rn(w0, w1);
          const float2 f = __bfloat1622float2(h);
          const __nv_bfloat162 rest = __floats2bfloat162_rn(w0 - f.x, w1 - f.y);
          l[n][0] += w0;
          l[n][1] += w1;
          uint32_t bits;
          memcpy(&bits, &h, 4);
          hi[n][r] = transpose8x8(bits);
          memcpy(&bits, &rest, 4);
          mid[n][r] = transpose8x8(bits);
          const float2 f2 = __bfloat1622float2(rest);
          const __nv_bfloat162 last = __floats2bfloat162_rn((w0 - f.x) - f2.x, (w1 - f.y) - f2.y);
          memcpy(&bits, &last, 4);
          lo[n][r] = transpose8x8(bits);
        }
#pragma unroll
      for (int c = 0; c < kVv; ++c) {
        const uint32_t v0[4] = {v[x][0][c].x, v[x][0][c].y, v[x][0][c].z, v[x][0][c].w};
        const uint32_t v1[4] = {v[x][1][c].x, v[x][1][c].y, v[x][1][c].z, v[x][1][c].w};
        const uint32_t v2[4] = {v[x][2][c].x, v[x][2][c].y, v[x][2][c].z, v[x][2][c].w};
        const uint32_t v3[4] = {v[x][3][c].x, v[x][3][c].y, v[x][3][c].z, v[x][3][c].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // rows g and g + 8 of the instruction are columns c * 64 + g * 8 + 2 i and the next
          const uint32_t a0 = __byte_perm(v0[i], v1[i], 0x5410), a1 = __byte_perm(v0[i], v1[i], 0x7632);
          const uint32_t a2 = __byte_perm(v2[i], v3[i], 0x5410), a3 = __byte_perm(v2[i], v3[i], 0x7632);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma16816(o[n][c * 4 + i], a0, a1, a2, a3, hi[n][0], hi[n][1]);
            mma16816(o[n][c * 4 + i], a0, a1, a2, a3, mid[n][0], mid[n][1]);
            mma16816(o[n][c * 4 + i], a0, a1, a2, a3, lo[n][0], lo[n][1]);
          }
        }
      }
    }
  }
  // the warp's sums, over the eight lanes of a column
  __device__ __forceinline__ void store(int nh, float* part_m, float* part_l, float* part_o) {
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], w);
        const int h = 8 * n + 2 * t() + e;
        if (h >= nh) continue;
        if (g() == 0) {
          part_m[warp * kHeads + h] = m[n][e];
          part_l[warp * kHeads + h] = l[n][e];
        }
        float* dst = part_o + (warp * kHeads + h) * D + g() * 8;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          *reinterpret_cast<float2*>(dst + (i >> 2) * 64 + 2 * (i & 3)) = make_float2(o[n][i][e], o[n][i][2 + e]);
      }
  }
};

// ---- fp32: 4 R keys at a time, eight lanes to a key, each with D / 8 of its columns --------------
template <int D, int NH>
struct CoreFp32 {
  static constexpr int kHeads = NH;
  static constexpr int R = 256 / D;  // keys per lane
  static constexpr int kKeys = 16;
  static constexpr int kSteps = 4 / R;
  static constexpr int kVec = D / 32;  // 16-byte pieces per lane and row

  float4 q[NH][kVec], k[R][kVec], v[R][kVec], o[NH][kVec];
  float gate[R], scale[NH], gain[NH], m[NH], l[NH], s[NH][R];

  static __device__ __forceinline__ int sub() { return threadIdx.x & 7; }          // the lane's columns
  static __device__ __forceinline__ int kg() { return (threadIdx.x & 31) >> 3; }   // its key of four
  static __device__ __forceinline__ float4 load4(const float* p) {
    const uint4 x = load_row16(p);
    return make_float4(__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w));
  }
  static __device__ __forceinline__ float4 zero() { return make_float4(0.0f, 0.0f, 0.0f, 0.0f); }

  __device__ __forceinline__ void load_q(const Plan& p, int b, int h0, int nh) {
    const float* qp = static_cast<const float*>(p.a.q) + (static_cast<int64_t>(b) * p.a.hq + h0) * D + sub() * 4;
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int c = 0; c < kVec; ++c) q[h][c] = h < nh ? load4(qp + h * D + c * 32) : zero();
  }
  __device__ __forceinline__ void begin(const float2* heads, int nh) {
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      const float2 x = h < nh ? heads[h] : make_float2(0.0f, 0.0f);
      scale[h] = x.x;
      gain[h] = x.y;
      m[h] = -INFINITY;
      l[h] = 0.0f;
#pragma unroll
      for (int c = 0; c < kVec; ++c) o[h][c] = zero();
    }
  }
  // one step of the warp's 16 keys: keys kg, kg + 4, ... of its 4 R on this lane
  __device__ __forceinline__ void load_k(const Plan& p, const Keys (&keys)[1], int step) {
    const Keys& at = keys[0];
    const float* src = static_cast<const float*>(p.a.k_pages) + (at.row + step * 4 * R + kg()) * D + sub() * 4;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int key = step * 4 * R + r * 4 + kg();
      const bool in = key < at.n;
#pragma unroll
      for (int c = 0; c < kVec; ++c) k[r][c] = in ? load4(src + r * 4 * D + c * 32) : zero();
      gate[r] = !in ? -INFINITY : p.a.logsig_pages ? p.a.logsig_pages[at.gate + key] : 0.0f;
    }
  }
  __device__ __forceinline__ void load_v(const Plan& p, const Keys (&keys)[1], int step) {
    const Keys& at = keys[0];
    const float* src = static_cast<const float*>(p.a.v_pages) + (at.row + step * 4 * R + kg()) * D + sub() * 4;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < kVec; ++c)
        v[r][c] = step * 4 * R + r * 4 + kg() < at.n ? load4(src + r * 4 * D + c * 32) : zero();
  }
  __device__ __forceinline__ void scores() {
    bool over = false;
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float2 a = make_float2(0.0f, 0.0f), b = a;
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
          a = __ffma2_rn(make_float2(q[h][c].x, q[h][c].y), make_float2(k[r][c].x, k[r][c].y), a);
          b = __ffma2_rn(make_float2(q[h][c].z, q[h][c].w), make_float2(k[r][c].z, k[r][c].w), b);
        }
        float x = (a.x + a.y) + (b.x + b.y);
#pragma unroll
        for (int w = 1; w < 8; w <<= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
        s[h][r] = gate[r] == -INFINITY ? -INFINITY : fmaf(x, scale[h], bias(gain[h], gate[r]));
        over |= s[h][r] > m[h] + kSlack;
      }
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (gate[r] == -INFINITY)
#pragma unroll
        for (int c = 0; c < kVec; ++c) v[r][c] = zero();  // 0 x NaN must not reach the sums
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        float x = m[h];
#pragma unroll
        for (int r = 0; r < R; ++r) x = fmaxf(x, s[h][r]);
        const float c = weight(m[h], x);
        m[h] = x;
        l[h] *= c;
#pragma unroll
        for (int i = 0; i < kVec; ++i) o[h][i] = make_float4(o[h][i].x * c, o[h][i].y * c, o[h][i].z * c, o[h][i].w * c);
      }
    }
  }
  __device__ __forceinline__ void accumulate() {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const float w = weight(s[h][r], m[h]);
        l[h] += w;
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
          const float2 a = __ffma2_rn(make_float2(w, w), make_float2(v[r][c].x, v[r][c].y), make_float2(o[h][c].x, o[h][c].y));
          const float2 b = __ffma2_rn(make_float2(w, w), make_float2(v[r][c].z, v[r][c].w), make_float2(o[h][c].z, o[h][c].w));
          o[h][c] = make_float4(a.x, a.y, b.x, b.y);
        }
      }
  }
  // the sums of the warp's four keys at a time, joined
  __device__ __forceinline__ void store(int nh, float* part_m, float* part_l, float* part_o) {
    const int warp = threadIdx.x >> 5;
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
        if (h < nh && kg() == 0) *reinterpret_cast<float4*>(part_o + (warp * NH + h) * D + sub() * 4 + i * 32) = y;
      }
      if (h < nh && (threadIdx.x & 31) == 0) {
        part_m[warp * NH + h] = x;
        part_l[warp * NH + h] = sum;
      }
    }
  }
};

__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void put4(__nv_bfloat16* p, float4 x) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
  uint2 u;
  memcpy(&u.x, &a, 4);
  memcpy(&u.y, &b, 4);
  *reinterpret_cast<uint2*>(p) = u;
}

// Shared memory of CTA `rank` of the cluster, at the place that p has in this one.
__device__ __forceinline__ float remote(const float* p, uint32_t rank) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(mapa_shared(smem_u32(p), rank)));
  return x;
}
__device__ __forceinline__ float4 remote4(const float* p, uint32_t rank) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "r"(mapa_shared(smem_u32(p), rank)));
  return x;
}

// a / b for 0 <= a, 0 < b; a 64-bit division takes ten times as long.
__device__ __forceinline__ int64_t quotient(int64_t a, int b) {
  return a <= UINT32_MAX ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}

// Four columns of one head, joined over the CTA's warps: the reference maximum, the sum of weights
// and the weighted v.
struct Joined {
  float top, l;
  float4 x;
};
template <int H, int D>
__device__ __forceinline__ Joined join_warps(const float* part_m, const float* part_l, const float* part_o, int h, int d) {
  Joined j = {-INFINITY, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
#pragma unroll
  for (int w = 0; w < kWarps; ++w) j.top = fmaxf(j.top, part_m[w * H + h]);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float c = weight(part_m[w * H + h], j.top);
    const float4 o = *reinterpret_cast<const float4*>(part_o + (w * H + h) * D + d);
    j.l = fmaf(part_l[w * H + h], c, j.l);
    j.x = make_float4(fmaf(o.x, c, j.x.x), fmaf(o.y, c, j.x.y), fmaf(o.z, c, j.x.z), fmaf(o.w, c, j.x.w));
  }
  return j;
}

// The output of four columns.  Nothing left of the sequence: 0 and -inf (a sum of nothing is 0, any
// other holds its reference's weight 1).
template <typename T, int D>
__device__ __forceinline__ void write_out(const Plan& p, int b, int head, int d, const Joined& j) {
  const float c = j.l == 0.0f ? 0.0f : 1.0f / j.l;
  put4(static_cast<T*>(p.a.out) + (static_cast<int64_t>(b) * p.a.hq + head) * D + d,
       make_float4(j.x.x * c, j.x.y * c, j.x.z * c, j.x.w * c));
  if (d == 0 && p.a.lse) p.a.lse[static_cast<int64_t>(head) * p.a.batch + b] = j.l == 0.0f ? -INFINITY : j.top + logf(j.l);
}

// A sequence without tokens.
template <typename T, int D>
__device__ __forceinline__ void write_nothing(const Plan& p, int b, int h0, int nh) {
  for (int x = threadIdx.x; x < nh * D; x += kThreads)
    put(static_cast<T*>(p.a.out) + (static_cast<int64_t>(b) * p.a.hq + h0) * D + x, 0.0f);
  if (p.a.lse)
    for (int h = threadIdx.x; h < nh; h += kThreads) p.a.lse[static_cast<int64_t>(h0 + h) * p.a.batch + b] = -INFINITY;
}

// The kv head, the first query head and the number of query heads of unit u of a sequence.
template <int H>
__device__ __forceinline__ void heads_of(const Plan& p, int u, int* hk, int* h0, int* nh) {
  *hk = p.blocks == 1 ? u : u / p.blocks;
  const int block = u - *hk * p.blocks;
  *h0 = *hk * p.group + block * H;
  *nh = min(H, p.group - block * H);
}

// A length as the table can hold it.
__device__ __forceinline__ int checked_length(const Plan& p, int len, bool* bad) {
  const int64_t most = static_cast<int64_t>(p.a.max_pages) << p.a.page_shift;
  if (len >= 0 && len <= most) return len;
  *bad = true;
  return len < 0 ? 0 : static_cast<int>(most);
}

// A place in the list of tiles: tile j of unit u of sequence b.
struct Place {
  int32_t b, u, j, tiles;  // tiles of every unit of the sequence
};

template <typename T, int D, typename Core>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(sizeof(T) == 2, Core::kHeads, D))
    paged_attn_kernel(const __grid_constant__ Plan p) {
  constexpr int H = Core::kHeads;
  constexpr int kGroups = Core::kKeys / 16;      // groups of 16 keys of a warp
  constexpr int kTile = Core::kKeys * kWarps;
  constexpr int kSlot = slot_floats(H, D);
  __shared__ int ends[kMaxSeqs];      // inclusive scan of the sequences' tiles (per unit)
  __shared__ int lens[kMaxSeqs];
  __shared__ float2 heads[kMaxHeads];  // 1 / (sqrt(d) temp) and the gain
  __shared__ int warp_sums[kWarps];
  __shared__ float part_m[kWarps * H], part_l[kWarps * H];
  __shared__ __align__(16) float part_o[kWarps * H * D];
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad = false;

  // Everything that does not depend on anything else is requested at once.
  const int batch = p.a.batch;
  const float temp0 = tid < p.a.hq ? p.a.temp[tid] : 1.0f, gain0 = tid < p.a.hq ? p.a.gain[tid] : 0.0f;
  // The tiles of every sequence, scanned.  Up to 32 sequences every warp does for itself; more are
  // shared among the threads, a run of them each.
  if (batch <= 32) {
    const int len = lane < batch ? checked_length(p, p.a.lens[lane], &bad) : 0;
    int scan = (len + kTile - 1) / kTile;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += y;
    }
    if (lane < batch) {  // (the same values from every warp)
      lens[lane] = len;
      ends[lane] = scan;
    }
    __syncwarp();
  } else {
    const int run = (batch + kThreads - 1) / kThreads;
    int sum = 0;
    for (int i = 0; i < run; ++i) {
      const int b = tid * run + i;
      if (b >= batch) break;
      const int len = checked_length(p, p.a.lens[b], &bad);
      lens[b] = len;
      sum += (len + kTile - 1) / kTile;
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
  }

  // this CTA's run of the list: an equal share with a workspace, whole units without
  const int64_t total = static_cast<int64_t>(ends[batch - 1]) * p.units;
  const int64_t per = quotient(total + gridDim.x - 1, static_cast<int>(gridDim.x));
  int64_t at = min(total, per * blockIdx.x), end = min(total, at + per);
  if (!p.shares) {
    const int64_t units = static_cast<int64_t>(batch) * p.units, share = (units + gridDim.x - 1) / gridDim.x;
    auto offset = [&](int64_t unit) {
      if (unit >= units) return total;
      const int b = static_cast<int>(unit / p.units), first = b > 0 ? ends[b - 1] : 0;
      return static_cast<int64_t>(first) * p.units + (unit - static_cast<int64_t>(b) * p.units) * (ends[b] - first);
    };
    at = offset(share * blockIdx.x);
    end = offset(share * (blockIdx.x + 1));
  }

  // The join of the warps' sums in shared memory, into the output or into a slot for the second kernel.
  auto finish = [&](int b, int h0, int nh, float* slot) {
    __syncthreads();
    for (int i = tid * 4; i < nh * D; i += kThreads * 4) {
      const int h = i / D, d = i - h * D;
      const Joined j = join_warps<H, D>(part_m, part_l, part_o, h, d);
      if (slot) {
        *reinterpret_cast<float4*>(slot + i) = j.x;
        if (d == 0) {
          slot[H * D + h] = j.top;
          slot[H * D + H + h] = j.l;
        }
      } else {
        write_out<T, D>(p, b, h0 + h, d, j);
      }
    }
    __syncthreads();
  };

  auto find = [&](int b, int hk, int tile, Keys (&keys)[kGroups]) {
#pragma unroll
    for (int x = 0; x < kGroups; ++x)
      keys[x] = locate(p, b, hk, lens[b], tile * kTile + (warp * kGroups + x) * 16, &bad);
  };
  if (at < end) {
    Place now;
    {
      int lo = 0, hi = batch - 1;  // the first sequence whose tiles reach past `at`
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (static_cast<int64_t>(ends[mid]) * p.units > at) hi = mid;
        else lo = mid + 1;
      }
      const int first = lo > 0 ? ends[lo - 1] : 0;
      const int64_t in_seq = at - static_cast<int64_t>(first) * p.units;
      now.b = lo;
      now.tiles = ends[lo] - first;
      now.u = static_cast<int>(quotient(in_seq, now.tiles));
      now.j = static_cast<int>(in_seq - static_cast<int64_t>(now.u) * now.tiles);
    }
    int hk, h0, nh;
    heads_of<H>(p, now.u, &hk, &h0, &nh);
    Core core;
    Keys keys[kGroups];
    find(now.b, hk, now.j, keys);
    core.load_k(p, keys, 0);
    core.load_v(p, keys, 0);
    core.load_q(p, now.b, h0, nh);
    if (tid < p.a.hq) heads[tid] = make_float2(1.0f / (sqrtf(static_cast<float>(D)) * temp0), gain0);
    for (int h = tid + kThreads; h < p.a.hq; h += kThreads)
      heads[h] = make_float2(1.0f / (sqrtf(static_cast<float>(D)) * p.a.temp[h]), p.a.gain[h]);
    __syncthreads();
    core.begin(heads + h0, nh);
    int j0 = now.j;  // where the present unit was entered
    for (;; ++at) {
      // the next tile, whose rows are requested before this one's are used up
      Place next = now;
      const bool more = at + 1 < end;
      bool turn = !more;
      int next_hk = hk, next_h0 = h0, next_nh = nh;
      Keys next_keys[kGroups] = {};
      if (more) {
        if (++next.j == next.tiles) {
          turn = true;
          next.j = 0;
          if (++next.u == p.units) {
            next.u = 0;
            do {
              ++next.b;
              next.tiles = ends[next.b] - ends[next.b - 1];
            } while (next.tiles == 0);
          }
          heads_of<H>(p, next.u, &next_hk, &next_h0, &next_nh);
        }
        find(next.b, next_hk, next.j, next_keys);
      }
#pragma unroll
      for (int step = 0; step < Core::kSteps; ++step) {
        const bool through = step == Core::kSteps - 1;
        core.scores();
        core.load_k(p, through ? next_keys : keys, through ? 0 : step + 1);
        if (through && turn && more) core.load_q(p, next.b, next_h0, next_nh);
        core.accumulate();
        core.load_v(p, through ? next_keys : keys, through ? 0 : step + 1);
      }
      if (turn) {
        core.store(nh, part_m, part_l, part_o);
        // slot 2c + 1: the unit begins in CTA c; slot 2c: it began before
        const bool whole = j0 == 0 && now.j == now.tiles - 1;
        finish(now.b, h0, nh, whole ? nullptr : p.partial + static_cast<int64_t>(2 * blockIdx.x + (j0 == 0)) * kSlot);
        if (j0 == 0 && p.shares && tid == 0) {
          const int64_t last = at - now.j + now.tiles - 1;  // the unit's last tile
          p.shares[static_cast<int64_t>(now.b) * p.units + now.u] =
              whole ? make_int2(0, -1) : make_int2(blockIdx.x, static_cast<int>(quotient(last, static_cast<int>(per))));
        }
        if (!more) break;
        core.begin(heads + next_h0, next_nh);
        j0 = 0;
      }
      now = next;
#pragma unroll
      for (int x = 0; x < kGroups; ++x) keys[x] = next_keys[x];
      hk = next_hk;
      h0 = next_h0;
      nh = next_nh;
    }
  }

  // sequences without tokens are in no run
  for (int i = blockIdx.x; i < batch; i += gridDim.x) {
    if (lens[i] != 0) continue;
    write_nothing<T, D>(p, i, 0, p.a.hq);
    if (p.shares)
      for (int u = tid; u < p.units; u += kThreads) p.shares[static_cast<int64_t>(i) * p.units + u] = make_int2(0, -1);
  }
  if (bad) atomicOr(p.a.status, kDevPageIndex);
}

// Few tiles: a cluster of CTAs for every unit, tile j in the CTA of rank j mod size, joined through
// distributed shared memory.  Neither a scan of the lengths nor a second launch.
template <typename T, int D, typename Core>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(sizeof(T) == 2, Core::kHeads, D))
    paged_cluster_kernel(const __grid_constant__ Plan p, int size) {
  constexpr int H = Core::kHeads;
  constexpr int kGroups = Core::kKeys / 16;
  constexpr int kTile = Core::kKeys * kWarps;
  __shared__ float2 heads[H];  // 1 / (sqrt(d) temp) and the gain
  __shared__ float part_m[kWarps * H], part_l[kWarps * H];
  __shared__ __align__(16) float part_o[kWarps * H * D];
  __shared__ __align__(16) float mine[H * D];  // the CTA's sums
  __shared__ float mine_m[H], mine_l[H];
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x, warp = tid >> 5;
  bool bad = false;
  const int unit = blockIdx.x / size, rank = blockIdx.x - unit * size;
  const int b = unit / p.units;
  int hk, h0, nh;
  heads_of<H>(p, unit - b * p.units, &hk, &h0, &nh);
  const int len = checked_length(p, p.a.lens[b], &bad);
  if (tid < nh) heads[tid] = make_float2(1.0f / (sqrtf(static_cast<float>(D)) * p.a.temp[h0 + tid]), p.a.gain[h0 + tid]);
  if (len == 0) {  // (all CTAs of the cluster)
    if (rank == 0) write_nothing<T, D>(p, b, h0, nh);
    if (bad) atomicOr(p.a.status, kDevPageIndex);
    return;
  }
  auto find = [&](int tile, Keys (&keys)[kGroups]) {
#pragma unroll
    for (int x = 0; x < kGroups; ++x)
      keys[x] = locate(p, b, hk, len, tile * kTile + (warp * kGroups + x) * 16, &bad);
  };
  Core core;
  Keys keys[kGroups];
  find(rank, keys);
  core.load_k(p, keys, 0);
  core.load_v(p, keys, 0);
  core.load_q(p, b, h0, nh);
  __syncthreads();
  core.begin(heads, nh);
  for (int j = rank; j * kTile < len; j += size) {
    Keys next_keys[kGroups];
    find(j + size, next_keys);
#pragma unroll
    for (int step = 0; step < Core::kSteps; ++step) {
      const bool through = step == Core::kSteps - 1;
      core.scores();
      core.load_k(p, through ? next_keys : keys, through ? 0 : step + 1);
      core.accumulate();
      core.load_v(p, through ? next_keys : keys, through ? 0 : step + 1);
    }
#pragma unroll
    for (int x = 0; x < kGroups; ++x) keys[x] = next_keys[x];
  }
  core.store(nh, part_m, part_l, part_o);
  __syncthreads();
  for (int i = tid * 4; i < nh * D; i += kThreads * 4) {
    const int h = i / D, d = i - h * D;
    const Joined j = join_warps<H, D>(part_m, part_l, part_o, h, d);
    if (size == 1) {
      write_out<T, D>(p, b, h0 + h, d, j);
    } else {
      *reinterpret_cast<float4*>(mine + i) = j.x;
      if (d == 0) {
        mine_m[h] = j.top;
        mine_l[h] = j.l;
      }
    }
  }
  if (bad) atomicOr(p.a.status, kDevPageIndex);
  if (size == 1) return;
  cluster_sync_all();
  // every CTA joins a part of the columns
  for (int i = (tid * size + rank) * 4; i < nh * D; i += kThreads * size * 4) {
    const int h = i / D, d = i - h * D;
    float m[kClusterMax], l[kClusterMax];
    float4 x[kClusterMax];
#pragma unroll
    for (int r = 0; r < kClusterMax; ++r) {
      if (r >= size) break;
      m[r] = remote(mine_m + h, r);
      l[r] = remote(mine_l + h, r);
      x[r] = remote4(mine + i, r);
    }
    Joined j = {-INFINITY, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
#pragma unroll
    for (int r = 0; r < kClusterMax; ++r)
      if (r < size) j.top = fmaxf(j.top, m[r]);
#pragma unroll
    for (int r = 0; r < kClusterMax; ++r) {
      if (r >= size) break;
      const float c = weight(m[r], j.top);
      j.l = fmaf(l[r], c, j.l);
      j.x = make_float4(fmaf(x[r].x, c, j.x.x), fmaf(x[r].y, c, j.x.y), fmaf(x[r].z, c, j.x.z), fmaf(x[r].w, c, j.x.w));
    }
    write_out<T, D>(p, b, h0 + h, d, j);
  }
  cluster_sync_all();  // no CTA leaves while another reads its sums
}

// The parts of a shared unit, joined in the order of the list.  With few parts the first block of a
// unit joins all its heads, a warp each; with many every block takes one head, and its warps every
// kJoinWarps-th part.  (With a block for every head in both cases a call of 61 sequences with 8 heads
// to a kv head took 32.6 us for 31.2.)
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kFewParts = 8;
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ Plan p, int heads) {
  constexpr int kPer = D / 32;
  __shared__ float part_m[kJoinWarps], part_l[kJoinWarps], part_o[kJoinWarps][D];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t unit = blockIdx.x;
  const int2 share = p.shares[unit];
  const bool few = share.y - share.x < kFewParts;
  if (share.y < share.x || (few && blockIdx.y > 0)) return;
  const int b = static_cast<int>(unit / p.units), u = static_cast<int>(unit - static_cast<int64_t>(b) * p.units);
  const int hk = u / p.blocks, block = u - hk * p.blocks;
  const int nh = min(heads, p.group - block * heads), h0 = hk * p.group + block * heads;
  const int64_t slot = slot_floats(heads, D);

  // head h of every `step`-th part from `first` on, four parts at a time; a lane has D / 32 columns
  float m, l, o[kPer];
  auto join = [&](int h, int first, int step) {
    m = -INFINITY;
    l = 0.0f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[e] = 0.0f;
    for (int c = first; c <= share.y; c += 4 * step) {
      float pm[4], pl[4], po[4][kPer];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int cc = c + x * step;
        const float* part = p.partial + (2 * cc + (cc == share.x)) * slot;
        pm[x] = cc <= share.y ? part[heads * D + h] : -INFINITY;
        pl[x] = cc <= share.y ? part[heads * D + heads + h] : 0.0f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) po[x][e] = cc <= share.y ? part[h * D + lane + 32 * e] : 0.0f;
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
  };
  auto out = [&](int h, int d, float x, float top, float sum) {
    put(static_cast<T*>(p.a.out) + (static_cast<int64_t>(b) * p.a.hq + h0 + h) * D + d, sum == 0.0f ? 0.0f : x / sum);
    if (d == 0 && p.a.lse)
      p.a.lse[static_cast<int64_t>(h0 + h) * p.a.batch + b] = sum == 0.0f ? -INFINITY : top + logf(sum);
  };
  if (few) {
    for (int h = warp; h < nh; h += kJoinWarps) {
      join(h, share.x, 1);
#pragma unroll
      for (int e = 0; e < kPer; ++e) out(h, lane + 32 * e, o[e], m, l);
    }
    return;
  }
  const int h = blockIdx.y;
  if (h >= nh) return;
  join(h, share.x + warp, kJoinWarps);
  if (lane == 0) {
    part_m[warp] = m;
    part_l[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) part_o[warp][lane + 32 * e] = o[e];
  __syncthreads();
  const int d = threadIdx.x;
  if (d >= D) return;
  float top = -INFINITY, sum = 0.0f, x = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, part_m[w]);
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    const float c = weight(part_m[w], top);
    sum = fmaf(part_l[w], c, sum);
    x = fmaf(part_o[w][d], c, x);
  }
  out(h, d, x, top, sum);
}

// CTAs of a cluster when the units are few and short, 0 when the list is the better way.  Clusters
// are as large as the GPU holds at once, at most a tile a CTA.  What a table can hold is all that
// the host knows of the lengths, so it decides: up to eight tiles a CTA when the clusters fill the
// GPU, up to four when they leave SMs idle that the list would use.  On the device, clusters and
// list, 16 query heads over 8 kv heads of 128 in bf16: 1 x 64 tokens 3.3 and 5.0 us, 1 x 1024 5.8 and
// 7.2, 1 x 2048 7.6 and 8.0, 1 x 4096 (eight tiles a CTA) 11.6 and 9.5, 33 x 256 10.4 and 14.1, 33 x 512
// 17.3 and 18.8.
int cluster_size(const Plan& p, int tile, int grid) {
  const int64_t tiles = ((static_cast<int64_t>(p.a.max_pages) << p.a.page_shift) + tile - 1) / tile;
  const int64_t units = static_cast<int64_t>(p.a.batch) * p.units;
  if (units > grid) return 0;
  int size = 1;
  while (size < kClusterMax && size < tiles && 2 * size * units <= grid) size *= 2;
  return tiles <= size * (2 * size * units <= grid ? 4 : 8) ? size : 0;
}

template <typename T, int D, typename Core>
cudaError_t launch_core(const Plan& p, int grid, cudaStream_t st) {
  if (const int size = cluster_size(p, Core::kKeys * kWarps, grid)) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.a.batch * p.units * size));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(size);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = size > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, paged_cluster_kernel<T, D, Core>, p, size);
  }
  const cudaError_t e = launch_pdl(paged_attn_kernel<T, D, Core>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, st, p);
  if (e != cudaSuccess || !p.shares) return e;
  const dim3 join(static_cast<unsigned>(static_cast<int64_t>(p.a.batch) * p.units),
                  static_cast<unsigned>(Core::kHeads < p.group ? Core::kHeads : p.group));
  return launch_pdl(paged_join_kernel<T, D>, join, dim3(kJoinThreads), 0, st, p, Core::kHeads);
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
  size_t share_bytes, slot_bytes;
};

Shape shape_of(bool bf16, int batch, int hq, int hkv, int head_dim) {
  Shape s;
  s.group = hq / hkv;
  s.heads = heads_per_unit(bf16, s.group);
  s.blocks = (s.group + s.heads - 1) / s.heads;
  s.units = hkv * s.blocks;
  s.grid = num_sms() * ctas_per_sm(bf16, s.heads, head_dim);
  s.share_bytes = (static_cast<size_t>(batch) * s.units * sizeof(int2) + 255) / 256 * 256;
  s.slot_bytes = sizeof(float) * slot_floats(s.heads, head_dim);
  return s;
}

}  // namespace

size_t paged_attention_workspace_bytes(tg_dtype dt, int batch, int hq, int hkv, int head_dim) {
  const Shape s = shape_of(dt == TG_BF16, batch, hq, hkv, head_dim);
  return s.share_bytes + 2 * s.grid * s.slot_bytes;
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
  p.shares = static_cast<int2*>(workspace);
  p.partial = workspace ? reinterpret_cast<float*>(static_cast<char*>(workspace) + s.share_bytes) : nullptr;
  return cuda_check(head_dim == 128 ? launch_dim<128>(p, bf16, s.heads, s.grid, st)
                                    : launch_dim<64>(p, bf16, s.heads, s.grid, st),
                    "paged attention launch");
}

}  // namespace tg
