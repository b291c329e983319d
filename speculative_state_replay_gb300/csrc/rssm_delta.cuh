// rssm_delta.cuh -- building blocks of the gated delta rule's kernels.
//
// Per (slot, value head) the state is S[dv][dk] (value rows, key columns; the
// layout of the selective-state checkpoints).  A token with key k, query q,
// value v, log decay g and rate beta does
//     S <- e^g S,   u = beta (v - S k),   S <- S + u k^T,   o = scale S q.
// Over a block of up to 8 tokens, with c_t the running sum of g,
//     u_t = beta_t (v_t - e^{c_t} S0 k_t - sum_{j<t} e^{c_t-c_j} (k_t.k_j) u_j)
//     o_t = scale (e^{c_t} S0 q_t + sum_{j<=t} e^{c_t-c_j} (q_t.k_j) u_j)
// so S0 is read once for all of them and S after a of them is
//     e^{c_{a-1}} S0 + sum_{j<a} e^{c_{a-1}-c_j} u_j k_j^T.
//
// The drafts that wait from the step before enter the same way, without
// forming the new state first: with E = e^{c_end} and e_j = e^{c_end - c_j},
//     S0' k = E (S0 k) + sum_j e_j w_j (k_j . k).
//
// A warp owns 16 value rows of S and all DK key columns as mma.sync fragments:
// lane (m = lane / 4, c = lane % 4) holds rows m and m + 8, and of each 32
// columns the eight 8c..8c+7 (the contraction index of two steps of 16 is
// permuted so that each lane's part is contiguous; keys and queries are loaded
// with the same permutation).  The first operand's 16 rows are the 8 keys and
// the 8 queries, so one instruction serves both products; the Gram products
// come from the same registers.  2-byte states go into the products as they
// are; fp32 states as three bf16 parts, which is all 24 bits of them: u = v - S k
// is what is left of values that the state predicts, and two parts (16 bits)
// leave 2^-18 of |S| |k| in it.
#pragma once

#include "rssm_device.cuh"
#include "rssm_host.h"

namespace rssm {

constexpr int kDeltaT = 8;       // tokens a block holds
// bytes between a block's keys (queries) in shared memory: 64 past the row, so
// that the two rows a quarter of a warp reads at a time fall on distinct banks
template <int DK>
constexpr int kTokenRow = DK * 2 + 64;
constexpr float kMinLog = -100.0f;  // log decays are held at this and above: e^-100 is zero to fp32 sums of O(1) values,
                                    // and a finite floor keeps differences of running sums defined (g = -inf resets a state)

constexpr float kMaxLog = 1000.0f;         // and at this and below (e^89 is infinite)
__device__ __forceinline__ float held_log(float g) { return g < kMinLog ? kMinLog : g > kMaxLog ? kMaxLog : g; }  // NaN stays NaN

// A sum as two floats, hi + lo: differences of running sums are exponents, and
// one float's rounding at a sum of 100 would be 2^-18.
struct LongSum {
  float hi, lo;
  __device__ __forceinline__ void add(float h, float l) {
    const float s = hi + h, b = s - hi;
    lo += l + ((hi - (s - b)) + (h - b));  // what the addition rounded off, exactly (Knuth's two-sum)
    hi = s;
  }
  __device__ __forceinline__ void settle() {  // hi: the sum rounded
    const float s = hi + lo;
    lo += hi - s;
    hi = s;
  }
};

// e^(hi + lo), lo what the rounding of hi left: expf's 2 units in the last place and one more, whatever hi (an infinite
// one stays infinite).  The hardware's power of two alone would be |hi| 2^-24 off, and a state keeps that of every commit.
__device__ __forceinline__ float exp_sum(float hi, float lo) { return expf(hi) * (1.0f + lo); }

struct DeltaCacheView {
  int S, Hk, Hv, rep, dv, np;
  int dtype, wide;  // wide: state rows start on 32 bytes
  void* state;
  long long state_stride;
  uint16_t* pend_k;
  long long pend_k_stride;
  float* pend_w;
  long long pend_w_stride;
  float* pend_c;
  long long pend_c_stride;
  float* pend_cl;  // or null
  long long pend_cl_stride;
  int* pend;
  unsigned* err;
};

struct DeltaTokens {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  long long q_stride, k_stride, v_stride;  // elements between tokens
  const float* g;
  const float* beta;
  uint16_t* out;  // [tok][Hv][dv]
  float scale;
  int l2norm;
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// (a, b) as bf16 hi + bf16 lo: 16 significant bits, the remainder's own
// rounding is at most 2^-18 of the value
__device__ __forceinline__ void split_bf16x2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = cvt_bf16x2(a, b);
  lo = cvt_bf16x2(a - bf16lo(hi), b - bf16hi(hi));
}

// Two fp32 values in one 64-bit register pair: packed instructions take and
// leave pairs, so values that go through them stay in this form.
using pair = unsigned long long;
__device__ __forceinline__ pair pack2(float lo, float hi) {
  pair d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpack2(pair d, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(d)); }
__device__ __forceinline__ void fma2(pair& d, pair a, pair b) { asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b)); }
__device__ __forceinline__ void add2(pair& d, pair a) { asm("add.rn.f32x2 %0, %0, %1;" : "+l"(d) : "l"(a)); }
__device__ __forceinline__ void mul2(pair& d, pair a) { asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(d) : "l"(a)); }
__device__ __forceinline__ uint32_t cvt_bf16x2(pair d) {
  float lo, hi;
  unpack2(d, lo, hi);
  return cvt_bf16x2(lo, hi);
}
__device__ __forceinline__ void split_bf16x2(pair d, uint32_t& h, uint32_t& l) {
  h = cvt_bf16x2(d);
  fma2(d, pack2(-1.0f, -1.0f), pack2(bf16lo(h), bf16hi(h)));  // the remainder, exact
  l = cvt_bf16x2(d);
}
// and as three parts, whose sum is the value
__device__ __forceinline__ void split_bf16x2(pair d, uint32_t& h, uint32_t& m, uint32_t& l) {
  h = cvt_bf16x2(d);
  fma2(d, pack2(-1.0f, -1.0f), pack2(bf16lo(h), bf16hi(h)));
  m = cvt_bf16x2(d);
  fma2(d, pack2(-1.0f, -1.0f), pack2(bf16lo(m), bf16hi(m)));
  l = cvt_bf16x2(d);
}

// Rows m (or m + 8) of a warp's state: a lane's 2 KS pairs of columns.
template <int DK, bool F32>
struct DeltaRow {
  static constexpr int KS = DK / 16;
  ulonglong2 s[KS];  // fp32 values; 2-byte states keep their words in `w` until they are needed as such
  uint4 w[KS / 2];

  // from the warp's rows in shared memory
  __device__ __forceinline__ void read(const uint8_t* buf, int row, int c) {
    if constexpr (F32) {
      const float* p = reinterpret_cast<const float*>(buf) + row * DK + 8 * c;
#pragma unroll
      for (int x = 0; x < KS; ++x) s[x] = *reinterpret_cast<const ulonglong2*>(p + 32 * (x >> 1) + 4 * (x & 1));
    } else {
      const uint16_t* p = reinterpret_cast<const uint16_t*>(buf) + row * DK + 8 * c;
#pragma unroll
      for (int y = 0; y < KS / 2; ++y) w[y] = *reinterpret_cast<const uint4*>(p + 32 * y);
    }
  }
  __device__ __forceinline__ void decay(float e) {
    const pair a = pack2(e, e);
#pragma unroll
    for (int x = 0; x < KS; ++x) {
      if constexpr (!F32) {
        const uint32_t p = (x & 1) ? w[x >> 1].z : w[x >> 1].x, q = (x & 1) ? w[x >> 1].w : w[x >> 1].y;
        s[x].x = pack2(bf16lo(p), bf16hi(p));
        s[x].y = pack2(bf16lo(q), bf16hi(q));
      }
      mul2(s[x].x, a);
      mul2(s[x].y, a);
    }
  }
  // += u k^T; `k`: the key in fp32, in shared memory
  __device__ __forceinline__ void add(float u, const float* k, int c) {
    const pair a = pack2(u, u);
#pragma unroll
    for (int x = 0; x < KS; ++x) {
      const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(k + 32 * (x >> 1) + 8 * c + 4 * (x & 1));
      fma2(s[x].x, a, y.x);
      fma2(s[x].y, a, y.y);
    }
  }
  // to memory; `p`: the lane's first column.  wide: rows start on 32 bytes,
  // and a lane writes a whole sector at a time
  __device__ __forceinline__ void store(void* p, bool wide) const {
    if constexpr (F32) {
#pragma unroll
      for (int y = 0; y < KS / 2; ++y) {
        float* to = static_cast<float*>(p) + 32 * y;
        if (wide) {
          asm volatile("st.global.v4.b64 [%0], {%1,%2,%3,%4};" ::"l"(to), "l"(s[2 * y].x), "l"(s[2 * y].y), "l"(s[2 * y + 1].x),
                       "l"(s[2 * y + 1].y)
                       : "memory");
        } else {
          *reinterpret_cast<ulonglong2*>(to) = s[2 * y];
          *reinterpret_cast<ulonglong2*>(to + 4) = s[2 * y + 1];
        }
      }
    } else {
#pragma unroll
      for (int y = 0; y < KS / 2; ++y)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + 32 * y) =
            make_uint4(cvt_bf16x2(s[2 * y].x), cvt_bf16x2(s[2 * y].y), cvt_bf16x2(s[2 * y + 1].x), cvt_bf16x2(s[2 * y + 1].y));
    }
  }
};

// A block of up to 8 tokens, and the drafts that wait before it.  Lane (t =
// lane / 4, c = lane % 4) has token t and, of pairs of tokens, j = 2c + {0, 1}.
// Keys and queries stay in shared memory, rows of DK bf16 at kTokenRow<DK>
// bytes, zeros past the last token, and come from there as the first operand of
// two steps of 16 at a time: 8 loads an item for 32 registers less.
template <int DK>
struct DeltaBlock {
  static constexpr int KS = DK / 16;
  const uint8_t *k, *q;  // this lane's part of its token's key and query
  float kk[4];           // k_t.k_j and q_t.k_j among the block's tokens, normalised and scaled
  float wk[4];           // k_t.k_j and q_t.k_j with the waiting keys, times 1 / |k_t| and scale / |q_t|
  float r, kq;           // 1 / |k_t| and scale / |q_t| (1 and scale without normalisation)

  __device__ __forceinline__ void set(const uint8_t* keys, const uint8_t* queries, int lane) {
    const int at = (lane >> 2) * kTokenRow<DK> + 16 * (lane & 3);
    k = keys + at;
    q = queries + at;
  }
  // first operands of steps 2 y and 2 y + 1: rows 0-7 keys, rows 8-15 queries
  __device__ __forceinline__ void operands(int y, uint32_t (&a)[4], uint32_t (&b)[4]) const {
    const uint4 kw = *reinterpret_cast<const uint4*>(k + 64 * y), qw = *reinterpret_cast<const uint4*>(q + 64 * y);
    a[0] = kw.x;
    a[1] = qw.x;
    a[2] = kw.y;
    a[3] = qw.y;
    b[0] = kw.z;
    b[1] = qw.z;
    b[2] = kw.w;
    b[3] = qw.w;
  }

  // the Gram products, the same for every value head of the key head;
  // `waiting`: the waiting keys, laid out like the keys
  __device__ __forceinline__ void gram(const DeltaTokens& tk, const uint8_t* waiting, int acc, int lane) {
    const int t = lane >> 2, cc = lane & 3;
    const unsigned full = 0xffffffffu;
    float qq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) kk[i] = wk[i] = 0.0f;
#pragma unroll
    for (int y = 0; y < KS / 2; ++y) {
      uint32_t a[4], b[4];
      operands(y, a, b);
      mma_bf16(kk, a, a[0], a[2]);
      mma_bf16(kk, b, b[0], b[2]);
      if (tk.l2norm) {
        mma_bf16(qq, a, a[1], a[3]);
        mma_bf16(qq, b, b[1], b[3]);
      }
      if (acc > 0) {
        const uint4 w = t < acc ? *reinterpret_cast<const uint4*>(waiting + t * kTokenRow<DK> + 16 * cc + 64 * y)
                                : make_uint4(0u, 0u, 0u, 0u);
        mma_bf16(wk, a, w.x, w.y);
        mma_bf16(wk, b, w.z, w.w);
      }
    }
    kq = tk.scale;
    r = 1.0f;
    if (tk.l2norm) {
      // the diagonal element (t, t) is in lane 4 t + t / 2, register t & 1
      const float dk = (t & 1) ? kk[1] : kk[0], dq = (t & 1) ? qq[3] : qq[2];
      r = rsqrtf(__shfl_sync(full, dk, t * 4 + (t >> 1)) + 1e-6f);
      kq = tk.scale * rsqrtf(__shfl_sync(full, dq, t * 4 + (t >> 1)) + 1e-6f);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float rj = __shfl_sync(full, r, (2 * cc + i) * 4);
      kk[i] *= r * rj;
      kk[2 + i] *= kq * rj;
      wk[i] *= r;
      wk[2 + i] *= kq;
    }
  }

  // d[i] = (keys; queries) times rows i of the warp's state, in short chains of products
  template <bool F32>
  __device__ __forceinline__ void product(const DeltaRow<DK, F32> (&S)[2], float (&d)[2][4]) const {
    float d1[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) d[i][e] = d1[i][e] = 0.0f;
    if constexpr (F32) {
      float l[2][4], l1[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) l[i][e] = l1[i][e] = 0.0f;
#pragma unroll
      for (int y = 0; y < KS / 2; ++y) {
        uint32_t a[4], b[4];
        operands(y, a, b);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t h[4], m[4], lo[4];
          split_bf16x2(S[i].s[2 * y].x, h[0], m[0], lo[0]);
          split_bf16x2(S[i].s[2 * y].y, h[1], m[1], lo[1]);
          split_bf16x2(S[i].s[2 * y + 1].x, h[2], m[2], lo[2]);
          split_bf16x2(S[i].s[2 * y + 1].y, h[3], m[3], lo[3]);
          mma_bf16(d[i], a, h[0], h[1]);
          mma_bf16(l[i], a, m[0], m[1]);
          mma_bf16(d1[i], b, h[2], h[3]);
          mma_bf16(l1[i], b, m[2], m[3]);
          mma_bf16(l[i], a, lo[0], lo[1]);
          mma_bf16(l1[i], b, lo[2], lo[3]);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) d[i][e] = (d[i][e] + d1[i][e]) + (l[i][e] + l1[i][e]);
    } else {
#pragma unroll
      for (int y = 0; y < KS / 2; ++y) {
        uint32_t a[4], b[4];
        operands(y, a, b);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mma_bf16(d[i], a, S[i].w[y].x, S[i].w[y].y);
          mma_bf16(d1[i], b, S[i].w[y].z, S[i].w[y].w);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) d[i][e] += d1[i][e];
    }
  }
};

// Scratch: counters of the steps' rows first, of a fixed number of rows, so that
// no prompt's data reaches them whatever the sizes of the calls that share it.
constexpr int kDeltaRows = 65536;
constexpr size_t kDeltaHead = kDeltaRows * sizeof(unsigned);

// host side
bool delta_view(const rssm_delta_cache* c, DeltaCacheView* out, rssm_status* st);
rssm_status delta_tokens(const DeltaCacheView& c, int dk, const void* q, const void* k, const void* v, int64_t q_stride,
                         int64_t k_stride, int64_t v_stride, const float* g, const float* beta, float scale, int l2norm,
                         void* out, DeltaTokens* tk);

}  // namespace rssm
