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
// A warp owns 16 value rows of S and all DK key columns, in registers, as
// mma.sync fragments: lane (m = lane / 4, c = lane % 4) holds rows m and m + 8,
// and of each 16 columns the four 4c..4c+3 (the contraction index of a step of
// 16 is permuted so that each lane's part is contiguous; keys and queries are
// loaded with the same permutation).  The first operand's 16 rows are the 8
// keys and the 8 queries, so one instruction serves both products; the Gram
// products k.k and q.k come from the same registers.  No shared memory and no
// barriers are involved.
#pragma once

#include "rssm_device.cuh"

namespace rssm {

constexpr int kDeltaT = 8;       // tokens a block holds
// bytes between a block's keys (queries) in shared memory: 32 past the row, so
// that the four rows half a warp reads at a time fall on distinct banks
template <int DK>
constexpr int kTokenRow = DK * 2 + 32;
constexpr float kMinLog = -100.0f;  // log decays are held at this and above: e^-100 is zero to fp32 sums of O(1) values,
                                    // and a finite floor keeps differences of running sums defined (g = -inf resets a state)

struct DeltaCacheView {
  int S, Hk, Hv, rep, dv, np;
  int dtype;
  void* state;
  long long state_stride;
  uint16_t* pend_k;
  long long pend_k_stride;
  float* pend_w;
  long long pend_w_stride;
  float* pend_c;
  long long pend_c_stride;
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
  asm volatile(
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

// (x, y) += a * (p, q), two fp32 FMAs in one instruction
__device__ __forceinline__ void fma2(float& x, float& y, float2 a, float p, float q) {
  float2 d = make_float2(x, y);
  const float2 b = make_float2(p, q);
  asm("fma.rn.f32x2 %0, %1, %2, %0;"
      : "+l"(*reinterpret_cast<unsigned long long*>(&d))
      : "l"(*reinterpret_cast<const unsigned long long*>(&a)), "l"(*reinterpret_cast<const unsigned long long*>(&b)));
  x = d.x;
  y = d.y;
}

// the state rows of one warp
template <int DK>
struct DeltaState {
  static constexpr int KS = DK / 16;
  float4 s[2][KS];

  // `head`: element offset of the warp's first row
  __device__ __forceinline__ void load(const void* state, long long head, int dtype, int lane) {
    const int m = lane >> 2, c = lane & 3;
    if (dtype == RSSM_F32) {
      const float* p = static_cast<const float*>(state) + head + m * DK + 4 * c;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int x = 0; x < KS; ++x) s[i][x] = *reinterpret_cast<const float4*>(p + i * 8 * DK + 16 * x);
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(state) + head + m * DK + 4 * c;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int x = 0; x < KS; ++x) {
          const uint2 w = *reinterpret_cast<const uint2*>(p + i * 8 * DK + 16 * x);
          s[i][x] = make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
        }
    }
  }
  __device__ __forceinline__ void store(void* state, long long head, int dtype, int lane) const {
    const int m = lane >> 2, c = lane & 3;
    if (dtype == RSSM_F32) {
      float* p = static_cast<float*>(state) + head + m * DK + 4 * c;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int x = 0; x < KS; ++x) *reinterpret_cast<float4*>(p + i * 8 * DK + 16 * x) = s[i][x];
    } else {
      uint16_t* p = static_cast<uint16_t*>(state) + head + m * DK + 4 * c;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int x = 0; x < KS; ++x)
          *reinterpret_cast<uint2*>(p + i * 8 * DK + 16 * x) =
              make_uint2(cvt_bf16x2(s[i][x].x, s[i][x].y), cvt_bf16x2(s[i][x].z, s[i][x].w));
    }
  }
  __device__ __forceinline__ void decay(float e) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        s[i][x].x *= e;
        s[i][x].y *= e;
        s[i][x].z *= e;
        s[i][x].w *= e;
      }
  }
  // S += (u0, u1) k^T for rows m and m + 8; `k`: the key in fp32, in shared memory
  __device__ __forceinline__ void add(float u0, float u1, const float* k, int lane) {
    const float2 a = make_float2(u0, u0), b = make_float2(u1, u1);
#pragma unroll
    for (int x = 0; x < KS; ++x) {
      const float4 w = *reinterpret_cast<const float4*>(k + 16 * x + 4 * (lane & 3));
      fma2(s[0][x].x, s[0][x].y, a, w.x, w.y);
      fma2(s[0][x].z, s[0][x].w, a, w.z, w.w);
      fma2(s[1][x].x, s[1][x].y, b, w.x, w.y);
      fma2(s[1][x].z, s[1][x].w, b, w.z, w.w);
    }
  }
};

// A block of up to 8 tokens against the warp's state rows.
template <int DK>
struct DeltaBlock {
  static constexpr int KS = DK / 16;
  uint32_t a[KS][4];  // first operand: rows 0-7 keys, rows 8-15 queries
  float c;            // running sum of g at this lane's token t = lane / 4
  float r, rq;        // 1 / |k_t|, scale / |q_t| (1 and scale without normalisation)
  float beta;
  float A[2], P[2];   // coefficients of u_j in u_t and o_t for j = 2 (lane % 4) + {0, 1}
  float u[2][2];      // u_t of value rows r0 + 8 i + 2 (lane % 4) + {0, 1}

  // the block's tokens: keys and queries in shared memory, rows of DK bf16 at kTokenRow<DK> bytes
  __device__ __forceinline__ void load(const uint8_t* keys, const uint8_t* queries, int T, int lane) {
    const int t = lane >> 2, cc = lane & 3;
    const bool live = t < T;
    const uint8_t *kp = keys + t * kTokenRow<DK> + 8 * cc, *qp = queries + t * kTokenRow<DK> + 8 * cc;
#pragma unroll
    for (int x = 0; x < KS; ++x) {
      const uint2 kw = live ? *reinterpret_cast<const uint2*>(kp + 32 * x) : make_uint2(0u, 0u);
      const uint2 qw = live ? *reinterpret_cast<const uint2*>(qp + 32 * x) : make_uint2(0u, 0u);
      a[x][0] = kw.x;
      a[x][1] = qw.x;
      a[x][2] = kw.y;
      a[x][3] = qw.y;
    }
  }

  // running decays, norms and the coefficients among the block's own tokens
  __device__ __forceinline__ void prepare(const DeltaTokens& tk, float g, float b, int lane) {
    const int t = lane >> 2, cc = lane & 3;
    const unsigned full = 0xffffffffu;
    c = g;
    beta = b;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      const float y = __shfl_up_sync(full, c, o);
      if (lane >= o) c += y;
    }
    float kk[4] = {0.f, 0.f, 0.f, 0.f};  // k_t.k_j, then q_t.k_j, j = 2 cc + {0, 1}
#pragma unroll
    for (int x = 0; x < KS; ++x) mma_bf16(kk, a[x], a[x][0], a[x][2]);
    r = 1.0f;
    rq = tk.scale;
    if (tk.l2norm) {
      float qq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int x = 0; x < KS; ++x) mma_bf16(qq, a[x], a[x][1], a[x][3]);
      // the diagonal element (t, t) is in lane 4 t + t / 2, register t & 1
      const float dk = (t & 1) ? kk[1] : kk[0], dq = (t & 1) ? qq[3] : qq[2];
      r = rsqrtf(__shfl_sync(full, dk, t * 4 + (t >> 1)) + 1e-6f);
      rq = tk.scale * rsqrtf(__shfl_sync(full, dq, t * 4 + (t >> 1)) + 1e-6f);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = 2 * cc + i;
      const float cj = __shfl_sync(full, c, j * 4), rj = __shfl_sync(full, r, j * 4);
      const float e = j <= t ? expf(c - cj) * rj : 0.0f;
      A[i] = j < t ? beta * r * e * kk[i] : 0.0f;
      P[i] = e * rq * kk[2 + i];
    }
  }

  // products of the state rows with the keys and queries, then the triangular
  // solve; vw: the lane's token's values of value rows r0 + 8 i + 2 (lane % 4)
  // + {0, 1}; o gets the outputs of the same rows
  __device__ __forceinline__ void solve(const DeltaState<DK>& S, const uint32_t (&vw)[2], int T, int lane, float (&o)[2][2]) {
    const int t = lane >> 2, cc = lane & 3;
    const unsigned full = 0xffffffffu;
    const float ec = expf(c);
    const float fu = -beta * ec * r, fo = ec * rq;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        uint32_t h0, l0, h1, l1;
        split_bf16x2(S.s[i][x].x, S.s[i][x].y, h0, l0);
        split_bf16x2(S.s[i][x].z, S.s[i][x].w, h1, l1);
        mma_bf16(d, a[x], h0, h1);
        mma_bf16(d, a[x], l0, l1);
      }
      u[i][0] = fmaf(fu, d[0], beta * bf16lo(vw[i]));
      u[i][1] = fmaf(fu, d[1], beta * bf16hi(vw[i]));
      o[i][0] = fo * d[2];
      o[i][1] = fo * d[3];
    }
#pragma unroll
    for (int j = 0; j < kDeltaT; ++j) {
      if (j >= T) break;
      // u_j is final in the lanes of token j once every earlier token's share is in
      const float Aj = __shfl_sync(full, A[j & 1], t * 4 + (j >> 1)), Pj = __shfl_sync(full, P[j & 1], t * 4 + (j >> 1));
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float uj = __shfl_sync(full, u[i][e], j * 4 + cc);
          // selected, not multiplied by zero: a later token's NaN stays out of the earlier ones
          if (t > j) u[i][e] = fmaf(-Aj, uj, u[i][e]);
          if (t >= j) o[i][e] = fmaf(Pj, uj, o[i][e]);
        }
    }
  }

  __device__ __forceinline__ void store_out(const float (&o)[2][2], uint16_t* out, long long stride, int T, int lane) const {
    const int t = lane >> 2, cc = lane & 3;
    if (t < T) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<uint32_t*>(out + t * stride + 8 * i + 2 * cc) = cvt_bf16x2(o[i][0], o[i][1]);
    }
  }
};

// host side
bool delta_view(const rssm_delta_cache* c, DeltaCacheView* out, rssm_status* st);
rssm_status delta_tokens(const DeltaCacheView& c, int dk, const void* q, const void* k, const void* v, int64_t q_stride,
                         int64_t k_stride, int64_t v_stride, const float* g, const float* beta, float scale, int l2norm,
                         void* out, DeltaTokens* tk);

}  // namespace rssm
