// rssm_delta_prefill.cu -- the gated delta rule over whole prompts, in chunks
// of 64 tokens on the tensor cores.
//
// Within a chunk, with c the running sum of g, r = 1/|k| (1 without
// normalisation) and the keys as given,
//     A[i][j] = beta_i e^{c_i - c_j} r_i r_j (k_i . k_j)      (j < i)
//     T'      = (I + A)^-1 diag(beta)
//     P[i][j] = scale e^{c_i - c_j} rq_i r_j (q_i . k_j)      (j <= i)
// and, with S the state before the chunk (X = K S^T, Y = Q S^T),
//     R = V - diag(e^c r) X,   U = T' R,   O = diag(scale e^c rq) Y + (P T') R
//     S <- e^{c_end} S + (diag(e^{c_end - c} r) U)^T K.
// T', P T' and the decay vectors do not depend on the state: delta_chunk_kernel
// forms them for every chunk at once (scratch).  delta_scan_kernel then walks
// each prompt's chunks in order; its chain per chunk is three products, X (with
// Y on top: one product of 128 rows), U (with (P T') R on top) and the state's
// update, on tcgen05 with accumulators in TMEM.
//
// Precision: products run in bf16 with fp32 accumulation.  Keys, queries and
// values are exact; fp32 factors (S, T', R, U) are carried as bf16 hi + lo,
// 16 significant bits, and the product of two lo parts (2^-18 of the term) is
// dropped: states and outputs keep about 5 decimal digits, and the outputs are
// rounded to bf16 once.  (P T' rounded to bf16 would save a quarter of the
// scratch traffic, but of a prompt of few tokens all outputs would share its
// error: up to 2^-8 more.)
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "rssm_delta.cuh"

namespace rssm {
namespace {

constexpr int kC = 64;                   // tokens of a chunk
constexpr int kImgHi = 128 * 128;        // bytes: T' (64 rows), then P T' (64 rows), rows of 64 bf16: the hi parts
constexpr int kImg = 2 * kImgHi;         // and the lo parts
constexpr int kVec = 1024;               // bytes: e^c r [64], e^{c_end-c} r [64], scale e^c rq [64], e^{c_end}
constexpr int kUnit = kImg + kVec;       // scratch of one (chunk, value head)

struct DeltaPrefillArgs {
  DeltaCacheView c;
  DeltaTokens tk;
  const int* slot_idx;
  const int* cu;
  const int* initial;
  int batch, tiles;
  long long tokens;
  uint8_t* units;  // scratch [chunk slot][Hv][kUnit]
};

// A prompt's chunks are in scratch from slot cu / 64 + b on: no two prompts
// share a slot, and the last slot is below tokens / 64 + batch.
__device__ __forceinline__ bool row_bounds(const DeltaPrefillArgs& a, int b, int& start, int& n) {
  start = a.cu[b];
  n = a.cu[b + 1] - start;
  return start >= 0 && n >= 0 && start + static_cast<long long>(n) <= a.tokens;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// 16-byte piece `ch` of row r of a matrix with 128-byte rows, 128-byte swizzle
__device__ __forceinline__ uint32_t sw128(int r, int ch) { return static_cast<uint32_t>(r * 128 + ((ch ^ (r & 7)) << 4)); }

// d (two n-tiles) += a * b with both split into hi + lo, the lo * lo part dropped
__device__ __forceinline__ void mma_split(float (&d)[2][4], const uint32_t (&ah)[4], const uint32_t (&al)[4],
                                          const uint32_t (&bh)[4], const uint32_t (&bl)[4]) {
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    mma_bf16(d[t], ah, bh[2 * t], bh[2 * t + 1]);
    mma_bf16(d[t], ah, bl[2 * t], bl[2 * t + 1]);
    mma_bf16(d[t], al, bh[2 * t], bh[2 * t + 1]);
  }
}
// the accumulators of two adjacent n-tiles as a first operand of the next product
__device__ __forceinline__ void as_operand(const float (&d)[2][4], uint32_t (&h)[4], uint32_t (&l)[4]) {
  split_bf16x2(d[0][0], d[0][1], h[0], l[0]);
  split_bf16x2(d[0][2], d[0][3], h[1], l[1]);
  split_bf16x2(d[1][0], d[1][1], h[2], l[2]);
  split_bf16x2(d[1][2], d[1][3], h[3], l[3]);
}

// --------------------------------------------------------------------------
// delta_chunk_kernel: one block of 4 warps per (chunk, key head); warp w has
// the chunk's tokens 16 w .. 16 w + 15.
// --------------------------------------------------------------------------
struct ChunkSmem {
  static constexpr int kA = 0;                   // A hi, lo: 2 x 8 KB
  static constexpr int kImage = kA + 2 * 8192;   // as in scratch
  static constexpr int kD = kImage + kImg;       // inverses of the diagonal blocks, hi and lo: 2 x 4 x 512
  static constexpr int kF = kD + 4096;           // diagonal blocks in fp32: 4 x 16 x 17, then the inverses
  static constexpr int kS = kF + 2 * 4 * 16 * 17 * 4;
  static constexpr int kScalars = kS;            // c hi, c lo, beta, r, rq: 5 x 64 floats
  static constexpr int kTokens = (kScalars + 5 * 64 * 4 + 127) / 128 * 128;  // K then Q
};

template <int DK>
__global__ void __launch_bounds__(128) delta_chunk_kernel(const DeltaPrefillArgs a) {
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ int sh[3];
  constexpr int RB = DK * 2, CH = DK / 8, KS = DK / 16;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hk = blockIdx.y;
  const unsigned full = 0xffffffffu;
  pdl_wait();
  if (tid == 0) sh[0] = -1;
  __syncthreads();
  for (int b = tid; b < a.batch; b += 128) {
    int start, n;
    if (!row_bounds(a, b, start, n)) continue;
    const int i = static_cast<int>(blockIdx.x) - (start / kC + b);
    if (i >= 0 && i < (n + kC - 1) / kC && a.slot_idx[b] > 0 && a.slot_idx[b] < a.c.S) {
      sh[0] = b;
      sh[1] = start + i * kC;
      sh[2] = min(n - i * kC, kC);
    }
  }
  __syncthreads();
  if (sh[0] < 0) return;  // an unused slot
  const long long tok0 = sh[1];
  const int n = sh[2];
  uint8_t* sk = sm + ChunkSmem::kTokens;
  uint8_t* sq = sk + kC * RB;
  float* s_ch = reinterpret_cast<float*>(sm + ChunkSmem::kScalars);
  float *s_cl = s_ch + 64, *s_beta = s_cl + 64, *s_r = s_beta + 64, *s_rq = s_r + 64;
  // tokens past the chunk's end are zeros: they add nothing anywhere
  for (int i = tid; i < kC * CH; i += 128) {
    const int r = i / CH, ch = i % CH;
    const uint32_t to = static_cast<uint32_t>(r * RB + ((ch ^ (r & 7)) << 4));
    if (r < n) {
      cp_async16(sk + to, a.tk.k + (tok0 + r) * a.tk.k_stride + hk * DK + ch * 8);
      cp_async16(sq + to, a.tk.q + (tok0 + r) * a.tk.q_stride + hk * DK + ch * 8);
    } else {
      *reinterpret_cast<uint4*>(sk + to) = make_uint4(0u, 0u, 0u, 0u);
      *reinterpret_cast<uint4*>(sq + to) = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  for (int i = tid; i < kImg / 16; i += 128)  // the upper triangles stay zero
    reinterpret_cast<uint4*>(sm + ChunkSmem::kImage)[i] = make_uint4(0u, 0u, 0u, 0u);
  cp_async_wait_all();
  __syncthreads();

  // k.k and q.k of the warp's 16 rows (n-tiles up to its own), q.q of its diagonal tile
  const int m = lane >> 2, cc = lane & 3;
  float kk[8][4], qk[8][4], qq[2][4];
#pragma unroll
  for (int t = 0; t < 8; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) kk[t][e] = qk[t][e] = 0.0f;
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) qq[t][e] = 0.0f;
  const uint32_t ak = smem_addr(sk), aq = smem_addr(sq);
  const auto tok_addr = [&](uint32_t base, int row, int ch) {
    return base + static_cast<uint32_t>(row * RB + ((ch ^ (row & 7)) << 4));
  };
  const int arow = (lane & 7) + ((lane >> 3) & 1) * 8, ach = lane >> 4;   // first operand, or a transposed second one
  const int brow = (lane & 7) + ((lane >> 4) << 3), bch = (lane >> 3) & 1;  // second operand, two n-tiles
#pragma unroll
  for (int x = 0; x < KS; ++x) {
    uint32_t fk[4], fq[4], b[4];
    ldsm4(fk, tok_addr(ak, 16 * warp + arow, 2 * x + ach));
    ldsm4(fq, tok_addr(aq, 16 * warp + arow, 2 * x + ach));
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (t <= warp) {
        ldsm4(b, tok_addr(ak, 16 * t + brow, 2 * x + bch));
        mma_bf16(kk[2 * t], fk, b[0], b[1]);
        mma_bf16(kk[2 * t + 1], fk, b[2], b[3]);
        mma_bf16(qk[2 * t], fq, b[0], b[1]);
        mma_bf16(qk[2 * t + 1], fq, b[2], b[3]);
      }
    }
    if (a.tk.l2norm) {
      ldsm4(b, tok_addr(aq, 16 * warp + brow, 2 * x + bch));
      mma_bf16(qq[0], fq, b[0], b[1]);
      mma_bf16(qq[1], fq, b[2], b[3]);
    }
  }
  if (cc == (m >> 1)) {  // the lanes that hold the diagonal
    float k0 = 0.f, k1 = 0.f;
#pragma unroll
    for (int t = 0; t < 4; ++t)
      if (t == warp) {
        k0 = (m & 1) ? kk[2 * t][1] : kk[2 * t][0];
        k1 = (m & 1) ? kk[2 * t + 1][3] : kk[2 * t + 1][2];
      }
    const float q0 = (m & 1) ? qq[0][1] : qq[0][0], q1 = (m & 1) ? qq[1][3] : qq[1][2];
    const int row = 16 * warp + m;
    s_r[row] = a.tk.l2norm ? rsqrtf(k0 + 1e-6f) : 1.0f;
    s_r[row + 8] = a.tk.l2norm ? rsqrtf(k1 + 1e-6f) : 1.0f;
    s_rq[row] = a.tk.scale * (a.tk.l2norm ? rsqrtf(q0 + 1e-6f) : 1.0f);
    s_rq[row + 8] = a.tk.scale * (a.tk.l2norm ? rsqrtf(q1 + 1e-6f) : 1.0f);
  }

  const uint32_t a_hi = smem_addr(sm + ChunkSmem::kA), a_lo = a_hi + 8192;
  const uint32_t img = smem_addr(sm + ChunkSmem::kImage);
  float* fd = reinterpret_cast<float*>(sm + ChunkSmem::kF) + warp * 16 * 17;  // the warp's diagonal block
  float* fi = fd + 4 * 16 * 17;                                              // and its inverse
  const uint32_t d_hi = smem_addr(sm + ChunkSmem::kD) , d_lo = d_hi + 2048;

#pragma unroll 1
  for (int rep = 0; rep < a.c.rep; ++rep) {
    const int h = hk * a.c.rep + rep;
    uint8_t* unit = a.units + (static_cast<long long>(blockIdx.x) * a.c.Hv + h) * kUnit;
    if (warp == 0) {
      // running sums of g in fp64, kept as two floats: differences of them are
      // exponents, and one float's rounding at a sum of 100 would be 2^-18
      double c[2];
      float g[2], be[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = 2 * lane + e;
        g[e] = i < n ? fmaxf(a.tk.g[(tok0 + i) * a.c.Hv + h], kMinLog) : 0.0f;
        be[e] = i < n ? a.tk.beta[(tok0 + i) * a.c.Hv + h] : 0.0f;
      }
      c[0] = g[0];
      c[1] = static_cast<double>(g[0]) + g[1];
      double run = c[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(full, run, o);
        if (lane >= o) run += y;
      }
      const double before = run - c[1];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const double x = before + c[e];
        const float hi = static_cast<float>(x);
        s_ch[2 * lane + e] = hi;
        s_cl[2 * lane + e] = static_cast<float>(x - hi);
        s_beta[2 * lane + e] = be[e];
      }
    }
    __syncthreads();
    if (tid < 64) {
      float* vec = reinterpret_cast<float*>(unit + kImg);
      const float ec = expf(s_ch[tid]), ed = expf((s_ch[63] - s_ch[tid]) + (s_cl[63] - s_cl[tid]));
      vec[tid] = ec * s_r[tid];
      vec[64 + tid] = ed * s_r[tid];
      vec[128 + tid] = ec * s_rq[tid];
      if (tid == 63) vec[192] = ec;
    }
    // A and P of the warp's rows
    uint32_t ph[4][4], pl[4][4];
    {
      const int i0 = 16 * warp + m, i1 = i0 + 8;
      const float ch0 = s_ch[i0], cl0 = s_cl[i0], ch1 = s_ch[i1], cl1 = s_cl[i1];
      const float br0 = s_beta[i0] * s_r[i0], br1 = s_beta[i1] * s_r[i1], rq0 = s_rq[i0], rq1 = s_rq[i1];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if (t > warp) break;
        float p[2][4];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int j = 16 * t + 8 * y + 2 * cc;
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = e < 2 ? i0 : i1, jj = j + (e & 1);
            const float dc = (e < 2 ? ch0 : ch1) - s_ch[jj] + ((e < 2 ? cl0 : cl1) - s_cl[jj]);
            const float w = jj <= i ? __expf(dc) * s_r[jj] : 0.0f;
            v[e] = jj < i ? (e < 2 ? br0 : br1) * w * kk[2 * t + y][e] : 0.0f;
            p[y][e] = jj <= i ? (e < 2 ? rq0 : rq1) * w * qk[2 * t + y][e] : 0.0f;
          }
          if (t == warp) {  // the diagonal block in fp32
            fd[m * 17 + 8 * y + 2 * cc] = v[0];
            fd[m * 17 + 8 * y + 2 * cc + 1] = v[1];
            fd[(m + 8) * 17 + 8 * y + 2 * cc] = v[2];
            fd[(m + 8) * 17 + 8 * y + 2 * cc + 1] = v[3];
          } else {
            uint32_t h0, l0, h1, l1;
            split_bf16x2(v[0], v[1], h0, l0);
            split_bf16x2(v[2], v[3], h1, l1);
            const uint32_t o0 = sw128(i0, 2 * t + y) + 4 * cc, o1 = sw128(i1, 2 * t + y) + 4 * cc;
            *reinterpret_cast<uint32_t*>(sm + ChunkSmem::kA + o0) = h0;
            *reinterpret_cast<uint32_t*>(sm + ChunkSmem::kA + o1) = h1;
            *reinterpret_cast<uint32_t*>(sm + ChunkSmem::kA + 8192 + o0) = l0;
            *reinterpret_cast<uint32_t*>(sm + ChunkSmem::kA + 8192 + o1) = l1;
          }
        }
        as_operand(p, ph[t], pl[t]);
      }
    }
    __syncwarp();
    // inverse of the warp's unit lower triangular diagonal block: a lane per column
    if (lane < 16) {
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float s0 = i == lane ? 1.0f : 0.0f, s1 = 0.0f;
#pragma unroll
        for (int j = 0; j < i; ++j) {
          if (j & 1)
            s1 = fmaf(-fd[i * 17 + j], x[j], s1);
          else
            s0 = fmaf(-fd[i * 17 + j], x[j], s0);
        }
        x[i] = s0 + s1;
        fi[i * 17 + lane] = x[i];
      }
    }
    __syncwarp();
    // its bf16 parts, rows of 32 bytes, and its transpose as this warp's first operand
    uint32_t yh[4][4], yl[4][4];
    {
      const int r = lane >> 1, c0 = (lane & 1) * 8;
      uint32_t hw[4], lw[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) split_bf16x2(fi[r * 17 + c0 + 2 * e], fi[r * 17 + c0 + 2 * e + 1], hw[e], lw[e]);
      const uint32_t to = static_cast<uint32_t>(warp * 512 + r * 32 + c0 * 2);
      *reinterpret_cast<uint4*>(sm + ChunkSmem::kD + to) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
      *reinterpret_cast<uint4*>(sm + ChunkSmem::kD + 2048 + to) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
    }
    float yd[2][4];  // D^T: row = column m of D, column = row of D
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int e = 0; e < 4; ++e) yd[y][e] = fi[(8 * y + 2 * cc + (e & 1)) * 17 + m + (e >> 1) * 8];
    __syncthreads();
    // column block `warp` of the inverse, transposed: Y_i = -(sum_l Y_l A_il^T) D_i^T, l from the diagonal down
    const float bt0 = s_beta[16 * warp + m], bt1 = s_beta[16 * warp + m + 8];
    uint8_t* im = sm + ChunkSmem::kImage;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < warp) continue;
      if (i > warp) {
        float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int l = 0; l < 3; ++l) {
          if (l < warp || l >= i) continue;
          uint32_t bh[4], bl[4];
          ldsm4(bh, a_hi + sw128(16 * i + brow, 2 * l + bch));
          ldsm4(bl, a_lo + sw128(16 * i + brow, 2 * l + bch));
          mma_split(acc, yh[l], yl[l], bh, bl);
        }
        uint32_t h[4], l4[4], bh[4], bl[4];
        as_operand(acc, h, l4);
        ldsm4(bh, d_hi + i * 512 + brow * 32 + bch * 16);
        ldsm4(bl, d_lo + i * 512 + brow * 32 + bch * 16);
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e) yd[y][e] = 0.0f;
        mma_split(yd, h, l4, bh, bl);
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e) yd[y][e] = -yd[y][e];
      }
      as_operand(yd, yh[i], yl[i]);
      // T'[row][column] = Y[column][row] beta[column]
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = 16 * i + 8 * y + 2 * cc + (e & 1), col = 16 * warp + m + (e >> 1) * 8;
          const float v = yd[y][e] * (e < 2 ? bt0 : bt1);
          const __nv_bfloat16 hi = __float2bfloat16_rn(v);
          const uint32_t to = sw128(row, col >> 3) + (col & 7) * 2;
          *reinterpret_cast<__nv_bfloat16*>(im + to) = hi;
          *reinterpret_cast<__nv_bfloat16*>(im + kImgHi + to) = __float2bfloat16_rn(v - __bfloat162float(hi));
        }
    }
    __syncthreads();
    // P T' of the warp's rows
    {
      float o[8][4];
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][e] = 0.0f;
#pragma unroll
      for (int l = 0; l < 4; ++l) {
        if (l > warp) break;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          if (t > l) break;
          uint32_t bh[4], bl[4];
          ldsm4_t(bh, img + sw128(16 * l + arow, 2 * t + ach));
          ldsm4_t(bl, img + kImgHi + sw128(16 * l + arow, 2 * t + ach));
          float(&d)[2][4] = *reinterpret_cast<float(*)[2][4]>(&o[2 * t]);
          mma_split(d, ph[l], pl[l], bh, bl);
        }
      }
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        if (t > 2 * warp + 1) break;
        uint32_t h0, l0, h1, l1;
        split_bf16x2(o[t][0], o[t][1], h0, l0);
        split_bf16x2(o[t][2], o[t][3], h1, l1);
        const uint32_t o0 = sw128(64 + 16 * warp + m, t) + 4 * cc, o1 = sw128(64 + 16 * warp + m + 8, t) + 4 * cc;
        *reinterpret_cast<uint32_t*>(im + o0) = h0;
        *reinterpret_cast<uint32_t*>(im + o1) = h1;
        *reinterpret_cast<uint32_t*>(im + kImgHi + o0) = l0;
        *reinterpret_cast<uint32_t*>(im + kImgHi + o1) = l1;
      }
    }
    __syncthreads();
    for (int i = tid; i < kImg / 16; i += 128) reinterpret_cast<uint4*>(unit)[i] = reinterpret_cast<const uint4*>(im)[i];
    __syncthreads();
  }
  pdl_trigger();
}

// --------------------------------------------------------------------------
// tcgen05 (PTX ISA: 5th generation tensor core instructions)
// --------------------------------------------------------------------------
// Shared-memory operand: start address, leading and stride byte offsets in 16-byte units, version 1, swizzle mode.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lbo, uint32_t sbo, uint64_t swizzle) {
  return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
         (static_cast<uint64_t>(sbo >> 4) << 32) | (1ull << 46) | (swizzle << 61);
}
constexpr uint64_t kSw128 = 2;
// kind::f16, bf16 operands, fp32 accumulators, M = 128
__host__ __device__ constexpr uint32_t instruction(int n, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
         (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_ld8(float* v, uint32_t addr) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tc_st8(uint32_t addr, const float* v) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}

// --------------------------------------------------------------------------
// delta_scan_kernel: one block per (prompt, value head, NDV value columns).
//
// A product's time here is its operands' way out of shared memory (128 bytes a
// cycle: 32 cycles for the 128 rows of a step of 16), so the hi and lo parts of
// S, R and U stand side by side and one instruction takes both: X, U and S have
// a column for each part, added when they are read.
// --------------------------------------------------------------------------
template <int DK, int NDV>
struct ScanSmem {
  static constexpr int kHalves = DK / 64;
  static constexpr int kStages = 2;
  static constexpr int kKQ = 0;  // per 64 key columns: K (64 rows of 128 bytes), then Q
  static constexpr int kHi = kKQ + kHalves * 16384;
  static constexpr int kLo = kHi + kImgHi;
  static constexpr int kV = kLo + kImgHi;
  static constexpr int kVecs = kV + kC * NDV * 2;
  static constexpr int kStage = kVecs + kVec;
  // operands: rows of 128 bytes, for 32 columns hi and lo in one row, for 64 in one block each
  static constexpr int kBlocks = NDV / 32;
  static constexpr int kS = kStages * kStage;
  static constexpr int kR = kS + kBlocks * DK * 128;  // R, then U in its place
  static constexpr int kBars = kR + kBlocks * kC * 128;
  static constexpr int kBytes = kBars + 128 + 1024;  // barriers, and room to start on 1024 bytes
  static constexpr uint32_t kTx = kHalves * 16384 + kImg + kC * NDV * 2 + kVec;
};

constexpr int kWorkWarps = 16;

// Roles.  Warps 0-15 turn accumulators into the next product's operands: warp w
// reads TMEM lanes 32 (w % 4) .. + 31, and a quarter of the value columns by
// w / 4.  In X and U the first 64 lanes are the chunk's tokens (warps with
// w % 4 < 2 make R, then U), the other 64 the same tokens' outputs (the other
// warps store them); of S a lane is a key column.  Warp 16 issues the copies,
// warp 17 the products.
template <int DK, int NDV>
__global__ void __launch_bounds__(kWorkWarps * 32 + 64, 1)
    delta_scan_kernel(const DeltaPrefillArgs a, const __grid_constant__ CUtensorMap mq,
                      const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using L = ScanSmem<DK, NDV>;
  constexpr int CN = NDV / 4;
  constexpr int kTmem = NDV == 32 ? 256 : 512;
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  __shared__ uint32_t tmem_base;
  __shared__ volatile int dead;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tile = blockIdx.x % a.tiles;
  const int h = (blockIdx.x / a.tiles) % a.c.Hv;
  const int b = blockIdx.x / a.tiles / a.c.Hv;
  pdl_wait();
  pdl_trigger();
  int start, n;
  const bool fits = row_bounds(a, b, start, n);
  const int s = a.slot_idx[b];
  const int dv = a.c.dv, dv0 = tile * NDV;
  const long long ostride = static_cast<long long>(a.c.Hv) * dv;
  if (!fits) {
    if (h == 0 && tile == 0 && tid == 0) set_error(a.c.err, RSSM_ERRBIT_SEQLEN);
    return;
  }
  if (s <= 0 || s >= a.c.S) {  // padding: zeros
    const int w = min(NDV, dv - dv0) / 8;
    for (long long i = tid; i < static_cast<long long>(n) * w; i += blockDim.x)
      *reinterpret_cast<uint4*>(a.tk.out + (start + i / w) * ostride + h * dv + dv0 + static_cast<int>(i % w) * 8) =
          make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::kBars);
  uint64_t *b_full = bars, *b_empty = bars + L::kStages, *b_s = bars + 2 * L::kStages, *b_x = b_s + 1, *b_r = b_s + 2,
           *b_u = b_s + 3, *b_up = b_s + 4, *b_new = b_s + 5;
  if (warp == kWorkWarps + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_base)),
                 "n"(kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    dead = 0;
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(b_full + i, 1);
      mbar_init(b_empty + i, 1);
    }
    mbar_init(b_s, kWorkWarps);       // S as an operand
    mbar_init(b_x, 1);                // X, and Y under it
    mbar_init(b_r, kWorkWarps / 2);   // R as an operand
    mbar_init(b_u, 1);                // U, and the outputs' part under it
    mbar_init(b_up, kWorkWarps);      // U as an operand, and S decayed in place
    mbar_init(b_new, 1);              // S after the chunk
    fence_barrier_init();
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tm_s = tmem_base, tm_x = tm_s + 2 * NDV, tm_u = tm_s + 4 * NDV;
  const int chunks = (n + kC - 1) / kC;
  // the chain is a few hundred cycles long between waits: poll before sleeping
  const auto wait = [&](uint64_t* bar, uint32_t parity) {
    for (int i = 0; i < 4096; ++i)
      if (mbar_test(bar, parity)) return true;
    if (dead) return false;
    if (mbar_wait(bar, parity)) return true;
    dead = 1;
    return false;
  };
  // the work warps' waits: a warp goes on, or gives up, as a whole
  const auto wait_warp = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
  const uint8_t* units = a.units + (static_cast<long long>(start / kC + b) * a.c.Hv + h) * kUnit;

  if (warp == kWorkWarps) {
    if (lane == 0) {
      const int hx = (h / a.c.rep) * DK;
      int c = 0;
      for (; c < chunks; ++c) {
        const int st = c % L::kStages;
        if (c >= L::kStages && !wait(b_empty + st, (c / L::kStages - 1) & 1)) break;
        uint8_t* p = sm + st * L::kStage;
        uint64_t* f = b_full + st;
        mbar_arrive_expect_tx(f, L::kTx);
        const uint8_t* unit = units + static_cast<long long>(c) * a.c.Hv * kUnit;
        const int y = start + c * kC;
#pragma unroll
        for (int x = 0; x < L::kHalves; ++x) {
          tma_2d(p + L::kKQ + x * 16384, &mk, hx + 64 * x, y, f);
          tma_2d(p + L::kKQ + x * 16384 + 8192, &mq, hx + 64 * x, y, f);
        }
        tma_2d(p + L::kV, &mv, h * dv + dv0, y, f);
        bulk_g2s(p + L::kHi, unit, kImg, f);
        bulk_g2s(p + L::kVecs, unit + kImg, kVec, f);
      }
      for (int i = max(0, c - L::kStages); i < c; ++i)  // also after a wait that gave up: no copy is in flight at the end
        mbar_wait(b_full + i % L::kStages, (i / L::kStages) & 1);
    }
  } else if (warp == kWorkWarps + 1) {
    if (lane == 0) {
      constexpr uint32_t i_x = instruction(2 * NDV, false, true), i_lo = instruction(NDV, false, true),
                         i_s = instruction(2 * NDV, true, true);
      const uint32_t base = smem_addr(sm);
      // addresses are in the operands' low bits, in units of 16 bytes: offsets are added to them
      const uint64_t d_s = operand(base + L::kS, DK * 128, 1024, kSw128), d_r = operand(base + L::kR, kC * 128, 1024, kSw128);
      const uint64_t d_k = operand(base + L::kKQ, 16, 1024, kSw128);
      // of 64 key columns the second 64 rows of the update are made from the queries, and nobody reads them
      const uint64_t d_kt = operand(base + L::kKQ, DK == 128 ? 16384 : 8192, 1024, kSw128);
      const uint64_t d_hi = operand(base + L::kHi, 16, 1024, kSw128), d_lo = operand(base + L::kLo, 16, 1024, kSw128);
      for (int c = 0; c < chunks; ++c) {
        const int st = c % L::kStages;
        const uint64_t p = static_cast<uint64_t>(st * L::kStage) >> 4;
        if (!wait(b_full + st, (c / L::kStages) & 1) || !wait(b_s, c & 1)) break;
        tc_after();
#pragma unroll
        for (int x = 0; x < DK / 16; ++x)
          tc_mma(tm_x, d_k + p + (((x >> 2) * 16384 + (x & 3) * 32) >> 4), d_s + ((x * 2048) >> 4), i_x, x > 0);
        tc_commit(b_x);
        if (!wait(b_r, c & 1)) break;
        tc_after();
#pragma unroll
        for (int x = 0; x < kC / 16; ++x) tc_mma(tm_u, d_hi + p + ((x * 32) >> 4), d_r + ((x * 2048) >> 4), i_x, x > 0);
#pragma unroll
        for (int x = 0; x < kC / 16; ++x) tc_mma(tm_u, d_lo + p + ((x * 32) >> 4), d_r + ((x * 2048) >> 4), i_lo, true);
        tc_commit(b_u);
        if (!wait(b_up, c & 1)) break;
        tc_after();
#pragma unroll
        for (int x = 0; x < kC / 16; ++x) tc_mma(tm_s, d_kt + p + ((x * 2048) >> 4), d_r + ((x * 2048) >> 4), i_s, true);
        tc_commit(b_new);
        tc_commit(b_empty + st);
      }
    }
  } else {
    const int q = warp & 3, row = 32 * q + lane, c0 = (warp >> 2) * CN;
    const uint32_t at = (static_cast<uint32_t>(32 * q) << 16) + c0;  // this warp's lanes and columns of an accumulator
    const bool is_tok = q < 2, has_s = row < DK;
    const int t = row & 63;
    // v (two sums of parts) from an accumulator's two halves
    const auto get = [&](float* v, uint32_t from) {
      float y[CN];
#pragma unroll
      for (int i = 0; i < CN; i += 8) {
        tc_ld8(v + i, from + at + i);
        tc_ld8(y + i, from + at + NDV + i);
      }
      tc_wait_ld();
#pragma unroll
      for (int i = 0; i < CN; ++i) v[i] += y[i];
    };
    const auto put = [&](int to, int rows, int r, const float* v) {  // as an operand of `rows` rows
#pragma unroll
      for (int i = 0; i < CN; i += 8) {
        uint32_t hw[4], lw[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split_bf16x2(v[i + 2 * e], v[i + 2 * e + 1], hw[e], lw[e]);
        const int ch = (c0 + i) >> 3;
        uint8_t* p = sm + to;
        *reinterpret_cast<uint4*>(p + sw128(r, ch)) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
        *reinterpret_cast<uint4*>(p + (NDV == 32 ? sw128(r, ch + 4) : rows * 128 + sw128(r, ch))) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
      }
    };
    const auto arrive = [&](uint64_t* bar) {
      tc_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    const long long head = s * a.c.state_stride + (static_cast<long long>(h) * dv + dv0 + c0) * DK + row;
    const int cols = min(CN, dv - dv0 - c0);  // of this warp's columns those that exist (may be negative)
    float v[CN];
    const bool go_on = a.initial && a.initial[b] != 0;
#pragma unroll
    for (int i = 0; i < CN; ++i) {
      v[i] = 0.0f;
      if (go_on && has_s && i < cols)
        v[i] = a.c.dtype == RSSM_F32 ? static_cast<const float*>(a.c.state)[head + static_cast<long long>(i) * DK]
                                     : bf16f(static_cast<const uint16_t*>(a.c.state)[head + static_cast<long long>(i) * DK]);
    }
    bool ok = true;
    for (int c = 0; c < chunks; ++c) {
      const int st = c % L::kStages;
      uint8_t* p = sm + st * L::kStage;
      const float* vec = reinterpret_cast<const float*>(p + L::kVecs);
      const int live = min(n - c * kC, kC);
      ok = wait_warp(b_full + st, (c / L::kStages) & 1);
      ok = ok && (c == 0 || wait_warp(b_new, (c - 1) & 1));
      if (!ok) break;
      if (live < kC) {  // keys past the prompt's end may be another prompt's: whatever they are, they must not count
        for (int i = tid; i < (kC - live) * L::kHalves * 8; i += kWorkWarps * 32) {
          const int r = live + i / (L::kHalves * 8), x = i % (L::kHalves * 8);
          *reinterpret_cast<uint4*>(p + L::kKQ + (x >> 3) * 16384 + r * 128 + (x & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      if (has_s) {
        if (c > 0) {
          tc_after();
          get(v, tm_s);
        }
        put(L::kS, DK, row, v);
      }
      fence_async();
      arrive(b_s);
      // while X is formed: the decayed S in place, and what this thread needs of the decay vectors
      const float w0 = vec[is_tok ? t : 128 + t], w1 = vec[64 + t], ec = vec[192];
      if (has_s) {
        float zero[CN];
#pragma unroll
        for (int i = 0; i < CN; ++i) {
          v[i] *= ec;
          zero[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < CN; i += 8) {
          tc_st8(tm_s + at + i, v + i);
          tc_st8(tm_s + at + NDV + i, zero + i);
        }
        tc_wait_st();
      }
      uint32_t xw[CN / 2];
      if (is_tok) {
#pragma unroll
        for (int i = 0; i < CN; i += 8) {
          const int ch = (c0 + i) >> 3;
          const uint4 x = *reinterpret_cast<const uint4*>(
              p + L::kV + (NDV == 32 ? t * 64 + ((ch ^ ((t >> 1) & 3)) << 4) : static_cast<int>(sw128(t, ch))));
          xw[i / 2] = x.x;
          xw[i / 2 + 1] = x.y;
          xw[i / 2 + 2] = x.z;
          xw[i / 2 + 3] = x.w;
        }
      } else {
        arrive(b_up);
      }
      if (!(ok = wait_warp(b_x, c & 1))) break;
      tc_after();
      get(v, tm_x);
      if (is_tok) {
#pragma unroll
        for (int i = 0; i < CN; i += 2) {
          v[i] = t < live ? fmaf(-w0, v[i], bf16lo(xw[i / 2])) : 0.0f;
          v[i + 1] = t < live ? fmaf(-w0, v[i + 1], bf16hi(xw[i / 2])) : 0.0f;
        }
        put(L::kR, kC, t, v);
        fence_async();
        arrive(b_r);
      }
      if (!(ok = wait_warp(b_u, c & 1))) break;
      tc_after();
      float u[CN];
      get(u, tm_u);
      if (is_tok) {
#pragma unroll
        for (int i = 0; i < CN; ++i) u[i] *= w1;
        put(L::kR, kC, t, u);
        fence_async();
        arrive(b_up);
      } else if (t < live) {
        uint16_t* o = a.tk.out + (start + c * kC + t) * ostride + h * dv + dv0 + c0;
#pragma unroll
        for (int i = 0; i < CN; i += 8) {
          if (i < cols) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = cvt_bf16x2(fmaf(w0, v[i + 2 * e], u[i + 2 * e]), fmaf(w0, v[i + 2 * e + 1], u[i + 2 * e + 1]));
            *reinterpret_cast<uint4*>(o + i) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    }
    if (ok && chunks > 0) {
      ok = wait_warp(b_new, (chunks - 1) & 1);
      if (ok && has_s) {
        tc_after();
        get(v, tm_s);
      }
    }
    if (ok && has_s) {
#pragma unroll
      for (int i = 0; i < CN; ++i) {
        if (i >= cols) break;
        if (a.c.dtype == RSSM_F32)
          static_cast<float*>(a.c.state)[head + static_cast<long long>(i) * DK] = v[i];
        else
          static_cast<__nv_bfloat16*>(a.c.state)[head + static_cast<long long>(i) * DK] = __float2bfloat16_rn(v[i]);
      }
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == kWorkWarps + 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "n"(kTmem) : "memory");
  if (tid == 0) {
    if (dead) set_error(a.c.err, RSSM_ERRBIT_TIMEOUT);
    if (h == 0 && tile == 0) reinterpret_cast<int2*>(a.c.pend)[s] = make_int2(0, 0);
  }
}

bool al(const void* p, unsigned n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// token rows of `width` bf16, boxes of 64 tokens x `cols` columns, swizzled over the box's row
bool token_map(CUtensorMap* map, const void* p, long long width, long long tokens, long long stride, int cols) {
  auto enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(cols), kC}, estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename K>
cudaError_t grow_smem(K kernel, size_t bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}

template <int DK>
cudaError_t launch_chunks(const DeltaPrefillArgs& a, cudaStream_t st) {
  constexpr size_t smem = ChunkSmem::kTokens + 2 * kC * DK * 2;
  const cudaError_t e = grow_smem(delta_chunk_kernel<DK>, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(delta_chunk_kernel<DK>, dim3(static_cast<unsigned>(a.tokens / kC + a.batch), a.c.Hk), dim3(128), smem, st, a);
}

template <int DK, int NDV>
cudaError_t launch_scan(DeltaPrefillArgs a, cudaStream_t st) {
  CUtensorMap mq = {}, mk = {}, mv = {};
  if (a.tokens > 0 && (!token_map(&mq, a.tk.q, a.c.Hk * DK, a.tokens, a.tk.q_stride, 64) ||
                       !token_map(&mk, a.tk.k, a.c.Hk * DK, a.tokens, a.tk.k_stride, 64) ||
                       !token_map(&mv, a.tk.v, a.c.Hv * a.c.dv, a.tokens, a.tk.v_stride, NDV)))
    return cudaErrorInvalidValue;
  constexpr size_t smem = ScanSmem<DK, NDV>::kBytes;
  const cudaError_t e = grow_smem(delta_scan_kernel<DK, NDV>, smem);
  if (e != cudaSuccess) return e;
  a.tiles = (a.c.dv + NDV - 1) / NDV;
  return launch_pdl(delta_scan_kernel<DK, NDV>, dim3(static_cast<unsigned>(static_cast<long long>(a.batch) * a.c.Hv * a.tiles)),
                    dim3(kWorkWarps * 32 + 64), smem, st, a, mq, mk, mv);
}

size_t ticket_bytes(int batch) { return align_up(static_cast<size_t>(batch) * sizeof(unsigned) + 1, 256); }

}  // namespace
}  // namespace rssm

using namespace rssm;

extern "C" size_t rssm_delta_scratch_bytes(const rssm_delta_cache* cache, int32_t batch, int64_t tokens) {
  DeltaCacheView c;
  rssm_status st;
  if (!delta_view(cache, &c, &st) || batch < 0 || tokens < 0) return 0;
  return ticket_bytes(batch) + static_cast<size_t>(tokens / kC + batch) * c.Hv * kUnit;
}

extern "C" rssm_status rssm_delta_prefill(const rssm_delta_cache* cache, const void* q, int64_t q_stride, const void* k,
                                          int64_t k_stride, const void* v, int64_t v_stride, const float* g,
                                          const float* beta, float scale, int32_t l2norm, const int32_t* slot_idx,
                                          const int32_t* cu_seqlens, const int32_t* initial, int32_t batch,
                                          int64_t tokens, void* out, void* scratch, size_t scratch_bytes, void* stream) {
  DeltaPrefillArgs a = {};
  rssm_status st;
  if (!delta_view(cache, &a.c, &st)) return st;
  if (batch < 0 || tokens < 0 || tokens > 0x7fffffffll - kC) return RSSM_ERR_INVALID_ARGUMENT;
  if (batch == 0) return RSSM_OK;
  if (!al(slot_idx, 4) || !al(cu_seqlens, 4) || (initial && !al(initial, 4)) || !al(scratch, 16)) return RSSM_ERR_INVALID_ARGUMENT;
  if (tokens > 0) {
    st = delta_tokens(a.c, cache->dkey, q, k, v, q_stride, k_stride, v_stride, g, beta, scale, l2norm, out, &a.tk);
    if (st != RSSM_OK) return st;
  }
  if (scratch_bytes < rssm_delta_scratch_bytes(cache, batch, tokens)) return RSSM_ERR_SCRATCH_TOO_SMALL;
  if (static_cast<long long>(batch) * a.c.Hv * ((a.c.dv + 31) / 32) > 0x7fffffffll || a.c.Hk > 65535) return RSSM_ERR_UNSUPPORTED;
  a.slot_idx = slot_idx;
  a.cu = cu_seqlens;
  a.initial = initial;
  a.batch = batch;
  a.tokens = tokens;
  a.units = static_cast<uint8_t*>(scratch) + ticket_bytes(batch);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  // Value columns of a block.  A chunk's chain takes little longer for 64 than
  // for 32, so 32 only where the blocks then still run all at once.
  const int sms = num_sms();
  if (sms == 0) return RSSM_ERR_CUDA;
  const bool narrow = a.c.dv <= 32 || static_cast<long long>(batch) * a.c.Hv * ((a.c.dv + 31) / 32) <= sms;
  cudaError_t e;
  if (cache->dkey == 128) {
    e = launch_chunks<128>(a, cs);
    if (e == cudaSuccess) e = narrow ? launch_scan<128, 32>(a, cs) : launch_scan<128, 64>(a, cs);
  } else {
    e = launch_chunks<64>(a, cs);
    if (e == cudaSuccess) e = narrow ? launch_scan<64, 32>(a, cs) : launch_scan<64, 64>(a, cs);
  }
  return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}
