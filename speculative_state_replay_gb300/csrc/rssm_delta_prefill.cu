// rssm_delta_prefill.cu -- the gated delta rule over whole prompts, in chunks
// of 64 tokens on the tensor cores.
//
// Within a chunk, with c the running sum of g, r = 1/|k| (1 without
// normalisation) and the keys as given,
//     A[i][j] = beta_i e^{c_i - c_j} r_i r_j (k_i . k_j)      (j < i)
//     T       = (I + A)^-1
//     P[i][j] = scale e^{c_i - c_j} rq_i r_j (q_i . k_j)      (j <= i)
// and, with S the state before the chunk (X = K S^T, Y = Q S^T),
//     R = diag(beta) (V - diag(e^c r) X),   U = T R,
//     O = diag(scale e^c rq) Y + (P T) R,
//     S <- e^{c_end} S + (diag(e^{c_end - c} r) U)^T K.
// T, P T and the decay vectors do not depend on the state: delta_chunk_kernel
// forms them for every chunk at once (scratch).  delta_scan_kernel then walks
// each prompt's chunks in order; its chain per chunk is three products, X (with
// Y on top: one product of 128 rows), U (with (P T) R on top) and the state's
// update.  The large products of both kernels are tcgen05's, with accumulators
// in TMEM.
//
// Precision: products run in bf16 with fp32 accumulation.  Keys, queries and
// values are exact; fp32 factors (S, A, T, P T, R, U) are carried as bf16 hi +
// lo, 16 significant bits, and the product of two lo parts (2^-18 of the term)
// is dropped.  For an fp32 state U is R + (T - I) R, R added in fp32, and U, which
// the state sums, goes in three parts, which is all of it.  Of a prompt of 16384
// tokens with random keys the state is then 2.3e-7 of its norm off, 638 us; without
// both it was 3e-6 off in 602 us, which is enough for a bf16 state: that is rounded
// to 2^-9.  What is left comes from T - I, R and S alike, and grows with T - I:
// 1000 tokens whose keys are correlated by 0.7 (0.95) leave the state 1.5e-6
// (2e-6) off, and with rates above 0.9 and hardly a decay 6e-6 (1.5e-5), where
// fp32 token by token is 1e-7 .. 3e-7.  Three parts of all of them would be as
// exact, with half as many operand bytes again for the chain and 32 KB more shared
// memory, which blocks of 64 value columns do not have: rssm_delta_step is the call
// for that.  Outputs are rounded to bf16 once.  (P T rounded to bf16 would save a
// quarter of the scratch traffic, but of a prompt of few tokens all outputs would
// share its error: up to 2^-8 more.)
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "rssm_delta.cuh"

namespace rssm {
namespace {

constexpr int kC = 64;                   // tokens of a chunk
constexpr int kImgHi = 128 * 128;        // bytes: T (fp32 states: T - I; 64 rows), then P T (64 rows), rows of 64 bf16: the hi parts
constexpr int kImg = 2 * kImgHi;         // and the lo parts
constexpr int kVec = 1040;               // bytes: beta e^c r [64], e^{c_end-c} r [64], scale e^c rq [64], beta [64], e^{c_end}
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

// A prompt's chunks are in scratch from slot cu / 64 + b on: of bounds that never
// fall no two prompts share a slot, and the last slot is below tokens / 64 +
// batch.  Where bounds fall, a row that begins before an earlier bound is skipped
// (begins_inside), so that what is left of them never falls either.
__device__ __forceinline__ bool row_bounds(const DeltaPrefillArgs& a, int b, int& start, int& n) {
  start = a.cu[b];
  const long long m = static_cast<long long>(a.cu[b + 1]) - start;
  n = static_cast<int>(m);
  return start >= 0 && m >= 0 && start + m <= a.tokens;
}
// whether one of the bounds i0, i0 + step, .. up to row b's own lies past its start (bounds that are none do not count)
__device__ __forceinline__ bool begins_inside(const DeltaPrefillArgs& a, int b, int start, int i0, int step) {
  bool inside = false;
  for (int i = i0; i < b; i += step) inside |= a.cu[i] > start && a.cu[i] <= a.tokens;
  return inside;
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
__device__ __forceinline__ void stsm4_t(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3])
               : "memory");
}
// bulk copy shared -> global (16-byte boundaries and multiples), and the wait until this thread's have left shared memory
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_addr(src)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_s2g_wait() {
  asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
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
// 8 columns of the warp's lanes: the registers hold them only after
// tc_wait_ld and are not to be touched before (tc_landed)
__device__ __forceinline__ void tc_ld8(uint32_t (&r)[8], uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr)
               : "memory");
}
// after tc_wait_ld: uses of r stay behind it
__device__ __forceinline__ void tc_landed(uint32_t (&r)[8]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]));
}
__device__ __forceinline__ void tc_st8(uint32_t addr, const pair* v) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack2(v[i], f[2 * i], f[2 * i + 1]);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "f"(f[0]), "f"(f[1]),
               "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
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
// delta_chunk_kernel: one block of 4 warps per (chunk, value head).
//
// The Gram products of the keys and of the queries with the keys are one
// product of 128 rows; a thread then has a row of A (threads 0-63) or of P.
// The inverse goes by blocks of 16: the diagonal ones by substitution, then
// joined twice, [T1 0; -T2 A21 T1  T2].  The block chain is a string of small
// dependent steps, so what matters is how many blocks an SM holds: four, for
// which A and P take the place of the keys and queries in shared memory, and
// P T that of A.
// --------------------------------------------------------------------------
struct ChunkSmem {
  static constexpr int kHi = 0;                   // K and Q per 64 columns as in the scan; A (64 rows) and P, the hi parts,
  static constexpr int kLo = kImgHi;              // and the lo parts; P T for A
  static constexpr int kT = 2 * kImgHi;           // T (64 rows), hi and lo parts
  static constexpr int kDiag = kT + 2 * 8192;     // diagonal blocks of A in fp32, then their inverses: 4 x 16 x 20
  static constexpr int kScalars = kDiag + 4 * 16 * 20 * 4;  // c hi, c lo, beta, r, rq, column factors: 6 x 64 floats
  static constexpr int kBars = kScalars + 6 * 64 * 4;
  static constexpr int kBytes = kBars + 64 + 1024;
};

template <int DK>
__global__ void __launch_bounds__(128, 4)
    delta_chunk_kernel(const DeltaPrefillArgs a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk) {
  extern __shared__ uint8_t raw[];
  uint8_t* sm = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  __shared__ int sh[3];
  __shared__ uint32_t tmem_base;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.y, hk = h / a.c.rep;
  const unsigned full = 0xffffffffu;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + ChunkSmem::kBars);  // copies, Gram products, P T
  if (tid == 0) {
    sh[0] = -1;
    mbar_init(bars, 1);
    mbar_init(bars + 1, 1);
    mbar_init(bars + 2, 1);
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_base)), "n"(128) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  const auto holds = [&](int b, int& start, int& n) {  // whether this slot is one of row b's
    if (!row_bounds(a, b, start, n)) return false;
    const int i = static_cast<int>(blockIdx.x) - (start / kC + b);
    return i >= 0 && i < (n + kC - 1) / kC && a.slot_idx[b] > 0 && a.slot_idx[b] < a.c.S;
  };
  const auto take = [&](int b, int start, int n) {
    const int i = static_cast<int>(blockIdx.x) - (start / kC + b);
    sh[0] = b;
    sh[1] = start + i * kC;
    sh[2] = min(n - i * kC, kC);
  };
  bool malformed = false;
  for (int b = tid; b < a.batch; b += 128) {
    int start, n;
    if (holds(b, start, n)) take(b, start, n);
    malformed |= !row_bounds(a, b, start, n);
  }
  tc_before();
  if (__syncthreads_or(malformed)) {  // more than one row may have taken the slot: the one that is not skipped has it
    if (tid == 0) sh[0] = -1;
    __syncthreads();
    for (int b = tid; b < a.batch; b += 128) {
      int start, n;
      if (holds(b, start, n) && !begins_inside(a, b, start, 0, 1)) take(b, start, n);
    }
    __syncthreads();
  }
  tc_after();
  const uint32_t tm = tmem_base;
  const auto release = [&]() {
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "n"(128) : "memory");
  };
  if (sh[0] < 0) {  // an unused slot
    release();
    return;
  }
  const int tok0 = sh[1], n = sh[2];
  float* s_ch = reinterpret_cast<float*>(sm + ChunkSmem::kScalars);
  float *s_cl = s_ch + 64, *s_beta = s_cl + 64, *s_r = s_beta + 64, *s_rq = s_r + 64, *s_col = s_rq + 64;
  uint8_t *kq = sm, *s_t = sm + ChunkSmem::kT;  // T
  const uint32_t base = smem_addr(sm);
  if (tid == 0) {
    mbar_arrive_expect_tx(bars, DK * 2 * 128);
#pragma unroll
    for (int x = 0; x < DK / 64; ++x) {
      tma_2d(kq + x * 16384, &mk, hk * DK + 64 * x, tok0, bars);
      tma_2d(kq + x * 16384 + 8192, &mq, hk * DK + 64 * x, tok0, bars);
    }
  }
  constexpr uint32_t i_gram = instruction(64, false, false), i_pt = instruction(64, false, true);
  if (warp == 2) {
    // running sums of g, two tokens a lane
    float g[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * lane + e;
      const long long at = static_cast<long long>(tok0 + i) * a.c.Hv + h;
      g[e] = i < n ? held_log(a.tk.g[at]) : 0.0f;
      s_beta[i] = i < n ? a.tk.beta[at] : 0.0f;
    }
    LongSum run = {g[0], 0.0f};
    run.add(g[1], 0.0f);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float yh = __shfl_up_sync(full, run.hi, o), yl = __shfl_up_sync(full, run.lo, o);
      if (lane >= o) run.add(yh, yl);
    }
    LongSum c = {__shfl_up_sync(full, run.hi, 1), __shfl_up_sync(full, run.lo, 1)};
    if (lane == 0) c = {0.0f, 0.0f};
    c.add(g[0], 0.0f);
    c.settle();
    run.settle();
    s_ch[2 * lane] = c.hi;
    s_cl[2 * lane] = c.lo;
    s_ch[2 * lane + 1] = run.hi;
    s_cl[2 * lane + 1] = run.lo;
  }
  bool ok = mbar_wait(bars, 0);
  if (tid == 32 && ok) {
    const uint64_t d = operand(base, 16, 1024, kSw128);
#pragma unroll
    for (int x = 0; x < DK / 16; ++x) {
      const uint64_t k = d + (((x >> 2) * 16384 + (x & 3) * 32) >> 4);
      tc_mma(tm, k, k, i_gram, x > 0);
    }
    tc_commit(bars + 1);
  }
  __syncwarp();
  // meanwhile the norm of the thread's key (query)
  const int i = tid & 63;
  const bool is_key = tid < 64, live = i < n;
  {
    float ss = 0.0f, s1 = 0.0f;
    if (a.tk.l2norm) {
#pragma unroll
      for (int x = 0; x < DK / 64; ++x)
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
          const uint4 w = *reinterpret_cast<const uint4*>(kq + x * 16384 + sw128(tid, ch));
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ss = fmaf(bf16lo(u[e]), bf16lo(u[e]), ss);
            s1 = fmaf(bf16hi(u[e]), bf16hi(u[e]), s1);
          }
        }
    }
    float r = a.tk.l2norm ? rsqrtf(ss + s1 + 1e-6f) : 1.0f;
    if (!live) r = 0.0f;  // whatever is past the chunk's end must not count
    (is_key ? s_r : s_rq)[i] = is_key ? r : a.tk.scale * r;
  }
  __syncthreads();
  uint8_t* unit = a.units + (static_cast<long long>(blockIdx.x) * a.c.Hv + h) * kUnit;
  const float ch = s_ch[i], cl = s_cl[i];
  if (is_key) {
    // decays of a row go through the end of the column's block: a factor of the column, at most 1, and one of the row
    const int end = i | 15;
    s_col[i] = live ? expf((s_ch[end] - ch) + (s_cl[end] - cl)) * s_r[i] : 0.0f;
    float* vec = reinterpret_cast<float*>(unit + kImg);
    const float ec = exp_sum(ch, cl);
    vec[i] = s_beta[i] * ec * s_r[i];
    vec[64 + i] = expf((s_ch[63] - ch) + (s_cl[63] - cl)) * s_r[i];
    vec[128 + i] = ec * s_rq[i];
    vec[192 + i] = s_beta[i];
    if (i == 63) vec[256] = ec;
  }
  __syncthreads();
  ok = ok && mbar_wait(bars + 1, 0);
  tc_after();
  // the thread's row of A (P), in blocks of 16 columns
  {
    const float rf = live ? (is_key ? s_beta[i] * s_r[i] : s_rq[i]) : 0.0f;
    float* fd = reinterpret_cast<float*>(sm + ChunkSmem::kDiag) + i * 20;
    const uint32_t lanes = tm + (static_cast<uint32_t>(32 * warp) << 16);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      pair v[8];
      if (b <= ((32 * warp + 31) & 63) / 16) {  // some row of the warp reaches the block
        uint32_t x[2][8];
        tc_ld8(x[0], lanes + 16 * b);
        tc_ld8(x[1], lanes + 16 * b + 8);
        tc_wait_ld();
        tc_landed(x[0]);
        tc_landed(x[1]);
        // the row's factor is at most 1 past the block, and in its own block as
        // large as the block's decay is small: up to e^60 the factors serve there too
        const float up = (ch - s_ch[16 * b + 15]) + (cl - s_cl[16 * b + 15]);
        const float f = expf(up) * rf;
        const pair f2 = pack2(f, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[e] = *reinterpret_cast<const pair*>(s_col + 16 * b + 2 * e);
          mul2(v[e], f2);
          mul2(v[e], pack2(__uint_as_float(x[e >> 2][2 * (e & 3)]), __uint_as_float(x[e >> 2][2 * (e & 3) + 1])));
        }
        const int d = i - 16 * b;  // the row's diagonal column
        if (d < 16) {
          float y[16];
#pragma unroll
          for (int e = 0; e < 8; ++e) unpack2(v[e], y[2 * e], y[2 * e + 1]);
          if (up > 60.0f && d >= 0) {
#pragma unroll 1
            for (int e = 0; e < 16; ++e) {
              const float w = expf((ch - s_ch[16 * b + e]) + (cl - s_cl[16 * b + e])) * (rf * s_r[16 * b + e]);
#pragma unroll
              for (int k = 0; k < 16; ++k)
                if (k == e) y[k] = w * __uint_as_float(x[k >> 3][k & 7]);
            }
          }
          const int last = is_key ? d : d + 1;
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = pack2(2 * e < last ? y[2 * e] : 0.0f, 2 * e + 1 < last ? y[2 * e + 1] : 0.0f);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0ull;
      }
      if (!live) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0ull;
      }
      if (is_key && b == (i >> 4)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) *reinterpret_cast<ulonglong2*>(fd + 4 * e) = make_ulonglong2(v[2 * e], v[2 * e + 1]);
      }
      uint32_t hw[8], lw[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) split_bf16x2(v[e], hw[e], lw[e]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t to = sw128(tid, 2 * b + e);
        *reinterpret_cast<uint4*>(sm + ChunkSmem::kHi + to) = make_uint4(hw[4 * e], hw[4 * e + 1], hw[4 * e + 2], hw[4 * e + 3]);
        *reinterpret_cast<uint4*>(sm + ChunkSmem::kLo + to) = make_uint4(lw[4 * e], lw[4 * e + 1], lw[4 * e + 2], lw[4 * e + 3]);
      }
    }
  }
  // T is zero above its diagonal
  for (int x = tid; x < 2 * 64 * 8; x += 128) *reinterpret_cast<uint4*>(s_t + x * 16) = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
  {
    // inverse of the warp's unit lower triangular diagonal block: a lane per column
    float* fd = reinterpret_cast<float*>(sm + ChunkSmem::kDiag) + warp * 16 * 20;
    float x[16];
    if (lane < 16) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        float s0 = r == lane ? 1.0f : 0.0f, s1 = 0.0f;
#pragma unroll
        for (int j = 0; j < r; j += 4) {
          const float4 w = *reinterpret_cast<const float4*>(fd + r * 20 + j);
          s0 = fmaf(-w.x, x[j], s0);
          if (j + 1 < r) s1 = fmaf(-w.y, x[j + 1], s1);
          if (j + 2 < r) s0 = fmaf(-w.z, x[j + 2], s0);
          if (j + 3 < r) s1 = fmaf(-w.w, x[j + 3], s1);
        }
        x[r] = s0 + s1;
      }
    }
    __syncwarp();
    if (lane < 16) {
#pragma unroll
      for (int r = 0; r < 16; ++r) fd[r * 20 + lane] = x[r];
    }
    __syncwarp();
    const int r = lane >> 1, c0 = (lane & 1) * 8;
    uint32_t hw[4], lw[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) split_bf16x2(fd[r * 20 + c0 + 2 * e], fd[r * 20 + c0 + 2 * e + 1], hw[e], lw[e]);
    const uint32_t to = sw128(16 * warp + r, 2 * warp + (lane & 1));
    *reinterpret_cast<uint4*>(s_t + to) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
    *reinterpret_cast<uint4*>(s_t + 8192 + to) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
  }
  // block (br, bc) of a 64 x 64 matrix as a second operand (its transpose: rows of it are columns), or, with .trans,
  // its transpose as a first operand; the same addresses store a transposed accumulator
  const auto block = [&](uint32_t m, int br, int bc) {
    return m + sw128(16 * br + (lane & 7) + ((lane >> 4) << 3), 2 * bc + ((lane >> 3) & 1));
  };
  const uint32_t t_hi = base + ChunkSmem::kT, t_lo = t_hi + 8192, a_hi = base + ChunkSmem::kHi, a_lo = base + ChunkSmem::kLo;
  // d += (T_lc)^T (A_il)^T for one l
  const auto first = [&](float (&d)[2][4], int l, int c, int r) {
    uint32_t th[4], tl[4], bh[4], bl[4];
    ldsm4_t(th, block(t_hi, l, c));
    ldsm4_t(tl, block(t_lo, l, c));
    ldsm4(bh, block(a_hi, r, l));
    ldsm4(bl, block(a_lo, r, l));
    mma_split(d, th, tl, bh, bl);
  };
  // d -= y (T_rl)^T
  const auto second = [&](float (&d)[2][4], const uint32_t (&yh)[4], const uint32_t (&yl)[4], int r, int l) {
    uint32_t bh[4], bl[4];
    ldsm4(bh, block(t_hi, r, l));
    ldsm4(bl, block(t_lo, r, l));
    mma_split(d, yh, yl, bh, bl);
  };
  const auto save = [&](float (&d)[2][4], int r, int c) {
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int e = 0; e < 4; ++e) d[y][e] = -d[y][e];
    uint32_t h4[4], l4[4];
    as_operand(d, h4, l4);
    stsm4_t(block(t_hi, r, c), h4);
    stsm4_t(block(t_lo, r, c), l4);
  };
  __syncthreads();
  if (warp < 2) {  // blocks (1, 0) and (3, 2)
    const int c = 2 * warp;
    float y[2][4] = {}, z[2][4] = {};
    uint32_t yh[4], yl[4];
    first(y, c, c, c + 1);
    as_operand(y, yh, yl);
    second(z, yh, yl, c + 1, c + 1);
    save(z, c + 1, c);
  }
  __syncthreads();
  if (warp < 2) {  // blocks (2, c) and (3, c): the lower left 32 x 32, a column of blocks each
    const int c = warp;
    uint32_t yh[2][4], yl[2][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float y[2][4] = {};
      if (c == 0) first(y, 0, c, 2 + r);
      first(y, 1, c, 2 + r);
      as_operand(y, yh[r], yl[r]);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float z[2][4] = {};
      second(z, yh[0], yl[0], 2 + r, 2);
      if (r == 1) second(z, yh[1], yl[1], 3, 3);
      save(z, 2 + r, c);
    }
  }
  fence_async();
  tc_before();
  __syncthreads();
  tc_after();
  // P T: P is rows 64-127 of its operand, so that the result is in the lanes of the threads that store it
  if (tid == 0 && ok) {
    const uint64_t ph = operand(a_hi, 16, 1024, kSw128), pl = operand(a_lo, 16, 1024, kSw128);
    const uint64_t bh = operand(t_hi, 16, 1024, kSw128), bl = operand(t_lo, 16, 1024, kSw128);
#pragma unroll
    for (int part = 0; part < 3; ++part)
#pragma unroll
      for (int x = 0; x < 4; ++x)
        tc_mma(tm + 64, (part == 1 ? pl : ph) + ((x * 32) >> 4), (part == 2 ? bl : bh) + ((x * 2048) >> 4), i_pt, part || x);
    tc_commit(bars + 2);
  }
  ok = ok && mbar_wait(bars + 2, 0);
  tc_after();
  if (warp < 2) {
    // for an fp32 state the scan's product takes T - I: what the ones would add it adds itself
    if (a.c.dtype == RSSM_F32) *reinterpret_cast<uint16_t*>(s_t + sw128(tid, tid >> 3) + (tid & 7) * 2) = 0;
  } else {
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      uint32_t x[8], hw[4], lw[4];
      tc_ld8(x, tm + 64 + (static_cast<uint32_t>(32 * warp) << 16) + 8 * b);
      tc_wait_ld();
      tc_landed(x);
#pragma unroll
      for (int e = 0; e < 4; ++e) split_bf16x2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]), hw[e], lw[e]);
      const uint32_t to = sw128(i, b);
      *reinterpret_cast<uint4*>(sm + ChunkSmem::kHi + to) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
      *reinterpret_cast<uint4*>(sm + ChunkSmem::kLo + to) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
    }
  }
  fence_async();
  tc_before();
  const bool all_ok = __syncthreads_and(ok) != 0;
  if (!all_ok) {  // once more, with their limits: neither copies nor products must outlive the block
    if (tid == 0)
      for (int x = 0; x < 3; ++x) mbar_wait(bars + x, 0);
    __syncthreads();
  }
  tc_after();
  release();
  if (tid == 0) {
    if (!all_ok) set_error(a.c.err, RSSM_ERRBIT_TIMEOUT);
    bulk_s2g(unit, s_t, 8192);
    bulk_s2g(unit + 8192, sm + ChunkSmem::kHi, 8192);
    bulk_s2g(unit + kImgHi, s_t + 8192, 8192);
    bulk_s2g(unit + kImgHi + 8192, sm + ChunkSmem::kLo, 8192);
    bulk_s2g_wait();
  }
  pdl_trigger();
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
  static constexpr int kStage = kVecs + 2048;  // the next one starts on 1024 bytes too
  // operands: rows of 128 bytes, for 32 columns hi and lo in one row, for 64 in one block each
  static constexpr int kBlocks = NDV / 32;
  static constexpr int kS = kStages * kStage;
  static constexpr int kR = kS + kBlocks * DK * 128;  // R, then U in its place
  static constexpr int kRest = kR + kBlocks * kC * 128;  // what of U hi and lo leave
  static constexpr int kBars = kRest + kC * 128;
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
template <int DK, int NDV, bool F32>
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
  if (__syncthreads_or(begins_inside(a, b, start, tid, blockDim.x)) || !fits) {
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
  // (polling with test_wait instead of try_wait, or by one lane for its warp, is slower: 618 and 639 us where this took 602)
  const auto wait = [&](uint64_t* bar, uint32_t parity) {
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
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
                         i_s = instruction(2 * NDV, true, true), i_rest = instruction(NDV, true, true);
      const uint32_t base = smem_addr(sm);
      // addresses are in the operands' low bits, in units of 16 bytes: offsets are added to them
      const uint64_t d_s = operand(base + L::kS, DK * 128, 1024, kSw128), d_r = operand(base + L::kR, kC * 128, 1024, kSw128);
      const uint64_t d_rest = operand(base + L::kRest, kC * 128, 1024, kSw128);
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
        if (F32) {
#pragma unroll
          for (int x = 0; x < kC / 16; ++x) tc_mma(tm_s, d_kt + p + ((x * 2048) >> 4), d_rest + ((x * 2048) >> 4), i_rest, true);
        }
        tc_commit(b_new);
        tc_commit(b_empty + st);
      }
    }
  } else {
    const int q = warp & 3, row = 32 * q + lane, c0 = (warp >> 2) * CN;
    const uint32_t at = (static_cast<uint32_t>(32 * q) << 16) + c0;  // this warp's lanes and columns of an accumulator
    const bool is_tok = q < 2, has_s = row < DK;
    const int t = row & 63;
    // CN values as pairs, an accumulator's two halves added
    const auto get = [&](pair* v, uint32_t from) {
      uint32_t x[CN / 8][8], y[CN / 8][8];
#pragma unroll
      for (int i = 0; i < CN / 8; ++i) {
        tc_ld8(x[i], from + at + 8 * i);
        tc_ld8(y[i], from + at + NDV + 8 * i);
      }
      tc_wait_ld();
#pragma unroll
      for (int i = 0; i < CN / 8; ++i) {
        tc_landed(x[i]);
        tc_landed(y[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[4 * i + e] = pack2(__uint_as_float(x[i][2 * e]), __uint_as_float(x[i][2 * e + 1]));
          add2(v[4 * i + e], pack2(__uint_as_float(y[i][2 * e]), __uint_as_float(y[i][2 * e + 1])));
        }
      }
    };
    const auto put = [&](int to, int rows, int r, const pair* v) {  // as an operand of `rows` rows
#pragma unroll
      for (int i = 0; i < CN; i += 8) {
        uint32_t hw[4], lw[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split_bf16x2(v[i / 2 + e], hw[e], lw[e]);
        const int ch = (c0 + i) >> 3;
        uint8_t* p = sm + to;
        *reinterpret_cast<uint4*>(p + sw128(r, ch)) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
        *reinterpret_cast<uint4*>(p + (NDV == 32 ? sw128(r, ch + 4) : rows * 128 + sw128(r, ch))) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
      }
    };
    const auto put_rest = [&](int r, const pair* v) {  // the third part
#pragma unroll
      for (int i = 0; i < CN; i += 8) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t hw, lw;
          pair d = v[i / 2 + e];
          split_bf16x2(d, hw, lw);
          fma2(d, pack2(-1.0f, -1.0f), pack2(bf16lo(hw), bf16hi(hw)));
          fma2(d, pack2(-1.0f, -1.0f), pack2(bf16lo(lw), bf16hi(lw)));
          w[e] = cvt_bf16x2(d);
        }
        *reinterpret_cast<uint4*>(sm + L::kRest + sw128(r, (c0 + i) >> 3)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    };
    const auto arrive = [&](uint64_t* bar) {
      tc_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    const long long head = s * a.c.state_stride + (static_cast<long long>(h) * dv + dv0 + c0) * DK + row;
    const int cols = min(CN, dv - dv0 - c0);  // of this warp's columns those that exist (may be negative)
    pair v[CN / 2];
    const bool go_on = a.initial && a.initial[b] != 0;
    const auto state_in = [&](int i) {
      if (!go_on || !has_s || i >= cols) return 0.0f;
      const long long x = head + static_cast<long long>(i) * DK;
      return F32 ? static_cast<const float*>(a.c.state)[x] : bf16f(static_cast<const uint16_t*>(a.c.state)[x]);
    };
    const auto state_out = [&](int i, float y) {
      if (i >= cols) return;
      const long long x = head + static_cast<long long>(i) * DK;
      if (F32)
        static_cast<float*>(a.c.state)[x] = y;
      else
        static_cast<__nv_bfloat16*>(a.c.state)[x] = __float2bfloat16_rn(y);
    };
#pragma unroll
    for (int i = 0; i < CN / 2; ++i) v[i] = pack2(state_in(2 * i), state_in(2 * i + 1));
    bool ok = true;
    for (int c = 0; c < chunks; ++c) {
      const int st = c % L::kStages;
      uint8_t* p = sm + st * L::kStage;
      const float* vec = reinterpret_cast<const float*>(p + L::kVecs);
      const int live = min(n - c * kC, kC);
      ok = wait_warp(b_full + st, (c / L::kStages) & 1);
      ok = ok && (c == 0 || wait_warp(b_new, (c - 1) & 1));
      if (!ok) break;
      if (live < kC) {  // rows past the prompt's end may be another prompt's: whatever they are, they must not count
        for (int i = tid; i < (kC - live) * L::kHalves * 8; i += kWorkWarps * 32) {
          const int r = live + i / (L::kHalves * 8), x = i % (L::kHalves * 8);
          *reinterpret_cast<uint4*>(p + L::kKQ + (x >> 3) * 16384 + r * 128 + (x & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      const bool past = t >= live;
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
      const float w0 = vec[is_tok ? t : 128 + t], w1 = vec[64 + t], be = vec[192 + t], ec = vec[256];
      if (has_s) {
        const pair e2 = pack2(ec, ec);
        const pair zero[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int i = 0; i < CN / 2; ++i) mul2(v[i], e2);
#pragma unroll
        for (int i = 0; i < CN; i += 8) {
          tc_st8(tm_s + at + i, v + i / 2);
          tc_st8(tm_s + at + NDV + i, zero);
        }
        tc_wait_st();
      }
      pair val[CN / 2];
      if (is_tok) {
#pragma unroll
        for (int i = 0; i < CN; i += 8) {
          const int ch = (c0 + i) >> 3;
          const uint4 x = *reinterpret_cast<const uint4*>(
              p + L::kV + (NDV == 32 ? t * 64 + ((ch ^ ((t >> 1) & 3)) << 4) : static_cast<int>(sw128(t, ch))));
          const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) val[i / 2 + e] = past ? 0ull : pack2(bf16lo(xw[e]), bf16hi(xw[e]));
        }
      } else {
        arrive(b_up);
      }
      if (!(ok = wait_warp(b_x, c & 1))) break;
      tc_after();
      get(v, tm_x);
      if (is_tok) {
        const pair m = pack2(-w0, -w0), m1 = pack2(be, be);
#pragma unroll
        for (int i = 0; i < CN / 2; ++i) {
          mul2(val[i], m1);
          fma2(val[i], m, v[i]);  // past the end X is zero: its key was
        }
        put(L::kR, kC, t, val);
        fence_async();
        arrive(b_r);
      }
      if (!(ok = wait_warp(b_u, c & 1))) break;
      tc_after();
      pair u[CN / 2];
      get(u, tm_u);
      if (is_tok) {
        const pair m = pack2(w1, w1);
#pragma unroll
        for (int i = 0; i < CN / 2; ++i) {
          if (F32) add2(u[i], val[i]);
          mul2(u[i], m);
        }
        put(L::kR, kC, t, u);
        if (F32) put_rest(t, u);
        fence_async();
        arrive(b_up);
      } else if (t < live) {
        const pair m = pack2(w0, w0);
#pragma unroll
        for (int i = 0; i < CN / 2; ++i) fma2(u[i], m, v[i]);
        uint16_t* o = a.tk.out + (start + c * kC + t) * ostride + h * dv + dv0 + c0;
#pragma unroll
        for (int i = 0; i < CN; i += 8) {
          if (i < cols)
            *reinterpret_cast<uint4*>(o + i) =
                make_uint4(cvt_bf16x2(u[i / 2]), cvt_bf16x2(u[i / 2 + 1]), cvt_bf16x2(u[i / 2 + 2]), cvt_bf16x2(u[i / 2 + 3]));
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
      for (int i = 0; i < CN / 2; ++i) {
        float lo, hi;
        unpack2(v[i], lo, hi);
        state_out(2 * i, lo);
        state_out(2 * i + 1, hi);
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
  CUtensorMap mq, mk;
  if (a.tokens == 0) return cudaSuccess;
  if (!token_map(&mq, a.tk.q, a.c.Hk * DK, a.tokens, a.tk.q_stride, 64) || !token_map(&mk, a.tk.k, a.c.Hk * DK, a.tokens, a.tk.k_stride, 64))
    return cudaErrorInvalidValue;
  const cudaError_t e = grow_smem(delta_chunk_kernel<DK>, ChunkSmem::kBytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(delta_chunk_kernel<DK>, dim3(static_cast<unsigned>(a.tokens / kC + a.batch), a.c.Hv), dim3(128), ChunkSmem::kBytes, st,
                    a, mq, mk);
}

template <int DK, int NDV, bool F32>
cudaError_t launch_scan(DeltaPrefillArgs a, cudaStream_t st) {
  CUtensorMap mq = {}, mk = {}, mv = {};
  if (a.tokens > 0 && (!token_map(&mq, a.tk.q, a.c.Hk * DK, a.tokens, a.tk.q_stride, 64) ||
                       !token_map(&mk, a.tk.k, a.c.Hk * DK, a.tokens, a.tk.k_stride, 64) ||
                       !token_map(&mv, a.tk.v, a.c.Hv * a.c.dv, a.tokens, a.tk.v_stride, NDV)))
    return cudaErrorInvalidValue;
  constexpr size_t smem = ScanSmem<DK, NDV>::kBytes;
  const cudaError_t e = grow_smem(delta_scan_kernel<DK, NDV, F32>, smem);
  if (e != cudaSuccess) return e;
  a.tiles = (a.c.dv + NDV - 1) / NDV;
  return launch_pdl(delta_scan_kernel<DK, NDV, F32>, dim3(static_cast<unsigned>(static_cast<long long>(a.batch) * a.c.Hv * a.tiles)),
                    dim3(kWorkWarps * 32 + 64), smem, st, a, mq, mk, mv);
}

template <int DK>
cudaError_t scan(const DeltaPrefillArgs& a, bool narrow, cudaStream_t st) {
  if (a.c.dtype == RSSM_F32) return narrow ? launch_scan<DK, 32, true>(a, st) : launch_scan<DK, 64, true>(a, st);
  return narrow ? launch_scan<DK, 32, false>(a, st) : launch_scan<DK, 64, false>(a, st);
}

}  // namespace
}  // namespace rssm

using namespace rssm;

extern "C" size_t rssm_delta_scratch_bytes(const rssm_delta_cache* cache, int32_t batch, int64_t tokens) {
  DeltaCacheView c;
  rssm_status st;
  if (!delta_view(cache, &c, &st) || batch < 0 || tokens < 0) return 0;
  return kDeltaHead + static_cast<size_t>(tokens / kC + batch) * c.Hv * kUnit;
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
  if (static_cast<long long>(batch) * a.c.Hv * ((a.c.dv + 31) / 32) > 0x7fffffffll || a.c.Hv > 65535) return RSSM_ERR_UNSUPPORTED;
  a.slot_idx = slot_idx;
  a.cu = cu_seqlens;
  a.initial = initial;
  a.batch = batch;
  a.tokens = tokens;
  a.units = static_cast<uint8_t*>(scratch) + kDeltaHead;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  // Value columns of a block.  A chunk's chain takes little longer for 64 than
  // for 32, so 32 only where the blocks then still run all at once.
  const int sms = num_sms();
  if (sms == 0) return RSSM_ERR_CUDA;
  const bool narrow = a.c.dv <= 32 || static_cast<long long>(batch) * a.c.Hv * ((a.c.dv + 31) / 32) <= sms;
  cudaError_t e;
  if (cache->dkey == 128) {
    e = launch_chunks<128>(a, cs);
    if (e == cudaSuccess) e = scan<128>(a, narrow, cs);
  } else {
    e = launch_chunks<64>(a, cs);
    if (e == cudaSuccess) e = scan<64>(a, narrow, cs);
  }
  return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}
