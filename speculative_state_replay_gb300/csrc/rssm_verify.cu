// rssm_verify.cu -- verification of drafted tokens against the target's
// probabilities from given random numbers.
#include <cooperative_groups.h>

#include "rssm_device.cuh"
#include "rssm_host.h"

namespace cg = cooperative_groups;

namespace rssm {
namespace {

struct VerifyArgs {
  const void* target;
  const void* draft;  // null: the drafts are certain (a lookup's)
  long long target_stride, draft_stride;
  int vocab;
  const int* tokens;
  const float* u;
  const float* u_next;
  const int* cu;
  int batch, T;
  long long ntok;
  int* accepted;
  int* next;
  unsigned* err;
};

constexpr int kVerifyThreads = 256;
constexpr int kVerifyBlocks = 4;  // an SM: 3 took 15 us for 12 (64 rows) and 64 for 48 (512 rows, now 42)
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxParts = 8;  // blocks of a cluster (the portable most)
constexpr int kRuns = 8;      // a warp's part of a row is summed in 8 runs
constexpr int kMaxVocab = 1 << 25;
constexpr int kMaxPart = 1 << 24;  // values of a block: its 8 warps' lanes then sum about 2^13 in a run, fewer than 2^14

template <typename P>
__device__ __forceinline__ float prob(P x);
template <>
__device__ __forceinline__ float prob<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ float prob<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
template <>
__device__ __forceinline__ float prob<__half>(__half x) {
  return __half2float(x);
}

// Sampling weights in fixed point, 36 fraction bits: sums of integers do not
// depend on their order, so the drawn token is a function of the inputs
// whatever the grid.  floor(2^36 r) of r in [0, 1] comes from two additions
// rounded toward zero: r + 32, whose last bit is 2^-18, leaves floor(2^18 r)
// in its fraction, and the remainder (exact) + 2^-13 the next 18 bits.  The
// sums' words are added as they are, two values an instruction, and the
// constants' bits taken off at the end: a lane's part of a row has fewer than
// 2^14 values (kMaxPart), so neither sum passes 32 bits even where all are 1.
// (The 64-bit conversion instruction runs at a fraction of these rates.)
using pair = unsigned long long;
__device__ __forceinline__ pair pack2(float lo, float hi) {
  pair d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
struct Weight {
  uint32_t hi = 0, lo = 0;  // in units of 2^-18 and 2^-36, less the constants' bits
  __device__ __forceinline__ void add(float r0, float r1) {  // both in [0, 1]
    const pair r = pack2(r0, r1), c = pack2(32.0f, 32.0f), f = pack2(1.220703125e-4f, 1.220703125e-4f), m = pack2(-1.0f, -1.0f);
    pair t, d;
    asm("add.rz.f32x2 %0, %1, %2;" : "=l"(t) : "l"(r), "l"(c));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(t), "l"(m), "l"(c));
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(d) : "l"(r));
    asm("add.rz.f32x2 %0, %0, %1;" : "+l"(d) : "l"(f));
    hi += static_cast<uint32_t>(t) + static_cast<uint32_t>(t >> 32) - 2u * 0x42000000u;
    lo += static_cast<uint32_t>(d) + static_cast<uint32_t>(d >> 32) - 2u * 0x39000000u;
  }
  __device__ __forceinline__ void add(float r) { add(r, 0.0f); }
  __device__ __forceinline__ void add(const Weight& w) {
    hi += w.hi;
    lo += w.lo;
  }
  __device__ __forceinline__ unsigned long long value() const {
    return (static_cast<unsigned long long>(hi) << 18) + lo;
  }
};

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One row's distribution to draw from: max(p - q, 0), q from the draft's row,
// or 1 at the draft's token (certain drafts), or nothing.  Pieces of VEC values
// start on 16 bytes of p's row: positions j are counted from `off` values
// before its first, so that rows of any alignment are read 16 bytes a lane.
// A row of q with another alignment (an odd vocabulary's) is read 16 bytes a
// lane as well, and a piece cut out of the two that hold it (94 rows of 15635
// fp16 values and their drafts': 11.9 us, value by value 16.8).
template <typename P>
struct Residual {
  static constexpr int VEC = 16 / sizeof(P);
  const P* p;
  const P* q;
  int token, vocab, off;
  unsigned long long certain;  // what a certain draft takes off the target's weight at `token`: all of it, of an entry up to 1
  int skew;  // values of q's 16 bytes before a piece: 0 if q's row has p's alignment

  __device__ __forceinline__ void set(const P* target, const P* draft, int tok, float at_tok, int v) {
    p = target;
    q = draft;
    token = tok;
    Weight all, left;
    all.add(__saturatef(at_tok));
    left.add(__saturatef(at_tok - 1.0f));
    certain = all.value() - left.value();
    vocab = v;
    off = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(P));
    skew = q ? static_cast<int>((reinterpret_cast<uintptr_t>(q - off) & 15u) / sizeof(P)) : 0;
  }
  // the target's row without anything taken off
  __device__ __forceinline__ void alone() {
    q = nullptr;
    token = -1;
    skew = 0;
  }
  // weights of the piece at position j, value by value: what lies past the
  // row's ends is 0, as NaN and what is negative are; at most 1
  __device__ __forceinline__ void values(int j, float (&r)[VEC]) const {
    const int i = j - off;
    P x[VEC], y[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const bool in = static_cast<unsigned>(i + e) < static_cast<unsigned>(vocab);
      x[e] = in ? p[i + e] : P(0.0f);
      y[e] = in && q ? q[i + e] : P(i + e == token ? 1.0f : 0.0f);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) r[e] = __saturatef(prob<P>(x[e]) - prob<P>(y[e]));
  }
  // whether the 32 pieces from position j on can be read 16 bytes a lane: all of
  // them (and of what lies around q's) is in the row
  __device__ __forceinline__ bool plain(int j) const {
    const int i = j - off;
    return i >= skew && i + 32 * VEC + (skew ? VEC - skew : 0) <= vocab;
  }
  __device__ __forceinline__ void add(Weight& w, const uint4& a, const uint4& c) const {
    const P *x = reinterpret_cast<const P*>(&a), *y = reinterpret_cast<const P*>(&c);
    if (q) {
#pragma unroll
      for (int e = 0; e < VEC; e += 2)
        w.add(__saturatef(prob<P>(x[e]) - prob<P>(y[e])), __saturatef(prob<P>(x[e + 1]) - prob<P>(y[e + 1])));
    } else {
#pragma unroll
      for (int e = 0; e < VEC; e += 2) w.add(__saturatef(prob<P>(x[e])), __saturatef(prob<P>(x[e + 1])));
    }
  }
  // the 16 bytes that start `skew` values into lo, hi
  __device__ __forceinline__ uint4 cut(const uint4& lo, const uint4& hi) const {
    const int bytes = skew * static_cast<int>(sizeof(P));
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int k = 0; k < 6; ++k) w[k] = bytes & 8 ? w[k + 2] : w[k];
#pragma unroll
    for (int k = 0; k < 5; ++k) w[k] = bytes & 4 ? w[k + 1] : w[k];
    const int bits = bytes % 4 * 8;
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                      __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
  }
  __device__ __forceinline__ static uint4 read(const P* at) { return __ldcs(reinterpret_cast<const uint4*>(at)); }
  // Weights of the lane's pieces of four steps that are `gap` positions apart:
  // their loads first, then the sums; where the row ends, one step at a time.
  __device__ __forceinline__ void steps(Weight (&w)[4], int j, int gap, int lane, int end) const {
    const int i = j - off + lane * VEC;
    const bool all = j + 3 * gap < end && plain(j) && plain(j + 3 * gap);
    if (all && skew == 0) {
      uint4 a[4], c[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        a[x] = read(p + i + x * gap);
        if (q) c[x] = read(q + i + x * gap);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) add(w[x], a[x], c[x]);
    } else if (all) {
#pragma unroll
      for (int x0 = 0; x0 < 4; x0 += 2) {
        uint4 a[2], lo[2], hi[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const P* at = q + i + (x0 + x) * gap - skew;
          a[x] = read(p + i + (x0 + x) * gap);
          lo[x] = *reinterpret_cast<const uint4*>(at);
          hi[x] = *reinterpret_cast<const uint4*>(at + VEC);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) add(w[x0 + x], a[x], cut(lo[x], hi[x]));
      }
    } else {
#pragma unroll 1
      for (int x = 0; x < 4; ++x) {
        const int k = j + x * gap;
        if (k >= end) break;
        Weight v;
        if (skew == 0 && plain(k)) {
          const uint4 a = read(p + i + x * gap);
          add(v, a, q ? read(q + i + x * gap) : a);
        } else {
          float r[VEC];
          values(k + lane * VEC, r);
#pragma unroll
          for (int e = 0; e < VEC; e += 2) v.add(r[e], r[e + 1]);
        }
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if (y == x) w[y].add(v);
      }
    }
  }
  // what to take off the lane's weight of the step at position j that holds a
  // certain draft's token: steps() does not look for it where it reads 16 bytes
  // a lane
  __device__ __forceinline__ unsigned long long taken(int j, int lane) const {
    const bool mine = static_cast<unsigned>(token - (j - off + lane * VEC)) < static_cast<unsigned>(VEC);
    return token >= 0 && mine && plain(j) ? certain : 0ull;
  }
};

// One cluster per row.  The row's tests come from single values; then the one
// row of the target (and of the draft) the next token is drawn from is read
// once, a part per block and warp, and summed in 64 bits; the sums of a
// warp's 8 runs are kept lane by lane, so the warp that holds the drawn mass finds
// the run, then the piece and the value, from them and a second look at that
// run alone.
template <typename P>
__global__ void __launch_bounds__(kVerifyThreads, kVerifyBlocks) verify_kernel(const VerifyArgs a) {
  constexpr int VEC = Residual<P>::VEC, kStep = 32 * VEC;
  __shared__ unsigned long long part[kVerifyWarps], runs[kRuns][kVerifyThreads];
  __shared__ unsigned long long sums[2][kMaxParts];
  __shared__ int sh_count, sh_bad, sh_token;
  __shared__ float sh_p;
  cg::cluster_group cl = cg::this_cluster();
  const int parts = cl.num_blocks(), rank = cl.block_rank();
  const int b = blockIdx.x / parts;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (parts > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this block runs: its sums can be written
  pdl_wait();
  pdl_trigger();
  const long long tok0 = a.cu ? a.cu[b] : static_cast<long long>(b) * a.T;
  const int n = a.cu ? a.cu[b + 1] - a.cu[b] : a.T;
  const bool empty = n <= 0 || n > a.T || tok0 < 0 || tok0 + n > a.ntok;  // the same in every block of the cluster
  if (empty) {
    if (rank == 0 && threadIdx.x == 0) {
      a.accepted[b] = 0;
      a.next[b] = -1;
      if (n != 0) set_error(a.err, RSSM_ERRBIT_SEQLEN);
    }
    if (parts > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    return;
  }
  const P* target = static_cast<const P*>(a.target);
  const P* draft = static_cast<const P*>(a.draft);
  const float u_next = a.u_next[b];
  if (warp == 0) {
    // draft t is tested against the target's probabilities after token t - 1
    bool pass = lane == 0, bad = false;
    int tok = -1;
    float p = 0.0f;
    if (lane > 0 && lane < n) {
      tok = a.tokens[tok0 + lane];
      const float u = a.u[tok0 + lane];
      bad = tok < 0 || tok >= a.vocab;
      if (!bad) {
        p = prob<P>(target[(tok0 + lane - 1) * a.target_stride + tok]);
        const float q = draft ? prob<P>(draft[(tok0 + lane) * a.draft_stride + tok]) : 1.0f;
        pass = __fmul_rn(u, q) < p;
      }
    }
    const unsigned failed = ~__ballot_sync(0xffffffffu, pass);
    const unsigned any_bad = __ballot_sync(0xffffffffu, bad);
    const int count = failed ? __ffs(failed) - 1 : 32;
    if (lane == 0) {
      sh_count = count;
      sh_bad = any_bad != 0u;
    }
    if (lane == count) {
      sh_token = tok;
      sh_p = p;
    }
  }
  __syncthreads();
  const int count = sh_count;
  Residual<P> res;
  res.set(target + (tok0 + count - 1) * a.target_stride,
          draft && count < n ? draft + (tok0 + count) * a.draft_stride : nullptr,
          !draft && count < n ? sh_token : -1, !draft && count < n ? sh_p : 0.0f, a.vocab);
  if (rank == 0 && threadIdx.x == 0 && sh_bad) set_error(a.err, RSSM_ERRBIT_TOKEN);

  // a warp's part: kRuns runs of `len` steps of 32 pieces
  const int len = (a.vocab + res.off + parts * kVerifyWarps * kRuns * kStep - 1) / (parts * kVerifyWarps * kRuns * kStep);
  const int span = kRuns * len * kStep, first = (rank * kVerifyWarps + warp) * span, end = a.vocab + res.off;
  unsigned long long total = 0, before = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    unsigned long long w = 0;
    const int place = res.token + res.off - first, held = place / kStep;  // the part's step that holds a certain token
    const unsigned long long off = place >= 0 && place < span ? res.taken(first + held * kStep, lane) : 0ull;
#pragma unroll 1
    for (int r = 0; r < kRuns; r += 4) {
      Weight run[4];
#pragma unroll 1
      for (int k = 0; k < len; ++k) res.steps(run, first + (r * len + k) * kStep, len * kStep, lane, end);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const unsigned long long y = run[x].value() - (held / len == r + x ? off : 0ull);
        runs[r + x][threadIdx.x] = y;
        w += y;
      }
    }
    w = warp_sum(w);
    if (lane == 0) part[warp] = w;
    __syncthreads();
    if (parts == 1) {
      total = 0;
#pragma unroll
      for (int x = 0; x < kVerifyWarps; ++x) total += part[x];
    } else {
      if (pass == 0) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
      if (threadIdx.x < parts) {
        unsigned long long mine = 0;
#pragma unroll
        for (int x = 0; x < kVerifyWarps; ++x) mine += part[x];
        *cl.map_shared_rank(&sums[pass][rank], threadIdx.x) = mine;
      }
      cl.sync();
      total = before = 0;
      for (int x = 0; x < parts; ++x) {
        const unsigned long long y = sums[pass][x];
        total += y;
        if (x < rank) before += y;
      }
    }
    if (total || (!res.q && res.token < 0)) break;
    // nothing left of the target above the draft: draw from the target itself
    res.alone();
    __syncthreads();
  }
  if (total == 0) {
    if (rank == 0 && threadIdx.x == 0) {
      a.accepted[b] = count;
      a.next[b] = -1;
      set_error(a.err, RSSM_ERRBIT_TOKEN);
    }
    return;
  }
  // floor(total * u) with u in 24 bits
  const unsigned long long u24 = static_cast<unsigned long long>(__float2ll_rz(fminf(fmaxf(u_next, 0.0f), 0.99999994f) * 16777216.0f));
  const unsigned long long aim = (total >> 24) * u24 + (((total & 0xffffffull) * u24) >> 24);
  for (int x = 0; x < warp; ++x) before += part[x];
  if (aim < before || aim >= before + part[warp]) return;
  // this warp's part holds the token: the run that does, then the step of 32 pieces
  unsigned long long left = aim - before;
  int at = first;
  bool found = false;
#pragma unroll
  for (int r = 0; r < kRuns; ++r) {
    const unsigned long long w = warp_sum(runs[r][threadIdx.x]);
    if (!found) {
      if (left < w) {
        found = true;
        at = first + r * len * kStep;
      } else {
        left -= w;
      }
    }
  }
#pragma unroll 1
  for (int k0 = 0; k0 < len; k0 += 4) {  // four steps' values on their way at a time
    Weight part4[4];
    res.steps(part4, at + k0 * kStep, kStep, lane, min(end, at + len * kStep));
    unsigned long long own[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) own[x] = part4[x].value() - (k0 + x < len ? res.taken(at + (k0 + x) * kStep, lane) : 0ull);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const unsigned long long all = warp_sum(own[x]);
      if (left >= all) {
        left -= all;
        continue;
      }
      unsigned long long upto = own[x];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      unsigned long long base = upto - own[x];
      if (left >= base && left < upto) {
        const int j = at + (k0 + x) * kStep + lane * VEC;
        float r[VEC];
        res.values(j, r);
        int e = 0;  // the first value whose running sum passes `left`; the piece's last one does
#pragma unroll
        for (int y = 0; y < VEC; ++y) {
          Weight w;
          w.add(r[y]);
          base += w.value();
          e += left >= base;
        }
        a.accepted[b] = count;
        a.next[b] = j - res.off + e;
      }
      return;
    }
  }
}

template <typename P>
cudaError_t launch_verify(const VerifyArgs& a, int parts, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.batch) * parts);
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = parts;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_kernel<P>, a);
}

}  // namespace
}  // namespace rssm

using namespace rssm;

extern "C" rssm_status rssm_verify(const void* target, int64_t target_stride, const void* draft, int64_t draft_stride,
                                   int32_t prob_dtype, int32_t vocab, const int32_t* tokens, const float* u,
                                   const float* u_next, const int32_t* cu_seqlens, int32_t batch, int32_t T,
                                   int64_t ntok, int32_t* accepted, int32_t* next, uint32_t* error_word, void* stream) {
  const auto al4 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; };
  if (batch < 0 || T < 1 || vocab < 1 || ntok < 0) return RSSM_ERR_INVALID_ARGUMENT;
  if (prob_dtype != RSSM_F32 && prob_dtype != RSSM_BF16 && prob_dtype != RSSM_F16) return RSSM_ERR_INVALID_ARGUMENT;
  if (T > 32 || vocab > kMaxVocab) return RSSM_ERR_UNSUPPORTED;
  if (batch == 0) return RSSM_OK;
  if ((ntok > 0 && (!target || !tokens || !u)) || !u_next || !accepted || !next) return RSSM_ERR_INVALID_ARGUMENT;
  if (!al4(tokens) || !al4(u) || !al4(u_next) || !al4(cu_seqlens) || !al4(accepted) || !al4(next) || !al4(error_word))
    return RSSM_ERR_INVALID_ARGUMENT;
  const int esz = prob_dtype == RSSM_F32 ? 4 : 2;
  if (target_stride < vocab || (draft && draft_stride < vocab)) return RSSM_ERR_INVALID_ARGUMENT;
  if (reinterpret_cast<uintptr_t>(target) % esz || reinterpret_cast<uintptr_t>(draft) % esz) return RSSM_ERR_INVALID_ARGUMENT;
  if (!cu_seqlens && ntok < static_cast<int64_t>(batch) * T) return RSSM_ERR_INVALID_ARGUMENT;
  if (batch > (1 << 27)) return RSSM_ERR_UNSUPPORTED;
  VerifyArgs a;
  a.target = target;
  a.draft = draft;
  a.target_stride = target_stride;
  a.draft_stride = draft_stride;
  a.vocab = vocab;
  a.tokens = tokens;
  a.u = u;
  a.u_next = u_next;
  a.cu = cu_seqlens;
  a.batch = batch;
  a.T = T;
  a.ntok = ntok;
  a.accepted = accepted;
  a.next = next;
  a.err = error_word;
  // blocks of a row: as many as still run all at once, each with 4096 values at
  // least; and two where one would have more than kMaxPart
  const int sms = num_sms();
  if (sms == 0) return RSSM_ERR_CUDA;
  int parts = 1;
  while (parts < kMaxParts && static_cast<long long>(batch) * parts * 2 <= kVerifyBlocks * sms && vocab > parts * 4096) parts *= 2;
  if (vocab > kMaxPart && parts == 1) parts = 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = prob_dtype == RSSM_F32    ? launch_verify<float>(a, parts, st)
                        : prob_dtype == RSSM_BF16 ? launch_verify<__nv_bfloat16>(a, parts, st)
                                                  : launch_verify<__half>(a, parts, st);
  return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}
