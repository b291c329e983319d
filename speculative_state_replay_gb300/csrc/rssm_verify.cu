// rssm_verify.cu -- verification of drafted tokens against the target's
// probabilities from given random numbers.
#include <cooperative_groups.h>

#include "rssm_device.cuh"

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

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;

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

// Sampling weight in fixed point, 36 fraction bits: sums of integers do not
// depend on their order, so the drawn token is a function of the inputs
// whatever the grid.  Comparisons send NaN to zero.
__device__ __forceinline__ unsigned long long weight(float r) {
  return r > 0.0f ? static_cast<unsigned long long>(__float2ll_rz(fminf(r, 1.0f) * 68719476736.0f)) : 0ull;
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One row's distribution to draw from: max(p - q, 0), q from the draft's row,
// or 1 at the draft's token (certain drafts), or nothing.
template <typename P>
struct Residual {
  const P* p;
  const P* q;
  int token;
  template <int VEC>
  __device__ __forceinline__ unsigned long long sum(int i) const {
    P a[VEC];
    unsigned long long w = 0;
    if constexpr (VEC == 1) {
      return at(i);
    } else {
      *reinterpret_cast<uint4*>(a) = *reinterpret_cast<const uint4*>(p + i);
      if (q) {
        P c[VEC];
        *reinterpret_cast<uint4*>(c) = *reinterpret_cast<const uint4*>(q + i);
#pragma unroll
        for (int e = 0; e < VEC; ++e) w += weight(prob<P>(a[e]) - prob<P>(c[e]));
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) w += weight(prob<P>(a[e]) - (i + e == token ? 1.0f : 0.0f));
      }
      return w;
    }
  }
  __device__ __forceinline__ unsigned long long at(int i) const {
    const float b = q ? prob<P>(q[i]) : (i == token ? 1.0f : 0.0f);
    return weight(prob<P>(p[i]) - b);
  }
};

// One cluster per row.  The row's tests come from single values; then the one
// row of the target (and of the draft) the next token is drawn from is read
// once in slices, one per CTA and warp, and summed; the CTA whose slice holds
// the drawn mass reads it again, in ever smaller parts, to find the token.
template <typename P, int VEC>
__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const VerifyArgs a) {
  __shared__ unsigned long long part[kVerifyWarps];
  __shared__ unsigned long long cta_sum;
  __shared__ int sh_count, sh_bad;
  cg::cluster_group cl = cg::this_cluster();
  const int parts = cl.num_blocks(), rank = cl.block_rank();
  const int b = blockIdx.x / parts;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  const long long tok0 = a.cu ? a.cu[b] : static_cast<long long>(b) * a.T;
  const int n = a.cu ? a.cu[b + 1] - a.cu[b] : a.T;
  if (n <= 0 || n > a.T || tok0 < 0 || tok0 + n > a.ntok) {  // the same in every CTA of the cluster
    if (rank == 0 && threadIdx.x == 0) {
      a.accepted[b] = 0;
      a.next[b] = -1;
      if (n != 0) set_error(a.err, RSSM_ERRBIT_SEQLEN);
    }
    return;
  }
  const P* target = static_cast<const P*>(a.target);
  const P* draft = static_cast<const P*>(a.draft);
  if (warp == 0) {
    // draft t is tested against the target's probabilities after token t - 1
    bool pass = lane == 0, bad = false;
    if (lane > 0 && lane < n) {
      const int tok = a.tokens[tok0 + lane];
      bad = tok < 0 || tok >= a.vocab;
      if (!bad) {
        const float p = prob<P>(target[(tok0 + lane - 1) * a.target_stride + tok]);
        const float q = draft ? prob<P>(draft[(tok0 + lane) * a.draft_stride + tok]) : 1.0f;
        pass = __fmul_rn(a.u[tok0 + lane], q) < p;
      }
    }
    const unsigned failed = ~__ballot_sync(0xffffffffu, pass);
    const unsigned any_bad = __ballot_sync(0xffffffffu, bad);
    if (lane == 0) {
      sh_count = failed ? __ffs(failed) - 1 : 32;
      sh_bad = any_bad != 0u;
    }
  }
  __syncthreads();
  const int count = sh_count;
  Residual<P> res;
  res.p = target + (tok0 + count - 1) * a.target_stride;
  res.q = draft && count < n ? draft + (tok0 + count) * a.draft_stride : nullptr;
  res.token = !draft && count < n ? a.tokens[tok0 + count] : -1;
  if (rank == 0 && threadIdx.x == 0 && sh_bad) set_error(a.err, RSSM_ERRBIT_TOKEN);

  // slices in whole vectors, the last one ragged
  const int step = kVerifyWarps * VEC * 32;
  const int slice = (a.vocab + parts * step - 1) / (parts * step) * step;  // a multiple of every warp's 32 vectors
  unsigned long long total = 0, before = 0, mine = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    const int lo = rank * slice + warp * (slice / kVerifyWarps), hi = min(lo + slice / kVerifyWarps, a.vocab);
    unsigned long long w = 0;
#pragma unroll 4
    for (int i = lo + lane * VEC; i < hi; i += 32 * VEC) {
      if (i + VEC <= hi) {
        w += res.template sum<VEC>(i);
      } else {
        for (int e = i; e < hi; ++e) w += res.at(e);
      }
    }
    w = warp_sum(w);
    if (lane == 0) part[warp] = w;
    __syncthreads();
    mine = 0;
#pragma unroll
    for (int x = 0; x < kVerifyWarps; ++x) mine += part[x];
    if (parts == 1) {
      total = mine;
    } else {
      if (threadIdx.x == 0) cta_sum = mine;
      cl.sync();
      total = before = 0;
      for (int x = 0; x < parts; ++x) {
        const unsigned long long y = *cl.map_shared_rank(&cta_sum, x);
        total += y;
        if (x < rank) before += y;
      }
      cl.sync();  // nobody leaves, or writes its sum again, before all have read
    }
    if (total || (!res.q && res.token < 0)) break;
    // nothing left of the target above the draft: draw from the target itself
    res.q = nullptr;
    res.token = -1;
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
  const unsigned long long u24 = static_cast<unsigned long long>(__float2ll_rz(fminf(fmaxf(a.u_next[b], 0.0f), 0.99999994f) * 16777216.0f));
  const unsigned long long aim = (total >> 24) * u24 + (((total & 0xffffffull) * u24) >> 24);
  if (aim < before || aim >= before + mine) return;
  // this CTA's slice holds the token: the warp's part that does, then parts of parts
  unsigned long long left = aim - before;
  int lo = rank * slice, width = slice / kVerifyWarps;
  while (true) {
    int x = 0;
    while (x < kVerifyWarps - 1 && left >= part[x]) left -= part[x++];
    lo += x * width;
    if (width <= 32 * VEC) break;
    __syncthreads();  // part is read
    const int next_width = (width + step - 1) / step * (step / kVerifyWarps);
    const int l = lo + warp * next_width, h = min(min(l + next_width, lo + width), a.vocab);
    unsigned long long w = 0;
    for (int i = l + lane * VEC; i < h; i += 32 * VEC) {
      if (i + VEC <= h) {
        w += res.template sum<VEC>(i);
      } else {
        for (int e = i; e < h; ++e) w += res.at(e);
      }
    }
    w = warp_sum(w);
    if (lane == 0) part[warp] = w;
    __syncthreads();
    width = next_width;
  }
  if (warp == 0) {
    const int i0 = lo + lane * VEC, i1 = min(i0 + VEC, a.vocab);
    unsigned long long w[VEC], own = 0;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      w[e] = i0 + e < i1 ? res.at(i0 + e) : 0ull;
      own += w[e];
    }
    unsigned long long upto = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    unsigned long long base = upto - own;
    if (left >= base && left < upto) {
      int e = 0;
#pragma unroll
      for (int x = 0; x < VEC - 1; ++x) {
        if (e == x && left >= base + w[x]) {
          base += w[x];
          e = x + 1;
        }
      }
      a.accepted[b] = count;
      a.next[b] = i0 + e;
    }
  }
}

template <typename P>
cudaError_t launch_verify(const VerifyArgs& a, bool vec, int parts, cudaStream_t st) {
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
  if (vec) return cudaLaunchKernelEx(&cfg, verify_kernel<P, 16 / static_cast<int>(sizeof(P))>, a);
  return cudaLaunchKernelEx(&cfg, verify_kernel<P, 1>, a);
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
  if (T > 32 || vocab > (1 << 28)) return RSSM_ERR_UNSUPPORTED;
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
  // rows that start on 16 bytes are read 16 bytes a lane
  const bool vec = reinterpret_cast<uintptr_t>(target) % 16 == 0 && target_stride * esz % 16 == 0 &&
                   (!draft || (reinterpret_cast<uintptr_t>(draft) % 16 == 0 && draft_stride * esz % 16 == 0));
  int parts = 1;
  while (parts < 8 && batch * parts < 304 && vocab > parts * 4096) parts *= 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = prob_dtype == RSSM_F32    ? launch_verify<float>(a, vec, parts, st)
                        : prob_dtype == RSSM_BF16 ? launch_verify<__nv_bfloat16>(a, vec, parts, st)
                                                  : launch_verify<__half>(a, vec, parts, st);
  return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}
