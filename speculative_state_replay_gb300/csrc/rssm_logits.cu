// rssm_logits.cu -- from logits to the probabilities that the verification
// takes: penalties for repeated tokens, biases, grammar masks, temperature.
//
// Bound by memory: a row is read once and written once.  A cluster of blocks takes a
// row, each a slice of the vocabulary that it keeps in shared memory, one 32-bit word
// an id.  A word is first the id's count in the request's text -- every block goes over
// the whole history and keeps what falls into its slice, integer additions in shared
// memory, whose order does not matter -- then the processed logit.  Maximum and sum
// meet through the cluster's shared memory.
#include <cooperative_groups.h>

#include "rssm_kv.cuh"

namespace cg = cooperative_groups;

namespace rssm {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxParts = 8;            // blocks of a cluster (the portable most)
constexpr int kMaxSlice = 1 << 15;      // words of a block: 128 KB
constexpr int kMaxVocab = kMaxParts * kMaxSlice;
constexpr unsigned kSeen = 1u << 31;    // a count's bit for ids of the prompt

struct LogitsArgs {
  rssm_logits_args a;
  int slice;  // ids of a block, a multiple of 32
};

template <typename P>
__device__ __forceinline__ float value(P x);
template <>
__device__ __forceinline__ float value<float>(float x) { return x; }
template <>
__device__ __forceinline__ float value<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float value<__half>(__half x) { return __half2float(x); }
template <typename P>
__device__ __forceinline__ P rounded(float x);
template <>
__device__ __forceinline__ float rounded<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half rounded<__half>(float x) { return __float2half_rn(x); }

// `N` values from p on, 16 bytes at a time if p allows; those past `n` are zeros (not written)
template <typename P, int N>
__device__ __forceinline__ void load(const P* p, int n, bool wide, float (&f)[N]) {
  constexpr int VEC = 16 / sizeof(P);
  if (wide && n >= N) {
#pragma unroll
    for (int i = 0; i < N; i += VEC) {
      const uint4 w = __ldcs(reinterpret_cast<const uint4*>(p + i));
      const P* x = reinterpret_cast<const P*>(&w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[i + e] = value<P>(x[e]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = i < n ? value<P>(p[i]) : 0.0f;
  }
}
template <typename P, int N>
__device__ __forceinline__ void store(P* p, int n, bool wide, const float (&f)[N]) {
  constexpr int VEC = 16 / sizeof(P);
  if (wide && n >= N) {
#pragma unroll
    for (int i = 0; i < N; i += VEC) {
      P x[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[e] = rounded<P>(f[i + e]);
      __stcs(reinterpret_cast<uint4*>(p + i), *reinterpret_cast<const uint4*>(x));
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) p[i] = rounded<P>(f[i]);
  }
}

// largest value, and of equal ones the lowest id, as one number that orders like them
__device__ __forceinline__ unsigned long long top_key(float x, int id) {
  const uint32_t u = __float_as_uint(x == 0.0f ? 0.0f : x);  // -0 is 0
  const uint32_t o = u & 0x80000000u ? ~u : u | 0x80000000u;
  return static_cast<unsigned long long>(o) << 32 | (0xffffffffu - static_cast<uint32_t>(id));
}

constexpr int kRun = 8;  // ids of a lane's step

template <typename IN, typename OUT>
__global__ void __launch_bounds__(kThreads) logits_kernel(const LogitsArgs k) {
  extern __shared__ __align__(16) uint32_t word[];  // [slice]
  __shared__ float sh_part[kWarps];
  __shared__ unsigned long long sh_key[kWarps];
  __shared__ float sh_all[2][kMaxParts];
  __shared__ unsigned long long sh_top[kMaxParts];
  __shared__ int sh_fed[kTreeT];
  __shared__ int sh_id[kThreads], sh_kept[kWarps];  // a part of the biases: those of this block's ids, in order
  __shared__ float sh_bias[kThreads];
  const rssm_logits_args& a = k.a;
  cg::cluster_group cl = cg::this_cluster();
  const int parts = cl.num_blocks(), rank = cl.block_rank();
  const int item = blockIdx.x / parts, b = item / a.T, t = item - b * a.T;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned full = 0xffffffffu;
  pdl_wait();
  pdl_trigger();
  long long first = static_cast<long long>(b) * a.T;
  int n = a.T;
  if (a.cu_seqlens) {
    const int lo = a.cu_seqlens[b], hi = a.cu_seqlens[b + 1];
    const long long m = static_cast<long long>(hi) - lo;
    if (m < 0 || m > a.T || lo < 0 || hi > a.ntok) {
      if (t == 0 && rank == 0 && threadIdx.x == 0) set_error(a.error_word, RSSM_ERRBIT_SEQLEN);
      return;  // the same in every block of the cluster
    }
    first = lo;
    n = static_cast<int>(m);
  }
  if (t >= n) return;
  const long long tok = first + t;
  const int from = rank * k.slice, size = min(k.slice, a.vocab - from);  // this block's ids; none: size <= 0
  const IN* x = static_cast<const IN*>(a.logits) + tok * a.logits_stride + from;
  OUT* out = static_cast<OUT*>(a.out) + tok * a.out_stride + from;
  const bool wide_in = (reinterpret_cast<uintptr_t>(x) & 15u) == 0, wide_out = (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
  float temp = a.temperature ? a.temperature[b] : 1.0f;
  if (!(temp >= 0.0f)) temp = 1.0f;
  float rep = a.repetition ? a.repetition[b] : 1.0f;
  if (!(rep > 0.0f)) rep = 1.0f;
  const float presence = a.presence ? a.presence[b] : 0.0f, frequency = a.frequency ? a.frequency[b] : 0.0f;
  const bool counted = rep != 1.0f || presence != 0.0f || frequency != 0.0f;

  // ---- this lane's entry of the first biases, asked for early
  const bool biased = a.bias_id != nullptr;
  long long bias_lo = 0, bias_hi = 0;
  int bias_id = -1;
  float bias_value = 0.0f;
  auto bias_entry = [&](long long e0) {
    const long long e = e0 + threadIdx.x;
    bias_id = -1;
    if (e < bias_hi) {
      const int id = a.bias_id[e];
      bias_id = id >= from ? id - from : -1;
      bias_value = a.bias_value[e];
    }
  };
  if (biased) {
    bias_lo = max(0, a.bias_start[b]);
    bias_hi = min(static_cast<long long>(a.bias_start[b + 1]), static_cast<long long>(a.biases));
    bias_entry(bias_lo);
  }

  // ---- counts
  if (counted) {
    for (int i = threadIdx.x; i < k.slice; i += kThreads) word[i] = 0u;
    if (warp == 0 && a.tokens) {
      // the fed tokens on the path to this one
      unsigned long long mask = (2ull << t) - 1ull;  // a chain: all up to it
      if (a.parents) {
        unsigned long long m[2];
        if (tree_masks(a.parents + first, n, lane, m)) {
          const unsigned long long m0 = __shfl_sync(full, m[0], t & 31), m1 = __shfl_sync(full, m[1], t & 31);
          mask = t < 32 ? m0 : m1;
        } else {
          mask = 1ull << t;
          if (lane == 0 && rank == 0) set_error(a.error_word, RSSM_ERRBIT_TREE);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int j = lane + 32 * i;
        sh_fed[j] = mask >> j & 1 && j < n ? a.tokens[first + j] : -1;
      }
    }
    __syncthreads();
    if (a.history) {
      const int* h = a.history + b * a.history_stride;
      const int len = min(max(a.history_len[b], 0), a.history_max);
      const int prompt = a.prompt_len ? min(max(a.prompt_len[b], 0), len) : 0;
#pragma unroll 4
      for (int i = threadIdx.x; i < len; i += kThreads) {
        const int id = h[i];
        if (id >= from && id < from + size) {
          if (i < prompt) atomicOr(word + id - from, kSeen);
          else atomicAdd(word + id - from, 1u);
        }
      }
    }
    if (a.tokens && threadIdx.x < kTreeT) {
      const int id = sh_fed[threadIdx.x];  // -1: none
      if (id >= from && id < from + size) atomicAdd(word + id - from, 1u);
    }
    __syncthreads();
  }

  // ---- the logits with their penalties, into the words
  const uint32_t* mask = a.mask ? a.mask + tok * a.mask_stride : nullptr;
  float top = -INFINITY;
  unsigned long long key = 0ull;
  // an id's last steps; a softmax divides by the temperature later, what is left of the largest: that stays in range
  auto finish = [&](float y, uint32_t allowed) {
    if (!allowed || y != y) y = -INFINITY;
    return temp > 0.0f && !a.probs ? __fdiv_rn(y, temp) : y;
  };
  auto take = [&](float y, int id) {
    top = fmaxf(top, y);
    if (temp == 0.0f && y > -INFINITY) key = max(key, top_key(y, id));
  };
  auto bits = [&](int i) {  // the mask's bits of ids from + i ..
    if (!mask) return 0xffffffffu;
    const int id = from + i;
    return mask[id >> 5] >> (id & 31);
  };
  for (int i = threadIdx.x * kRun; i < size; i += kThreads * kRun) {
    float f[kRun];
    load<IN, kRun>(x + i, size - i, wide_in, f);
    if (counted) {
      uint32_t w[kRun];
      *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(word + i);
      *reinterpret_cast<uint4*>(w + 4) = *reinterpret_cast<const uint4*>(word + i + 4);
#pragma unroll
      for (int e = 0; e < kRun; ++e) {
        if (w[e]) {
          f[e] = f[e] > 0.0f ? __fdiv_rn(f[e], rep) : f[e] * rep;
          const unsigned c = w[e] & ~kSeen;
          if (c) f[e] -= presence + frequency * static_cast<float>(c);
        }
      }
    }
    if (!biased) {
      const uint32_t ok = bits(i);
#pragma unroll
      for (int e = 0; e < kRun; ++e) {
        f[e] = i + e < size ? finish(f[e], ok >> e & 1u) : -INFINITY;
        take(f[e], from + i + e);
      }
    }
    *reinterpret_cast<float4*>(word + i) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(word + i + 4) = make_float4(f[4], f[5], f[6], f[7]);
  }
  if (biased) {
    for (long long e0 = bias_lo; e0 < bias_hi; e0 += kThreads) {  // (a barrier with the dense pass inside)
      if (e0 > bias_lo) bias_entry(e0);
      const bool mine = bias_id >= 0 && bias_id < size;
      const unsigned kept = __ballot_sync(full, mine);
      if (lane == 0) sh_kept[warp] = __popc(kept);
      __syncthreads();
      int at = __popc(kept & ((1u << lane) - 1u)), all = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        if (i < warp) at += sh_kept[i];
        all += sh_kept[i];
      }
      if (mine) {
        sh_id[at] = bias_id;
        sh_bias[at] = bias_value;
      }
      __syncthreads();
      if (warp == 0) {
        // of 32 entries at a time, the first lane of those with one id adds them up, in order
        float* y = reinterpret_cast<float*>(word);
        for (int i0 = 0; i0 < all; i0 += 32) {
          const bool on = i0 + lane < all;
          const int id = on ? sh_id[i0 + lane] : -1 - lane;
          const float v = on ? sh_bias[i0 + lane] : 0.0f;
          const unsigned same = __match_any_sync(full, id);
          const int count = __popc(same), most = __reduce_max_sync(full, count);
          float sum = on ? y[id] : 0.0f;
          for (int j = 0; j < most; ++j) {
            const float add = __shfl_sync(full, v, j < count ? static_cast<int>(__fns(same, 0, j + 1)) : lane);
            if (j < count) sum += add;
          }
          if (on && lane == __ffs(same) - 1) y[id] = sum;
          __syncwarp();
        }
      }
      __syncthreads();
    }
    if (bias_lo >= bias_hi) __syncthreads();
    for (int i = threadIdx.x * kRun; i < size; i += kThreads * kRun) {
      float f[kRun];
      *reinterpret_cast<float4*>(f) = *reinterpret_cast<const float4*>(word + i);
      *reinterpret_cast<float4*>(f + 4) = *reinterpret_cast<const float4*>(word + i + 4);
      const uint32_t ok = bits(i);
#pragma unroll
      for (int e = 0; e < kRun; ++e) {
        f[e] = i + e < size ? finish(f[e], ok >> e & 1u) : -INFINITY;
        take(f[e], from + i + e);
      }
      *reinterpret_cast<float4*>(word + i) = make_float4(f[0], f[1], f[2], f[3]);
      *reinterpret_cast<float4*>(word + i + 4) = make_float4(f[4], f[5], f[6], f[7]);
    }
  }
  // (a lane reads back what it wrote itself)
  if (!a.probs) {
    for (int i = threadIdx.x * kRun; i < size; i += kThreads * kRun) {
      float f[kRun];
      *reinterpret_cast<float4*>(f) = *reinterpret_cast<const float4*>(word + i);
      *reinterpret_cast<float4*>(f + 4) = *reinterpret_cast<const float4*>(word + i + 4);
      store<OUT, kRun>(out + i, size - i, wide_out, f);
    }
    return;
  }

  // ---- the row's maximum
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    top = fmaxf(top, __shfl_xor_sync(full, top, o));
    key = max(key, __shfl_xor_sync(full, key, o));
  }
  if (lane == 0) {
    sh_part[warp] = top;
    sh_key[warp] = key;
  }
  __syncthreads();
  top = sh_part[lane % kWarps];
  key = sh_key[lane % kWarps];
#pragma unroll
  for (int o = kWarps / 2; o; o >>= 1) {
    top = fmaxf(top, __shfl_xor_sync(full, top, o));
    key = max(key, __shfl_xor_sync(full, key, o));
  }
  if (parts > 1) {
    cl.sync();  // all blocks run
    if (threadIdx.x < parts) {
      *cl.map_shared_rank(&sh_all[0][rank], threadIdx.x) = top;
      *cl.map_shared_rank(&sh_top[rank], threadIdx.x) = key;
    }
    cl.sync();
    for (int i = 0; i < parts; ++i) {
      top = fmaxf(top, sh_all[0][i]);
      key = max(key, sh_top[i]);
    }
  }
  float scale = 0.0f;
  if (temp > 0.0f) {
    // ---- and its sum
    const float cool = __fdiv_rn(1.0f, temp);
    float sum = 0.0f;
    if (top > -INFINITY) {
      for (int i = threadIdx.x * kRun; i < size; i += kThreads * kRun) {
        float f[kRun];
        *reinterpret_cast<float4*>(f) = *reinterpret_cast<const float4*>(word + i);
        *reinterpret_cast<float4*>(f + 4) = *reinterpret_cast<const float4*>(word + i + 4);
#pragma unroll
        for (int e = 0; e < kRun; ++e) {
          const float d = f[e] - top;
          f[e] = f[e] == top ? 1.0f : d == -INFINITY ? 0.0f : expf(d * cool);  // (infinite ones too, and any temperature)
          sum += f[e];
        }
        *reinterpret_cast<float4*>(word + i) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4*>(word + i + 4) = make_float4(f[4], f[5], f[6], f[7]);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(full, sum, o);
    __syncthreads();  // sh_part is read
    if (lane == 0) sh_part[warp] = sum;
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) sum += sh_part[i];
    if (parts > 1) {
      if (threadIdx.x < parts) *cl.map_shared_rank(&sh_all[1][rank], threadIdx.x) = sum;
      cl.sync();
      sum = 0.0f;
      for (int i = 0; i < parts; ++i) sum += sh_all[1][i];
    }
    scale = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
  }
  const int best = key ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(key)) : -1;
  for (int i = threadIdx.x * kRun; i < size; i += kThreads * kRun) {
    float f[kRun];
    if (temp > 0.0f) {
      *reinterpret_cast<float4*>(f) = *reinterpret_cast<const float4*>(word + i);
      *reinterpret_cast<float4*>(f + 4) = *reinterpret_cast<const float4*>(word + i + 4);
#pragma unroll
      for (int e = 0; e < kRun; ++e) f[e] = scale == 0.0f ? 0.0f : f[e] * scale;
    } else {
#pragma unroll
      for (int e = 0; e < kRun; ++e) f[e] = from + i + e == best ? 1.0f : 0.0f;
    }
    store<OUT, kRun>(out + i, size - i, wide_out, f);
  }
}

template <typename IN, typename OUT>
cudaError_t launch(const LogitsArgs& k, int parts, cudaStream_t st) {
  static bool ready[64] = {};  // per device: the attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(logits_kernel<IN, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSlice * 4);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(k.a.batch) * k.a.T * parts);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(k.slice) * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = parts;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, logits_kernel<IN, OUT>, k);
}

template <typename IN>
cudaError_t launch_out(const LogitsArgs& k, int parts, cudaStream_t st) {
  return k.a.out_dtype == RSSM_F32    ? launch<IN, float>(k, parts, st)
         : k.a.out_dtype == RSSM_BF16 ? launch<IN, __nv_bfloat16>(k, parts, st)
                                      : launch<IN, __half>(k, parts, st);
}

}  // namespace
}  // namespace rssm

using namespace rssm;

extern "C" rssm_status rssm_logits(const rssm_logits_args* args, void* stream) {
  if (!args) return RSSM_ERR_INVALID_ARGUMENT;
  const rssm_logits_args& a = *args;
  const auto known = [](int d) { return d == RSSM_F32 || d == RSSM_BF16 || d == RSSM_F16; };
  const auto al = [](const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
  if (a.batch < 0 || a.T < 1 || a.vocab < 1 || a.ntok < 0 || !known(a.logits_dtype) || !known(a.out_dtype)) return RSSM_ERR_INVALID_ARGUMENT;
  if (a.probs != 0 && a.probs != 1) return RSSM_ERR_INVALID_ARGUMENT;
  if (a.vocab > kMaxVocab || a.T > kTreeT || a.ntok > INT32_MAX) return RSSM_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(a.batch) * a.T > (1 << 27)) return RSSM_ERR_UNSUPPORTED;
  if (!al(a.logits, a.logits_dtype == RSSM_F32 ? 4 : 2) || !al(a.out, a.out_dtype == RSSM_F32 ? 4 : 2)) return RSSM_ERR_INVALID_ARGUMENT;
  for (const void* p : {static_cast<const void*>(a.cu_seqlens), static_cast<const void*>(a.temperature), static_cast<const void*>(a.repetition),
                        static_cast<const void*>(a.presence), static_cast<const void*>(a.frequency), static_cast<const void*>(a.history),
                        static_cast<const void*>(a.history_len), static_cast<const void*>(a.prompt_len), static_cast<const void*>(a.tokens),
                        static_cast<const void*>(a.parents), static_cast<const void*>(a.bias_start), static_cast<const void*>(a.bias_id),
                        static_cast<const void*>(a.bias_value), static_cast<const void*>(a.mask), static_cast<const void*>(a.error_word)})
    if (!al(p, 4)) return RSSM_ERR_INVALID_ARGUMENT;
  if (a.history && (!a.history_len || a.history_max < 0 || a.history_stride < a.history_max)) return RSSM_ERR_INVALID_ARGUMENT;
  if (a.bias_id && (!a.bias_start || !a.bias_value || a.biases < 0)) return RSSM_ERR_INVALID_ARGUMENT;
  if (a.mask && a.mask_stride < (static_cast<int64_t>(a.vocab) + 31) / 32) return RSSM_ERR_INVALID_ARGUMENT;
  if (a.logits_stride < a.vocab || a.out_stride < a.vocab) return RSSM_ERR_INVALID_ARGUMENT;
  if (!a.cu_seqlens && static_cast<int64_t>(a.batch) * a.T > a.ntok) return RSSM_ERR_INVALID_ARGUMENT;
  if (a.batch == 0 || a.ntok == 0) return RSSM_OK;
  if (!a.logits || !a.out) return RSSM_ERR_INVALID_ARGUMENT;
  const int sms = num_sms();
  if (sms == 0) return RSSM_ERR_CUDA;
  // blocks of a row: while all rows' still run at once, and each has 2048 ids; and as many as a slice's words need
  int parts = 1;
  while (parts < kMaxParts && ((static_cast<int64_t>(a.batch) * a.T * parts * 2 <= 2 * sms && a.vocab > parts * 2048) || a.vocab > parts * (kMaxSlice / 2)))
    parts *= 2;
  LogitsArgs k;
  k.a = a;
  k.slice = ((a.vocab + parts - 1) / parts + 31) / 32 * 32;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a.logits_dtype == RSSM_F32    ? launch_out<float>(k, parts, st)
                        : a.logits_dtype == RSSM_BF16 ? launch_out<__nv_bfloat16>(k, parts, st)
                                                      : launch_out<__half>(k, parts, st);
  return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}
