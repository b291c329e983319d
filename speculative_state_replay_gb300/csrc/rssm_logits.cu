// rssm_logits.cu -- from logits to the probabilities that the verification
// takes: penalties for repeated tokens, biases, grammar masks, temperature.
//
// Bound by memory: a row is read once and written once.  A cluster of blocks takes a
// row, each a slice of the vocabulary that it keeps in shared memory, one 32-bit word
// an id.  A word is first the id's count in the request's text -- every block goes over
// the whole history and keeps what falls into its slice, integer additions in shared
// memory, whose order does not matter -- then the processed logit, then its
// exponential.  Each block takes them against its own maximum; maxima and sums meet once
// through the cluster's shared memory.  Rows of any alignment are read 16 bytes a lane:
// places are counted from the 16-byte boundary before the row's first value.  252 rows
// of 131073 bf16 values, 132 MB: 52 us without options, 106 us with a history of 8192
// tokens (25 us: every block reads all of it), a mask and 100 biases a request.  Threads
// a block: 256 take 52 us where 128 take 71 and 512 take 78 (no options, 131072 values).
#include <cooperative_groups.h>

#include "rssm_kv.cuh"

namespace cg = cooperative_groups;

namespace rssm {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBlocks = 3;              // an SM
constexpr int kMaxParts = 8;            // blocks of a cluster (the portable most)
constexpr int kMaxVocab = 1 << 18;
constexpr int kRun = 8;                 // ids of a lane's step
constexpr int kAhead = 4;               // steps whose loads are on their way at a time
constexpr int kStride = kThreads * kRun;
constexpr int kMaxSlice = kMaxVocab / kMaxParts + 32;  // words of a block: 128 KB
constexpr unsigned kSeen = 1u << 31;    // bits of a count: the prompt holds the id,
constexpr unsigned kBiased = 1u << 30;  // it has a bias

struct LogitsArgs {
  rssm_logits_args a;
  int slice;  // words of a block, a multiple of 32
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

// largest value, and of equal ones the lowest id, as one number that orders like them
__device__ __forceinline__ unsigned long long top_key(float x, int id) {
  const uint32_t u = __float_as_uint(x == 0.0f ? 0.0f : x);  // -0 is 0
  const uint32_t o = u & 0x80000000u ? ~u : u | 0x80000000u;
  return static_cast<unsigned long long>(o) << 32 | (0xffffffffu - static_cast<uint32_t>(id));
}

template <typename IN, typename OUT>
__global__ void __launch_bounds__(kThreads, kBlocks) logits_kernel(const LogitsArgs k) {
  constexpr int VEC = 16 / sizeof(IN), PIECES = kRun / VEC;  // 16-byte pieces of a step
  extern __shared__ __align__(16) uint32_t word[];  // [slice]
  __shared__ float sh_part[kWarps];
  __shared__ unsigned long long sh_key[kWarps];
  __shared__ float sh_top[kMaxParts], sh_sum[kMaxParts];
  __shared__ unsigned long long sh_best[kMaxParts];
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
  if (parts > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this block runs: its sums can be written
  const long long tok = first + t;
  const IN* x = static_cast<const IN*>(a.logits) + tok * a.logits_stride;
  OUT* out = static_cast<OUT*>(a.out) + tok * a.out_stride;
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(IN));
  const int base = rank * k.slice - off;  // the id of word 0
  const int words = min(k.slice, a.vocab - base);  // up to the last id's; none: <= 0
  // where word w lies: a step's first four and last four words in planes of their own, so that a warp's 16-byte accesses neighbour
  const int plane = k.slice / 2;
  auto at = [&](int w) { return (w >> 3) * 4 + (w & 3) + (w & 4 ? plane : 0); };
  // (an id may be any 32 bits: id - base of the largest would pass them where the row begins up to seven places in)
  auto holds = [&](int id) { return id >= max(base, 0) && id < base + words; };

  // ---- the first logits, asked for early
  uint4 raw[kAhead][PIECES];
  auto ask = [&](int w0) {
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      const int w = w0 + s * kStride + threadIdx.x * kRun, id = base + w;
      if (w < words && id >= 0 && w + kRun <= words) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) raw[s][i] = __ldcs(reinterpret_cast<const uint4*>(x + id) + i);
      }
    }
  };
  ask(0);

  // a request's parents, whatever its penalties
  if (a.parents && t == 0 && rank == 0 && warp == 0) {
    bool fine = true;
#pragma unroll
    for (int i = lane; i < kTreeT; i += 32)
      if (i < n) {
        const int up = a.parents[first + i];
        fine = fine && up >= -1 && up < i;
      }
    if (!__all_sync(full, fine) && lane == 0) set_error(a.error_word, RSSM_ERRBIT_TREE);
  }

  float temp = a.temperature ? a.temperature[b] : 1.0f;
  if (!(temp >= 0.0f)) temp = 1.0f;
  float rep = a.repetition ? a.repetition[b] : 1.0f;
  if (!(rep > 0.0f)) rep = 1.0f;
  const float less = __fdiv_rn(1.0f, rep);  // x / repetition is x times this: one rounding more
  const float presence = a.presence ? a.presence[b] : 0.0f, frequency = a.frequency ? a.frequency[b] : 0.0f;
  const bool counted = rep != 1.0f || presence != 0.0f || frequency != 0.0f;
  long long bias_lo = 0, bias_hi = 0;
  if (a.bias_id) {
    bias_lo = max(0, a.bias_start[b]);
    bias_hi = min(static_cast<long long>(a.bias_start[b + 1]), static_cast<long long>(a.biases));
  }
  const bool biased = bias_lo < bias_hi, marked = counted || biased;

  // ---- counts, and marks of ids with a bias
  if (marked) {
    for (int i = threadIdx.x * 4; i < k.slice; i += kThreads * 4) *reinterpret_cast<uint4*>(word + i) = make_uint4(0u, 0u, 0u, 0u);
    if (counted && warp == 0 && a.tokens) {
      // the fed tokens on the path to this one
      unsigned long long mask = (2ull << t) - 1ull;  // a chain: all up to it
      if (a.parents) {
        unsigned long long m[2];
        if (tree_masks(a.parents + first, n, lane, m)) {
          const unsigned long long m0 = __shfl_sync(full, m[0], t & 31), m1 = __shfl_sync(full, m[1], t & 31);
          mask = t < 32 ? m0 : m1;
        } else {
          mask = 1ull << t;
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int j = lane + 32 * i;
        sh_fed[j] = mask >> j & 1 && j < n ? a.tokens[first + j] : -1;
      }
    }
    __syncthreads();
    if (counted && a.history) {
      const int* h = a.history + b * a.history_stride;
      const int len = min(max(a.history_len[b], 0), a.history_max);
      const int prompt = a.prompt_len ? min(max(a.prompt_len[b], 0), len) : 0;
      for (int i0 = threadIdx.x; i0 < len; i0 += 8 * kThreads) {
        int id[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) id[e] = i0 + e * kThreads < len ? h[i0 + e * kThreads] : -1;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (holds(id[e])) {
            if (i0 + e * kThreads < prompt) atomicOr(word + at(id[e] - base), kSeen);
            else atomicAdd(word + at(id[e] - base), 1u);
          }
        }
      }
    }
    if (counted && a.tokens && threadIdx.x < kTreeT && holds(sh_fed[threadIdx.x])) atomicAdd(word + at(sh_fed[threadIdx.x] - base), 1u);
    for (long long e = bias_lo + threadIdx.x; e < bias_hi; e += kThreads) {
      const int id = a.bias_id[e];
      if (holds(id)) atomicOr(word + at(id - base), kBiased);
    }
    __syncthreads();
  }

  // ---- the logits with their penalties, masked, into the words
  const uint32_t* mask = a.mask ? a.mask + tok * a.mask_stride : nullptr;
  float top = -INFINITY;
  unsigned long long key = 0ull;
  const bool greedy = temp == 0.0f;
  auto take = [&](float y, int id) {
    top = fmaxf(top, y);
    if (greedy && y > -INFINITY) key = max(key, top_key(y, id));
  };
  auto allowed = [&](int id) {  // the mask's bits of eight ids, the first of which may be before the row's
    if (!mask) return 0xffu;
    if (id < 0) return mask[0] << -id;
    const uint32_t lo = mask[id >> 5], hi = (id & 31) > 24 && (id | 31) + 1 < a.vocab ? mask[(id >> 5) + 1] : 0u;
    return __funnelshift_r(lo, hi, id & 31);
  };
  for (int w0 = 0; w0 < words; w0 += kAhead * kStride) {
    if (w0) ask(w0);
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
      const int w = w0 + s * kStride + threadIdx.x * kRun, id = base + w;
      if (w >= words) continue;
      const bool all = id >= 0 && w + kRun <= words;
      float f[kRun];
      if (all) {
#pragma unroll
        for (int e = 0; e < kRun; ++e) f[e] = value<IN>(reinterpret_cast<const IN*>(raw[s])[e]);
      } else {
#pragma unroll
        for (int e = 0; e < kRun; ++e) f[e] = id + e >= 0 && w + e < words ? value<IN>(x[id + e]) : -INFINITY;
      }
      const uint32_t ok = allowed(id);
      uint4* const p0 = reinterpret_cast<uint4*>(word + (w >> 1));
      uint4* const p1 = reinterpret_cast<uint4*>(word + plane + (w >> 1));
      uint32_t later = 0u;  // ids with a bias: their turn comes with that
      if (marked) {
        const uint4 c0 = *p0, c1 = *p1;
        if (c0.x | c0.y | c0.z | c0.w | c1.x | c1.y | c1.z | c1.w) {
          const uint32_t c[kRun] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
          for (int e = 0; e < kRun; ++e) {
            // (no branches: of a warp's 256 ids some mostly count)
            const unsigned m = c[e] & ~(kSeen | kBiased);
            const float y = f[e] * (f[e] > 0.0f ? less : rep);
            f[e] = c[e] & ~kBiased ? y : f[e];
            f[e] -= m ? presence + frequency * static_cast<float>(m) : 0.0f;
            later |= (c[e] & kBiased) >> (30 - e);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < kRun; ++e) f[e] = ok >> e & 1u ? f[e] : -INFINITY;
      *p0 = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
      *p1 = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
      if (later || greedy) {
#pragma unroll
        for (int e = 0; e < kRun; ++e)
          if (!(later >> e & 1u)) take(f[e], id + e);
      } else {
        top = fmaxf(fmaxf(fmaxf(top, fmaxf(f[0], f[1])), fmaxf(f[2], f[3])), fmaxf(fmaxf(f[4], f[5]), fmaxf(f[6], f[7])));  // (not of NaN)
      }
    }
  }
  float* const val = reinterpret_cast<float*>(word);
  if (biased) {
    // ---- the biases: those of this block's ids, in order, a part of the entries at a time
    __syncthreads();
    for (long long e0 = bias_lo; e0 < bias_hi; e0 += kThreads) {
      const long long e = e0 + threadIdx.x;
      const int id = e < bias_hi ? a.bias_id[e] : -1;
      const bool mine = holds(id);
      const unsigned kept = __ballot_sync(full, mine);
      if (lane == 0) sh_kept[warp] = __popc(kept);
      __syncthreads();
      int place = __popc(kept & ((1u << lane) - 1u)), all = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        if (i < warp) place += sh_kept[i];
        all += sh_kept[i];
      }
      if (mine) {
        sh_id[place] = id - base;
        sh_bias[place] = a.bias_value[e];
      }
      __syncthreads();
      if (warp == 0) {
        // of 32 entries at a time, the first lane of those with one id adds them up
        for (int i0 = 0; i0 < all; i0 += 32) {
          const bool on = i0 + lane < all;
          const int w = on ? sh_id[i0 + lane] : -1 - lane;
          const float v = on ? sh_bias[i0 + lane] : 0.0f;
          const unsigned same = __match_any_sync(full, w);
          const int most = __reduce_max_sync(full, __popc(same));
          float sum = on ? val[at(w)] : 0.0f;
          unsigned rest = same;
          for (int j = 0; j < most; ++j) {
            const float add = __shfl_sync(full, v, rest ? __ffs(rest) - 1 : lane);
            if (rest) sum += add;
            rest &= rest - 1u;
          }
          if (on && lane == __ffs(same) - 1) val[at(w)] = sum;
          __syncwarp();
        }
      }
      __syncthreads();
    }
    // (entries of one id look at the same value)
    for (long long e = bias_lo + threadIdx.x; e < bias_hi; e += kThreads) {
      const int id = a.bias_id[e];
      if (holds(id) && val[at(id - base)] == val[at(id - base)]) take(val[at(id - base)], id);
    }
  }

  const bool wide = ((reinterpret_cast<uintptr_t>(out) - off * sizeof(OUT)) & 15u) == 0;
  // the words, times `scale`, to the row: 16 bytes a lane where its alignment goes with the logits', else neighbouring values by neighbouring lanes
  auto write = [&](auto result) {  // result(word, its id)
    if (wide) {
      constexpr int OV = 16 / sizeof(OUT);
      for (int w = threadIdx.x * kRun; w < words; w += kStride) {
        const int id = base + w;
        const float4 v0 = *reinterpret_cast<const float4*>(val + (w >> 1)), v1 = *reinterpret_cast<const float4*>(val + plane + (w >> 1));
        const float v[kRun] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
        OUT y[kRun];
#pragma unroll
        for (int e = 0; e < kRun; ++e) y[e] = rounded<OUT>(result(v[e], id + e));
        if (id >= 0 && w + kRun <= words) {
#pragma unroll
          for (int i = 0; i < kRun; i += OV) __stcs(reinterpret_cast<uint4*>(out + id + i), *reinterpret_cast<const uint4*>(y + i));
        } else {
#pragma unroll
          for (int e = 0; e < kRun; ++e)
            if (id + e >= 0 && w + e < words) out[id + e] = y[e];
        }
      }
    } else {
      for (int w = threadIdx.x + max(0, -base); w < words; w += kThreads) out[base + w] = rounded<OUT>(result(val[at(w)], base + w));
    }
  };
  if (!a.probs) {
    __syncthreads();
    write([&](float y, int) {
      if (y != y) y = -INFINITY;
      return temp > 0.0f ? __fdiv_rn(y, temp) : y;
    });
    if (parts > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    return;
  }

  // ---- the block's maximum, its exponentials and their sum; then the row's
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
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    top = fmaxf(top, sh_part[i]);
    key = max(key, sh_key[i]);
  }
  float sum = 0.0f;
  const float cool = __fdiv_rn(1.0f, temp);  // the temperature divides what is left of the largest: that stays in range
  auto weight = [&](float y, float most) {   // (infinite ones too, and any temperature; NaN: 0)
    const float d = y - most;
    return y == most ? 1.0f : d > -INFINITY ? expf(d * cool) : 0.0f;
  };
  if (temp > 0.0f && top > -INFINITY) {
    // by the hardware's power of two, of the difference from the maximum: a value of e^x is off by 2^-23 (1 + |x|) of
    // itself, and what has large |x| is small.  (Of NaN the maximum takes 0.)
    const float by = cool * 1.4426950408889634f;
    const bool plain = top < INFINITY && by > 0.0f && by < INFINITY;
    auto power = [&](float y) {
      float e;
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"((y - top) * by));
      return fmaxf(e, 0.0f);
    };
    float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int w = threadIdx.x * kRun; w < words; w += kStride) {
      float4* const q0 = reinterpret_cast<float4*>(val + (w >> 1));
      float4* const q1 = reinterpret_cast<float4*>(val + plane + (w >> 1));
      float4 f = *q0, g = *q1;
      if (plain) {
        f = make_float4(power(f.x), power(f.y), power(f.z), power(f.w));
        g = make_float4(power(g.x), power(g.y), power(g.z), power(g.w));
      } else {
        f = make_float4(weight(f.x, top), weight(f.y, top), weight(f.z, top), weight(f.w, top));
        g = make_float4(weight(g.x, top), weight(g.y, top), weight(g.z, top), weight(g.w, top));
      }
      s4[0] += f.x + g.x;
      s4[1] += f.y + g.y;
      s4[2] += f.z + g.z;
      s4[3] += f.w + g.w;
      *q0 = f;
      *q1 = g;
    }
    sum = (s4[0] + s4[1]) + (s4[2] + s4[3]);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(full, sum, o);
  }
  __syncthreads();  // sh_part is read
  if (lane == 0) sh_part[warp] = sum;
  __syncthreads();
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) sum += sh_part[i];
  float most = top;
  if (parts > 1) {
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (threadIdx.x < parts) {
      *cl.map_shared_rank(&sh_top[rank], threadIdx.x) = top;
      *cl.map_shared_rank(&sh_sum[rank], threadIdx.x) = sum;
      *cl.map_shared_rank(&sh_best[rank], threadIdx.x) = key;
    }
    cl.sync();
    for (int i = 0; i < parts; ++i) {
      most = fmaxf(most, sh_top[i]);
      key = max(key, sh_best[i]);
    }
    sum = 0.0f;
    for (int i = 0; i < parts; ++i) sum += sh_sum[i] > 0.0f ? sh_sum[i] * weight(sh_top[i], most) : 0.0f;
  }
  if (temp > 0.0f) {
    // (a block whose values are all -inf has them in the words still)
    const float scale = top > -INFINITY && sum > 0.0f ? weight(top, most) * __fdiv_rn(1.0f, sum) : 0.0f;
    if (scale > 0.0f) write([&](float y, int) { return y * scale; });
    else write([&](float, int) { return 0.0f; });
  } else {
    const int best = key ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(key)) : -1;
    write([&](float, int id) { return id == best ? 1.0f : 0.0f; });
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
  // blocks of a row: while all rows' still run at once, and each has 2048 ids; and as many as let three blocks' words be on an SM
  int parts = 1;
  while (parts < kMaxParts && ((static_cast<int64_t>(a.batch) * a.T * parts * 2 <= kBlocks * sms && a.vocab > parts * 2048) || a.vocab > parts * 16384))
    parts *= 2;
  LogitsArgs k;
  k.a = a;
  k.slice = ((a.vocab + 7 + parts - 1) / parts + 31) / 32 * 32;  // (a row begins up to seven places in)
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a.logits_dtype == RSSM_F32    ? launch_out<float>(k, parts, st)
                        : a.logits_dtype == RSSM_BF16 ? launch_out<__nv_bfloat16>(k, parts, st)
                                                      : launch_out<__half>(k, parts, st);
  return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}
