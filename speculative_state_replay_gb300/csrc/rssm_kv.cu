// rssm_kv.cu -- the paged cache of keys and values: writing new tokens,
// reading tokens back, and the commit of a tree's accepted drafts.
#include "rssm_kv.cuh"

#include <type_traits>

namespace rssm {
namespace {

constexpr int kWarps = 8;  // a block of the append and read kernels: a warp takes a token

struct KvPlace {
  long long page;
  int slot;
};

// Whether the bounds of all rows are sound, by a whole block; sets the error bit if not.
__device__ __forceinline__ bool bounds_sound(const KvRows& r, unsigned* err) {
  int bad = 0;
  for (int b = threadIdx.x; b < r.batch; b += blockDim.x) bad |= row_span(r, b).count < 0;
  if (!__syncthreads_or(bad)) return true;
  if (threadIdx.x == 0) set_error(err, RSSM_ERRBIT_SEQLEN);
  return false;
}

// Where position `pos` of row b is: false if it is past the row's table or in no page.
__device__ __forceinline__ bool kv_place(const KvView& c, const KvRows& r, int b, long long pos, KvPlace& at) {
  if (pos >= static_cast<long long>(r.max_pages) * c.page_size) return false;
  const unsigned p = static_cast<unsigned>(pos), page = p / static_cast<unsigned>(c.page_size);
  at.slot = static_cast<int>(p - page * c.page_size);
  at.page = r.pages[b * r.pages_stride + page];
  return at.page >= 0 && at.page < c.pages;
}

// --------------------------------------------------------------------------
// Writing.  Bound by memory: a token's heads are read once (2 bytes a value) and
// written once.  A warp takes a token, its keys' heads and then its values', D / 8
// lanes a head with 8 values each, four heads' loads a lane on their way at a time
// (they do not depend on where the token goes, so the first four leave before the
// token's row and page are looked up).  The largest magnitude of a head is found on
// the bits: magnitudes order as integers, and what is not finite is at 0x7f80 and above.
// A token's row is found by the rows' ends, which order where all bounds are sound.  The
// first block looks whether they are, and goes over the sound rows itself if not, since
// some of their tokens may then have been found in no row, or in another.
// Measured: 16411 tokens of 8 heads of 128 as int8, 102 MB, 22.7 us, 4.5 TB/s; issue slots
// are 70 % taken, and the two ends of so short a launch are in it.
// --------------------------------------------------------------------------
struct AppendArgs {
  KvView c;
  KvRows r;
  const uint16_t* k;
  const uint16_t* v;
  long long k_stride, v_stride;
};

// Codes of eight values times 1 / scale.  int8 ones need no limits: no magnitude is above the head's largest, which
// three roundings of 2^-24 take to no more than 127 (1 + 2^-22).
template <int FMT>
__device__ __forceinline__ uint2 quantize8(const uint4& x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t out[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float v[4];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      v[2 * q] = __fmul_rn(bf16lo(w[2 * h + q]), inv);
      v[2 * q + 1] = __fmul_rn(bf16hi(w[2 * h + q]), inv);
    }
    if constexpr (FMT == RSSM_I8) {
      // adding 1.5 2^23 rounds to an integer, to even; its low byte is the code
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = __fadd_rn(v[q], 12582912.0f);
      out[h] = __byte_perm(__byte_perm(__float_as_uint(v[0]), __float_as_uint(v[1]), 0x0040u),
                           __byte_perm(__float_as_uint(v[2]), __float_as_uint(v[3]), 0x0040u), 0x5410u);
    } else {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE, __NV_E4M3);
      out[h] = lo | hi << 16;
    }
  }
  return make_uint2(out[0], out[1]);
}

// token `tok`, of row `row` or (-1) of the one that it is found in, by a warp; RUN heads' loads of a lane on their way at a time
template <int D, int FMT, int RUN>
__device__ __forceinline__ void append_token(const AppendArgs& a, long long tok, int row) {
  constexpr int G = D / 8, AT_ONCE = 32 / G;
  const KvView& c = a.c;
  const int lane = threadIdx.x & 31, mine = lane / G, part = lane % G;
  const int items = 2 * c.heads;
  constexpr int ESZ = FMT == RSSM_BF16 ? 2 : 1;
  const uint16_t* const from_k = a.k + tok * a.k_stride + part * 8;
  const uint16_t* const from_v = a.v + tok * a.v_stride + part * 8 - c.heads * D;
  uint8_t *to_k = nullptr, *to_v = nullptr;  // of the token's place in head 0 (to_v: of head -heads)
  float *scale_k = nullptr, *scale_v = nullptr;
  const unsigned stride = static_cast<unsigned>(c.page_size) * (D * ESZ);  // bytes between heads
#pragma unroll 1
  for (int i0 = 0; i0 < items; i0 += RUN * AT_ONCE) {
    uint4 x[RUN];
#pragma unroll
    for (int u = 0; u < RUN; ++u) {
      const int i = i0 + u * AT_ONCE + mine;
      x[u] = i < items ? __ldcs(reinterpret_cast<const uint4*>((i >= c.heads ? from_v : from_k) + i * D)) : make_uint4(0u, 0u, 0u, 0u);
    }
    if (i0 == 0) {
      const int b = row < 0 ? find_row(a.r, tok, lane) : row;
      if (b < 0) return;
      const RowSpan s = row_span(a.r, b);
      const long long t = tok - s.first;
      if (t < 0 || t >= s.count) return;  // (bounds that are not sound: the first block says so)
      const int len = a.r.lengths[b];
      if (len < 0) return;
      KvPlace at;
      if (!kv_place(c, a.r, b, len + t, at)) {
        if (lane == 0) set_error(c.err, RSSM_ERRBIT_PAGE);
        return;
      }
      to_k = c.k + at.page * c.k_page + at.slot * (D * ESZ) + part * (8 * ESZ);
      to_v = c.v + at.page * c.v_page + at.slot * (D * ESZ) + part * (8 * ESZ) - static_cast<long long>(c.heads) * stride;
      if constexpr (FMT != RSSM_BF16) {
        scale_k = c.ks + at.page * c.ks_page + at.slot;
        scale_v = c.vs + at.page * c.vs_page + at.slot - static_cast<long long>(c.heads) * c.page_size;
      }
    }
#pragma unroll
    for (int u = 0; u < RUN; ++u) {
      const int i = i0 + u * AT_ONCE + mine;
      const bool values = i >= c.heads;
      uint8_t* const to = (values ? to_v : to_k) + static_cast<unsigned long long>(i) * stride;
      if constexpr (FMT == RSSM_BF16) {
        if (i < items) *reinterpret_cast<uint4*>(to) = x[u];
      } else {
        uint32_t m = __vmaxu2(__vmaxu2(x[u].x & 0x7fff7fffu, x[u].y & 0x7fff7fffu), __vmaxu2(x[u].z & 0x7fff7fffu, x[u].w & 0x7fff7fffu));
#pragma unroll
        for (int o = 1; o < G; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
        const uint32_t most = max(m & 0xffffu, m >> 16);
        const float amax = __uint_as_float(most << 16);
        const bool finite = most < 0x7f80u;
        const float scale = !finite ? __uint_as_float(0x7fffffffu)
                            : amax < 7.888609052210118e-31f /* 2^-100 */ ? 1.0f
                                                                         : __fmul_rn(amax, FMT == RSSM_I8 ? 1.0f / 127.0f : 1.0f / 448.0f);
        const uint2 codes = quantize8<FMT>(x[u], __frcp_rn(scale));
        if (i < items) {
          *reinterpret_cast<uint2*>(to) = finite ? codes : make_uint2(0u, 0u);
          if (part == 0) (values ? scale_v : scale_k)[static_cast<long long>(i) * c.page_size] = scale;
        }
      }
    }
  }
}
template <int D, int FMT>
__global__ void __launch_bounds__(kWarps * 32) append_kernel(const __grid_constant__ AppendArgs a) {
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5;
  if (a.r.cu && blockIdx.x == 0) {
    if (bounds_sound(a.r, a.c.err)) return;
    for (int b = 0; b < a.r.batch; ++b) {
      const RowSpan s = row_span(a.r, b);
      for (int t = warp; t < s.count; t += kWarps) append_token<D, FMT, 1>(a, s.first + t, b);
    }
    return;
  }
  const long long tok = static_cast<long long>(blockIdx.x - (a.r.cu ? 1 : 0)) * kWarps + warp;
  if (tok < a.r.tokens) append_token<D, FMT, 4>(a, tok, -1);
}

// --------------------------------------------------------------------------
// Reading back: the same cut, the other way.  51584 tokens of 8 heads of 128, e4m3 to
// bf16, 320 MB: 51.0 us, 6.3 TB/s (92 % of a copy).
// --------------------------------------------------------------------------
struct ReadArgs {
  KvView c;
  KvRows r;
  void* k;
  void* v;
  long long k_stride, v_stride;  // elements
};

template <int FMT>
__device__ __forceinline__ void decode8(const uint4& x, float scale, float (&f)[8]) {
  if constexpr (FMT == RSSM_BF16) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f[2 * q] = bf16lo(w[q]);
      f[2 * q + 1] = bf16hi(w[q]);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t w = h ? x.y : x.x;
      if constexpr (FMT == RSSM_I8) {
        // code + 128 in the low byte of 2^23: 2^23 + 128 + code
        const uint32_t y = w ^ 0x80808080u;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          f[4 * h + q] = __fmul_rn(__fsub_rn(__uint_as_float(__byte_perm(y, 0x4b000000u, 0x7440u + q)), 8388736.0f), scale);
      } else {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const __half2_raw y = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(q ? w >> 16 : w & 0xffffu), __NV_E4M3);
          const float2 z = __half22float2(__half2(y));
          f[4 * h + 2 * q] = __fmul_rn(z.x, scale);
          f[4 * h + 2 * q + 1] = __fmul_rn(z.y, scale);
        }
      }
    }
  }
}

__device__ __forceinline__ uint32_t two_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t two_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// (as append_token)
template <int D, int FMT, int OUT, int RUN>
__device__ __forceinline__ void read_token(const ReadArgs& a, long long tok, int row) {
  constexpr int G = D / 8, AT_ONCE = 32 / G, ESZ = FMT == RSSM_BF16 ? 2 : 1;
  const KvView& c = a.c;
  const int lane = threadIdx.x & 31, mine = lane / G, part = lane % G;
  const int b = row < 0 ? find_row(a.r, tok, lane) : row;
  if (b < 0) return;
  const RowSpan s = row_span(a.r, b);
  const long long t = tok - s.first;
  if (t < 0 || t >= s.count) return;
  const int start = a.r.lengths ? a.r.lengths[b] : 0;
  KvPlace at = {0, 0};
  bool have = start >= 0;
  if (have && !kv_place(c, a.r, b, start + t, at)) {
    have = false;
    if (lane == 0) set_error(c.err, RSSM_ERRBIT_PAGE);
  }
  const int items = 2 * c.heads;
  // of the token's place in head 0 (values: of head -heads), read and written
  const unsigned stride = static_cast<unsigned>(c.page_size) * (D * ESZ);
  const uint8_t* const from_k = c.k + at.page * c.k_page + at.slot * (D * ESZ) + part * (8 * ESZ);
  const uint8_t* const from_v = c.v + at.page * c.v_page + at.slot * (D * ESZ) + part * (8 * ESZ) - static_cast<long long>(c.heads) * stride;
  const float *scale_k = nullptr, *scale_v = nullptr;
  if constexpr (FMT != RSSM_BF16) {
    scale_k = c.ks + at.page * c.ks_page + at.slot;
    scale_v = c.vs + at.page * c.vs_page + at.slot - static_cast<long long>(c.heads) * c.page_size;
  }
  using Out = typename std::conditional<OUT == RSSM_F32, float, uint16_t>::type;
  Out* const to_k = static_cast<Out*>(a.k) + tok * a.k_stride + part * 8;
  Out* const to_v = static_cast<Out*>(a.v) + tok * a.v_stride + part * 8 - c.heads * D;
#pragma unroll 1
  for (int i0 = 0; i0 < items; i0 += RUN * AT_ONCE) {
    uint4 x[RUN];
    float scale[RUN];
#pragma unroll
    for (int u = 0; u < RUN; ++u) {
      const int i = i0 + u * AT_ONCE + mine;
      const bool values = i >= c.heads;
      const uint8_t* p = (values ? from_v : from_k) + static_cast<unsigned long long>(i) * stride;
      x[u] = make_uint4(0u, 0u, 0u, 0u);
      scale[u] = 0.0f;
      if (have && i < items) {
        if constexpr (FMT == RSSM_BF16) {
          x[u] = __ldcs(reinterpret_cast<const uint4*>(p));
        } else {
          const uint2 y = __ldcs(reinterpret_cast<const uint2*>(p));
          x[u].x = y.x;
          x[u].y = y.y;
          scale[u] = (values ? scale_v : scale_k)[static_cast<long long>(i) * c.page_size];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < RUN; ++u) {
      const int i = i0 + u * AT_ONCE + mine;
      if (i >= items) continue;
      Out* const p = (i >= c.heads ? to_v : to_k) + i * D;
      float f[8];
      decode8<FMT>(x[u], scale[u], f);
      if constexpr (OUT == RSSM_F32) {
        __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
        __stcs(reinterpret_cast<float4*>(p + 4), make_float4(f[4], f[5], f[6], f[7]));
      } else {
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = OUT == RSSM_BF16 ? two_bf16(f[2 * q], f[2 * q + 1]) : two_f16(f[2 * q], f[2 * q + 1]);
        __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
      }
    }
  }
}
template <int D, int FMT, int OUT>
__global__ void __launch_bounds__(kWarps * 32) read_kernel(const __grid_constant__ ReadArgs a) {
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5;
  if (blockIdx.x == 0) {
    if (bounds_sound(a.r, a.c.err)) return;
    for (int b = 0; b < a.r.batch; ++b) {
      const RowSpan s = row_span(a.r, b);
      for (int t = warp; t < s.count; t += kWarps) read_token<D, FMT, OUT, 1>(a, s.first + t, b);
    }
    return;
  }
  const long long tok = static_cast<long long>(blockIdx.x - 1) * kWarps + warp;
  if (tok < a.r.tokens) read_token<D, FMT, OUT, 4>(a, tok, -1);
}

// --------------------------------------------------------------------------
// The commit of a tree.  A block per (row, layer); each walks the row's tree by its
// first warp (a step down is two ballots), so no block waits for another.  Entries
// move to positions not after their own, and paths rise, so a thread that takes the
// same 16 bytes of every entry in order never overwrites what it still has to read;
// their loads leave eight at a time.  64 rows' trees of up to 48 tokens take 7.5 us, one
// row's of 8 6.9: the call.
// --------------------------------------------------------------------------
struct AcceptArgs {
  KvView c;  // k null: no cache
  KvRows r;
  const int* tokens;
  const int* parents;  // or null: a chain
  const int* drawn;
  int* accepted;
  int* next;
  int* path;
};

constexpr int kAcceptThreads = 256;

__global__ void __launch_bounds__(kAcceptThreads) accept_kernel(const AcceptArgs a) {
  __shared__ int sh_path[kTreeT];
  __shared__ long long sh_page[2][kTreeT];  // where an accepted token lies, and where it goes
  __shared__ int sh_slot[2][kTreeT];
  __shared__ int sh_count;
  const int b = blockIdx.x, layer = blockIdx.y, lane = threadIdx.x & 31;
  const unsigned full = 0xffffffffu;
  pdl_wait();
  pdl_trigger();
  const KvView& c = a.c;
  if (threadIdx.x < 32) {
    const RowSpan s = row_span(a.r, b);
    const int len = a.r.lengths ? a.r.lengths[b] : 0;
    unsigned bad = s.count < 0 ? RSSM_ERRBIT_SEQLEN : 0u;
    const int n = len < 0 || bad ? 0 : s.count;
    int up[2], tok[2], drawn[2];
    bool ok = true;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = lane + 32 * i;
      up[i] = -2;
      tok[i] = drawn[i] = -1;
      if (t < n) {
        up[i] = a.parents ? a.parents[s.first + t] : t - 1;
        tok[i] = a.tokens[s.first + t];
        drawn[i] = a.drawn[s.first + t];
        ok = ok && up[i] >= -1 && up[i] < t;
      }
    }
    if (!__all_sync(full, ok)) bad = RSSM_ERRBIT_TREE;
    int count = 0, next = -1;
    if (n > 0 && !bad) {
      int cur = 0;
      while (true) {
        if (lane == 0) sh_path[count] = cur;
        ++count;
        const int d0 = __shfl_sync(full, drawn[0], cur & 31), d1 = __shfl_sync(full, drawn[1], cur & 31);
        next = cur < 32 ? d0 : d1;
        const unsigned m0 = __ballot_sync(full, up[0] == cur && tok[0] == next), m1 = __ballot_sync(full, up[1] == cur && tok[1] == next);
        if (next < 0 || !(m0 | m1)) break;
        cur = m0 ? __ffs(m0) - 1 : __ffs(m1) + 31;  // after its parent: the walk ends
      }
    }
    __syncwarp();
    // where the accepted tokens lie and where they go
    if (c.k && count > 0) {
      bool found = static_cast<long long>(len) + n <= static_cast<long long>(a.r.max_pages) * c.page_size;
      if (found) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int j = lane + 32 * i;
          if (j < count) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const unsigned pos = static_cast<unsigned>(len) + (e ? j : sh_path[j]), page = pos / static_cast<unsigned>(c.page_size);
              const long long pg = a.r.pages[b * a.r.pages_stride + page];
              sh_page[e][j] = pg;
              sh_slot[e][j] = static_cast<int>(pos - page * c.page_size);
              found = found && pg >= 0 && pg < c.pages;
            }
          }
        }
      }
      if (!__all_sync(full, found)) bad = RSSM_ERRBIT_PAGE;
    }
    if (bad) count = 0, next = -1;
    if (lane == 0) {
      sh_count = count;
      if (layer == 0) {
        a.accepted[b] = count;
        a.next[b] = next;
        if (bad) set_error(c.err, bad);
      }
    }
  }
  __syncthreads();
  const int count = sh_count;
  if (layer == 0 && threadIdx.x < a.r.T)
    a.path[static_cast<long long>(b) * a.r.T + threadIdx.x] = threadIdx.x < count ? sh_path[threadIdx.x] : -1;
  // the first tokens of a path often are where they belong
  int from = 0;
  while (from < count && sh_path[from] == from) ++from;
  if (!c.k || from == count) return;
  const int chunks = c.dim * c.esz / 16, columns = 2 * c.heads * chunks;
  for (int col = threadIdx.x; col < columns; col += kAcceptThreads) {
    const bool values = col >= c.heads * chunks;
    const int x = values ? col - c.heads * chunks : col, head = x / chunks;
    uint8_t* base = (values ? c.v + layer * c.v_layer : c.k + layer * c.k_layer) + static_cast<long long>(head) * c.page_size * c.dim * c.esz +
                    (x - head * chunks) * 16;
    const long long page = values ? c.v_page : c.k_page;
    const int row = c.dim * c.esz;
    for (int j0 = from; j0 < count; j0 += 8) {
      uint4 w[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (j0 + u < count) w[u] = *reinterpret_cast<const uint4*>(base + sh_page[0][j0 + u] * page + static_cast<long long>(sh_slot[0][j0 + u]) * row);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (j0 + u < count) *reinterpret_cast<uint4*>(base + sh_page[1][j0 + u] * page + static_cast<long long>(sh_slot[1][j0 + u]) * row) = w[u];
    }
  }
  if (c.ks) {
    for (int col = threadIdx.x; col < 2 * c.heads; col += kAcceptThreads) {
      const bool values = col >= c.heads;
      const int head = values ? col - c.heads : col;
      float* base = (values ? c.vs + layer * c.vs_layer : c.ks + layer * c.ks_layer) + static_cast<long long>(head) * c.page_size;
      const long long page = values ? c.vs_page : c.ks_page;
      for (int j0 = from; j0 < count; j0 += 8) {
        float w[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (j0 + u < count) w[u] = base[sh_page[0][j0 + u] * page + sh_slot[0][j0 + u]];
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (j0 + u < count) base[sh_page[1][j0 + u] * page + sh_slot[1][j0 + u]] = w[u];
      }
    }
  }
}

bool al(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// a warp a token, and a block for the bounds, if there are any
template <typename A>
cudaError_t launch(void (*kernel)(A), const A& a, cudaStream_t st) {
  const unsigned blocks = static_cast<unsigned>((a.r.tokens + kWarps - 1) / kWarps) + (a.r.cu ? 1u : 0u);
  return launch_pdl(kernel, dim3(blocks), dim3(kWarps * 32), 0, st, a);
}

template <int D>
cudaError_t append_dim(const AppendArgs& a, cudaStream_t st) {
  return launch(a.c.fmt == RSSM_BF16 ? append_kernel<D, RSSM_BF16> : a.c.fmt == RSSM_I8 ? append_kernel<D, RSSM_I8> : append_kernel<D, RSSM_E4M3>, a, st);
}
template <int D, int FMT>
cudaError_t read_format(const ReadArgs& a, int out, cudaStream_t st) {
  return launch(out == RSSM_F32 ? read_kernel<D, FMT, RSSM_F32> : out == RSSM_BF16 ? read_kernel<D, FMT, RSSM_BF16> : read_kernel<D, FMT, RSSM_F16>, a, st);
}
template <int D>
cudaError_t read_dim(const ReadArgs& a, int out, cudaStream_t st) {
  return a.c.fmt == RSSM_BF16 ? read_format<D, RSSM_BF16>(a, out, st)
         : a.c.fmt == RSSM_I8 ? read_format<D, RSSM_I8>(a, out, st)
                              : read_format<D, RSSM_E4M3>(a, out, st);
}

}  // namespace

// Strides from layer to layer and page to page must keep every row on 16 bytes.
rssm_status kv_view(const rssm_kv_cache* c, int layer, KvView* out) {
  if (!c) return RSSM_ERR_INVALID_ARGUMENT;
  if (c->num_pages < 1 || c->nlayers < 1 || c->nheads < 1 || c->page_size < 1) return RSSM_ERR_INVALID_ARGUMENT;
  if (c->format != RSSM_BF16 && c->format != RSSM_I8 && c->format != RSSM_E4M3) return RSSM_ERR_INVALID_ARGUMENT;
  if (layer < 0 || layer >= c->nlayers) return RSSM_ERR_INVALID_ARGUMENT;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return RSSM_ERR_UNSUPPORTED;
  if (c->page_size % 16 || c->page_size > 65536 || c->nheads > 1024) return RSSM_ERR_UNSUPPORTED;
  const bool q8 = c->format != RSSM_BF16;
  const int esz = q8 ? 1 : 2;
  if (!c->k || !c->v || !c->error_word || (q8 && (!c->k_scale || !c->v_scale))) return RSSM_ERR_INVALID_ARGUMENT;
  if (!al(c->k, 16) || !al(c->v, 16) || !al(c->error_word, 4) || (q8 && (!al(c->k_scale, 16) || !al(c->v_scale, 16))))
    return RSSM_ERR_INVALID_ARGUMENT;
  const long long page = static_cast<long long>(c->nheads) * c->page_size * c->head_dim;
  const long long scales = static_cast<long long>(c->nheads) * c->page_size;
  const auto strides = [&](int64_t p, int64_t l, long long dense, int size) {
    return p >= dense && (p * size) % 16 == 0 && (l * size) % 16 == 0 && (c->nlayers == 1 || l >= dense);
  };
  if (!strides(c->k_page_stride, c->k_layer_stride, page, esz) || !strides(c->v_page_stride, c->v_layer_stride, page, esz))
    return RSSM_ERR_INVALID_ARGUMENT;
  if (q8 && (!strides(c->k_scale_page_stride, c->k_scale_layer_stride, scales, 4) ||
             !strides(c->v_scale_page_stride, c->v_scale_layer_stride, scales, 4)))
    return RSSM_ERR_INVALID_ARGUMENT;
  KvView& v = *out;
  v.esz = esz;
  v.k_page = c->k_page_stride * esz;
  v.v_page = c->v_page_stride * esz;
  v.k_layer = c->k_layer_stride * esz;
  v.v_layer = c->v_layer_stride * esz;
  v.k = static_cast<uint8_t*>(c->k) + layer * v.k_layer;
  v.v = static_cast<uint8_t*>(c->v) + layer * v.v_layer;
  v.ks = v.vs = nullptr;
  v.ks_page = v.vs_page = v.ks_layer = v.vs_layer = 0;
  if (q8) {
    v.ks_page = c->k_scale_page_stride;
    v.vs_page = c->v_scale_page_stride;
    v.ks_layer = c->k_scale_layer_stride;
    v.vs_layer = c->v_scale_layer_stride;
    v.ks = c->k_scale + layer * v.ks_layer;
    v.vs = c->v_scale + layer * v.vs_layer;
  }
  v.pages = c->num_pages;
  v.layers = c->nlayers;
  v.heads = c->nheads;
  v.dim = c->head_dim;
  v.page_size = c->page_size;
  v.fmt = c->format;
  v.err = c->error_word;
  return RSSM_OK;
}

rssm_status kv_rows(const int32_t* pages, int64_t pages_stride, int32_t max_pages, const int32_t* lengths, const int32_t* cu, int32_t batch, int32_t T,
                    int64_t tokens, KvRows* out) {
  if (batch < 0 || T < 1 || tokens < 0 || max_pages < 0) return RSSM_ERR_INVALID_ARGUMENT;
  if (tokens > INT32_MAX || batch > (1 << 24)) return RSSM_ERR_UNSUPPORTED;
  if (batch > 0 && (!pages || pages_stride < max_pages)) return RSSM_ERR_INVALID_ARGUMENT;
  if (!al(pages, 4) || !al(lengths, 4) || !al(cu, 4)) return RSSM_ERR_INVALID_ARGUMENT;
  if (!cu && static_cast<int64_t>(batch) * T > tokens) return RSSM_ERR_INVALID_ARGUMENT;
  out->pages = pages;
  out->pages_stride = pages_stride;
  out->max_pages = max_pages;
  out->lengths = lengths;
  out->cu = cu;
  out->batch = batch;
  out->T = T;
  out->tokens = tokens;
  return RSSM_OK;
}

}  // namespace rssm

using namespace rssm;

namespace {
// token rows of a caller's tensor: heads of `dim` elements each
bool token_rows(const void* p, int64_t stride, int64_t tokens, int heads, int dim, int esz) {
  if (tokens > 0 && !p) return false;
  return al(p, 16) && stride >= static_cast<int64_t>(heads) * dim && (stride * esz) % 16 == 0;
}
}  // namespace

extern "C" rssm_status rssm_kv_append(const rssm_kv_cache* cache, int32_t layer, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                      const int32_t* pages, int64_t pages_stride, int32_t max_pages, const int32_t* lengths,
                                      const int32_t* cu_seqlens, int32_t batch, int32_t T, int64_t tokens, void* stream) {
  AppendArgs a;
  rssm_status st = kv_view(cache, layer, &a.c);
  if (st == RSSM_OK) st = kv_rows(pages, pages_stride, max_pages, lengths, cu_seqlens, batch, T, tokens, &a.r);
  if (st != RSSM_OK) return st;
  if (!token_rows(k, k_stride, tokens, a.c.heads, a.c.dim, 2) || !token_rows(v, v_stride, tokens, a.c.heads, a.c.dim, 2)) return RSSM_ERR_INVALID_ARGUMENT;
  if (batch > 0 && !lengths) return RSSM_ERR_INVALID_ARGUMENT;
  if (batch == 0 || tokens == 0) return RSSM_OK;
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a.c.dim == 64 ? append_dim<64>(a, s) : a.c.dim == 128 ? append_dim<128>(a, s) : append_dim<256>(a, s);
  return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}

extern "C" rssm_status rssm_kv_read(const rssm_kv_cache* cache, int32_t layer, const int32_t* pages, int64_t pages_stride, int32_t max_pages,
                                    const int32_t* starts, const int32_t* cu_seqlens, int32_t batch, int64_t tokens, int32_t out_dtype, void* k_out,
                                    int64_t k_stride, void* v_out, int64_t v_stride, void* stream) {
  ReadArgs a;
  rssm_status st = kv_view(cache, layer, &a.c);
  if (st == RSSM_OK && !cu_seqlens) st = RSSM_ERR_INVALID_ARGUMENT;
  if (st == RSSM_OK) st = kv_rows(pages, pages_stride, max_pages, starts, cu_seqlens, batch, INT32_MAX, tokens, &a.r);
  if (st != RSSM_OK) return st;
  if (out_dtype != RSSM_F32 && out_dtype != RSSM_BF16 && out_dtype != RSSM_F16) return RSSM_ERR_INVALID_ARGUMENT;
  const int esz = out_dtype == RSSM_F32 ? 4 : 2;
  if (!token_rows(k_out, k_stride, tokens, a.c.heads, a.c.dim, esz) || !token_rows(v_out, v_stride, tokens, a.c.heads, a.c.dim, esz))
    return RSSM_ERR_INVALID_ARGUMENT;
  if (batch == 0 || tokens == 0) return RSSM_OK;
  a.k = k_out;
  a.v = v_out;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a.c.dim == 64 ? read_dim<64>(a, out_dtype, s) : a.c.dim == 128 ? read_dim<128>(a, out_dtype, s) : read_dim<256>(a, out_dtype, s);
  return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}

extern "C" rssm_status rssm_tree_accept(const rssm_kv_cache* cache, const int32_t* pages, int64_t pages_stride, int32_t max_pages,
                                        const int32_t* lengths, const int32_t* tokens, const int32_t* parents, const int32_t* drawn,
                                        const int32_t* cu_seqlens, int32_t batch, int32_t T, int64_t ntok, int32_t* accepted, int32_t* next,
                                        int32_t* path, uint32_t* error_word, void* stream) {
  static const int32_t none = 0;
  AcceptArgs a;
  rssm_status st = RSSM_OK;
  if (cache) {
    st = kv_view(cache, 0, &a.c);
    if (st == RSSM_OK && batch > 0 && !lengths) st = RSSM_ERR_INVALID_ARGUMENT;
  } else {
    a.c = KvView{};
    a.c.layers = 1;
    a.c.err = error_word;
    pages = &none;  // not read
    pages_stride = max_pages = 0;
  }
  if (st == RSSM_OK) st = kv_rows(pages, pages_stride, max_pages, lengths, cu_seqlens, batch, T, ntok, &a.r);
  if (st != RSSM_OK) return st;
  if (T > kTreeT || a.c.layers > 65535) return RSSM_ERR_UNSUPPORTED;
  if (!al(tokens, 4) || !al(parents, 4) || !al(drawn, 4) || !al(accepted, 4) || !al(next, 4) || !al(path, 4) || !al(error_word, 4))
    return RSSM_ERR_INVALID_ARGUMENT;
  if ((ntok > 0 && (!tokens || !drawn)) || (batch > 0 && (!accepted || !next || !path))) return RSSM_ERR_INVALID_ARGUMENT;
  if (batch == 0) return RSSM_OK;
  a.tokens = tokens;
  a.parents = parents;
  a.drawn = drawn;
  a.accepted = accepted;
  a.next = next;
  a.path = path;
  const cudaError_t e = launch_pdl(accept_kernel, dim3(batch, a.c.layers), dim3(kAcceptThreads), 0, static_cast<cudaStream_t>(stream), a);
  return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}
