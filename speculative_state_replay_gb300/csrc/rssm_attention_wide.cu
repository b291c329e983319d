// rssm_attention_wide.cu -- attention of many queries of a head: trees of many
// tokens, prompts.
//
// With 256 queries over the same tokens the products are what bounds it, and they are
// tcgen05's: of two tiles of 128 queries, S = Q K' of 128 tokens into tensor memory,
// the softmax in registers, a query a thread, its weights P back into tensor memory in
// S's place, O += P V with O in tensor memory throughout.  Keys and values come in
// turn through a ring of shared-memory buffers, 8-bit codes as fp16, exactly.  The two
// tiles alternate: while one's scores are turned into weights the products of the other
// run.  The running maximum that weights are taken against follows the true one only
// when that is more than 2^4 times past it, so that O is rarely touched (weights are
// then at most 2^4: of a bf16 cache as bf16; fp16 ones are times 2^11).
//
// Work is cut as in rssm_attention.cu, or, where there are segments enough for all
// blocks, a segment a block with the longest first: a prompt's late queries see more.
#include "rssm_attention.cuh"
#include "rssm_tcgen05.cuh"

namespace rssm {
namespace {

constexpr int kQ = 128;                    // queries of a tile: the product's rows
constexpr int kTiles = 2;                  // tiles of a block
constexpr int kRows = kTiles * kQ;
constexpr int kTok = 128;                  // tokens of a step
constexpr int kSoftWarps = 4 * kTiles;     // a thread has a query
constexpr int kLoadWarps = 4;
constexpr int kThreads = (kSoftWarps + kLoadWarps + 1) * 32;
constexpr int kRing = 4;                   // buffers of a tile of keys or values
constexpr int kInfo = 3;                   // and what goes with them: K of step j + 3 waits until K of j + 1 is used, which
                                           // is after the weights of j
constexpr float kLazy = 4.0f;              // log2 of how far the true maximum may be past the one in use
constexpr float kShift = 11.0f;            // fp16 weights are times 2^11: 2^15 at most
constexpr int kTmem = 512;                 // columns: two of S, two of O

struct Wait {  // a wait that gives up is for all of the block
  volatile int* dead;
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*dead) return false;
    if (mbar_wait(bar, parity)) return true;
    *dead = 1;
    return false;
  }
};

template <int D_, int FMT_>
struct Shape {
  static constexpr int D = D_, FMT = FMT_;
  static constexpr bool Q8 = FMT != RSSM_BF16;
  static constexpr int RB = D * (Q8 ? 1 : 2);     // bytes of a cached head
  static constexpr int NC = RB / 16;              // and its 16-byte chunks
  static constexpr int kTile = kTok * D * 2;      // bytes of a tile as an operand: per 64 dimensions, rows of 128 bytes
  static constexpr int kRingAt = kTiles * kTile;  // queries first
  static constexpr int kInfoAt = kRingAt + kRing * kTile;
  static constexpr int kBarsAt = kInfoAt + (Q8 ? kInfo * 3 * kTok * 4 : 0);
  static constexpr int kSmem = kBarsAt + 256 + 1024;  // and room to start on 1024 bytes
};

__device__ __forceinline__ uint32_t sw(int r, int ch) { return static_cast<uint32_t>(r * 128 + ((ch ^ (r & 7)) << 4)); }

__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {  // first operand in tensor memory
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}
#define R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define S8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
__device__ __forceinline__ void tc_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,"
      "%27,%28,%29,%30,%31}, [%32];"
      : R8(r, 0), R8(r, 8), R8(r, 16), R8(r, 24)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,"
      "%26,%27,%28,%29,%30,%31};" ::S8(r, 0),
      S8(r, 8), S8(r, 16), S8(r, 24), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::S8(r, 0), S8(r, 8), "r"(addr)
               : "memory");
}
#undef R8
#undef S8
// after tc_wait_ld: uses of r stay behind it
__device__ __forceinline__ void landed(uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}

template <typename S>
__global__ void __launch_bounds__(kThreads, 1) wide_kernel(const AttnArgs a) {
  constexpr int D = S::D, RB = S::RB, NC = S::NC;
  constexpr bool Q8 = S::Q8;
  extern __shared__ uint8_t raw[];
  uint8_t* const sm = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  __shared__ uint32_t tmem_base;
  __shared__ volatile int dead;
  __shared__ int sh_bad, sh_odd;
  __shared__ unsigned long long sh_mask[kTreeT];
  __shared__ float sh_back[kRows];
  __shared__ unsigned sh_valid[kInfo];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const unsigned full = 0xffffffffu;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(sm + S::kBarsAt);
  uint64_t *const b_full = bars, *const b_empty = bars + kRing, *const b_s = bars + 2 * kRing, *const b_p = b_s + kTiles, *const b_o = b_p + kTiles,
           *const b_info = b_o + kTiles;
  const uint32_t base = smem_addr(sm);
  if (warp == kSoftWarps + kLoadWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_base)), "n"(kTmem) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    dead = 0;
    for (int i = 0; i < kRing; ++i) {
      mbar_init(b_full + i, kLoadWarps * 32);
      mbar_init(b_empty + i, 1);
    }
    for (int i = 0; i < kTiles; ++i) {
      mbar_init(b_s + i, 1);
      mbar_init(b_p + i, 4);
      mbar_init(b_o + i, 1);
    }
    for (int i = 0; i < kInfo; ++i) mbar_init(b_info + i, kLoadWarps * 32);
    fence_barrier_init();
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tm = tmem_base;
  const Wait wait{&dead};
  pdl_wait();
  pdl_trigger();

  Line line;
  if (a.whole) {
    // segments of the longest prompts' last queries first; a row's tokens are not known here, so its place is by T
    const int per = a.r.batch * a.c.heads;
    const int mt = static_cast<int>(gridDim.x / per) - 1 - static_cast<int>(blockIdx.x / per);
    const int x = static_cast<int>(blockIdx.x % per);
    line.b = x / a.c.heads;
    const RowWork w = row_work<kRows, kTok>(a, line.b);
    if (blockIdx.x == 0) {
      for (int i = tid; i < a.r.batch; i += kThreads) {
        const RowWork y = row_work<kRows, kTok>(a, i);
        if (y.s.count < 0) set_error(a.c.err, RSSM_ERRBIT_SEQLEN);
        if (y.len == -2) set_error(a.c.err, RSSM_ERRBIT_PAGE);
      }
    }
    line.base = 0;
    line.share = 1;
    line.lo = mt < w.mtiles ? static_cast<long long>(mt * a.c.heads + x % a.c.heads) * w.tiles : 0;
    line.hi = mt < w.mtiles ? line.lo + w.tiles : 0;
  } else {
    line = cut_line<kRows, kTok, kThreads>(a);
  }
  int b = line.b;
  long long rbase = line.base;
  int items = 0, steps = 0, used[kTiles] = {0, 0}, done[kTiles] = {0, 0};  // how often the ring, and what goes with it, the scores, the sums came round
  bool ok = true;

#pragma unroll 1
  for (long long u = line.lo; u < line.hi;) {
    const RowWork w = row_work<kRows, kTok>(a, b);
    const long long units = static_cast<long long>(w.tiles) * w.mtiles * a.c.heads;
    if (u >= rbase + units) {
      rbase += units;
      ++b;
      continue;
    }
    const long long at = u - rbase;
    const int seg = static_cast<int>(at / w.tiles), t0 = static_cast<int>(at - static_cast<long long>(seg) * w.tiles);
    const int t1 = static_cast<int>(min(static_cast<long long>(w.tiles), t0 + (line.hi - u)));
    const int mtile = seg / a.c.heads, head = seg - mtile * a.c.heads;
    const long long seg0 = u - t0;
    u += t1 - t0;
    const int row0 = mtile * kRows, rows = min(kRows, w.s.count * a.group - row0);
    const int nq = rows > kQ ? 2 : 1;
    __syncthreads();  // the last piece's shared memory is free
    if (tid == 0) sh_bad = sh_odd = 0;
    const bool flip = a.scale2 < 0.0f;  // the maximum is taken before the scale
    const float scale2 = fabsf(a.scale2);
    {
      constexpr int G = D / 8, AT = 32 / G;  // lanes of a row, rows of a warp
#pragma unroll 1
      for (int r0 = warp * AT; r0 < nq * kQ; r0 += kThreads / 32 * AT) {
        const int r = r0 + lane / G, part = lane % G;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows) {
          const int t = (row0 + r) / a.group, h = head * a.group + (row0 + r) - t * a.group;
          x = *reinterpret_cast<const uint4*>(a.q + (w.s.first + t) * a.q_stride + static_cast<long long>(h) * D + part * 8);
          if (flip) x = make_uint4(x.x ^ 0x80008000u, x.y ^ 0x80008000u, x.z ^ 0x80008000u, x.w ^ 0x80008000u);
        }
        if constexpr (Q8) {
          float back;
          x = query_f16<G>(x, back);
          if (part == 0) sh_back[r] = scale2 * back;
        }
        *reinterpret_cast<uint4*>(sm + (r / kQ) * S::kTile + (part / 8) * 16384 + sw(r % kQ, part % 8)) = x;
      }
    }
    __syncthreads();
    if (a.parents && warp == 0 && w.len >= 0) {
      unsigned long long mask[2];
      const bool fine = tree_masks(a.parents + w.s.first, w.s.count, lane, mask);
      sh_mask[lane] = mask[0];
      sh_mask[lane + 32] = mask[1];
      if (!fine && lane == 0) {
        sh_bad = 1;
        set_error(a.c.err, RSSM_ERRBIT_TREE);
      }
    }
    fence_async();
    __syncthreads();
    const int last = (row0 + rows - 1) / a.group;
    const long long end = w.len < 0 || sh_bad ? 0 : static_cast<long long>(w.len) + (a.parents ? w.s.count : last + 1);
    // from here on there are tokens that not every query of the tile sees, or none
    const long long some = static_cast<long long>(w.len) + (a.parents ? 0 : row0 / a.group + 1);
    const int stop = static_cast<int>(min(static_cast<long long>(t1), (end + kTok - 1) / kTok));
    const int nt = max(0, stop - t0);
    const int* table = a.r.pages + b * a.r.pages_stride;
    const uint8_t* kbase = a.c.k + static_cast<long long>(head) * a.c.page_size * RB;
    const uint8_t* vbase = a.c.v + static_cast<long long>(head) * a.c.page_size * RB;

    float ref = -INFINITY, sum = 0.0f;
    if (warp < kSoftWarps) {
      // ---- scores into weights
      const int tile = warp >> 2;
      if (tile < nq) {
        const int r = tid;  // its query
        const int t = (row0 + min(r, rows - 1)) / a.group;
        const unsigned long long path = a.parents ? sh_mask[t & 63] : 0ull;
        const float back = Q8 ? sh_back[r] : scale2;
        const uint32_t s_at = tm + tile * kTok + ((warp & 3) << 21), o_at = tm + kTiles * kTok + tile * D + ((warp & 3) << 21);
#pragma unroll 1
        for (int j = 0; j < nt; ++j) {
          const int slot = (steps + j) % kInfo;
          ok = ok && wait(b_info + slot, ((steps + j) / kInfo) & 1);
          ok = __all_sync(full, ok && wait(b_s + tile, (used[tile] + j) & 1)) != 0;
          if (!ok) break;
          tc_after();
          const long long pos = static_cast<long long>(t0 + j) * kTok;
          const unsigned valid = sh_valid[slot];
          const bool edge = pos + kTok > some || valid != 0xffu;
          const float* ks = reinterpret_cast<const float*>(sm + S::kInfoAt) + slot * 3 * kTok;
          // scores in units of log2 (8-bit: with their values' scales)
          auto units_of = [&](uint32_t (&x)[32], int c) {
            if constexpr (Q8) {
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const float4 k4 = *reinterpret_cast<const float4*>(ks + 32 * c + i), l4 = *reinterpret_cast<const float4*>(ks + kTok + 32 * c + i);
                x[i] = __float_as_uint(__uint_as_float(x[i]) * back * k4.x + l4.x);
                x[i + 1] = __float_as_uint(__uint_as_float(x[i + 1]) * back * k4.y + l4.y);
                x[i + 2] = __float_as_uint(__uint_as_float(x[i + 2]) * back * k4.z + l4.z);
                x[i + 3] = __float_as_uint(__uint_as_float(x[i + 3]) * back * k4.w + l4.w);
              }
            }
          };
          float top = -INFINITY;
          if (edge) {
#pragma unroll 1
            for (int c = 0; c < kTok / 32; ++c) {
              uint32_t x[32];
              tc_ld32(x, s_at + 32 * c);
              tc_wait_ld();
              landed(x);
              units_of(x, c);
              // which of the 32 this query sees
              const long long j0 = pos + 32 * c - w.len;
              uint32_t see;
              if (a.parents) {
                see = j0 <= -32 ? full : j0 < 0 ? static_cast<uint32_t>(path << -j0) | ((1u << -j0) - 1u) : j0 < 64 ? static_cast<uint32_t>(path >> j0) : 0u;
              } else {
                const long long n = t - j0;  // the last one's place
                see = n >= 31 ? full : n < 0 ? 0u : (2u << n) - 1u;
              }
              see &= (valid >> (2 * c) & 1u ? 0xffffu : 0u) | (valid >> (2 * c + 1) & 1u ? 0xffff0000u : 0u);
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float y = Q8 ? __uint_as_float(x[i]) : __uint_as_float(x[i]) * back;
                x[i] = __float_as_uint(see >> i & 1u ? y : -INFINITY);
                top = fmaxf(top, __uint_as_float(x[i]));
              }
              tc_st32(s_at + 32 * c, x);
            }
            tc_wait_st();
          } else {
#pragma unroll
            for (int c = 0; c < kTok / 32; ++c) {
              uint32_t x[32];
              tc_ld32(x, s_at + 32 * c);
              tc_wait_ld();
              landed(x);
              units_of(x, c);
#pragma unroll
              for (int i = 0; i < 32; ++i) top = fmaxf(top, __uint_as_float(x[i]));
            }
            if constexpr (!Q8) top *= back;
          }
          // the maximum in use follows where it has to; the products before this step's are done (its scores came after them)
          if (__any_sync(full, top > ref + kLazy)) {
            const float now = fmaxf(ref, top);
            const float f = now == -INFINITY ? 1.0f : exp2_fast(ref - now);
            ref = now;
            sum *= f;
            if (j > 0) {
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t x[32];
                tc_ld32(x, o_at + 32 * c);
                tc_wait_ld();
                landed(x);
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
                tc_st32(o_at + 32 * c, x);
              }
            }
          }
          const float off = (ref == -INFINITY ? 0.0f : ref) - (Q8 ? kShift : 0.0f);
          float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          auto weights = [&](auto is_edge) {
            constexpr bool E = decltype(is_edge)::value;
#pragma unroll
            for (int c = 0; c < kTok / 32; ++c) {
              uint32_t x[32], p[16];
              tc_ld32(x, s_at + 32 * c);
              tc_wait_ld();
              landed(x);
              if constexpr (!E) units_of(x, c);
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float y = __uint_as_float(x[i]);
                x[i] = __float_as_uint(exp2_fast(Q8 || E ? y - off : y * back - off));
              }
              if constexpr (Q8) {
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                  const float4 i4 = *reinterpret_cast<const float4*>(ks + 2 * kTok + 32 * c + i);
                  const float v4[4] = {i4.x, i4.y, i4.z, i4.w};
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const float y = __uint_as_float(x[i + e]);
                    if (!E || y > 0.0f) s4[e] += y * v4[e];
                  }
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) p[i] = pack_f16(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) s4[i & 3] += __uint_as_float(x[i]);
#pragma unroll
                for (int i = 0; i < 16; ++i) p[i] = pack_bf16(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
              }
              tc_st16(s_at + 16 * c, p);
            }
          };
          if (edge) weights(std::true_type{});
          else weights(std::false_type{});
          sum += (s4[0] + s4[1]) + (s4[2] + s4[3]);
          tc_wait_st();
          tc_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(b_p + tile);
        }
        if (nt > 0) {
          ok = __all_sync(full, ok && wait(b_o + tile, done[tile] & 1)) != 0;
          tc_after();
        }
      }
    } else if (warp < kSoftWarps + kLoadWarps) {
      // ---- keys and values, in turn
      const int lt = tid - kSoftWarps * 32;
      int pending = -1;  // an item whose copies are on their way
      bool pending_odd = false;
      // this thread's copies have landed: its values are looked at where not every query sees them, then the buffer is announced
      auto announce = [&]() {
        if (pending < 0) return;
        const int buf = pending % kRing;
        if constexpr (!Q8) {
          if (pending_odd) {
            uint8_t* p = sm + S::kRingAt + buf * S::kTile;
#pragma unroll 4
            for (int x = 0; x < NC; ++x) {
              const int i = lt + 128 * x, r = i / NC, ch = i % NC;
              uint4* q = reinterpret_cast<uint4*>(p + (ch / 8) * 16384 + sw(r, ch % 8));
              uint4 y = *q;
              if (take_out_odd(y)) {
                *q = y;
                sh_odd = 1;
              }
            }
          }
        }
        fence_async();
        mbar_arrive(b_full + buf);
        pending = -1;
      };
      auto page_id = [&](int j) {
        const long long p = static_cast<long long>(t0 + j) * kTok + 16 * lane;
        return lane < 8 && j < nt && p < end ? table[static_cast<unsigned>(p) / static_cast<unsigned>(a.c.page_size)] : -1;
      };
      int next_id = page_id(0);
#pragma unroll 1
      for (int j = 0; j < nt; ++j) {
        const long long pos = static_cast<long long>(t0 + j) * kTok;
        const long long mine = pos + 16 * lane;
        const int id = next_id;
        next_id = page_id(j + 1);
        const bool have = lane < 8 && mine < end && id >= 0 && id < a.c.pages;
        if (lane < 8 && mine < end && !have) set_error(a.c.err, RSSM_ERRBIT_PAGE);
        const unsigned missing = __ballot_sync(full, lane < 8 && mine < end && !have) & 0xffu;
        const unsigned place = static_cast<unsigned>(mine) % static_cast<unsigned>(a.c.page_size);
        const long long koff = have ? id * a.c.k_page + static_cast<long long>(place) * RB : 0;
        const long long voff = have ? id * a.c.v_page + static_cast<long long>(place) * RB : 0;
        const int live = have ? static_cast<int>(min(16ll, end - mine)) : 0;
        const int slot = (steps + j) % kInfo;
        float ksv = 0.0f, vsv = 0.0f;
        if constexpr (Q8) {  // a token a thread
          const int sl = lt / 16;
          const long long row = static_cast<long long>(head) * a.c.page_size + __shfl_sync(full, place, sl) + (lt & 15);
          const int pg = __shfl_sync(full, have ? id : 0, sl);
          if ((lt & 15) < __shfl_sync(full, live, sl)) {
            ksv = a.c.ks[pg * a.c.ks_page + row];
            vsv = a.c.vs[pg * a.c.vs_page + row];
          }
        }
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          const int item = items + 2 * j + kv, buf = item % kRing;
          const uint8_t* src = kv ? vbase : kbase;
          const long long off = kv ? voff : koff;
          uint4 codes[Q8 ? NC : 1];
          if constexpr (Q8) {  // asked for before the buffer is free
#pragma unroll
            for (int x = 0; x < NC; ++x) {
              const int i = lt + 128 * x, r = i / NC, ch = i % NC, sl = r / 16;
              const long long o = __shfl_sync(full, off, sl);
              codes[x] = r % 16 < __shfl_sync(full, live, sl) ? __ldcg(reinterpret_cast<const uint4*>(src + o + (r % 16) * RB + ch * 16)) : make_uint4(0u, 0u, 0u, 0u);
            }
          }
          if (item >= kRing && !mbar_try_wait(b_empty + buf, (item / kRing - 1) & 1)) {
            if constexpr (!Q8) {
              copy_wait<0>();
              announce();
            }
            ok = ok && wait(b_empty + buf, (item / kRing - 1) & 1);
          }
          ok = __all_sync(full, ok) != 0;
          if (!ok) break;
          uint8_t* to = sm + S::kRingAt + buf * S::kTile;
          if (kv == 0) {  // what goes with the step: the place is free since K of two steps before is
            if (lt == 0) sh_valid[slot] = 0xffu & ~missing;
            if constexpr (Q8) {
              float* info = reinterpret_cast<float*>(sm + S::kInfoAt) + slot * 3 * kTok;
              vsv = vsv < 7.7037197775489434e-34f ? 7.7037197775489434e-34f : vsv;  // 2^-110: a scale of 0 stands for zeros all the same
              info[lt] = ksv;
              info[kTok + lt] = __log2f(vsv);
              info[2 * kTok + lt] = __frcp_rn(vsv) * kShift8;
            }
            mbar_arrive(b_info + slot);
          }
          if constexpr (Q8) {
#pragma unroll
            for (int x = 0; x < NC; ++x) {
              const int i = lt + 128 * x, r = i / NC, ch = i % NC;
              const uint32_t c4[4] = {codes[x].x, codes[x].y, codes[x].z, codes[x].w};
              uint32_t h[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t y = S::FMT == RSSM_I8 ? c4[e] ^ 0x80808080u : c4[e];
                h[2 * e] = codes_f16<S::FMT>(y, 0x4140u, 0x4410u);
                h[2 * e + 1] = codes_f16<S::FMT>(y, 0x4342u, 0x4432u);
              }
              uint8_t* p = to + (ch / 4) * 16384;
              *reinterpret_cast<uint4*>(p + sw(r, (2 * ch) % 8)) = make_uint4(h[0], h[1], h[2], h[3]);
              *reinterpret_cast<uint4*>(p + sw(r, (2 * ch + 1) % 8)) = make_uint4(h[4], h[5], h[6], h[7]);
            }
            pending = item;
            announce();
          } else {
#pragma unroll
            for (int x = 0; x < NC; ++x) {
              const int i = lt + 128 * x, r = i / NC, ch = i % NC, sl = r / 16;
              const long long o = __shfl_sync(full, off, sl);
              copy16(base + S::kRingAt + buf * S::kTile + (ch / 8) * 16384 + sw(r, ch % 8), src + o + (r % 16) * RB + ch * 16,
                     r % 16 < __shfl_sync(full, live, sl));
            }
            copy_commit();
            if (pending >= 0) {
              copy_wait<1>();
              announce();
            }
            pending = item;
            pending_odd = kv && pos + kTok > some;
          }
        }
        if (!ok) break;
      }
      if constexpr (!Q8) {
        copy_wait<0>();
        announce();
      }
    } else if (lane == 0) {
      // ---- products
      constexpr uint32_t kind = Q8 ? (1u << 7) | (1u << 10) : 0u;  // fp16 operands: without bf16's bits
      constexpr uint32_t i_s = instruction(kTok, false, false) & ~kind, i_o = instruction(D, false, true) & ~kind;
      auto scores = [&](int tile, int buf) {
        const uint64_t q = operand(base + tile * S::kTile, 16, 1024, kSw128), k = operand(base + S::kRingAt + buf * S::kTile, 16, 1024, kSw128);
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const uint64_t o = (x / 4) * (16384 / 16) + (x % 4) * 2;
          tc_mma(tm + tile * kTok, q + o, k + o, i_s, x > 0);
        }
        tc_commit(b_s + tile);
      };
      if (nt > 0) {
        const int buf = items % kRing;
        ok = ok && wait(b_full + buf, (items / kRing) & 1);
        if (ok) {
          tc_after();
          for (int x = 0; x < nq; ++x) scores(x, buf);
          tc_commit(b_empty + buf);
        }
      }
#pragma unroll 1
      for (int j = 0; ok && j < nt; ++j) {
        const int iv = items + 2 * j + 1, bv = iv % kRing, ik = iv + 1, bk = ik % kRing;
        const bool more = j + 1 < nt;
        ok = ok && wait(b_full + bv, (iv / kRing) & 1);
        if (more) ok = ok && wait(b_full + bk, (ik / kRing) & 1);
        for (int x = 0; x < nq; ++x) {
          ok = ok && wait(b_p + x, (used[x] + j) & 1);
          if (!ok) break;
          tc_after();
          const uint64_t v = operand(base + S::kRingAt + bv * S::kTile, 16384, 1024, kSw128);
#pragma unroll
          for (int y = 0; y < kTok / 16; ++y) tc_mma_ts(tm + kTiles * kTok + x * D, tm + x * kTok + 8 * y, v + y * (2048 / 16), i_o, j > 0 || y > 0);
          if (more) scores(x, bk);
          else tc_commit(b_o + x);
        }
        if (ok) {
          tc_commit(b_empty + bv);
          if (more) tc_commit(b_empty + bk);
        }
      }
    }
    ok = __syncthreads_and(ok);
    if (!ok) break;
    items += 2 * nt;
    steps += nt;
#pragma unroll
    for (int x = 0; x < kTiles; ++x)
      if (x < nq) used[x] += nt, done[x] += nt > 0;

    // ---- the queries' sums
    const bool whole = t0 == 0 && t1 == w.tiles;
    constexpr float kUnit = Q8 ? kShift8 : 1.0f;
    if (warp < kSoftWarps && (warp >> 2) < nq) {
      const int r = tid, tile = warp >> 2, t = (row0 + min(r, rows - 1)) / a.group;
      float* const left = piece_place<kRows, D>(a, blockIdx.x, t0 == 0);
      const float inv = sum == 0.0f ? 0.0f : kUnit / sum;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t x[32];
        if (nt > 0) {
          tc_ld32(x, tm + kTiles * kTok + tile * D + ((warp & 3) << 21) + 32 * c);
          tc_wait_ld();
          landed(x);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = 0u;
        }
        if (r < rows) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            float y0[4] = {__uint_as_float(x[i]), __uint_as_float(x[i + 1]), __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])};
            float y1[4] = {__uint_as_float(x[i + 4]), __uint_as_float(x[i + 5]), __uint_as_float(x[i + 6]), __uint_as_float(x[i + 7])};
            if constexpr (!Q8) {
              if (sh_odd) {
                const long long from = max(static_cast<long long>(t0) * kTok, some / kTok * kTok), to = min(static_cast<long long>(t1) * kTok, end);
                const unsigned long long path = a.parents ? sh_mask[t & 63] : 0ull;
                add_odd(a, w, table, vbase, RB, from, to, t, path, 32 * c + i, y0);
                add_odd(a, w, table, vbase, RB, from, to, t, path, 32 * c + i + 4, y1);
              }
            }
            if (whole) {
              const int h = head * a.group + (row0 + r) - t * a.group;
              *reinterpret_cast<uint4*>(a.out + (w.s.first + t) * a.out_stride + static_cast<long long>(h) * D + 32 * c + i) =
                  make_uint4(pack_bf16(y0[0] * inv, y0[1] * inv), pack_bf16(y0[2] * inv, y0[3] * inv), pack_bf16(y1[0] * inv, y1[1] * inv),
                             pack_bf16(y1[2] * inv, y1[3] * inv));
            } else {
              __stcg(reinterpret_cast<float4*>(left + r * D + 32 * c + i), make_float4(y0[0], y0[1], y0[2], y0[3]));
              __stcg(reinterpret_cast<float4*>(left + r * D + 32 * c + i + 4), make_float4(y1[0], y1[1], y1[2], y1[3]));
            }
          }
        }
        __syncwarp();  // the next load is the whole warp's
      }
      if (!whole && r < rows) {
        __stcg(left + kRows * D + r, ref);
        __stcg(left + kRows * D + kRows + r, sum);
      }
      tc_before();
    }
    if (!whole) join_pieces<kRows, D, kThreads>(a, w, head, row0, rows, seg0, line.share, kUnit);
  }
  // a wait that gave up: what was started ends before the memory is given back
  if (!ok && warp == kSoftWarps + kLoadWarps && lane == 0) {
    mbar_init(b_info, 1);
    fence_barrier_init();
    tc_commit(b_info);
    mbar_wait(b_info, 0);
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == kSoftWarps + kLoadWarps) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "n"(kTmem) : "memory");
  if (tid == 0 && dead) set_error(a.c.err, RSSM_ERRBIT_TIMEOUT);
}

template <int D, int FMT>
cudaError_t launch(const AttnArgs& a, int grid, cudaStream_t st) {
  using S = Shape<D, FMT>;
  static bool ready[64] = {};  // per device: the attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(wide_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev] = true;
  }
  return launch_pdl(wide_kernel<S>, dim3(grid), dim3(kThreads), S::kSmem, st, a);
}
template <int D>
cudaError_t launch_format(const AttnArgs& a, int grid, cudaStream_t st) {
  return a.c.fmt == RSSM_BF16 ? launch<D, RSSM_BF16>(a, grid, st) : a.c.fmt == RSSM_I8 ? launch<D, RSSM_I8>(a, grid, st) : launch<D, RSSM_E4M3>(a, grid, st);
}

}  // namespace

// More than 32 queries a head go through here; a head of 256 dimensions leaves no room for two tiles.
bool wide_takes(const KvView& c, int64_t queries) { return c.dim <= 128 && queries > 32; }

size_t wide_scratch(const KvView& c, int sms) { return c.dim <= 128 ? static_cast<size_t>(sms) * 2 * kRows * (c.dim + 2) * sizeof(float) : 0; }

cudaError_t run_wide(const AttnArgs& args, int sms, cudaStream_t st) {
  AttnArgs a = args;
  const int64_t mtiles = (static_cast<int64_t>(a.r.T) * a.group + kRows - 1) / kRows, segments = mtiles * a.r.batch * a.c.heads;
  a.whole = segments >= 2 * sms && segments < (1ll << 30);
  const int grid = a.whole ? static_cast<int>(segments) : sms;
  return a.c.dim == 64 ? launch_format<64>(a, grid, st) : launch_format<128>(a, grid, st);
}

}  // namespace rssm
