// rssm_attention_wide.cu -- attention of many queries of a head: trees of many
// tokens, prompts.
//
// With 256 queries over the same tokens the products are what bounds it, and they are
// tcgen05's: of two tiles of 128 queries, S = Q K' of 128 tokens into tensor memory,
// the softmax in registers, its weights P back into tensor memory in S's place (bf16: a query
// for two threads; 8-bit: four queries for eight, each with a quarter of a half's tokens, as
// their scales are read along), O += P V with O in tensor memory throughout.  Keys and values come in
// turn through a ring of shared-memory buffers, 8-bit codes as fp16, exactly.  The two
// tiles alternate: while one's scores are turned into weights the products of the other
// run.  Where a segment has 128 queries or fewer, both take the same ones and every
// other step of tokens, and are added at the end.  The running maximum that weights are
// taken against follows the true one only when that is more than 2^4 times past it, so
// that O is rarely touched (weights are then at most 2^4: of a bf16 cache as bf16; fp16
// ones are times 2^11).
//
// Work is cut as in rssm_attention.cu, or, where there are segments enough for all
// blocks, a segment a block with the longest first: a prompt's late queries see more.
//
// Measured: the second 4096 tokens of a prompt (32 heads over 8, of 128, bf16) 390 us, 1.06
// PFLOP/s.  A step of 256 queries over 128 tokens takes 4250 cycles, of which the tensor
// cores are at work 2050; issuing the products takes 2600 and a tile's softmax 2500, so the
// two tiles' softmax is what the products wait for.  16 trees of up to 48 tokens over 5000
// int8 ones each: 145 us; a step of 256 queries takes 5000 cycles, the two warps that
// convert codes taking 1900 for a tile of keys or values.
#include "rssm_attention.cuh"
#include "rssm_readout.cuh"
#include "rssm_tcgen05.cuh"

namespace rssm {
namespace {

constexpr int kQ = 128;                 // queries of a tile: the product's rows
constexpr int kTiles = 2;               // tiles of a block
constexpr int kRows = kTiles * kQ;
constexpr int kTok = 128;               // tokens of a step
constexpr int kInfo = 5;                // places of what goes with a step of tokens: K of step j + 5 waits for a buffer that is
                                        // free once the scores of j + 2 are made, which is after the weights of j
constexpr float kLazy = 4.0f;           // log2 of how far the true maximum may be past the one in use
constexpr float kShift = 11.0f;         // fp16 weights are times 2^11: 2^15 at most
constexpr int kTmem = 512;              // columns: two of S, two of O
constexpr int kPairs = 2;               // named barriers from here on: of the two warps with the same queries

struct Wait {  // a wait that gives up is for all of the block
  volatile int* dead;
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
    if (mbar_try_wait(bar, parity)) return true;
    for (uint32_t i = 0; i < kWaitTries; ++i) {
      if (mbar_try_wait_for(bar, parity, 1000000u)) return true;
      if (*dead) return false;
    }
    *dead = 1;
    return false;
  }
};

template <int D_, int FMT_>
struct Shape {
  static constexpr int D = D_, FMT = FMT_;
  static constexpr bool Q8 = FMT != RSSM_BF16;
  static constexpr int kParts = 2;                // threads of a query, each with a part of a step's tokens
  static constexpr int kSoftWarps = 4 * kTiles * kParts, kSoft = kSoftWarps * 32;
  static constexpr int kLoadWarps = 3;            // the first copies; 8-bit: the others convert, bf16: all look at tiles that not every query sees
  static constexpr int kWorkWarps = Q8 ? kLoadWarps - 1 : kLoadWarps, kWorkers = kWorkWarps * 32;
  static constexpr int kThreads = kSoft + kLoadWarps * 32 + 32;
  static constexpr int RB = D * (Q8 ? 1 : 2);     // bytes of a cached head
  static constexpr int NC = RB / 16;              // and its 16-byte chunks
  static constexpr int kTile = kTok * D * 2;      // bytes of a tile as an operand: per 64 dimensions, rows of 128 bytes
  static constexpr int kRing = Q8 ? 3 : 4;        // buffers of a tile of keys or values; 8-bit: as many of tiles as they come
  static constexpr int kRingAt = kTiles * kTile;  // queries first
  static constexpr int kRawAt = kRingAt + kRing * kTile;
  static constexpr int kInfoAt = kRawAt + (Q8 ? kRing * kTok * RB : 0);
  static constexpr int kBarsAt = kInfoAt + (Q8 ? kInfo * 3 * kTok * 4 : 0);
  static constexpr int kSmem = kBarsAt + 256 + 1024;  // and room to start on 1024 bytes
  static_assert(kSmem <= 226 * 1024 && kRing * kTile >= kQ * D * 4, "fits, and a tile's sums fit the ring");
};

struct Slice {  // 16 tokens of a step
  long long off[2];       // bytes from the head's first key (value)
  int page, place, live;  // its page, where it begins there, and how many of the tokens there are
};

__device__ __forceinline__ uint32_t sw(int r, int ch) { return static_cast<uint32_t>(r * 128 + ((ch ^ (r & 7)) << 4)); }

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst), "l"(map),
               "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
               : "memory");
}
// Products and their commits by one lane of a warp that runs as a whole: the descriptors are the warp's, and no branch
// stands between two products
__device__ __forceinline__ void mma_ss(bool mine, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "setp.ne.u32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "r"(static_cast<uint32_t>(mine))
      : "memory");
}
__device__ __forceinline__ void mma_ts(bool mine, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {  // first operand in tensor memory
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "setp.ne.u32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "r"(static_cast<uint32_t>(mine))
      : "memory");
}
__device__ __forceinline__ void commit(bool mine, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.u32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)),
      "r"(static_cast<uint32_t>(mine))
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
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::S8(r, 0), S8(r, 8), "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tc_stw8(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::S8(r, 0), "r"(addr) : "memory");
}
// 16 lanes by 64 columns as a fragment: registers 4 n, 4 n + 1 are columns 8 n + 2 (lane % 4), + 1 of lane / 4, the next two those
// of lane / 4 + 8
__device__ __forceinline__ void tc_ld64(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,"
      "%27,%28,%29,%30,%31}, [%32];"
      : R8(r, 0), R8(r, 8), R8(r, 16), R8(r, 24)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_ld16(uint32_t (&r)[8], uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];" : R8(r, 0) : "r"(addr) : "memory");
}
__device__ __forceinline__ void tc_st16f(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::S8(r, 0), "r"(addr) : "memory");
}
// and 32 columns: register 2 n is column 4 n + lane % 4 of lane / 4, the next that of lane / 4 + 8
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x8.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::S8(r, 0), S8(r, 8), "r"(addr)
               : "memory");
}
#undef R8
#undef S8
// what was asked for has landed; uses of r stay behind
__device__ __forceinline__ void landed(uint32_t (&r)[32]) {
  tc_wait_ld();
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}

// Two fp32 values in one 64-bit register pair
using pair = unsigned long long;
__device__ __forceinline__ pair pack2(float lo, float hi) {
  pair d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpack2(pair d, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(d)); }
__device__ __forceinline__ void add2(pair& d, pair a) { asm("add.rn.f32x2 %0, %0, %1;" : "+l"(d) : "l"(a)); }
__device__ __forceinline__ void fma2(pair& d, pair a, pair b) { asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b)); }
__device__ __forceinline__ pair fma2v(pair a, pair b, pair c) {
  pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
// two scores times the query's factor and their keys' scales, and the logarithms of their values' scales
__device__ __forceinline__ void scaled(uint32_t& x0, uint32_t& x1, pair back, pair keys, pair values) {
  pair y = pack2(__uint_as_float(x0), __uint_as_float(x1));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(y) : "l"(back));
  y = fma2v(y, keys, values);
  float y0, y1;
  unpack2(y, y0, y1);
  x0 = __float_as_uint(y0);
  x1 = __float_as_uint(y1);
}

template <int N>
__device__ __forceinline__ void soft_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}

// A block's part of a segment: what its warps have to know, in shared memory, so that their loops have the registers.
struct Piece {
  long long first;                   // the row's first new token
  int row, len, count, head;         // the row, its committed and new tokens, the head
  int row0, rows;                    // the tile's queries
  int t0, nt, t1;                    // its steps of tokens: from t0 on nt that any query sees, of t1 - t0
  int end, some;                     // the last token seen by any of its queries; from `some` on not every query sees all
  int items, steps, used[2], done[2], number;  // how often things came round so far: the ring, steps, by tile scores and sums, pieces
  int fixed[2];                      // and tiles whose values were looked at: where piece n finds them, n % 2, and leaves them for the
                                     // next (one place would be written while a late warp still has to read it)
  bool alt, whole, fine, over;       // both tiles have the same queries, and every other step; the whole segment; the row's tree; no piece
};

template <typename S>
__global__ void __launch_bounds__(S::kThreads, 1)
    wide_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  constexpr int D = S::D, RB = S::RB, NC = S::NC, kRing = S::kRing, kThreads = S::kThreads, kLoadWarps = S::kLoadWarps, kWorkWarps = S::kWorkWarps,
                kWorkers = S::kWorkers, kParts = S::kParts, kSoftWarps = S::kSoftWarps, kSoft = S::kSoft, kMmaWarp = kSoftWarps + kLoadWarps, kPart = kTok / kParts;
  constexpr bool Q8 = S::Q8;
  constexpr float kUnit = Q8 ? kShift8 : 1.0f;
  extern __shared__ uint8_t raw[];
  uint8_t* const sm = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  __shared__ uint32_t tmem_base;
  __shared__ volatile int dead;
  __shared__ int sh_odd;  // the last piece (counted from 1) with values that are not finite among its new tokens
  __shared__ Piece sh_piece;
  __shared__ unsigned long long sh_mask[kTreeT];
  __shared__ float sh_back[kRows], sh_top[kTiles][kParts][kQ], sh_sum[kTiles][kParts][kQ], sh_ref[kTiles][kQ];
  __shared__ unsigned sh_valid[kInfo];
  constexpr int kFinders = Q8 ? 1 : kLoadWarps, kFound = Q8 ? 4 : 2;  // warps that look up where steps are; steps kept (8-bit: converted up to two steps behind the copies)
  __shared__ Slice sh_slice[kFinders][kFound][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned full = 0xffffffffu;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(sm + S::kBarsAt);
  uint64_t *const b_full = bars, *const b_empty = b_full + kRing, *const b_raw = b_empty + kRing, *const b_free = b_raw + kRing,
           *const b_s = b_free + kRing, *const b_p = b_s + kTiles, *const b_o = b_p + kTiles, *const b_info = b_o + kTiles, *const b_q = b_info + kInfo;
  const uint32_t base = smem_addr(sm);
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_base)), "n"(kTmem) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 0) {
    dead = sh_odd = 0;
    for (int i = 0; i < kRing; ++i) {
      mbar_init(b_full + i, kWorkWarps);
      mbar_init(b_empty + i, 1);
      mbar_init(b_raw + i, 1);
      mbar_init(b_free + i, kWorkWarps);
    }
    for (int i = 0; i < kTiles; ++i) {
      mbar_init(b_s + i, 1);
      mbar_init(b_p + i, kSoftWarps / kTiles);
      mbar_init(b_o + i, 1);
    }
    for (int i = 0; i < kInfo; ++i) mbar_init(b_info + i, Q8 ? 32 : kWorkers);
    mbar_init(b_q, kSoft);
    fence_barrier_init();
    Piece& p = sh_piece;
    p.items = p.steps = p.used[0] = p.used[1] = p.done[0] = p.done[1] = p.number = p.fixed[0] = p.fixed[1] = 0;
    p.nt = 0;
    p.alt = p.over = false;
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tm = tmem_base;
  const Wait wait{&dead};
  pdl_wait();
  pdl_trigger();

  __shared__ Line sh_line;
  {
    Line line;
    if (a.whole) {
      // segments of the longest prompts' last queries first; a row's tokens are not known here, so its place is by T
      const int per = a.r.batch * a.c.heads;
      const int mt = static_cast<int>(gridDim.x / per) - 1 - static_cast<int>(blockIdx.x / per);
      const int x = static_cast<int>(blockIdx.x % per);
      line.b = x / a.c.heads;
      const RowWork w = row_work<kRows, kTok>(a, line.b);
      if (blockIdx.x == 0) {
        for (int i = threadIdx.x; i < a.r.batch; i += kThreads) {
          const RowWork y = row_work<kRows, kTok>(a, i);
          if (y.s.count < 0) set_error(a.c.err, RSSM_ERRBIT_SEQLEN);
          if (y.len == -2) set_error(a.c.err, RSSM_ERRBIT_PAGE);
        }
      }
      line.base = 0;
      line.share = 1;
      line.lo = mt < w.mtiles ? static_cast<long long>(mt * a.c.heads + x % a.c.heads) * w.seg : 0;
      line.hi = mt < w.mtiles ? line.lo + w.seg : 0;
    } else {
      line = cut_line<kRows, kTok, kThreads>(a, blockIdx.x, gridDim.x);
    }
    if (threadIdx.x == 0) sh_line = line;
  }
  bool ok = true;

#pragma unroll 1
  while (true) {
    __syncthreads();  // the last piece's shared memory is free
    if (warp == 0) {
      // ---- the next piece, by the first warp: line.lo is the unit that it begins at or before
      Piece& p = sh_piece;
      Line& line = sh_line;
      RowWork w;
      bool over = true;
      int seg = 0, t0 = 0, t1 = 0;
      long long lo = line.lo, row_at = line.base;
      int row = line.b;
      while (lo < line.hi) {
        w = row_work<kRows, kTok>(a, row);
        if (lo >= row_at + w.units) {
          row_at += w.units;
          ++row;
          continue;
        }
        seg = static_cast<int>((lo - row_at) / w.seg);
        const int in = static_cast<int>(lo - row_at - static_cast<long long>(seg) * w.seg);
        const int to = static_cast<int>(min(static_cast<long long>(w.seg), in + (line.hi - lo)));
        t0 = tiles_before<kRows>(w, in);
        t1 = tiles_before<kRows>(w, to);
        lo += to - in;
        over = t0 == t1;  // (only what is done once: that is for who has the first tile)
        if (!over) break;
      }
      __syncwarp();
      if (lane == 0) {
        line.lo = lo;
        line.base = row_at;
        line.b = row;
      }
      bool fine = true;
      if (!over && a.parents && w.len >= 0) {
        unsigned long long masks[2];
        fine = tree_masks(a.parents + w.s.first, w.s.count, lane, masks);
        sh_mask[lane] = masks[0];
        sh_mask[lane + 32] = masks[1];
        if (!fine && lane == 0) set_error(a.c.err, RSSM_ERRBIT_TREE);
      }
      __syncwarp();
      if (lane == 0) {
        // what the last piece used
        p.items += 2 * p.nt;
        p.steps += p.nt;
        p.used[0] += p.alt ? (p.nt + 1) / 2 : p.nt;
        p.used[1] += p.alt ? p.nt / 2 : p.nt;
        p.done[0] += p.nt > 0;
        p.done[1] += p.nt > (p.alt ? 1 : 0);
        ++p.number;
        p.over = over;
        if (!over) {
          p.t0 = t0;
          p.t1 = t1;
          p.whole = t0 == 0 && t1 == w.tiles;
          const int mtile = seg / a.c.heads;
          p.head = seg - mtile * a.c.heads;
          p.row = row;
          p.first = w.s.first;
          p.len = w.len;
          p.count = w.s.count;
          p.row0 = mtile * kRows;
          p.rows = min(kRows, w.s.count * a.group - p.row0);
          p.alt = p.rows <= kQ;
          p.fine = fine;
          p.end = w.len < 0 || !fine ? 0 : w.len + (a.parents ? w.s.count : (p.row0 + p.rows - 1) / a.group + 1);
          p.some = w.len + (a.parents ? 0 : p.row0 / a.group + 1);
          p.nt = max(0, min(p.t1, (p.end + kTok - 1) / kTok) - p.t0);
        }
      }
    }
    __syncthreads();
    const Piece& p = sh_piece;
    if (p.over) break;

    if (warp < kSoftWarps) {
      // ---- queries
      const float scale2 = fmaxf(fabsf(a.scale2), 1e-30f);  // (times -inf it stays that)
      {
        const bool flip = a.scale2 < 0.0f;            // the maximum is taken before the scale
        constexpr int G = D / 8, AT = 32 / G, N = 2;  // lanes of a row, rows of a warp; rows on their way at a time (all eight at once: 8 us more for 16 trees)
        const int row0 = p.row0, rows = p.rows, head = p.head;
        const long long first = p.first;
#pragma unroll 1
        for (int r0 = warp * AT; r0 < (p.alt ? kQ : kRows); r0 += N * kSoftWarps * AT) {
          uint4 x[N];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int r = r0 + i * kSoftWarps * AT + lane / G;
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            if (r < rows) {
              const int tq = (row0 + r) / a.group, h = head * a.group + (row0 + r) - tq * a.group;
              x[i] = *reinterpret_cast<const uint4*>(a.q + (first + tq) * a.q_stride + static_cast<long long>(h) * D + lane % G * 8);
              if (flip) x[i] = make_uint4(x[i].x ^ 0x80008000u, x[i].y ^ 0x80008000u, x[i].z ^ 0x80008000u, x[i].w ^ 0x80008000u);
            }
          }
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int r = r0 + i * kSoftWarps * AT + lane / G, part = lane % G;
            if constexpr (Q8) {
              float back;
              x[i] = query_f16<G>(x[i], back);
              if (part == 0) sh_back[r] = scale2 * back;
            }
            *reinterpret_cast<uint4*>(sm + (r / kQ) * S::kTile + (part / 8) * 16384 + sw(r % kQ, part % 8)) = x[i];
          }
        }
      }
      fence_async();
      mbar_arrive(b_q);
      if constexpr (Q8) soft_sync<kSoft>();
      // ---- scores into weights: a warp's tile, half of a step's tokens, lanes of tensor memory; a thread's query in the tile
      const int tile = warp / (4 * kParts), half = (warp >> 2) % kParts, mine = (warp & 3) * 32 + lane;
      const bool alt = p.alt;
      const uint32_t s_at = tm + ((warp & 3) << 21) + tile * kTok + half * kPart;
      const int n0 = p.used[tile], nt = p.nt, len = p.len, some = p.some;
      int n = n0, j = alt ? tile : 0, step = p.steps + j, pos = (p.t0 + j) * kTok + half * kPart;
      auto pass = [&] {
        __syncwarp();
        if (lane == 0) mbar_arrive(b_p + tile);
        const int by = alt ? 2 : 1;
        j += by;
        step += by;
        pos += by * kTok;
      };
      if constexpr (!Q8) {
        const int r = alt ? mine : tile * kQ + mine;
        const int t = (p.row0 + min(r, p.rows - 1)) / a.group;
        const unsigned long long path = a.parents ? sh_mask[t & 63] : 0ull;
        float ref = -INFINITY, sum = 0.0f;
#pragma unroll 1
        for (; j < nt; ++n) {
          const int slot = step % kInfo;
          ok = ok && wait(b_info + slot, (step / kInfo) & 1);
          ok = __all_sync(full, ok && wait(b_s + tile, n & 1)) != 0;
          if (!ok) {
            pair_leave(kPairs + (warp & 3 | tile << 2));
            break;
          }
          tc_after();
          uint32_t x[kPart / 32][32];
#pragma unroll
          for (int c = 0; c < kPart / 32; ++c) tc_ld32(x[c], s_at + 32 * c);
          const unsigned valid = sh_valid[slot] >> (8 / kParts * half);
          const bool edge = pos + kPart > some || (valid & (0xffu >> (8 - 8 / kParts))) != 0xffu >> (8 - 8 / kParts);
#pragma unroll
          for (int c = 0; c < kPart / 32; ++c) landed(x[c]);
          float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < kPart / 32; ++c) {
            uint32_t(&y)[32] = x[c];
            if (edge) {
              // which of the 32 this query sees
              const int j0 = pos + 32 * c - len;
              uint32_t see;
              if (a.parents) {
                see = j0 <= -32 ? full : j0 < 0 ? static_cast<uint32_t>(path << -j0) | ((1u << -j0) - 1u) : j0 < 64 ? static_cast<uint32_t>(path >> j0) : 0u;
              } else {
                const int m = t - j0;  // the last one's place
                see = m >= 31 ? full : m < 0 ? 0u : (2u << m) - 1u;
              }
              see &= (valid >> (2 * c) & 1u ? 0xffffu : 0u) | (valid >> (2 * c + 1) & 1u ? 0xffff0000u : 0u);
#pragma unroll
              for (int i = 0; i < 32; ++i) y[i] = see >> i & 1u ? y[i] : 0xff800000u;  // -inf
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) t4[i & 3] = fmaxf(t4[i & 3], __uint_as_float(y[i]));
          }
          float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
          top = top == -INFINITY ? top : top * scale2;
          // the other half's; after this the other half's scores are in registers too, and P may take their place
          sh_top[tile][half][mine] = top;
          tc_before();
          pair_sync(kPairs + (warp & 3 | tile << 2));
          tc_after();
          top = fmaxf(top, sh_top[tile][half ^ 1][mine]);
          // the maximum in use follows where it has to; the products before this step's are done (its scores came after them)
          if (__any_sync(full, top > ref + kLazy)) {
            const float now = fmaxf(ref, top);
            const float f = now == -INFINITY ? 1.0f : exp2_fast(ref - now);
            ref = now;
            sum *= f;
            if (n > n0) {
              const uint32_t o_at = tm + ((warp & 3) << 21) + kTiles * kTok + tile * D + half * (D / kParts);
#pragma unroll 1
              for (int c = 0; c < D / (8 * kParts); ++c) {
                uint32_t y[8];
                tc_ld8(y, o_at + 8 * c);
                tc_wait_ld();
                tc_landed(y);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
                tc_stw8(o_at + 8 * c, y);
              }
            }
          }
          const float lift = ref == -INFINITY ? 0.0f : -ref;
          const pair lift2 = pack2(lift, lift), scale22 = pack2(scale2, scale2);
          pair s2[2] = {0ull, 0ull};
#pragma unroll
          for (int c = 0; c < kPart / 32; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                pair y = pack2(__uint_as_float(x[c][i + 2 * e]), __uint_as_float(x[c][i + 2 * e + 1]));
                y = fma2v(y, scale22, lift2);
                float y0, y1;
                unpack2(y, y0, y1);
                y0 = exp2_fast(y0);
                y1 = exp2_fast(y1);
                add2(s2[e], pack2(y0, y1));
                w[i / 2 + e] = bf16_pair(y0, y1);
              }
            }
            tc_st16(s_at - half * (kPart / 2) + 16 * c, w);
          }
          add2(s2[0], s2[1]);
          float u0, u1;
          unpack2(s2[0], u0, u1);
          sum += u0 + u1;
          tc_wait_st();
          tc_before();
          pass();
        }
        sh_sum[tile][half][mine] = sum;
        if (half == 0) sh_ref[tile][mine] = ref;
      } else {
        // A thread has a quarter of the half's tokens, of four queries: what goes with a token is read from shared memory once
        // for the four (a query a thread would read 12 bytes for every score, 3100 cycles of shared memory a step of 256 queries)
        const int g = lane >> 2, c2 = 2 * (lane & 3), r0 = (warp & 3) * 32 + g;  // queries r0 + 8 i
        float back[4], ref[4];
        pair s2[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          back[i] = sh_back[(alt ? 0 : tile * kQ) + r0 + 8 * i];
          ref[i] = -INFINITY;
          s2[i] = 0ull;
        }
#pragma unroll 1
        for (; j < nt; ++n) {
          const int slot = step % kInfo;
          ok = ok && wait(b_info + slot, (step / kInfo) & 1);
          ok = __all_sync(full, ok && wait(b_s + tile, n & 1)) != 0;
          if (!ok) {
            pair_leave(kPairs + (warp & 3 | tile << 2));
            break;
          }
          tc_after();
          uint32_t x[2][32];  // of query i token 8 y + c2 + e: [i / 2][4 y + 2 (i % 2) + e]
          tc_ld64(x[0], s_at);
          tc_ld64(x[1], s_at + (16u << 16));
          const unsigned valid = sh_valid[slot] >> (4 * half);
          const bool edge = pos + kPart > some || (valid & 0xfu) != 0xfu;
          const float* info = reinterpret_cast<const float*>(sm + S::kInfoAt) + slot * 3 * kTok + half * kPart + c2;
          landed(x[0]);
          landed(x[1]);
          // in units of log2, with their values' scales
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const pair k2 = *reinterpret_cast<const pair*>(info + 8 * y), l2 = *reinterpret_cast<const pair*>(info + kTok + 8 * y);
#pragma unroll
            for (int i = 0; i < 4; ++i) scaled(x[i / 2][4 * y + 2 * (i & 1)], x[i / 2][4 * y + 2 * (i & 1) + 1], pack2(back[i], back[i]), k2, l2);
          }
          if (edge) {
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              const int t = (p.row0 + min((alt ? 0 : tile * kQ) + r0 + 8 * i, p.rows - 1)) / a.group;
              const unsigned long long path = a.parents ? sh_mask[t & 63] : 0ull;
              uint32_t see = 0u;
#pragma unroll
              for (int y = 0; y < 16; ++y) {
                const int q = pos + 8 * (y >> 1) + c2 + (y & 1) - len;  // which new token this is
                const bool seen = (valid >> (y >> 2) & 1u) && (q < 0 || (a.parents ? q < 64 && (path >> (q & 63) & 1) : q <= t));
                see |= seen ? 1u << y : 0u;
              }
              // (i is not known to the compiler, and registers have no index)
#pragma unroll
              for (int z = 0; z < 4; ++z)
                if (z == i) {
#pragma unroll
                  for (int y = 0; y < 16; ++y) {
                    uint32_t& v = x[z / 2][4 * (y >> 1) + 2 * (z & 1) + (y & 1)];
                    v = see >> y & 1u ? v : 0xff800000u;  // -inf
                  }
                }
            }
          }
          float top[4];
          bool up = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float t2[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int y = 0; y < 16; ++y) t2[y & 1] = fmaxf(t2[y & 1], __uint_as_float(x[i / 2][4 * (y >> 1) + 2 * (i & 1) + (y & 1)]));
            top[i] = fmaxf(t2[0], t2[1]);
            top[i] = fmaxf(top[i], __shfl_xor_sync(full, top[i], 1));
            top[i] = fmaxf(top[i], __shfl_xor_sync(full, top[i], 2));
            if ((lane & 3) == 0) sh_top[tile][half][r0 + 8 * i] = top[i];
          }
          // the other half's; after this the other half's scores are in registers too, and P may take their place
          tc_before();
          pair_sync(kPairs + (warp & 3 | tile << 2));
          tc_after();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            top[i] = fmaxf(top[i], sh_top[tile][half ^ 1][r0 + 8 * i]);
            up = up || top[i] > ref[i] + kLazy;
          }
          // the maximum in use follows where it has to; the products before this step's are done (its scores came after them)
          if (__any_sync(full, up)) {
            float f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float now = fmaxf(ref[i], top[i]);
              f[i] = now == -INFINITY ? 1.0f : exp2_fast(ref[i] - now);
              ref[i] = now;
              s2[i] = fma2v(s2[i], pack2(f[i], f[i]), 0ull);
            }
            if (n > n0) {
              const uint32_t o_at = tm + ((warp & 3) << 21) + kTiles * kTok + tile * D + half * (D / kParts);
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll 1
                for (int c = 0; c < D / (16 * kParts); ++c) {
                  uint32_t y[8];
                  const uint32_t at = o_at + (static_cast<uint32_t>(16 * h) << 16) + 16 * c;
                  tc_ld16(y, at);
                  tc_wait_ld();
                  tc_landed(y);
#pragma unroll
                  for (int i = 0; i < 8; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * f[2 * h + (i >> 1 & 1)]);
                  tc_st16f(at, y);
                }
            }
          }
          float lift[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) lift[i] = kShift - (ref[i] == -INFINITY ? 0.0f : ref[i]);
          uint32_t w[2][16];
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const pair v2 = *reinterpret_cast<const pair*>(info + 2 * kTok + 8 * y);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float y0 = exp2_fast(__uint_as_float(x[i / 2][4 * y + 2 * (i & 1)]) + lift[i]);
              const float y1 = exp2_fast(__uint_as_float(x[i / 2][4 * y + 2 * (i & 1) + 1]) + lift[i]);
              fma2(s2[i], pack2(y0, y1), v2);
              w[i / 2][2 * y + (i & 1)] = f16_pair(y0, y1);
            }
          }
          tc_st32(s_at - half * (kPart / 2), w[0]);
          tc_st32(s_at - half * (kPart / 2) + (16u << 16), w[1]);
          tc_wait_st();
          tc_before();
          pass();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float u0, u1;
          unpack2(s2[i], u0, u1);
          u0 += u1;
          u0 += __shfl_xor_sync(full, u0, 1);
          u0 += __shfl_xor_sync(full, u0, 2);
          if ((lane & 3) == 0) {
            sh_sum[tile][half][r0 + 8 * i] = u0;
            if (half == 0) sh_ref[tile][r0 + 8 * i] = ref[i];
          }
        }
      }
      if (nt > (alt ? tile : 0)) {
        ok = __all_sync(full, ok && wait(b_o + tile, p.done[tile] & 1)) != 0;
        tc_after();
      }
    } else if (warp < kMmaWarp) {
      // ---- keys and values, in turn
      const int items = p.items, steps = p.steps, nt = p.nt, t0 = p.t0, end = p.end, head = p.head;
      const int* table = a.r.pages + p.row * a.r.pages_stride;
      const int lw = warp - kSoftWarps, lt = static_cast<int>(threadIdx.x) - kSoft - (kLoadWarps - kWorkWarps) * 32;  // lt: of those that look or convert
      // a tile is 128 NC chunks of 16 bytes; thread lt looks at chunk `ch` of rows r0, r0 + R, ..
      constexpr int R = kWorkers / NC;
      const int ch = (lt + kWorkers) % NC, r0 = lt / NC;
      // (asked for a step ahead, whether there is one or not: a load in a branch would be waited for there)
      const int most = max(0, end - 1);
      auto page_id = [&](int j) {
        const unsigned at = min(most, (t0 + j) * kTok + 16 * (lane & 7));
        return end > 0 ? table[at / static_cast<unsigned>(a.c.page_size)] : 0;
      };
      int next_id = page_id(0);
      unsigned missing = 0u;
      // where the slices of step j are, for this warp
      auto find = [&](int j) {
        const int mine = (t0 + j) * kTok + 16 * lane;
        const int id = next_id;
        next_id = page_id(j + 1);
        const bool wanted = lane < 8 && mine < end, have = wanted && id >= 0 && id < a.c.pages;
        missing = __ballot_sync(full, wanted && !have);
        if (missing && lane == 0) set_error(a.c.err, RSSM_ERRBIT_PAGE);
        if (lane < 8) {
          const unsigned place = static_cast<unsigned>(mine) % static_cast<unsigned>(a.c.page_size);
          Slice s;
          s.off[0] = have ? id * a.c.k_page + (static_cast<long long>(head) * a.c.page_size + place) * RB : 0;
          s.off[1] = have ? id * a.c.v_page + (static_cast<long long>(head) * a.c.page_size + place) * RB : 0;
          s.page = have ? id : 0;
          s.place = static_cast<int>(place);
          s.live = have ? min(16, end - mine) : 0;
          sh_slice[lw][j % kFound][lane] = s;
        }
        __syncwarp();
      };
      // the copies of item n, by the first of these warps: a lane takes the tokens that neighbour in a page
      auto copy = [&](int n, uint64_t* bar, uint32_t to) {
        const Slice* slices = sh_slice[lw][(n >> 1) % kFound];
        const int groups = kTok / a.box;
        const Slice sl = slices[lane < groups ? lane * a.box / 16 : 0];
        const bool mine = lane < groups && sl.live > 0;
        const int count = __popc(__ballot_sync(full, mine));
        if (lane == 0) mbar_arrive_expect_tx(bar, count * a.box * RB);
        __syncwarp();
        if (mine) {
          if constexpr (Q8) {
            const uint8_t* src = (n & 1 ? a.c.v : a.c.k) + sl.off[n & 1];
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to + lane * a.box * RB), "l"(src),
                         "r"(a.box * RB), "r"(smem_addr(bar))
                         : "memory");
          } else {
#pragma unroll
            for (int x = 0; x < D / 64; ++x) tma_4d(to + x * 16384 + lane * a.box * 128, n & 1 ? &map_v : &map_k, 64 * x, sl.place, head, sl.page, bar);
          }
        }
      };
      if constexpr (Q8) {
        if (lw == 0) {
          int n = 0;
          float ksv[4], vsv[4];  // the scales of the step's tokens lane + 32 e
#pragma unroll 1
          for (; n < 2 * nt; ++n) {
            const int item = items + n, buf = item % kRing, j = n >> 1;
            if (!(n & 1)) {
              find(j);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const Slice& sl = sh_slice[0][j % kFound][lane / 16 + 2 * e];
                const long long row = static_cast<long long>(head) * a.c.page_size + sl.place + (lane & 15);
                // (of page 0 where there is none: such a token's weight is 0.  Ordinary loads: this kernel may have begun before
                // the append that writes these ended, so they are not constant while it runs)
                ksv[e] = a.c.ks[sl.page * a.c.ks_page + row];
                vsv[e] = a.c.vs[sl.page * a.c.vs_page + row];
              }
            }
            ok = __all_sync(full, ok && (item < kRing || wait(b_free + buf, (item / kRing - 1) & 1))) != 0;
            if (!ok) break;
            copy(n, b_raw + buf, base + S::kRawAt + buf * kTok * RB);
            if (n & 1) {
              // what goes with the step: its place is free, by the buffer that K waited for
              const int slot = (steps + j) % kInfo;
              float* info = reinterpret_cast<float*>(sm + S::kInfoAt) + slot * 3 * kTok + lane;
              if (lane == 0) sh_valid[slot] = 0xffu & ~missing;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float y = vsv[e] < 7.7037197775489434e-34f ? 7.7037197775489434e-34f : vsv[e];  // 2^-110: a scale of 0 stands for zeros all the same
                info[32 * e] = ksv[e];
                info[kTok + 32 * e] = __log2f(y);
                info[2 * kTok + 32 * e] = y == y ? rcp_fast(y) * kShift8 : 0.0f;  // (a weight is NaN as it is, or 0 where the token is not seen)
              }
              mbar_arrive(b_info + slot);
            }
          }
          if (!ok)  // no copy is in flight at the end
            for (int i = max(0, n - kRing); i < n; ++i) mbar_wait(b_raw + (items + i) % kRing, ((items + i) / kRing) & 1);
        } else {
          // a row's 16 codes of chunk ch
          static_assert(R % 4 == 0, "the swizzle of row r0 + k R follows from r0's");
          const uint32_t to0 = (ch / 4) * 16384 + r0 * 128 + (((2 * ch % 8) ^ (r0 & 7)) << 4);
          auto fetch = [&](uint32_t (&c4)[4], uint32_t from, int k) {
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(c4[0]), "=r"(c4[1]), "=r"(c4[2]), "=r"(c4[3]) : "r"(from + k * R * RB));
          };
          auto store = [&](const uint32_t (&c4)[4], uint8_t* tile, int k, bool there) {
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t y = !there ? S::FMT == RSSM_I8 ? 0x80808080u : 0u : S::FMT == RSSM_I8 ? c4[e] ^ 0x80808080u : c4[e];
              codes_f16<S::FMT>(y, h[2 * e], h[2 * e + 1]);
            }
            uint8_t* const to = tile + k * R * 128;
            const uint32_t x = to0 ^ ((R * k & 4) << 4);
            *reinterpret_cast<uint4*>(to + x) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(to + (x ^ 16)) = make_uint4(h[4], h[5], h[6], h[7]);
          };
#pragma unroll 1
          for (int n = 0; n < 2 * nt; ++n) {
            const int item = items + n, buf = item % kRing;
            ok = __all_sync(full, ok && (item < kRing || wait(b_empty + buf, (item / kRing - 1) & 1))) != 0;
            if (!ok) break;
            ok = __all_sync(full, wait(b_raw + buf, (item / kRing) & 1)) != 0;
            if (!ok) break;
            const uint32_t from = base + S::kRawAt + buf * kTok * RB + r0 * RB + ch * 16;
            uint8_t* const tile = sm + S::kRingAt + buf * S::kTile;
            // kBatch rows at a time: a load does not pass the stores before it
            constexpr int kFull = kTok / R, kBatch = kFull % 5 == 0 ? 5 : kFull % 4 == 0 ? 4 : 2;
            static_assert(kFull % kBatch == 0 && R * (kFull + 1) > kTok, "batches, then one row for some");
            const Slice* slices = sh_slice[0][(n >> 1) % kFound];  // the first warp's: it wrote them before the copies
            if (__all_sync(full, slices[lane & 7].live == 16)) {
#pragma unroll
              for (int k0 = 0; k0 < kFull; k0 += kBatch) {
                uint32_t c4[kBatch][4];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) fetch(c4[k], from, k0 + k);
#pragma unroll
                for (int k = 0; k < kBatch; ++k) store(c4[k], tile, k0 + k, true);
              }
              if (r0 + kFull * R < kTok) {
                uint32_t c4[4];
                fetch(c4, from, kFull);
                store(c4, tile, kFull, true);
              }
            } else {
#pragma unroll 1
              for (int k = 0; r0 + k * R < kTok; ++k) {
                const int r = r0 + k * R;
                uint32_t c4[4];
                fetch(c4, from, k);
                store(c4, tile, k, r % 16 < slices[r / 16].live);  // what lies behind may be anything
              }
            }
            fence_async();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(b_full + buf);
              mbar_arrive(b_free + buf);
            }
          }
        }
      } else {
        int n = 0, fixed = p.fixed[p.number & 1];
#pragma unroll 1
        for (; n < 2 * nt; ++n) {
          const int item = items + n, buf = item % kRing, j = n >> 1;
          if (!(n & 1)) find(j);
          ok = __all_sync(full, ok && (item < kRing || wait(b_empty + buf, (item / kRing - 1) & 1))) != 0;
          if (!ok) break;
          if (!(n & 1)) {
            const int slot = (steps + j) % kInfo;
            if (lt == 0) sh_valid[slot] = 0xffu & ~missing;
            mbar_arrive(b_info + slot);
          }
          const uint32_t to = base + S::kRingAt + buf * S::kTile;
          // values that not every query sees are looked at before the product gets them, and what lies behind the last or in no
          // page is zero
          // (two barriers in turn: the ring lets the first warp be up to two such tiles ahead of another, which has
          // to find the phase that it waits for, and not the one after)
          const bool unseen = (t0 + j + 1) * kTok > p.some, fix = (n & 1) && (unseen || missing);
          if (lw == 0) copy(n, fix ? b_raw + (fixed & 1) : b_full + buf, to);
          if (fix) {
            ok = __all_sync(full, ok && wait(b_raw + (fixed & 1), (fixed >> 1) & 1)) != 0;
            ++fixed;
            if (!ok) break;
            uint8_t* tile = sm + S::kRingAt + buf * S::kTile + (ch / 8) * 16384;
            const Slice* slices = sh_slice[lw][j % kFound];
            for (int r = r0; r < kTok; r += R) {
              uint4* q = reinterpret_cast<uint4*>(tile + sw(r, ch % 8));
              if (r % 16 >= slices[r / 16].live) {
                *q = make_uint4(0u, 0u, 0u, 0u);
                continue;
              }
              if (!unseen) continue;  // every query sees the others, whatever they are
              uint4 y = *q;
              if (take_out_odd(y)) {
                *q = y;
                sh_odd = p.number;
              }
            }
            fence_async();
            __syncwarp();
          }
          if (lane == 0 && (fix || lw != 0)) mbar_arrive(b_full + buf);
        }
        if (lw == 0 && lane == 0) sh_piece.fixed[(p.number + 1) & 1] = fixed;
        if (!ok && lw == 0) {  // no copy is in flight at the end, that of a tile to be looked at neither
          for (int i = max(0, n - kRing); i < n; ++i) mbar_wait(b_full + (items + i) % kRing, ((items + i) / kRing) & 1);
          if (fixed > 0) mbar_wait(b_raw + ((fixed - 1) & 1), ((fixed - 1) >> 1) & 1);
        }
      }
    } else {
      // ---- products
      const int items = p.items, nt = p.nt, used0 = p.used[0], used1 = p.used[1];
      constexpr uint32_t kind = Q8 ? (1u << 7) | (1u << 10) : 0u;  // fp16 operands: without bf16's bits
      constexpr uint32_t i_s = instruction(kTok, false, false) & ~kind, i_o = instruction(D, false, true) & ~kind;
      auto scores = [&](int tile, int queries, int buf) {
        const uint64_t q = operand(base + queries * S::kTile, 16, 1024, kSw128), k = operand(base + S::kRingAt + buf * S::kTile, 16, 1024, kSw128);
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const uint64_t o = (x / 4) * (16384 / 16) + (x % 4) * 2;
          mma_ss(lane == 0, tm + tile * kTok, q + o, k + o, i_s, x > 0);
        }
        commit(lane == 0, b_s + tile);
      };
      auto sums = [&](int tile, int buf, bool more) {
        const uint64_t v = operand(base + S::kRingAt + buf * S::kTile, 16384, 1024, kSw128);
#pragma unroll
        for (int y = 0; y < kTok / 16; ++y) mma_ts(lane == 0, tm + kTiles * kTok + tile * D, tm + tile * kTok + 8 * y, v + y * (2048 / 16), i_o, more || y > 0);
      };
      auto filled = [&](int n) {  // item n of the piece is there
        const int item = items + n;
        ok = __all_sync(full, ok && wait(b_full + item % kRing, (item / kRing) & 1)) != 0;
        return item % kRing;
      };
      ok = __all_sync(full, ok && wait(b_q, (p.number - 1) & 1)) != 0;
      if (p.alt) {
        for (int j = 0; ok && j < min(nt, 2); ++j) {
          const int buf = filled(2 * j);
          if (!ok) break;
          tc_after();
          scores(j, 0, buf);
          commit(lane == 0, b_empty + buf);
        }
#pragma unroll 1
        for (int j = 0; ok && j < nt; ++j) {
          const int x = j & 1, bv = filled(2 * j + 1);
          ok = __all_sync(full, ok && wait(b_p + x, ((x ? used1 : used0) + j / 2) & 1)) != 0;
          if (!ok) break;
          tc_after();
          sums(x, bv, j > 1);
          commit(lane == 0, b_empty + bv);
          if (j + 2 < nt) {
            const int bk = filled(2 * j + 4);
            if (!ok) break;
            tc_after();
            scores(x, 0, bk);
            commit(lane == 0, b_empty + bk);
          } else {
            commit(lane == 0, b_o + x);
          }
        }
      } else {
        if (ok && nt > 0) {
          const int buf = filled(0);
          if (ok) {
            tc_after();
            for (int x = 0; x < kTiles; ++x) scores(x, x, buf);
            commit(lane == 0, b_empty + buf);
          }
        }
#pragma unroll 1
        for (int j = 0; ok && j < nt; ++j) {
          const bool more = j + 1 < nt;
          const int bv = filled(2 * j + 1), bk = more ? filled(2 * j + 2) : 0;
          for (int x = 0; x < kTiles; ++x) {
            ok = __all_sync(full, ok && wait(b_p + x, ((x ? used1 : used0) + j) & 1)) != 0;
            if (!ok) break;
            tc_after();
            sums(x, bv, j > 0);
            if (more) scores(x, x, bk);
            else commit(lane == 0, b_o + x);
          }
          if (ok) {
            commit(lane == 0, b_empty + bv);
            if (more) commit(lane == 0, b_empty + bk);
          }
        }
      }
    }
    ok = __syncthreads_and(ok);
    if (!ok) break;

    // ---- the queries' sums
    if (warp < kSoftWarps) {
      const int tile = warp / (4 * kParts), half = (warp >> 2) % kParts, mine = (warp & 3) * 32 + lane;
      const uint32_t o_at = tm + ((warp & 3) << 21) + kTiles * kTok + tile * D + half * (D / kParts);
      const bool alt = p.alt, whole = p.whole, both = alt && p.nt > 1;
      const int rows = p.rows, row0 = p.row0;
      float ref = sh_ref[tile][mine];
      float* const other = reinterpret_cast<float*>(sm + S::kRingAt);  // [dimension][query]
      if (both && tile == 1) {
        // the second tile's sums are the same queries'
#pragma unroll 1
        for (int c = 0; c < D / (32 * kParts); ++c) {
          uint32_t x[32];
          tc_ld32(x, o_at + 32 * c);
          landed(x);
#pragma unroll
          for (int i = 0; i < 32; ++i) other[(half * (D / kParts) + 32 * c + i) * kQ + mine] = __uint_as_float(x[i]);
        }
      }
      if (both) soft_sync<kSoft>();
      float sum = sh_sum[tile][0][mine] + (kParts == 2 ? sh_sum[tile][kParts - 1][mine] : 0.0f);
      if (tile == 0 || !alt) {
        float join0 = 1.0f, join1 = 0.0f;  // what the two tiles' sums are times
        if (both) {
          const float now = fmaxf(ref, sh_ref[1][mine]), at0 = now == -INFINITY ? 0.0f : now;
          join0 = exp2_fast(ref - at0);
          join1 = exp2_fast(sh_ref[1][mine] - at0);
          sum = sum * join0 + (sh_sum[1][0][mine] + (kParts == 2 ? sh_sum[1][kParts - 1][mine] : 0.0f)) * join1;
          ref = now;
        }
        const int r = tile * kQ + mine;
        float* const left = piece_place<kRows, D>(a, blockIdx.x, p.t0 == 0);
        const float inv = sum == 0.0f ? 0.0f : kUnit / sum;
#pragma unroll 1
        for (int c = 0; c < D / (32 * kParts); ++c) {
          const int d0 = half * (D / kParts) + 32 * c;
          uint32_t x[32];
          if (p.nt > 0) {
            tc_ld32(x, o_at + 32 * c);
            landed(x);
            if (both) {
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * join0 + other[(d0 + i) * kQ + mine] * join1);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = 0u;
          }
          if (r < rows) {
            if (whole) {
              // bf16, in the place of the tile's queries: rows leave from there side by side
              uint8_t* const q = sm + tile * S::kTile + d0 / 64 * 16384;
#pragma unroll
              for (int i = 0; i < 32; i += 8) {
                uint32_t y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = bf16_pair(__uint_as_float(x[i + 2 * e]) * inv, __uint_as_float(x[i + 2 * e + 1]) * inv);
                *reinterpret_cast<uint4*>(q + sw(mine, d0 % 64 / 8 + i / 8)) = make_uint4(y[0], y[1], y[2], y[3]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; i += 4) __stcg(reinterpret_cast<uint4*>(left + piece_at<kRows, D>(r, d0 + i)), make_uint4(x[i], x[i + 1], x[i + 2], x[i + 3]));
            }
          }
          __syncwarp();  // the next load is the whole warp's
        }
        if (!whole && r < rows && half == 0) {
          __stcg(left + kRows * D + r, ref);
          __stcg(left + kRows * D + kRows + r, sum);
        }
      }
      tc_before();
      fence_async();  // the next piece's copies come into the ring, where the second tile's sums were
      if (!Q8 && sh_odd == p.number) {
        // values that are not finite, to those queries that see them
        soft_sync<kSoft>();
        const int from = max(p.t0 * kTok, p.some / kTok * kTok), to = min(p.t1 * kTok, p.end);
        float* const left = piece_place<kRows, D>(a, blockIdx.x, p.t0 == 0);
#pragma unroll 1
        for (int i = threadIdx.x; i < rows * (D / 4); i += kSoft) {
          const int r = i / (D / 4), c = i % (D / 4) * 4, t = (row0 + r) / a.group;
          const float4 y = add_odd4(a, p.len, a.r.pages + p.row * a.r.pages_stride, a.c.v + static_cast<long long>(p.head) * a.c.page_size * RB, RB, from,
                                    to, t, a.parents ? sh_mask[t & 63] : 0ull, c, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
          if (y.x == 0.0f && y.y == 0.0f && y.z == 0.0f && y.w == 0.0f) continue;
          if (whole) {
            uint2* const q = reinterpret_cast<uint2*>(sm + (r / kQ) * S::kTile + c / 64 * 16384 + sw(r % kQ, c % 64 / 8) + c % 8 * 2);
            *q = make_uint2(bf16_pair(bf16lo(q->x) + y.x, bf16hi(q->x) + y.y), bf16_pair(bf16lo(q->y) + y.z, bf16hi(q->y) + y.w));
          } else {
            float4* const q = reinterpret_cast<float4*>(left + piece_at<kRows, D>(r, c));
            const float4 z = __ldcg(q);
            __stcg(q, make_float4(z.x + y.x, z.y + y.y, z.z + y.z, z.w + y.w));
          }
        }
      }
      if (whole) {
        soft_sync<kSoft>();
        constexpr int G = D / 8;
        for (int i = threadIdx.x; i < rows * G; i += kSoft) {
          const int r = i / G, ch = i % G, tq = (row0 + r) / a.group, h = p.head * a.group + (row0 + r) - tq * a.group;
          *reinterpret_cast<uint4*>(a.out + (p.first + tq) * a.out_stride + static_cast<long long>(h) * D + ch * 8) =
              *reinterpret_cast<const uint4*>(sm + (r / kQ) * S::kTile + (ch / 8) * 16384 + sw(r % kQ, ch % 8));
        }
      }
    }
  }
  // a wait that gave up: what was started ends before the memory is given back
  if (!ok && warp == kMmaWarp && lane == 0) {
    mbar_init(b_info, 1);
    fence_barrier_init();
    tc_commit(b_info);
    mbar_wait(b_info, 0);
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "n"(kTmem) : "memory");
  if (threadIdx.x == 0 && dead) set_error(a.c.err, RSSM_ERRBIT_TIMEOUT);
}

// a layer's keys or values as [page][head][place][dimension], boxes of 64 dimensions of `box` tokens
bool page_map(const KvView& c, bool values, int box, CUtensorMap* map) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t row = static_cast<cuuint64_t>(c.dim) * 2;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.dim), static_cast<cuuint64_t>(c.page_size), static_cast<cuuint64_t>(c.heads),
                              static_cast<cuuint64_t>(c.pages)};
  const cuuint64_t strides[3] = {row, row * c.page_size, static_cast<cuuint64_t>(values ? c.v_page : c.k_page)};
  const cuuint32_t shape[4] = {64, static_cast<cuuint32_t>(box), 1, 1}, one[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, values ? c.v : c.k, dims, strides, shape, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
  CUtensorMap k = {}, v = {};
  if (!S::Q8 && (!page_map(a.c, false, a.box, &k) || !page_map(a.c, true, a.box, &v))) return cudaErrorInvalidValue;
  e = launch_pdl(wide_kernel<S>, dim3(grid), dim3(S::kThreads), S::kSmem, st, a, k, v);
  if (e != cudaSuccess || a.whole || grid < 2) return e;
  return launch_join<kRows, kTok, D>(a, grid, S::Q8 ? kShift8 : 1.0f, st);
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
  a.box = 16;  // tokens that neighbour in a page, and in a step
  while (a.box < kTok && a.c.page_size % (2 * a.box) == 0) a.box *= 2;
  const int grid = a.whole ? static_cast<int>(segments) : sms;
  return a.c.dim == 64 ? launch_format<64>(a, grid, st) : launch_format<128>(a, grid, st);
}

}  // namespace rssm
