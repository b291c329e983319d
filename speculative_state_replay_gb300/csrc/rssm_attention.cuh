// rssm_attention.cuh -- what the two attention kernels share: arguments, how the
// work is cut, and how the pieces of a shared segment are joined.
//
// The queries of a (row, key head) are its new tokens times the heads of its group,
// `group` consecutive ones a token.  A segment is a tile of them over all of the
// row's tokens, tile by tile; work is measured in units.
#pragma once

#include "rssm_kv.cuh"

namespace rssm {

// 1 / (a value's scale) is summed times this, 2^-16.  Scales are at least 2^-109 (2^-100 / 448), at most 2^121 (bf16's largest
// / 127): the inverse of the largest keeps 12 bits, and 2^20 tokens of the smallest with weights of 2^15 stay in range.
constexpr float kShift8 = 1.52587890625e-05f;

struct AttnArgs {
  KvView c;
  KvRows r;
  const uint16_t* q;
  long long q_stride;
  uint16_t* out;
  long long out_stride;
  const int* parents;  // or null: a chain
  int group;
  float scale2;  // scale log2(e)
  int whole;     // a block takes one segment, the longest first, instead of an equal part of the line
  int box;           // tokens of one copy (the kernel for many queries)
  int apart;         // shared segments are joined by a launch of its own
  unsigned* ticket;  // [blocks]
  float* partial;    // [blocks][2][rows of a tile x (head_dim + 2)]
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The four codes of w (int8: with their sign bits turned) as two pairs of fp16 values, exactly: bytes 0 and 1, 2 and 3.
// int8: code + 128 under the exponent of 1024 is 1152 + code.
template <int FMT>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == RSSM_I8) {
    const uint32_t l = __byte_perm(w, 0x64646464u, 0x4140u), h = __byte_perm(w, 0x64646464u, 0x4342u);
    const __half2 off = __float2half2_rn(1152.0f), y = __hsub2(*reinterpret_cast<const __half2*>(&l), off),
                  z = __hsub2(*reinterpret_cast<const __half2*>(&h), off);
    lo = *reinterpret_cast<const uint32_t*>(&y);
    hi = *reinterpret_cast<const uint32_t*>(&z);
  } else {
    asm("{\n\t.reg .b16 x, z;\n\tmov.b32 {x, z}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, z;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

// 16 (4) bytes to shared memory, zeros if not `have`
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool have) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(have ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool have) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(have ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Eight values of a query for an 8-bit cache: fp16, times a power of two that takes the row's largest to
// 2^14 .. 2^15 (smaller ones keep all their bits down to 2^-28 of it).  G lanes hold a row; `back`: its inverse.
template <int G>
__device__ __forceinline__ uint4 query_f16(const uint4& x, float& back) {
  uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
#pragma unroll
  for (int o = 1; o < G; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
  const int e = static_cast<int>(max(m & 0xffffu, m >> 16) >> 7);  // exponent of the largest, 255: not finite
  const int by = e == 0 || e == 255 ? 0 : 141 - e, h1 = by / 2, h2 = by - h1;  // two factors, for exponents of any size
  const float f1 = __uint_as_float(static_cast<uint32_t>(127 + h1) << 23), f2 = __uint_as_float(static_cast<uint32_t>(127 + h2) << 23);
  back = __uint_as_float(static_cast<uint32_t>(127 - h1) << 23) * __uint_as_float(static_cast<uint32_t>(127 - h2) << 23);
  const uint32_t y[4] = {x.x, x.y, x.z, x.w};
  uint32_t z[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) z[i] = f16_pair(bf16lo(y[i]) * f1 * f2, bf16hi(y[i]) * f1 * f2);
  return make_uint4(z[0], z[1], z[2], z[3]);
}

// bf16 values that are not finite become zeros; whether there was one
__device__ __forceinline__ bool take_out_odd(uint4& x) {
  uint32_t z[4] = {x.x, x.y, x.z, x.w};
  bool odd = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if ((z[e] & 0x7f80u) == 0x7f80u) z[e] &= 0xffff0000u, odd = true;
    if ((z[e] & 0x7f800000u) == 0x7f800000u) z[e] &= 0xffffu, odd = true;
  }
  x = make_uint4(z[0], z[1], z[2], z[3]);
  return odd;
}

struct RowWork {
  RowSpan s;
  int len;    // committed tokens; < 0: nothing to see, zeros (-1: padding, -2: past the page table)
  int tiles;  // of tokens
  int mtiles; // of queries
  int cost;   // of a tile of tokens, in units
  int seg;    // units of a segment
  long long units;  // of the row
};

// What a segment costs, in units: a tile of tokens, and what is done once.  The kernel for few queries: a tile is a unit.
// The one for many: a tile of tokens costs about 5000 cycles where both query tiles have queries of their own (3 units),
// 3500 where they share them (2), and a segment's queries and sums 20000 (16 ragged trees over int8: 204 us with equal
// tiles, 145 so).  A part is at least what a tile costs, so that none between a segment's first tile and its end is
// without one.
template <int kRows>
constexpr int kOnce = kRows > 32 ? 12 : 0;
template <int kRows>
constexpr int kLeast = kRows > 32 ? 4 : 1;
// the tiles of tokens that begin before unit `at` of a segment
template <int kRows>
__device__ __forceinline__ int tiles_before(const RowWork& w, int at) {
  return at <= kOnce<kRows> ? 0 : (at - kOnce<kRows>) / w.cost;
}

template <int kRows, int kTile>
__device__ __forceinline__ RowWork row_work(const AttnArgs& a, int b) {
  RowWork w;
  w.s = row_span(a.r, b);
  w.tiles = w.mtiles = 0;
  w.cost = kRows > 32 ? 2 : 1;
  w.seg = 0;
  w.units = 0;
  w.len = -1;
  if (w.s.count <= 0) return w;
  w.len = max(a.r.lengths[b], -1);  // (any below 0 is padding)
  w.tiles = 1;
  w.mtiles = static_cast<int>((static_cast<long long>(w.s.count) * a.group + kRows - 1) / kRows);
  if (w.len >= 0) {
    const long long end = static_cast<long long>(w.len) + w.s.count;  // (positions are 31 bits from here on)
    if (end > min(static_cast<long long>(a.r.max_pages) * a.c.page_size, 0x7fffff00ll)) w.len = -2;
    else w.tiles = static_cast<int>((end + kTile - 1) / kTile);
  }
  if (kRows > 32 && static_cast<long long>(w.s.count) * a.group > kRows / 2) w.cost = 3;
  w.seg = kOnce<kRows> + w.tiles * w.cost;
  w.units = static_cast<long long>(w.seg) * w.mtiles * a.c.heads;
  return w;
}

// Part `block` of `blocks` of the line of all units, ordered by row, query tile, head and token tile: units lo .. hi of
// `share` a part, which begin in row b, whose units begin at `base`.  All threads of the block call it.
struct Line {
  long long lo, hi, share, base;
  int b;
};
template <int kRows, int kTile, int kThreads>
__device__ __forceinline__ Line cut_line(const AttnArgs& a, int block, int blocks) {
  constexpr int kWarps = kThreads / 32;
  __shared__ long long scan[kWarps], sh_base;
  __shared__ int sh_row;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (a.r.batch + kThreads - 1) / kThreads;
  const int r0 = min(a.r.batch, static_cast<int>(threadIdx.x) * per), r1 = min(a.r.batch, r0 + per);
  long long sum = 0;
  for (int i = r0; i < r1; ++i) {
    const RowWork w = row_work<kRows, kTile>(a, i);
    sum += w.units;
    if (block == 0) {
      if (w.s.count < 0) set_error(a.c.err, RSSM_ERRBIT_SEQLEN);
      if (w.len == -2) set_error(a.c.err, RSSM_ERRBIT_PAGE);
    }
  }
  long long upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) scan[warp] = upto;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int x = 0; x < kWarps; ++x) {
    if (x < warp) upto += scan[x];
    total += scan[x];
  }
  Line l;
  l.share = max(static_cast<long long>(kLeast<kRows>), (total + blocks - 1) / blocks);
  l.lo = l.share * block;
  l.hi = min(total, l.lo + l.share);
  long long at = upto - sum;
  if (l.lo < l.hi && l.lo >= at && l.lo < upto) {
    int i = r0;
    for (; i < r1; ++i) {
      const RowWork w = row_work<kRows, kTile>(a, i);
      if (l.lo < at + w.units) break;
      at += w.units;
    }
    sh_row = i;
    sh_base = at;
  }
  __syncthreads();
  l.b = sh_row;
  l.base = sh_base;
  return l;
}

// What values that are not finite add to four columns from x4 on of the query at new token t: the kernels take
// them out of the products from position `from` on, where tokens are that not every query sees, since they must not
// meet the weight 0 of one that does not.
static __device__ __noinline__ float4 add_odd4(const AttnArgs& a, int len, const int* table, const uint8_t* vbase, int row_bytes, long long from,
                                             long long to, int t, unsigned long long path, int x4, float4 y4) {
  float y[4] = {y4.x, y4.y, y4.z, y4.w};
  for (long long p = from; p < to; ++p) {
    const long long j = p - len;
    if (j >= 0 && !(a.parents ? path >> (j & 63) & 1 : j <= t)) continue;
    const unsigned pos = static_cast<unsigned>(p), page = pos / static_cast<unsigned>(a.c.page_size);
    const int pg = table[page];
    if (pg < 0 || pg >= a.c.pages) continue;
    const uint2 v = *reinterpret_cast<const uint2*>(vbase + pg * a.c.v_page + static_cast<long long>(pos - page * a.c.page_size) * row_bytes + x4 * 2);
    const float f[4] = {bf16lo(v.x), bf16hi(v.x), bf16lo(v.y), bf16hi(v.y)};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (!isfinite(f[e])) y[e] += f[e];
  }
  return make_float4(y[0], y[1], y[2], y[3]);
}

__device__ __forceinline__ void write_out(const AttnArgs& a, long long first, int head, int query, int D, int x4, const float (&y)[4], float inv) {
  const int t = query / a.group, h = head * a.group + query - t * a.group;
  *reinterpret_cast<uint2*>(a.out + (first + t) * a.out_stride + static_cast<long long>(h) * D + x4) =
      make_uint2(bf16_pair(y[0] * inv, y[1] * inv), bf16_pair(y[2] * inv, y[3] * inv));
}

// A segment that several blocks share: each leaves its sums, and they are joined in the
// segment's order.  A piece is kRows x D sums, then the rows' maxima and the rows' sums of
// weights; a block has two places, for a segment that began before it and for one that
// goes on after it.
template <int kRows, int D>
__device__ __forceinline__ float* piece_place(const AttnArgs& a, int block, bool begins) {
  return a.partial + (static_cast<long long>(block) * 2 + begins) * (kRows * (D + 2));
}
// where row r's columns from x4 on are in a piece: a tile of few rows has them one after another, one of many by four
// columns (there a thread has a row, and a warp writes 512 bytes that neighbour)
template <int kRows, int D>
__device__ __forceinline__ int piece_at(int r, int x4) {
  return kRows > 32 ? x4 * kRows + r * 4 : r * D + x4;
}
// The joined sums of a row's four columns.
struct JoinSum {
  float y[4] = {0.0f, 0.0f, 0.0f, 0.0f}, z = 0.0f, top = -INFINITY;
  __device__ __forceinline__ void add(const float4& v, float m, float l) {
    const float now = fmaxf(top, m), ref = now == -INFINITY ? 0.0f : now;
    const float f = exp2_fast(top - ref), g = exp2_fast(m - ref);
    top = now;
    y[0] = y[0] * f + v.x * g;
    y[1] = y[1] * f + v.y * g;
    y[2] = y[2] * f + v.z * g;
    y[3] = y[3] * f + v.w * g;
    z = z * f + l * g;
  }
};
// of row r's columns from x4 on, with the loads of kDeep pieces on their way at a time
template <int kRows, int D, int kDeep>
__device__ __forceinline__ JoinSum join_row(const AttnArgs& a, int first, int pieces, int r, int x4) {
  JoinSum s;
#pragma unroll 1
  for (int x0 = 0; x0 < pieces; x0 += kDeep) {
    float4 v[kDeep];
    float m[kDeep], l[kDeep];
#pragma unroll
    for (int e = 0; e < kDeep; ++e)
      if (x0 + e < pieces) {
        const float* p = piece_place<kRows, D>(a, first + x0 + e, x0 + e == 0);
        m[e] = __ldcg(p + kRows * D + r);
        l[e] = __ldcg(p + kRows * D + kRows + r);
        v[e] = __ldcg(reinterpret_cast<const float4*>(p + piece_at<kRows, D>(r, x4)));
      }
#pragma unroll
    for (int e = 0; e < kDeep; ++e)
      if (x0 + e < pieces) s.add(v[e], m[e], l[e]);
  }
  return s;
}

struct Joint {  // a segment that a block has a piece of
  long long first_token, seg0;  // its row's first new token, its first unit
  int tiles, head, row0, rows;
};
// Whoever leaves a segment's last piece joins them.  (After all of a block's pieces: in their loop it would take
// registers from it.)
template <int kRows, int D, int kThreads, int kDeep>
__device__ __forceinline__ void join_pieces(const AttnArgs& a, const Joint& j, long long share, float unit) {
  const long long first_token = j.first_token, seg0 = j.seg0;
  const int tiles = j.tiles, head = j.head, row0 = j.row0, rows = j.rows;
  __shared__ int last;
  const int first = static_cast<int>(seg0 / share), pieces = static_cast<int>((seg0 + tiles - 1) / share) - first + 1;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    last = atomicAdd(a.ticket + first, 1u) == static_cast<unsigned>(pieces - 1);
    if (last) a.ticket[first] = 0u;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  constexpr int D4 = D / 4;
#pragma unroll 1
  for (int i = threadIdx.x; i < rows * D4; i += kThreads) {
    const int r = i / D4, x4 = (i - r * D4) * 4;
    const JoinSum s = join_row<kRows, D, kDeep>(a, first, pieces, r, x4);
    write_out(a, first_token, head, row0 + r, D, x4, s.y, s.z == 0.0f ? 0.0f : unit / s.z);
  }
}

// The same by a launch of its own.  A piece has up to 256 x 128 sums, and where few segments meet many blocks, one block
// that joined all of a segment's pieces would take longer than the pieces themselves (one row's tree of 64 over 4096
// tokens, 8 heads, groups of 4: 152 us with it, 59 without when this came, now 39 in bf16 and 46 in int8).  Block
// (x, y): rows 16 y .. of the segment, if any, that cut x of the line is the first to go through.
constexpr int kJoinRows = 16, kJoinThreads = 256;
template <int kRows, int kTile, int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ AttnArgs a, int blocks, float unit) {
  pdl_wait();
  pdl_trigger();
  const int cut = blockIdx.x + 1;
  const Line line = cut_line<kRows, kTile, kJoinThreads>(a, cut, blocks);
  if (line.lo >= line.hi) return;
  const RowWork w = row_work<kRows, kTile>(a, line.b);
  const long long at = line.lo - line.base;
  const int seg = static_cast<int>(at / w.seg), in = static_cast<int>(at - static_cast<long long>(seg) * w.seg);
  // the first piece with a tile is of the part that unit `body` is in; this is the cut behind it, or there is nothing to do
  const long long body = line.lo - in + kOnce<kRows> + w.cost - 1;
  const int first = cut - 1, pieces = static_cast<int>((line.lo - in + w.seg - 1) / line.share) - first + 1;
  if (body >= line.lo || body < line.lo - line.share) return;
  const int mtile = seg / a.c.heads, head = seg - mtile * a.c.heads, row0 = mtile * kRows;
  const int r0 = blockIdx.y * kJoinRows, rows = min(kJoinRows, min(kRows, w.s.count * a.group - row0) - r0);
  constexpr int D4 = D / 4;
#pragma unroll 1
  for (int i = threadIdx.x; i < kJoinRows * D4; i += kJoinThreads) {
    // a warp: eight rows, four times four columns, which are 128 bytes that neighbour of a piece, 32 of a row's output
    const int at = i / (8 * D4) * 8 + (i & 7), r = r0 + at, x4 = i / 8 % D4 * 4;
    if (at >= rows) continue;
    const JoinSum s = join_row<kRows, D, 8>(a, first, pieces, r, x4);
    write_out(a, w.s.first, head, row0 + r, D, x4, s.y, s.z == 0.0f ? 0.0f : unit / s.z);
  }
}
template <int kRows, int kTile, int D>
cudaError_t launch_join(const AttnArgs& a, int blocks, float unit, cudaStream_t st) {
  const long long most = static_cast<long long>(a.r.T) * a.group;
  const int rows = static_cast<int>(most < kRows ? most : kRows);
  return launch_pdl(join_kernel<kRows, kTile, D>, dim3(blocks - 1, (rows + kJoinRows - 1) / kJoinRows), dim3(kJoinThreads), 0, st, a, blocks, unit);
}

// host side: the kernel for many queries of a head (rssm_attention_wide.cu)
bool wide_takes(const KvView& c, int64_t queries);
size_t wide_scratch(const KvView& c, int sms);
cudaError_t run_wide(const AttnArgs& a, int sms, cudaStream_t st);

}  // namespace rssm
