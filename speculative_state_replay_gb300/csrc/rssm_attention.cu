// rssm_attention.cu -- attention of a row's new tokens over its cached ones.
//
// The queries of a (row, key head) are its new tokens times the heads of its group,
// `group` consecutive ones a token; a tile of kRows of them goes over the row's
// cached tokens once, with the running maximum and sum of the softmax.  A warp takes
// 16 cached tokens at a time (a slice never crosses a page), by itself: its own
// copies into shared memory, its own statistics and sums, so that no warp waits for
// another until the pieces are joined.
//
// What bounds it is the cache's read: 64 rows of 8192 bf16 tokens, 8 heads of 128, 4
// queries each, take 311 us, 6.9 TB/s.  8-bit codes are bound by the instructions that
// make operands of them: the same in e4m3 197 us, 5.6 TB/s, in int8 223.  The scores'
// contraction index is permuted so that a lane's part of a key is 16 bytes as they lie
// in the cache; 8-bit codes become
// fp16 exactly, on their way into the products.  The values' tile is read by transposing
// loads; 8-bit ones come as pairs of neighbouring dimensions of two tokens, which two
// byte permutations turn into the even and the odd dimension's operands.  In units of
// log2, with scales a_i of keys and b_i of values,
//   s_i = q . k_i a_i scale log2(e),  m = max (s_i + log2 b_i),  w_i = 2^(s_i + log2 b_i - m),
//   out = (sum w_i code_i) / (sum w_i / b_i)
// so the values' scales enter the weights, which are at most 2^4 whatever the scales: the
// m in use follows the true maximum only when that is more than 2^4 times past it, so that
// the sums are rarely scaled.  8-bit caches take the weights to fp16 times 2^11 (those down
// to 2^-25 of the largest keep 11 bits), bf16 ones to bf16.
//
// Work is cut without regard to rows: all (row, tile, head) segments in one line of
// 64-token units, and every block takes an equal part of it.  A segment that several
// blocks share is joined by the one that finishes last, from what the others left in
// the scratch, in the segment's order: no block waits for another.  Of more than 8
// queries a launch of its own joins them.
#include <type_traits>

#include "rssm_attention.cuh"

namespace rssm {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kSlice = 16;              // tokens of a warp's step
constexpr int kTile = kWarps * kSlice;  // tokens of a unit of work
constexpr int kBlocks = 3;              // an SM, at most
constexpr int kMaxSms = 512;
constexpr float kShift = 11.0f;         // fp16 weights are times 2^11: 2^15 at most
constexpr float kLazy = 4.0f;           // log2 of how far the true maximum may be past the one that weights are taken against

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_b16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <bool Q8>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (Q8) mma_f16(d, a0, a1, a2, a3, b0, b1);
  else mma_b16(d, a0, a1, a2, a3, b0, b1);
}
__device__ __forceinline__ void ldmatrix_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
template <int D_, int FMT_, int MT_>
struct Shape {
  static constexpr int D = D_, FMT = FMT_, MT = MT_;
  static constexpr bool Q8 = FMT != RSSM_BF16;
  static constexpr int ESZ = Q8 ? 1 : 2;
  static constexpr int kRows = 16 * MT;    // queries of a tile
  static constexpr int RB = D * ESZ;       // bytes of a cached head
  static constexpr int NC = RB / 16;       // and its 16-byte chunks
  static constexpr int NL = NC / 4;        // chunks a lane takes of a key
  static constexpr int QS = D * 2 + (Q8 ? 16 : 64);  // bytes between queries: a quarter of a warp's reads fall on distinct banks
  // blocks an SM: 8-bit codes are bound by instructions, and eight warps issue in half of the
  // cycles only (64 rows of 8192 tokens, one query token, e4m3, heads of 128: two blocks 227 us,
  // three 197, of 64: 195, 133); bf16 keys of 128 are bound by bytes, and two blocks of three
  // stages are what fits (three of two stages took 341 us where these took 332)
  static constexpr int kSm = MT == 1 && D * ESZ <= 128 ? 3 : 2;
  static constexpr int STAGES = Q8 && D < 256 ? 4 : 3;
  static constexpr int SB = 2 * kSlice * RB + (Q8 ? 2 * kSlice * 4 : 0);  // bytes of a stage: keys, values, their scales
  static constexpr int OS = D + (Q8 ? 16 : 8);      // floats between rows where the warps' sums meet
  static constexpr int kStageBytes = kWarps * STAGES * SB;
  static constexpr int kMeetBytes = kWarps * kRows * (OS + 2) * 4;
  static constexpr int kSmem = kRows * QS + (kStageBytes > kMeetBytes ? kStageBytes : kMeetBytes);
  static constexpr int kGrid = kSm * (kSmem + 2560) <= 227 * 1024 ? kSm : 2 * (kSmem + 2560) <= 227 * 1024 ? 2 : 1;
};

// where chunk `ch` of a slice's row lies: eight rows' equal chunks on distinct banks, and
// four neighbouring chunks of two rows too
template <int NC>
__device__ __forceinline__ uint32_t chunk_at(int row, int ch) {
  if constexpr (NC == 4) return row * 64 + ((ch ^ ((row >> 1) & 3)) << 4);
  return row * (NC * 16) + ((ch ^ (((row & 1) << 2) | ((row >> 1) & 3))) << 4);
}

template <typename S>
__global__ void __launch_bounds__(kThreads, S::kSm) attention_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int D = S::D, MT = S::MT, kRows = S::kRows, NL = S::NL, RB = S::RB, NC = S::NC, QS = S::QS, OS = S::OS;
  constexpr bool Q8 = S::Q8;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int sh_bad;
  __shared__ unsigned long long sh_mask[kTreeT];
  __shared__ float sh_qscale[kRows];
  __shared__ int sh_odd;  // values that are not finite among the piece's new tokens
  __shared__ __align__(16) float sh_v[kWarps][2][kSlice];  // of a slice's values' scales: logarithms, inverses
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, cc = lane & 3;
  const unsigned full = 0xffffffffu;
  uint8_t* const stages = smem + kRows * QS;
  const uint32_t q_at = smem_addr(smem), st_at = smem_addr(stages) + warp * S::STAGES * S::SB;
  pdl_wait();
  pdl_trigger();

  const Line line = cut_line<kRows, kTile, kThreads>(a, blockIdx.x, gridDim.x);
  __shared__ Joint sh_joint[2];
  int joints = 0;
  constexpr float kUnit = Q8 ? kShift8 : 1.0f;
  int b = line.b;
  long long base = line.base;
#pragma unroll 1
  for (long long u = line.lo; u < line.hi;) {
    const RowWork w = row_work<kRows, kTile>(a, b);
    const long long units = static_cast<long long>(w.tiles) * w.mtiles * a.c.heads;
    if (u >= base + units) {
      base += units;
      ++b;
      continue;
    }
    const long long at = u - base;
    const int seg = static_cast<int>(at / w.tiles), t0 = static_cast<int>(at - static_cast<long long>(seg) * w.tiles);
    const int t1 = static_cast<int>(min(static_cast<long long>(w.tiles), t0 + (line.hi - u)));
    const int mtile = seg / a.c.heads, head = seg - mtile * a.c.heads;
    const long long seg0 = u - t0;  // the segment's first unit
    u += t1 - t0;
    const int row0 = mtile * kRows, rows = min(kRows, w.s.count * a.group - row0);  // queries of this tile
    __syncthreads();  // the last piece's shared memory is free
    if (threadIdx.x == 0) sh_bad = sh_odd = 0;

    // ---- queries: bf16 as they are, or fp16 for 8-bit caches
    {
      constexpr int G = D / 8;  // lanes of a row
#pragma unroll 1
      for (int r = threadIdx.x / G; r < kRows; r += kThreads / G) {
        const int part = threadIdx.x % G;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows) {
          const int t = (row0 + r) / a.group, h = head * a.group + (row0 + r) - t * a.group;
          x = *reinterpret_cast<const uint4*>(a.q + (w.s.first + t) * a.q_stride + static_cast<long long>(h) * D + part * 8);
        }
        if constexpr (Q8) {
          float back;
          x = query_f16<G>(x, back);
          if (part == 0) sh_qscale[r] = a.scale2 * back;
        }
        *reinterpret_cast<uint4*>(smem + r * QS + part * 16) = x;
      }
    }
    if (a.parents && warp == 0 && w.len >= 0) {
      unsigned long long mask[2];
      const bool ok = tree_masks(a.parents + w.s.first, w.s.count, lane, mask);
      sh_mask[lane] = mask[0];
      sh_mask[lane + 32] = mask[1];
      if (!ok && lane == 0) {
        sh_bad = 1;
        set_error(a.c.err, RSSM_ERRBIT_TREE);
      }
    }
    __syncthreads();

    // ---- the warp's slices: 4 k + warp of the piece's, up to the last token that any of its queries sees
    const int last = (row0 + rows - 1) / a.group;  // the tile's last token
    const long long end = w.len < 0 || sh_bad ? 0 : static_cast<long long>(w.len) + (a.parents ? w.s.count : last + 1);
    // from here on there are tokens that not every query of the tile sees, or none
    const long long some = static_cast<long long>(w.len) + (a.parents ? 0 : row0 / a.group + 1);
    const int first = t0 * kWarps + warp;  // in slices of 16
    const int stop = static_cast<int>(min(static_cast<long long>(t1) * kWarps, (end + kSlice - 1) / kSlice));
    const int count = stop > first ? (stop - first + kWarps - 1) / kWarps : 0;
    const int* table = a.r.pages + b * a.r.pages_stride;
    const uint8_t* kbase = a.c.k + static_cast<long long>(head) * a.c.page_size * RB;
    const uint8_t* vbase = a.c.v + static_cast<long long>(head) * a.c.page_size * RB;
    unsigned missing = 0;  // per stage: the slice is in no page
    // of the next slice to ask for: its first token's place in its page, tokens from there to the last one seen
    const int page_step = kTile % a.c.page_size;
    int slot = static_cast<int>(static_cast<unsigned>(first) * kSlice % static_cast<unsigned>(a.c.page_size));
    int behind = static_cast<int>(end - static_cast<long long>(first) * kSlice);

    // pages of the 32 slices from a multiple of 32 on, a lane each, and of the 32 after them
    auto look_up = [&](int k) {
      const int i = k + lane;
      if (i >= count) return -1;
      return table[static_cast<unsigned>(first + i * kWarps) * kSlice / static_cast<unsigned>(a.c.page_size)];
    };
    int page_now = look_up(0), page_next = look_up(32);
    auto issue = [&](int k) {
      if (k < count) {
        if (k && (k & 31) == 0) {
          page_now = page_next;
          page_next = look_up(k + 32);
        }
        const int stage = k % S::STAGES;
        const int page = __shfl_sync(full, page_now, k & 31);
        const bool have = page >= 0 && page < a.c.pages;
        const int live = have ? min(kSlice, behind) : 0;
        missing = (missing & ~(1u << stage)) | (have ? 0u : 1u << stage);
        const uint32_t to = st_at + stage * S::SB;
        const long long pg = have ? page : 0;
        const uint8_t* ksrc = kbase + pg * a.c.k_page + static_cast<long long>(slot) * RB;
        const uint8_t* vsrc = vbase + pg * a.c.v_page + static_cast<long long>(slot) * RB;
        auto both = [&](auto all) {
#pragma unroll
          for (int x = 0; x < kSlice * NC / 32; ++x) {
            const int i = lane + 32 * x, r = i / NC, ch = i % NC;
            copy16(to + chunk_at<NC>(r, ch), ksrc + i * 16, all.value || r < live);
          }
#pragma unroll
          for (int x = 0; x < kSlice * NC / 32; ++x) {
            const int i = lane + 32 * x, r = i / NC, ch = i % NC;
            copy16(to + kSlice * RB + chunk_at<NC>(r, ch), vsrc + i * 16, all.value || r < live);
          }
        };
        if (Q8 && live == kSlice) both(std::true_type());  // (bf16 ones are not bound by instructions)
        else both(std::false_type());
        if constexpr (Q8) {
          const int r = lane & 15;
          const long long row = static_cast<long long>(head) * a.c.page_size + slot + r;
          copy4(to + 2 * kSlice * RB + lane * 4, lane < 16 ? a.c.ks + pg * a.c.ks_page + row : a.c.vs + pg * a.c.vs_page + row, r < live);
        }
        behind -= kTile;
        slot += page_step;
        if (slot >= a.c.page_size) slot -= a.c.page_size;
      }
      copy_commit();
    };

    float o[MT][D / 8][4];
    float m[MT][2], l[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
#pragma unroll
      for (int x = 0; x < D / 8; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][x][e] = 0.0f;
      m[i][0] = m[i][1] = -INFINITY;
      l[i][0] = l[i][1] = 0.0f;
    }

#pragma unroll
    for (int k = 0; k < S::STAGES - 1; ++k) issue(k);
#pragma unroll 1
    for (int k = 0; k < count; ++k) {
      copy_wait<S::STAGES - 2>();
      __syncwarp();
      const int stage = k % S::STAGES;
      const uint32_t ks = st_at + stage * S::SB, vs = ks + kSlice * RB;
      const int pos = (first + k * kWarps) * kSlice;
      if (missing >> stage & 1) {  // not seen
        if (lane == 0) set_error(a.c.err, RSSM_ERRBIT_PAGE);
        __syncwarp();
        issue(k + S::STAGES - 1);
        continue;
      }
      const bool edge = pos + kSlice > some;
      if constexpr (Q8) {
        // a lane's token: the logarithm (lanes 0 .. 15) or the inverse of its values' scale
        float y;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(y) : "r"(ks + 2 * kSlice * RB + (16 + (lane & 15)) * 4) : "memory");
        y = y < 7.7037197775489434e-34f ? 7.7037197775489434e-34f : y;  // 2^-110: a scale of 0 stands for zeros all the same
        // NaN: the weight is that, or 0 if not seen
        const float inverse = y == y ? rcp_fast(y) * kShift8 : 0.0f;
        sh_v[warp][lane >> 4][lane & 15] = lane < 16 ? __log2f(y) : inverse;
        __syncwarp();
      }

      // scores
      float s[MT][2][4];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][n][e] = 0.0f;
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const uint4 k0 = lds16(ks + chunk_at<NC>(g, cc + 4 * i)), k1 = lds16(ks + chunk_at<NC>(8 + g, cc + 4 * i));
        const uint32_t kw[2][4] = {{k0.x, k0.y, k0.z, k0.w}, {k1.x, k1.y, k1.z, k1.w}};
        if constexpr (Q8) {
          uint32_t bf[2][4][2];
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              codes_f16<S::FMT>(S::FMT == RSSM_I8 ? kw[n][j] ^ 0x80808080u : kw[n][j], bf[n][j][0], bf[n][j][1]);
            }
#pragma unroll
          for (int x = 0; x < MT; ++x) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t qa = q_at + (16 * x + g) * QS + (cc + 4 * i) * 32 + h * 16;
              const uint4 q0 = lds16(qa), q1 = lds16(qa + 8 * QS);
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                mma<true>(s[x][n], q0.x, q1.x, q0.y, q1.y, bf[n][2 * h][0], bf[n][2 * h][1]);
                mma<true>(s[x][n], q0.z, q1.z, q0.w, q1.w, bf[n][2 * h + 1][0], bf[n][2 * h + 1][1]);
              }
            }
          }
        } else {
#pragma unroll
          for (int x = 0; x < MT; ++x) {
            const uint32_t qa = q_at + (16 * x + g) * QS + (cc + 4 * i) * 16;
            const uint4 q0 = lds16(qa), q1 = lds16(qa + 8 * QS);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              mma<false>(s[x][n], q0.x, q1.x, q0.y, q1.y, kw[n][0], kw[n][1]);
              mma<false>(s[x][n], q0.z, q1.z, q0.w, q1.w, kw[n][2], kw[n][3]);
            }
          }
        }
      }

      // weights
      float kf[2][2], lv[2][2], iv[2][2];
      if constexpr (Q8) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float2 l2 = *reinterpret_cast<const float2*>(&sh_v[warp][0][8 * n + 2 * cc]), i2 = *reinterpret_cast<const float2*>(&sh_v[warp][1][8 * n + 2 * cc]);
          asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(kf[n][0]), "=f"(kf[n][1]) : "r"(ks + 2 * kSlice * RB + (8 * n + 2 * cc) * 4) : "memory");
          lv[n][0] = l2.x, lv[n][1] = l2.y;
          iv[n][0] = i2.x, iv[n][1] = i2.y;
        }
      }
      uint32_t pa[MT][4];
#pragma unroll
      for (int x = 0; x < MT; ++x)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = 16 * x + g + 8 * h;
          float v[4];
          const float rf = Q8 ? sh_qscale[r] : a.scale2;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float y = s[x][n][2 * h + e] * rf;
              if constexpr (Q8) y = y * kf[n][e] + lv[n][e];
              v[2 * n + e] = y;
            }
          if (edge) {
            const int t = (row0 + r) / a.group;  // rows past the tile's last see what it sees
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int j = pos + 8 * n + 2 * cc + e - w.len;  // which new token this is
                const bool y = j < 0 || (j < w.s.count && (a.parents ? t < kTreeT && (sh_mask[t] >> (j & 63) & 1) : j <= t));
                if (!y) v[2 * n + e] = -INFINITY;
              }
          }
          float top = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
          top = fmaxf(top, __shfl_xor_sync(full, top, 1));
          top = fmaxf(top, __shfl_xor_sync(full, top, 2));
          if (__any_sync(full, top > m[x][h] + kLazy)) {
            const float now = fmaxf(m[x][h], top);
            const float alpha = now == -INFINITY ? 1.0f : exp2_fast(m[x][h] - now);
            m[x][h] = now;
            l[x][h] *= alpha;
#pragma unroll
            for (int y = 0; y < D / 8; ++y) {
              o[x][y][2 * h] *= alpha;
              o[x][y][2 * h + 1] *= alpha;
            }
          }
          const float ref = m[x][h] == -INFINITY ? 0.0f : m[x][h];  // nothing seen yet
          float p[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) p[y] = exp2_fast(v[y] - (Q8 ? ref - kShift : ref));
          if constexpr (Q8) {
#pragma unroll
            for (int y = 0; y < 4; ++y) l[x][h] += p[y] * iv[y >> 1][y & 1];
            pa[x][h] = f16_pair(p[0], p[1]);
            pa[x][2 + h] = f16_pair(p[2], p[3]);
          } else {
            l[x][h] += (p[0] + p[1]) + (p[2] + p[3]);
            pa[x][h] = bf16_pair(p[0], p[1]);
            pa[x][2 + h] = bf16_pair(p[2], p[3]);
          }
        }

      // values that are not finite must not meet the weight 0 of a query that does not see them: among the new
      // tokens they are taken out here and added at the piece's end, to those that do
      if constexpr (!Q8) {
        if (edge) {
          bool odd = false;
#pragma unroll
          for (int x = 0; x < kSlice * NC / 32; ++x) {
            const int i = lane + 32 * x;
            uint8_t* p = stages + (vs - smem_addr(stages)) + chunk_at<NC>(i / NC, i % NC);
            uint4 y = *reinterpret_cast<uint4*>(p);
            const bool mine = take_out_odd(y);
            if (mine) *reinterpret_cast<uint4*>(p) = y;
            odd = odd || mine;
          }
          if (__any_sync(full, odd) && lane == 0) sh_odd = 1;
          __syncwarp();
        }
      }

      // sums
      const int vr = lane & 15;  // the row of the slice whose chunk this lane names to the transposing loads
#pragma unroll
      for (int y = 0; y < NC / 2; ++y) {
        uint32_t f[4];  // tokens 0-7, 8-15 of chunk 2 y, and of chunk 2 y + 1
        ldmatrix_t(f, vs + chunk_at<NC>(vr, 2 * y + (lane >> 4)));
        if constexpr (Q8) {
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            uint32_t e0, e1, d0, d1;  // even and odd dimensions: bytes 0 and 2, 1 and 3
            codes_f16<S::FMT>(__byte_perm(f[2 * z], 0u, 0x3120u) ^ (S::FMT == RSSM_I8 ? 0x80808080u : 0u), e0, d0);
            codes_f16<S::FMT>(__byte_perm(f[2 * z + 1], 0u, 0x3120u) ^ (S::FMT == RSSM_I8 ? 0x80808080u : 0u), e1, d1);
#pragma unroll
            for (int x = 0; x < MT; ++x) {
              mma<true>(o[x][4 * y + 2 * z], pa[x][0], pa[x][1], pa[x][2], pa[x][3], e0, e1);
              mma<true>(o[x][4 * y + 2 * z + 1], pa[x][0], pa[x][1], pa[x][2], pa[x][3], d0, d1);
            }
          }
        } else {
#pragma unroll
          for (int z = 0; z < 2; ++z)
#pragma unroll
            for (int x = 0; x < MT; ++x) mma<false>(o[x][2 * y + z], pa[x][0], pa[x][1], pa[x][2], pa[x][3], f[2 * z], f[2 * z + 1]);
        }
      }
      __syncwarp();
      issue(k + S::STAGES - 1);
    }
    copy_wait<0>();
#pragma unroll
    for (int x = 0; x < MT; ++x)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[x][h] += __shfl_xor_sync(full, l[x][h], 1);
        l[x][h] += __shfl_xor_sync(full, l[x][h], 2);
      }

    // ---- the warps' sums meet
    __syncthreads();
    float* const meet = reinterpret_cast<float*>(stages);
    float* const meet_m = meet + kWarps * kRows * OS;
    float* const meet_l = meet_m + kWarps * kRows;
#pragma unroll
    for (int x = 0; x < MT; ++x)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 16 * x + g + 8 * h;
        float* to = meet + (warp * kRows + r) * OS;
        if constexpr (Q8) {
#pragma unroll
          for (int y = 0; y < D / 16; ++y)
            *reinterpret_cast<float4*>(to + 16 * y + 4 * cc) = make_float4(o[x][2 * y][2 * h], o[x][2 * y + 1][2 * h], o[x][2 * y][2 * h + 1], o[x][2 * y + 1][2 * h + 1]);
        } else {
#pragma unroll
          for (int y = 0; y < D / 8; ++y) *reinterpret_cast<float2*>(to + 8 * y + 2 * cc) = make_float2(o[x][y][2 * h], o[x][y][2 * h + 1]);
        }
        if (cc == 0) {
          meet_m[warp * kRows + r] = m[x][h];
          meet_l[warp * kRows + r] = l[x][h];
        }
      }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == w.tiles;
    float* const left = piece_place<kRows, D>(a, blockIdx.x, t0 == 0);
    constexpr int D4 = D / 4;
#pragma unroll 1
    for (int i = threadIdx.x; i < rows * D4; i += kThreads) {
      const int r = i / D4, x4 = (i - r * D4) * 4;
      float top = -INFINITY;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) top = fmaxf(top, meet_m[x * kRows + r]);
      const float ref = top == -INFINITY ? 0.0f : top;
      float y[4] = {0.0f, 0.0f, 0.0f, 0.0f}, z = 0.0f;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        const float f = exp2_fast(meet_m[x * kRows + r] - ref);
        const float4 v = *reinterpret_cast<const float4*>(meet + (x * kRows + r) * OS + x4);
        y[0] += f * v.x;
        y[1] += f * v.y;
        y[2] += f * v.z;
        y[3] += f * v.w;
        z += f * meet_l[x * kRows + r];
      }
      if constexpr (!Q8) {
        if (sh_odd) {
          const int t = (row0 + r) / a.group;
          const float4 z4 = add_odd4(a, w.len, table, vbase, RB, max(static_cast<long long>(t0) * kTile, some / kSlice * kSlice),
                                     min(static_cast<long long>(t1) * kTile, end), t, a.parents ? sh_mask[t] : 0ull, x4, make_float4(y[0], y[1], y[2], y[3]));
          y[0] = z4.x, y[1] = z4.y, y[2] = z4.z, y[3] = z4.w;
        }
      }
      if (whole) {
        write_out(a, w.s.first, head, row0 + r, D, x4, y, z == 0.0f ? 0.0f : kUnit / z);
      } else {
        __stcg(reinterpret_cast<float4*>(left + r * D + x4), make_float4(y[0], y[1], y[2], y[3]));
        if (x4 == 0) {
          __stcg(left + kRows * D + r, top);
          __stcg(left + kRows * D + kRows + r, z);
        }
      }
    }
    if (whole) continue;

    if (threadIdx.x == 0) sh_joint[joints & 1] = Joint{w.s.first, seg0, w.tiles, head, row0, rows};
    ++joints;
  }
  __syncthreads();
  if (a.apart) return;
  for (int i = 0; i < joints; ++i) join_pieces<kRows, D, kThreads, 8>(a, sh_joint[i], line.share, kUnit);
}

template <typename S>
cudaError_t run(const AttnArgs& args, int sms, cudaStream_t st) {
  static bool ready[64] = {};  // per device: the attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(attention_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev] = true;
  }
  AttnArgs a = args;
  const int grid = S::kGrid * sms;
  // up to 8 queries a head the joins are short, and a launch costs as much (one row of 8192 int8 tokens,
  // heads of 128: 4 queries 20 us, 25 apart; 8 queries 25, 26 apart; 16 34, 32 apart; 32 81, 40 apart)
  a.apart = grid > 1 && static_cast<long long>(a.r.T) * a.group > 8;
  e = launch_pdl(attention_kernel<S>, dim3(grid), dim3(kThreads), S::kSmem, st, a);
  if (e != cudaSuccess || !a.apart) return e;
  return launch_join<S::kRows, kTile, S::D>(a, grid, S::Q8 ? kShift8 : 1.0f, st);
}

template <int D, int FMT>
cudaError_t run_rows(const AttnArgs& a, int sms, cudaStream_t st) {
  if constexpr (D < 256) {
    if (static_cast<long long>(a.r.T) * a.group > 16) return run<Shape<D, FMT, 2>>(a, sms, st);
  }
  return run<Shape<D, FMT, 1>>(a, sms, st);
}
template <int D>
cudaError_t run_format(const AttnArgs& a, int sms, cudaStream_t st) {
  return a.c.fmt == RSSM_BF16 ? run_rows<D, RSSM_BF16>(a, sms, st)
         : a.c.fmt == RSSM_I8 ? run_rows<D, RSSM_I8>(a, sms, st)
                              : run_rows<D, RSSM_E4M3>(a, sms, st);
}

constexpr size_t kHead = 8192;  // bytes of tickets before the pieces
size_t scratch_need(const KvView& c, int sms) {
  const int rows = c.dim == 256 ? 16 : 32;
  const size_t narrow = static_cast<size_t>(kBlocks) * sms * 2 * rows * (c.dim + 2) * sizeof(float), wide = wide_scratch(c, sms);
  return kHead + (narrow > wide ? narrow : wide);
}
static_assert(kBlocks * kMaxSms * sizeof(unsigned) <= kHead, "a ticket a block");

}  // namespace
}  // namespace rssm

using namespace rssm;

extern "C" size_t rssm_attention_scratch_bytes(const rssm_kv_cache* cache, int32_t nqheads) {
  KvView c;
  if (kv_view(cache, 0, &c) != RSSM_OK || nqheads < 1 || nqheads % c.heads) return 0;
  const int sms = num_sms();
  const int n = sms > 0 && sms < kMaxSms ? sms : kMaxSms;
  return scratch_need(c, n);
}

extern "C" rssm_status rssm_tree_attention(const rssm_kv_cache* cache, int32_t layer, const void* q, int64_t q_stride, int32_t nqheads, float scale,
                                           const int32_t* pages, int64_t pages_stride, int32_t max_pages, const int32_t* lengths,
                                           const int32_t* parents, const int32_t* cu_seqlens, int32_t batch, int32_t T, int64_t tokens, void* out,
                                           int64_t out_stride, void* scratch, size_t scratch_bytes, void* stream) {
  AttnArgs a;
  rssm_status st = kv_view(cache, layer, &a.c);
  if (st == RSSM_OK) st = kv_rows(pages, pages_stride, max_pages, lengths, cu_seqlens, batch, T, tokens, &a.r);
  if (st != RSSM_OK) return st;
  if (nqheads < 1 || nqheads % a.c.heads) return RSSM_ERR_INVALID_ARGUMENT;
  const auto al = [](const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
  const int64_t dense = static_cast<int64_t>(nqheads) * a.c.dim;
  if (tokens > 0 && (!q || !out)) return RSSM_ERR_INVALID_ARGUMENT;
  if (!al(q, 16) || !al(out, 16) || q_stride < dense || out_stride < dense || q_stride % 8 || out_stride % 8) return RSSM_ERR_INVALID_ARGUMENT;
  if (!al(parents, 4) || !al(scratch, 16) || !(scale == scale)) return RSSM_ERR_INVALID_ARGUMENT;
  if (parents && T > kTreeT) return RSSM_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(T) * (nqheads / a.c.heads) > INT32_MAX / 2) return RSSM_ERR_UNSUPPORTED;
  if (batch > 0 && !lengths) return RSSM_ERR_INVALID_ARGUMENT;
  if (batch == 0 || tokens == 0) return RSSM_OK;
  const int sms = num_sms();
  if (sms == 0) return RSSM_ERR_CUDA;
  if (sms > kMaxSms) return RSSM_ERR_UNSUPPORTED;
  if (!scratch) return RSSM_ERR_INVALID_ARGUMENT;
  if (scratch_bytes < scratch_need(a.c, sms)) return RSSM_ERR_SCRATCH_TOO_SMALL;
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.out = static_cast<uint16_t*>(out);
  a.out_stride = out_stride;
  a.parents = parents;
  a.group = nqheads / a.c.heads;
  a.scale2 = scale * 1.4426950408889634f;
  a.ticket = static_cast<unsigned*>(scratch);
  a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + kHead);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  a.whole = 0;
  const cudaError_t e = wide_takes(a.c, static_cast<int64_t>(T) * a.group) ? run_wide(a, sms, s)
                        : a.c.dim == 64 ? run_format<64>(a, sms, s) : a.c.dim == 128 ? run_format<128>(a, sms, s) : run_format<256>(a, sms, s);
  return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}
