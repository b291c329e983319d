// rssm_kv.cuh -- the paged cache of keys and values: its device view, the
// layout of a page, and helpers that its kernels share.
#pragma once

#include "rssm_device.cuh"
#include "rssm_host.h"

namespace rssm {

constexpr int kTreeT = 64;  // most tokens of a tree: a path is a bit mask of one 64-bit word

// One layer of the cache (all layers for the acceptance).  Addresses are bytes.
struct KvView {
  uint8_t *k, *v;
  long long k_page, v_page;    // bytes between pages
  long long k_layer, v_layer;  // bytes between layers
  float *ks, *vs;              // null for a bf16 cache
  long long ks_page, vs_page, ks_layer, vs_layer;  // floats
  int pages, layers, heads, dim, page_size, fmt, esz;
  unsigned* err;
};

// A row's pages and what a call knows of the rows.
struct KvRows {
  const int* pages;
  long long pages_stride;
  int max_pages;
  const int* lengths;  // or null: 0
  const int* cu;       // or null: T tokens a row
  int batch, T;
  long long tokens;
};

// Token bounds of row b; count < 0: bad bounds.
struct RowSpan {
  long long first;
  int count;
};
__device__ __forceinline__ RowSpan row_span(const KvRows& r, int b) {
  RowSpan s;
  if (r.cu) {
    const int lo = r.cu[b], hi = r.cu[b + 1];
    const long long n = static_cast<long long>(hi) - lo;
    s.first = lo;
    s.count = n < 0 || n > r.T || lo < 0 || hi > r.tokens ? -1 : static_cast<int>(n);
  } else {
    s.first = static_cast<long long>(b) * r.T;
    s.count = r.T;
  }
  return s;
}

// The row that token `tok` of the packed ones lies in, by one warp: -1 behind the
// last.  Each step looks at 32 of the rows' ends at a time, so 1024 rows take two
// round trips to memory instead of ten.
__device__ __forceinline__ int find_row(const KvRows& r, long long tok, int lane) {
  if (!r.cu) {
    const int b = static_cast<int>(tok) / r.T;
    return b < r.batch ? b : -1;
  }
  int lo = 0, n = r.batch;  // the row is among lo .. lo + n - 1, or there is none
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int at = lo + min(n, (lane + 1) * step) - 1;  // the last row of this lane's part
    const unsigned past = __ballot_sync(0xffffffffu, r.cu[at + 1] > tok);
    if (!past) return -1;
    const int part = __ffs(past) - 1;
    const int first = part * step;
    if (step == 1) return tok >= r.cu[lo + first] ? lo + first : -1;
    lo += first;
    n = min(step, n - first);
  }
  return -1;
}

// the ancestors of a row's tokens (each its own too) as bit masks, by one warp: lane
// l has tokens l and l + 32 of `n`.  A token's mask takes in its pointer's, and the
// pointer jumps to its pointer's own: six rounds reach 64 steps up.  Returns whether
// every parent is before its token.
__device__ __forceinline__ bool tree_masks(const int* parents, int n, int lane, unsigned long long (&mask)[2]) {
  const unsigned full = 0xffffffffu;
  int up[2];
  bool ok = true;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = lane + 32 * i;
    up[i] = t < n ? parents[t] : -1;
    ok = ok && up[i] >= -1 && up[i] < t;
    mask[i] = 1ull << t;
  }
  if (!__all_sync(full, ok)) return false;
#pragma unroll 1
  for (int round = 0; round < 6; ++round) {
    unsigned long long add[2];
    int next[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int src = up[i] & 31;
      const unsigned long long m0 = __shfl_sync(full, mask[0], src), m1 = __shfl_sync(full, mask[1], src);
      const int u0 = __shfl_sync(full, up[0], src), u1 = __shfl_sync(full, up[1], src);
      add[i] = up[i] < 0 ? 0ull : up[i] < 32 ? m0 : m1;
      next[i] = up[i] < 0 ? -1 : up[i] < 32 ? u0 : u1;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mask[i] |= add[i];
      up[i] = next[i];
    }
    if (!__any_sync(full, up[0] >= 0 || up[1] >= 0)) break;
  }
  return true;
}

// host side
rssm_status kv_view(const rssm_kv_cache* c, int layer, KvView* out);
rssm_status kv_rows(const int32_t* pages, int64_t pages_stride, int32_t max_pages, const int32_t* lengths,
                    const int32_t* cu, int32_t batch, int32_t T, int64_t tokens, KvRows* out);

}  // namespace rssm
