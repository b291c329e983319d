// rssm_delta_prefill.cu -- the gated delta rule over whole prompts.
#include "rssm_delta.cuh"

namespace rssm {
namespace {

struct DeltaPrefillArgs {
  DeltaCacheView c;
  DeltaTokens tk;
  const int* slot_idx;
  const int* cu;
  const int* initial;
  int batch, tiles;
  long long tokens;
};

constexpr int kScanWarps = 4;

// One warp per 16 value rows of a (prompt, value head) walks the prompt in
// blocks of 8 tokens with its part of S in registers.
template <int DK>
__global__ void __launch_bounds__(kScanWarps * 32) delta_scan_kernel(const DeltaPrefillArgs a) {
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = blockIdx.x % a.tiles;
  const int h = (blockIdx.x / a.tiles) % a.c.Hv;
  const int b = blockIdx.x / a.tiles / a.c.Hv;
  const int r0 = (tile * kScanWarps + warp) * 16;
  if (r0 >= a.c.dv) return;
  const int s = a.slot_idx[b];
  const long long tok0 = a.cu[b];
  const int n = a.cu[b + 1] - a.cu[b];
  if (n < 0 || tok0 < 0 || tok0 + n > a.tokens) {
    if (h == 0 && r0 == 0 && lane == 0) set_error(a.c.err, RSSM_ERRBIT_SEQLEN);
    return;
  }
  const int dv = a.c.dv, Hv = a.c.Hv, hk = h / a.c.rep;
  const long long ostride = static_cast<long long>(Hv) * dv;
  uint16_t* out = a.tk.out + tok0 * ostride + h * dv + r0;
  DeltaBlock<DK> blk;
  float o[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
  if (s <= 0 || s >= a.c.S) {
    for (int t = 0; t < n; t += kDeltaT) blk.store_out(o, out + t * ostride, ostride, min(n - t, kDeltaT), lane);
    return;
  }
  DeltaState<DK> S;
  const long long head = s * a.c.state_stride + (static_cast<long long>(h) * dv + r0) * DK;
  if (a.initial && a.initial[b] != 0)
    S.load(a.c.state, head, a.c.dtype, lane);
  else
    S.zero();
  for (int t = 0; t < n; t += kDeltaT) {
    const int T = min(n - t, kDeltaT);
    blk.load(a.tk, tok0 + t, T, hk, h, Hv, lane);
    blk.prepare(a.tk, lane);
    blk.solve(S, a.tk.v + (tok0 + t) * a.tk.v_stride + h * dv + r0, a.tk.v_stride, T, lane, o);
    blk.store_out(o, out + t * ostride, ostride, T, lane);
    const float end = __shfl_sync(0xffffffffu, blk.c, (T - 1) * 4);
    S.decay(expf(end));
    for (int j = 0; j < T; ++j) {
      const float2 u = blk.rows_of(j, lane);
      const float e = expf(end - __shfl_sync(0xffffffffu, blk.c, j * 4)) * __shfl_sync(0xffffffffu, blk.r, j * 4);
      S.add(e * u.x, e * u.y, a.tk.k + (tok0 + t + j) * a.tk.k_stride + hk * DK, lane);
    }
  }
  S.store(a.c.state, head, a.c.dtype, lane);
  if (h == 0 && r0 == 0 && lane == 0) reinterpret_cast<int2*>(a.c.pend)[s] = make_int2(0, 0);
}

bool al(const void* p, unsigned n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace rssm

using namespace rssm;

extern "C" size_t rssm_delta_scratch_bytes(const rssm_delta_cache* cache, int32_t batch, int64_t tokens) {
  DeltaCacheView c;
  rssm_status st;
  if (!delta_view(cache, &c, &st) || batch < 0 || tokens < 0) return 0;
  return align_up(static_cast<size_t>(batch) * sizeof(unsigned) + 1, 256);
}

extern "C" rssm_status rssm_delta_prefill(const rssm_delta_cache* cache, const void* q, int64_t q_stride, const void* k,
                                          int64_t k_stride, const void* v, int64_t v_stride, const float* g,
                                          const float* beta, float scale, int32_t l2norm, const int32_t* slot_idx,
                                          const int32_t* cu_seqlens, const int32_t* initial, int32_t batch,
                                          int64_t tokens, void* out, void* scratch, size_t scratch_bytes, void* stream) {
  DeltaPrefillArgs a = {};
  rssm_status st;
  if (!delta_view(cache, &a.c, &st)) return st;
  if (batch < 0 || tokens < 0 || tokens > 0x7fffffffll) return RSSM_ERR_INVALID_ARGUMENT;
  if (batch == 0) return RSSM_OK;
  if (!al(slot_idx, 4) || !al(cu_seqlens, 4) || (initial && !al(initial, 4)) || !al(scratch, 16)) return RSSM_ERR_INVALID_ARGUMENT;
  if (tokens > 0) {
    st = delta_tokens(a.c, cache->dkey, q, k, v, q_stride, k_stride, v_stride, g, beta, scale, l2norm, out, &a.tk);
    if (st != RSSM_OK) return st;
  }
  if (scratch_bytes < rssm_delta_scratch_bytes(cache, batch, tokens)) return RSSM_ERR_SCRATCH_TOO_SMALL;
  a.slot_idx = slot_idx;
  a.cu = cu_seqlens;
  a.initial = initial;
  a.batch = batch;
  a.tokens = tokens;
  a.tiles = (a.c.dv + kScanWarps * 16 - 1) / (kScanWarps * 16);
  const long long blocks = static_cast<long long>(batch) * a.c.Hv * a.tiles;
  if (blocks > 0x7fffffffll) return RSSM_ERR_UNSUPPORTED;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->dkey == 128
                            ? launch_pdl(delta_scan_kernel<128>, dim3(static_cast<unsigned>(blocks)), dim3(kScanWarps * 32), 0, cs, a)
                            : launch_pdl(delta_scan_kernel<64>, dim3(static_cast<unsigned>(blocks)), dim3(kScanWarps * 32), 0, cs, a);
  return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}
