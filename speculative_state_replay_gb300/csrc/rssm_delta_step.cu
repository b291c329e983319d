// rssm_delta_step.cu -- the gated delta rule's decode step over drafted
// tokens, and the checks the delta rule's calls share.
#include "rssm_delta.cuh"

namespace rssm {
namespace {

struct DeltaStepArgs {
  DeltaCacheView c;
  DeltaTokens tk;
  const int* slot_idx;
  const int* accepted;
  const int* cu;
  int batch, T;
  long long tokens;
  int tiles;         // blocks per (row, value head)
  unsigned* ticket;  // scratch [batch]: blocks that have read the row's `pend` (zero between calls)
};

constexpr int kStepWarps = 4;
constexpr int kStepRows = kStepWarps * 16;  // value rows of a block

// One warp per 16 value rows of a (row, value head): reads its part of S once,
// adds the accepted drafts of the step before, writes it back if there were
// any, and forms the new drafts' outputs and corrections from registers.  The
// block's loads go out in three rounds -- the row's scalars; the state, the new
// tokens and `pend`; the waiting drafts -- and only the first two are waited for
// one after another: the state's, the longest, covers the third.
template <int DK>
__global__ void __launch_bounds__(kStepWarps * 32, 4) delta_step_kernel(const DeltaStepArgs a) {
  __shared__ int sh[2];
  __shared__ __align__(16) uint8_t s_k[kDeltaT * kTokenRow<DK>], s_q[kDeltaT * kTokenRow<DK>];
  __shared__ __align__(16) float s_p[kDeltaT * DK], s_w[kDeltaT * kStepRows], s_c[kDeltaT];  // the waiting drafts
  constexpr int CH = DK / 8;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, m = lane >> 2, cc = lane & 3;
  const int tile = blockIdx.x % a.tiles;
  const int h = (blockIdx.x / a.tiles) % a.c.Hv;
  const int b = blockIdx.x / a.tiles / a.c.Hv;
  const int s = a.slot_idx[b];
  const long long tok0 = a.cu ? a.cu[b] : static_cast<long long>(b) * a.T;
  const int n = a.cu ? a.cu[b + 1] - a.cu[b] : a.T;
  const int acc = a.accepted ? a.accepted[b] : 0;
  if (n < 0 || n > a.T || tok0 < 0 || tok0 + n > a.tokens) {  // the row's tokens are not known: nothing to write
    if (tid == 0 && blockIdx.x % (a.tiles * a.c.Hv) == 0) set_error(a.c.err, RSSM_ERRBIT_SEQLEN);
    return;
  }
  const int dv = a.c.dv, Hv = a.c.Hv, np = a.c.np, hk = h / a.c.rep;
  const int r0 = tile * kStepRows + warp * 16;
  const bool mine = r0 < dv;
  const long long ostride = static_cast<long long>(Hv) * dv;
  uint16_t* out = a.tk.out + tok0 * ostride + h * dv + r0;
  DeltaBlock<DK> blk;
  float o[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
  if (s <= 0 || s >= a.c.S) {
    if (mine) blk.store_out(o, out, ostride, n, lane);
    return;
  }
  DeltaState<DK> S;
  const long long head = s * a.c.state_stride + (static_cast<long long>(h) * dv + r0) * DK;
  if (mine) S.load(a.c.state, head, a.c.dtype, lane);
  for (int i = tid; i < n * CH; i += kStepWarps * 32) {
    const int t = i / CH, ch = i % CH;
    cp_async16(s_k + t * kTokenRow<DK> + ch * 16, a.tk.k + (tok0 + t) * a.tk.k_stride + hk * DK + ch * 8);
    cp_async16(s_q + t * kTokenRow<DK> + ch * 16, a.tk.q + (tok0 + t) * a.tk.q_stride + hk * DK + ch * 8);
  }
  float g = 0.0f, beta = 0.0f;
  uint32_t vw[2] = {0u, 0u};
  if (mine && m < n) {
    g = fmaxf(a.tk.g[(tok0 + m) * Hv + h], kMinLog);
    beta = a.tk.beta[(tok0 + m) * Hv + h];
    const uint16_t* v = a.tk.v + (tok0 + m) * a.tk.v_stride + h * dv + r0 + 2 * cc;
    vw[0] = *reinterpret_cast<const uint32_t*>(v);
    vw[1] = *reinterpret_cast<const uint32_t*>(v + 8);
  }
  if (tid == 0) {
    const int2 p = __ldcg(reinterpret_cast<const int2*>(a.c.pend) + s);
    sh[0] = p.x;
    sh[1] = p.y;
  }
  __syncthreads();
  const int side = sh[0] & 1;
  const bool ok = acc >= 0 && acc <= sh[1];
  // every block of the row takes a ticket once it has read (side, count); the
  // last one knows that all have, and turns the sides
  if (tid == 0) {
    __threadfence();
    const unsigned blocks = static_cast<unsigned>(a.tiles * Hv);
    if (atomicInc(a.ticket + b, blocks - 1u) == blocks - 1u) {
      if (ok)
        reinterpret_cast<int2*>(a.c.pend)[s] = make_int2(side ^ 1, n);
      else
        set_error(a.c.err, RSSM_ERRBIT_ACCEPT);
    }
  }
  if (!ok) {
    cp_async_wait_all();
    if (mine) blk.store_out(o, out, ostride, n, lane);
    return;
  }
  if (acc > 0) {
    const float* pc = a.c.pend_c + s * a.c.pend_c_stride + (static_cast<long long>(side) * Hv + h) * np;
    const float* pw = a.c.pend_w + s * a.c.pend_w_stride + (static_cast<long long>(side) * Hv + h) * np * dv + tile * kStepRows;
    const uint16_t* pk = a.c.pend_k + s * a.c.pend_k_stride + (static_cast<long long>(side) * a.c.Hk + hk) * np * DK;
    if (tid < acc) cp_async4(s_c + tid, pc + tid);
    for (int i = tid; i < acc * (kStepRows / 4); i += kStepWarps * 32) {
      const int j = i / (kStepRows / 4), r = i % (kStepRows / 4) * 4;
      if (tile * kStepRows + r < dv) cp_async16(s_w + j * kStepRows + r, pw + static_cast<long long>(j) * dv + r);
    }
    for (int i = tid; i < acc * CH; i += kStepWarps * 32) {
      const uint4 x = *reinterpret_cast<const uint4*>(pk + i * 8);
      float4* to = reinterpret_cast<float4*>(s_p + i * 8);
      to[0] = make_float4(bf16lo(x.x), bf16hi(x.x), bf16lo(x.y), bf16hi(x.y));
      to[1] = make_float4(bf16lo(x.z), bf16hi(x.z), bf16lo(x.w), bf16hi(x.w));
    }
  }
  cp_async_wait_all();
  __syncthreads();
  if (!mine) return;
  if (acc > 0) {
    const float end = s_c[acc - 1];
    S.decay(expf(end));
    for (int j = 0; j < acc; ++j) {
      const float e = expf(end - s_c[j]);
      S.add(e * s_w[j * kStepRows + warp * 16 + m], e * s_w[j * kStepRows + warp * 16 + m + 8], s_p + j * DK, lane);
    }
    S.store(a.c.state, head, a.c.dtype, lane);
  }
  if (n == 0) return;
  blk.load(s_k, s_q, n, lane);
  blk.prepare(a.tk, g, beta, lane);
  blk.solve(S, vw, n, lane, o);
  blk.store_out(o, out, ostride, n, lane);
  // the new drafts wait in the other half
  if (m < n) {
    const int to = side ^ 1;
    float* pw = a.c.pend_w + s * a.c.pend_w_stride + ((static_cast<long long>(to) * Hv + h) * np + m) * dv + r0 + 2 * cc;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<float2*>(pw + 8 * i) = make_float2(blk.u[i][0] * blk.r, blk.u[i][1] * blk.r);
    if (r0 == 0 && cc == 0) a.c.pend_c[s * a.c.pend_c_stride + (static_cast<long long>(to) * Hv + h) * np + m] = blk.c;
    if (r0 == 0 && h % a.c.rep == 0) {
      uint16_t* pk = a.c.pend_k + s * a.c.pend_k_stride + ((static_cast<long long>(to) * a.c.Hk + hk) * np + m) * DK + 4 * cc;
#pragma unroll
      for (int x = 0; x < DK / 16; ++x) *reinterpret_cast<uint2*>(pk + 16 * x) = make_uint2(blk.a[x][0], blk.a[x][2]);
    }
  }
}

bool al(const void* p, unsigned n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

bool delta_view(const rssm_delta_cache* c, DeltaCacheView* o, rssm_status* st) {
  *st = RSSM_ERR_INVALID_ARGUMENT;
  if (!c || c->num_slots < 1 || c->nkheads < 1 || c->nvheads < 1 || c->nvheads % c->nkheads) return false;
  if (c->dvalue < 1 || c->npredicted < 1) return false;
  if (c->state_dtype != RSSM_F32 && c->state_dtype != RSSM_BF16) return false;
  if ((c->dkey != 64 && c->dkey != 128) || c->dvalue % 16 || c->dvalue > 1024 || c->npredicted > kDeltaT) {
    *st = RSSM_ERR_UNSUPPORTED;
    return false;
  }
  if (!al(c->state, 16) || !al(c->pend_k, 16) || !al(c->pend_w, 16) || !al(c->pend_c, 4) || !al(c->pend, 8) || !al(c->error_word, 4))
    return false;
  const int64_t esz = c->state_dtype == RSSM_F32 ? 4 : 2;
  const int64_t kl = static_cast<int64_t>(2) * c->nkheads * c->npredicted * c->dkey;
  const int64_t cl = static_cast<int64_t>(2) * c->nvheads * c->npredicted;
  if (c->state_slot_stride < static_cast<int64_t>(c->nvheads) * c->dvalue * c->dkey || c->pend_k_slot_stride < kl ||
      c->pend_w_slot_stride < cl * c->dvalue || c->pend_c_slot_stride < cl)
    return false;
  if (c->state_slot_stride * esz % 16 || c->pend_k_slot_stride % 8 || c->pend_w_slot_stride % 4) return false;
  o->S = c->num_slots;
  o->Hk = c->nkheads;
  o->Hv = c->nvheads;
  o->rep = c->nvheads / c->nkheads;
  o->dv = c->dvalue;
  o->np = c->npredicted;
  o->dtype = c->state_dtype;
  o->state = c->state;
  o->state_stride = c->state_slot_stride;
  o->pend_k = static_cast<uint16_t*>(c->pend_k);
  o->pend_k_stride = c->pend_k_slot_stride;
  o->pend_w = c->pend_w;
  o->pend_w_stride = c->pend_w_slot_stride;
  o->pend_c = c->pend_c;
  o->pend_c_stride = c->pend_c_slot_stride;
  o->pend = c->pend;
  o->err = c->error_word;
  *st = RSSM_OK;
  return true;
}

rssm_status delta_tokens(const DeltaCacheView& c, int dk, const void* q, const void* k, const void* v, int64_t q_stride,
                         int64_t k_stride, int64_t v_stride, const float* g, const float* beta, float scale, int l2norm,
                         void* out, DeltaTokens* tk) {
  if (!al(q, 16) || !al(k, 16) || !al(v, 16) || !al(out, 16) || !al(g, 4) || !al(beta, 4)) return RSSM_ERR_INVALID_ARGUMENT;
  if (q_stride < static_cast<int64_t>(c.Hk) * dk || k_stride < static_cast<int64_t>(c.Hk) * dk ||
      v_stride < static_cast<int64_t>(c.Hv) * c.dv || q_stride % 8 || k_stride % 8 || v_stride % 8)
    return RSSM_ERR_INVALID_ARGUMENT;
  if (l2norm != 0 && l2norm != 1) return RSSM_ERR_INVALID_ARGUMENT;
  tk->q = static_cast<const uint16_t*>(q);
  tk->k = static_cast<const uint16_t*>(k);
  tk->v = static_cast<const uint16_t*>(v);
  tk->q_stride = q_stride;
  tk->k_stride = k_stride;
  tk->v_stride = v_stride;
  tk->g = g;
  tk->beta = beta;
  tk->out = static_cast<uint16_t*>(out);
  tk->scale = scale;
  tk->l2norm = l2norm;
  return RSSM_OK;
}

}  // namespace rssm

using namespace rssm;

extern "C" rssm_status rssm_delta_step(const rssm_delta_cache* cache, const void* q, int64_t q_stride, const void* k,
                                       int64_t k_stride, const void* v, int64_t v_stride, const float* g,
                                       const float* beta, float scale, int32_t l2norm, const int32_t* slot_idx,
                                       const int32_t* accepted, const int32_t* cu_seqlens, int32_t batch, int32_t T,
                                       int64_t tokens, void* out, void* scratch, size_t scratch_bytes, void* stream) {
  DeltaStepArgs a = {};
  rssm_status st;
  if (!delta_view(cache, &a.c, &st)) return st;
  if (batch < 0 || T < 1 || tokens < 0) return RSSM_ERR_INVALID_ARGUMENT;
  if (T > a.c.np) return RSSM_ERR_UNSUPPORTED;
  if (!cu_seqlens && tokens < static_cast<int64_t>(batch) * T) return RSSM_ERR_INVALID_ARGUMENT;
  if (batch == 0) return RSSM_OK;
  if (tokens > 0) {
    st = delta_tokens(a.c, cache->dkey, q, k, v, q_stride, k_stride, v_stride, g, beta, scale, l2norm, out, &a.tk);
    if (st != RSSM_OK) return st;
  }
  if (!al(slot_idx, 4) || (accepted && !al(accepted, 4)) || (cu_seqlens && !al(cu_seqlens, 4)) || !al(scratch, 16))
    return RSSM_ERR_INVALID_ARGUMENT;
  if (scratch_bytes < static_cast<size_t>(batch) * sizeof(unsigned)) return RSSM_ERR_SCRATCH_TOO_SMALL;
  a.slot_idx = slot_idx;
  a.accepted = accepted;
  a.cu = cu_seqlens;
  a.batch = batch;
  a.T = T;
  a.tokens = tokens;
  a.tiles = (a.c.dv + kStepRows - 1) / kStepRows;
  a.ticket = static_cast<unsigned*>(scratch);
  const long long blocks = static_cast<long long>(batch) * a.c.Hv * a.tiles;
  if (blocks > 0x7fffffffll) return RSSM_ERR_UNSUPPORTED;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->dkey == 128
                            ? launch_pdl(delta_step_kernel<128>, dim3(static_cast<unsigned>(blocks)), dim3(kStepWarps * 32), 0, cs, a)
                            : launch_pdl(delta_step_kernel<64>, dim3(static_cast<unsigned>(blocks)), dim3(kStepWarps * 32), 0, cs, a);
  return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}
