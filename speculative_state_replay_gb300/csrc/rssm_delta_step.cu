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
  int tiles;         // kStepRows value rows a head has
  int items;         // (value head, tile) items of a (row, key head)
  int whole, per;    // blocks that take all items of theirs; the (row, key head)s after them go `per` items to a block
  unsigned* ticket;  // scratch [batch]: blocks that have read the row's `pend` (zero between calls)
};

constexpr int kStepWarps = 4;
constexpr int kStepRows = kStepWarps * 16;  // value rows of a tile
// blocks an SM: 2-byte states 438 us with 4, 464 with 3, 454 with 5 (1024 rows);
// fp32 states keep 64 values a lane and spill with 4: 81 us, 58 with 3 (64 rows)
constexpr int step_blocks(bool f32) { return f32 ? 3 : 4; }

// A warp's item on its way from memory: its state rows (a bulk copy) and, for
// this item and the next in turn, of the waiting drafts the corrections of these
// rows and the running sums, of the new tokens the values of these rows, log
// decays and rates.
template <int DK, bool F32>
struct alignas(128) StepWarp {
  uint8_t s[16 * DK * (F32 ? 4 : 2)];
  struct alignas(16) Small {
    float w[kDeltaT][16];
    uint16_t v[kDeltaT][16];
    float c[kDeltaT], cl[kDeltaT], g[kDeltaT], beta[kDeltaT];
  } x[2];
  uint64_t bar;  // the state rows have landed
};
template <int DK, bool F32>
struct alignas(128) StepSmem {
  StepWarp<DK, F32> warp[kStepWarps];
  alignas(16) uint8_t k[kDeltaT * kTokenRow<DK>];  // the new tokens' keys and queries
  alignas(16) uint8_t q[kDeltaT * kTokenRow<DK>];
  alignas(16) uint8_t pk[kDeltaT * kTokenRow<DK>];  // the waiting drafts' keys, and in fp32
  alignas(16) float p[kDeltaT * DK];
};
// every destination of a 16-byte or bulk copy starts on 16 bytes
static_assert(sizeof(StepWarp<64, false>) % 128 == 0 && sizeof(StepWarp<128, true>) % 128 == 0, "a warp's part keeps the next one's alignment");
static_assert(sizeof(StepWarp<64, false>::Small) % 16 == 0 && kTokenRow<64> % 16 == 0 && kTokenRow<128> % 16 == 0, "rows start on 16 bytes");

// A block takes items -- 64 value rows of a value head each -- of a (row, key
// head); the tokens' keys and queries, their Gram products and the waiting
// keys serve all of them.  One warp per 16 value rows reads its part of S once
// (one bulk copy: the rows are contiguous), and with the rows in registers sends
// for its next item's; it forms the new drafts' outputs and corrections, adds the
// accepted drafts of the step before and writes the rows back if there were any.
template <int DK, bool F32>
__global__ void __launch_bounds__(kStepWarps * 32, step_blocks(F32)) delta_step_kernel(const DeltaStepArgs a) {
  extern __shared__ __align__(128) uint8_t raw[];
  StepSmem<DK, F32>& sm = *reinterpret_cast<StepSmem<DK, F32>*>(raw);
  __shared__ int sh[2];
  constexpr int CH = DK / 8, kRow = DK * (F32 ? 4 : 2);
  constexpr unsigned full = 0xffffffffu;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, t = lane >> 2, cc = lane & 3;
  StepWarp<DK, F32>& wm = sm.warp[warp];
  if (lane == 0) {
    mbar_init(&wm.bar, 1);
    fence_barrier_init();
  }
  __syncwarp();
  int unit = blockIdx.x, item0 = 0, left = a.items;
  const int groups = (a.items + a.per - 1) / a.per;
  if (unit >= a.whole) {
    const int x = unit - a.whole;
    unit = a.whole + x / groups;
    item0 = x % groups * a.per;
    left = min(a.per, a.items - item0);
  }
  const int b = unit / a.c.Hk, hk = unit - b * a.c.Hk;
  pdl_wait();
  pdl_trigger();
  const int s = a.slot_idx[b];
  const long long tok0 = a.cu ? a.cu[b] : static_cast<long long>(b) * a.T;
  const int n = a.cu ? a.cu[b + 1] - static_cast<int>(tok0) : a.T;
  const int acc = a.accepted ? a.accepted[b] : 0;
  if (n < 0 || n > a.T || tok0 < 0 || tok0 + n > a.tokens) {  // the row's tokens are not known: nothing to write
    if (tid == 0 && hk == 0 && item0 == 0) set_error(a.c.err, RSSM_ERRBIT_SEQLEN);
    return;
  }
  const int dv = a.c.dv, Hv = a.c.Hv, np = a.c.np;
  const bool live = t < n;
  // the item: value head hv, and the warp's first value row in it
  int hv = hk * a.c.rep + item0 / a.tiles, r0 = item0 % a.tiles * kStepRows + warp * 16;
  const auto step_on = [&](int& h, int& r) {
    r += kStepRows;
    if (r - warp * 16 >= dv) {
      r = warp * 16;
      ++h;
    }
  };
  uint16_t* out = a.tk.out + (tok0 + t) * Hv * dv + 2 * cc;
  const auto zeros = [&]() {
    for (; left > 0; --left, step_on(hv, r0))
      if (r0 < dv && live) {
        *reinterpret_cast<uint32_t*>(out + hv * dv + r0) = 0u;
        *reinterpret_cast<uint32_t*>(out + hv * dv + r0 + 8) = 0u;
      }
  };
  if (s <= 0 || s >= a.c.S) {
    zeros();
    return;
  }
  uint8_t* state = static_cast<uint8_t*>(a.c.state) + s * a.c.state_stride * (F32 ? 4 : 2);
  const uint16_t* vp = a.tk.v + (tok0 + t) * a.tk.v_stride + 8 * (cc & 1);
  const float* gp = (lane < 8 ? a.tk.g : a.tk.beta) + (tok0 + (lane & 7)) * Hv;
  int turn = 0;
  // an item's state rows, and the new tokens' part; a head's decays, rates and (below) running sums come with the first
  // of its items that the warp has
  const auto fetch = [&](int h, int r, int x, bool new_head) {
    if (r >= dv) return;
    if (lane == 0) {
      mbar_arrive_expect_tx(&wm.bar, 16 * kRow);
      bulk_g2s(wm.s, state + static_cast<long long>(h * dv + r) * kRow, 16 * kRow, &wm.bar);
    }
    if (live && cc < 2) cp_async16(&wm.x[x].v[t][8 * cc], vp + h * dv + r);
    if (new_head && lane < 16 && (lane & 7) < n) cp_async4(lane < 8 ? &wm.x[x].g[lane] : &wm.x[x].beta[lane & 7], gp + h);
  };
  fetch(hv, r0, 0, true);
  for (int i = tid; i < kDeltaT * CH; i += kStepWarps * 32) {
    const int r = i / CH, ch = i % CH, to = r * kTokenRow<DK> + ch * 16;
    if (r < n) {
      cp_async16(sm.k + to, a.tk.k + (tok0 + r) * a.tk.k_stride + hk * DK + ch * 8);
      cp_async16(sm.q + to, a.tk.q + (tok0 + r) * a.tk.q_stride + hk * DK + ch * 8);
    } else {
      *reinterpret_cast<uint4*>(sm.k + to) = *reinterpret_cast<uint4*>(sm.q + to) = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  if (tid == 0) {
    const int2 p = __ldcg(reinterpret_cast<const int2*>(a.c.pend) + s);
    sh[0] = p.x;
    sh[1] = p.y;
  }
  __syncthreads();
  const int side = sh[0] & 1, to = side ^ 1;
  const bool ok = acc >= 0 && acc <= sh[1] && acc <= np;
  // every block of the row takes a ticket once it has read (side, count); the
  // last one knows that all have, and turns the sides
  if (tid == 0) {
    __threadfence();
    const int wholes = min(max(a.whole - b * a.c.Hk, 0), a.c.Hk);  // of the row's blocks
    const unsigned blocks = static_cast<unsigned>(wholes + (a.c.Hk - wholes) * groups);
    if (atomicInc(a.ticket + b, blocks - 1u) == blocks - 1u) {
      if (ok)
        reinterpret_cast<int2*>(a.c.pend)[s] = make_int2(to, n);
      else
        set_error(a.c.err, RSSM_ERRBIT_ACCEPT);
    }
  }
  if (!ok) {
    cp_async_wait_all();
    if (r0 < dv && !mbar_wait(&wm.bar, 0)) {  // nothing is in flight at the end
      if (lane == 0) set_error(a.c.err, RSSM_ERRBIT_TIMEOUT);
      mbar_wait(&wm.bar, 0);
    }
    zeros();
    return;
  }
  const float* pw = a.c.pend_w + s * a.c.pend_w_stride + 4 * cc;
  const float* pc = a.c.pend_c + s * a.c.pend_c_stride + lane;
  const auto fetch_waiting = [&](int h, int r, int x, bool new_head) {
    const int at = (side * Hv + h) * np;
    if (r < dv && t < acc) cp_async16(&wm.x[x].w[t][4 * cc], pw + static_cast<long long>(at + t) * dv + r);
    if (new_head && lane < acc) {
      cp_async4(&wm.x[x].c[lane], pc + at);
      if (a.c.pend_cl)
        cp_async4(&wm.x[x].cl[lane], a.c.pend_cl + s * a.c.pend_cl_stride + at + lane);
      else
        wm.x[x].cl[lane] = 0.0f;
    }
  };
  if (acc > 0) {
    fetch_waiting(hv, r0, 0, true);
    const uint16_t* pk = a.c.pend_k + s * a.c.pend_k_stride + (static_cast<long long>(side) * a.c.Hk + hk) * np * DK;
    for (int i = tid; i < acc * CH; i += kStepWarps * 32) {
      const uint4 x = *reinterpret_cast<const uint4*>(pk + i * 8);
      *reinterpret_cast<uint4*>(sm.pk + i / CH * kTokenRow<DK> + i % CH * 16) = x;
      float4* d = reinterpret_cast<float4*>(sm.p + i * 8);
      d[0] = make_float4(bf16lo(x.x), bf16hi(x.x), bf16lo(x.y), bf16hi(x.y));
      d[1] = make_float4(bf16lo(x.z), bf16hi(x.z), bf16lo(x.w), bf16hi(x.w));
    }
  }
  cp_async_wait_all();
  __syncthreads();
  DeltaBlock<DK> blk;
  blk.set(sm.k, sm.q, lane);
  blk.gram(a.tk, sm.pk, acc, lane);
  if (item0 == 0 && warp == 0 && live) {  // the new drafts wait in the other half
    uint16_t* pk = a.c.pend_k + s * a.c.pend_k_stride + ((static_cast<long long>(to) * a.c.Hk + hk) * np + t) * DK + 8 * cc;
#pragma unroll
    for (int y = 0; y < DK / 32; ++y) *reinterpret_cast<uint4*>(pk + 32 * y) = *reinterpret_cast<const uint4*>(blk.k + 64 * y);
  }
  float* nw = a.c.pend_w + s * a.c.pend_w_stride + static_cast<long long>(to * Hv * np + t) * dv + 2 * cc;
  float* nc = a.c.pend_c + s * a.c.pend_c_stride + to * Hv * np + t;
  state += (t * DK + 8 * cc) * (F32 ? 4 : 2);
  uint32_t parity = 0;
  int head = -1;
  float beta = 0.0f, ec = 0.0f, E = 1.0f, ew = 0.0f, A[2], P[2], gk[2], gq[2];
#pragma unroll 1
  for (; left > 0; --left, turn ^= 1) {
    const typename StepWarp<DK, F32>::Small& x = wm.x[turn];
    const int h = hv, r = r0;
    step_on(hv, r0);
    cp_async_wait_all();
    __syncwarp();  // the other lanes' copies have landed too
    if (r >= dv) {
      if (left > 1) {
        fetch(hv, r0, turn ^ 1, r0 == warp * 16);
        if (acc > 0) fetch_waiting(hv, r0, turn ^ 1, r0 == warp * 16);
      }
      continue;
    }
    if (!__all_sync(full, mbar_wait(&wm.bar, parity))) {
      if (lane == 0) set_error(a.c.err, RSSM_ERRBIT_TIMEOUT);
      mbar_wait(&wm.bar, parity);  // once more, with its limit: the copy must not outlive the block
      return;
    }
    parity ^= 1;
    DeltaRow<DK, F32> S[2];
    S[0].read(wm.s, t, cc);
    S[1].read(wm.s, t + 8, cc);
    __syncwarp();  // the rows are read
    if (left > 1) {
      fetch(hv, r0, turn ^ 1, r0 == warp * 16);
      if (acc > 0) fetch_waiting(hv, r0, turn ^ 1, r0 == warp * 16);
    }
    if (h != head) {  // what the head's items share
      head = h;
      beta = live ? x.beta[t] : 0.0f;
      // running sums and the coefficients among the block's own tokens
      LongSum c = {live ? held_log(x.g[t]) : 0.0f, 0.0f};
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        const float yh = __shfl_up_sync(full, c.hi, o), yl = __shfl_up_sync(full, c.lo, o);
        if (lane >= o) c.add(yh, yl);
      }
      c.settle();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int j = 2 * cc + i;
        const float d = (c.hi - __shfl_sync(full, c.hi, j * 4)) + (c.lo - __shfl_sync(full, c.lo, j * 4));
        const float e = j <= t ? expf(d) : 0.0f;
        A[i] = j < t ? beta * e * blk.kk[i] : 0.0f;
        P[i] = e * blk.kk[2 + i];
      }
      ec = exp_sum(c.hi, c.lo);
      if (r == 0 && live && cc == 0) {  // they wait with the drafts
        nc[h * np] = c.hi;
        if (a.c.pend_cl) a.c.pend_cl[s * a.c.pend_cl_stride + (to * Hv + h) * np + t] = c.lo;
      }
      if (acc > 0) {
        const float end = x.c[acc - 1], rest = x.cl[acc - 1];
        E = exp_sum(end, rest);
        ew = lane < acc ? expf((end - x.c[lane]) + (rest - x.cl[lane])) : 0.0f;
        const float e0 = __shfl_sync(full, ew, 2 * cc), e1 = __shfl_sync(full, ew, 2 * cc + 1);
        gk[0] = blk.wk[0] * e0;
        gk[1] = blk.wk[1] * e1;
        gq[0] = blk.wk[2] * e0;
        gq[1] = blk.wk[3] * e1;
      }
    }
    // what the waiting drafts add to S0 k_t and S0 q_t
    float wu[2][2] = {{0.f, 0.f}, {0.f, 0.f}}, wo[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
    if (acc > 0) {
#pragma unroll
      for (int j = 0; j < kDeltaT; ++j) {
        if (j >= acc) break;
        const float xk = __shfl_sync(full, gk[j & 1], t * 4 + (j >> 1)), xq = __shfl_sync(full, gq[j & 1], t * 4 + (j >> 1));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 w = *reinterpret_cast<const float2*>(&x.w[j][8 * i + 2 * cc]);
          wu[i][0] = fmaf(xk, w.x, wu[i][0]);
          wu[i][1] = fmaf(xk, w.y, wu[i][1]);
          wo[i][0] = fmaf(xq, w.x, wo[i][0]);
          wo[i][1] = fmaf(xq, w.y, wo[i][1]);
        }
      }
    }
    const float fk = E * blk.r, fq = E * blk.kq, be = beta * ec;
    float u[2][2], o[2][2], d[2][4];
    blk.product(S, d);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t vw = live ? *reinterpret_cast<const uint32_t*>(&x.v[t][8 * i + 2 * cc]) : 0u;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        u[i][e] = fmaf(-be, fmaf(fk, d[i][e], wu[i][e]), beta * (e ? bf16hi(vw) : bf16lo(vw)));
        o[i][e] = ec * fmaf(fq, d[i][2 + e], wo[i][e]);
      }
    }
    if (acc > 0) {
      uint8_t* mine = state + static_cast<long long>(h * dv + r) * kRow;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        S[i].decay(E);
        for (int j = 0; j < acc; ++j) S[i].add(__shfl_sync(full, ew, j) * x.w[j][t + 8 * i], sm.p + j * DK, cc);
        S[i].store(mine + 8 * i * kRow, a.c.wide);
      }
    }
    if (n == 0) continue;
#pragma unroll
    for (int j = 0; j < kDeltaT; ++j) {
      if (j >= n) break;
      // u_j is final in the lanes of token j once every earlier token's share is in
      const float Aj = __shfl_sync(full, A[j & 1], t * 4 + (j >> 1)), Pj = __shfl_sync(full, P[j & 1], t * 4 + (j >> 1));
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float uj = __shfl_sync(full, u[i][e], j * 4 + cc);
          // selected, not multiplied by zero: a later token's NaN stays out of the earlier ones
          if (t > j) u[i][e] = fmaf(-Aj, uj, u[i][e]);
          if (t >= j) o[i][e] = fmaf(Pj, uj, o[i][e]);
        }
    }
    if (live) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        *reinterpret_cast<uint32_t*>(out + h * dv + r + 8 * i) = cvt_bf16x2(o[i][0], o[i][1]);
        *reinterpret_cast<float2*>(nw + static_cast<long long>(h * np) * dv + r + 8 * i) = make_float2(u[i][0] * blk.r, u[i][1] * blk.r);
      }
    }
  }
}

template <int DK, bool F32>
cudaError_t launch_step(const DeltaStepArgs& a, unsigned blocks, cudaStream_t st) {
  constexpr size_t smem = sizeof(StepSmem<DK, F32>);
  const cudaError_t e = cudaFuncSetAttribute(delta_step_kernel<DK, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  return e == cudaSuccess ? launch_pdl(delta_step_kernel<DK, F32>, dim3(blocks), dim3(kStepWarps * 32), smem, st, a) : e;
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
  if (c->pend_cl && (!al(c->pend_cl, 4) || c->pend_cl_slot_stride < cl)) return false;
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
  o->pend_cl = c->pend_cl;
  o->pend_cl_stride = c->pend_cl_slot_stride;
  o->pend = c->pend;
  o->err = c->error_word;
  o->wide = al(c->state, 32) && c->state_slot_stride * esz % 32 == 0;
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
  if (T > a.c.np || batch > kDeltaRows) return RSSM_ERR_UNSUPPORTED;
  if (!cu_seqlens && tokens < static_cast<int64_t>(batch) * T) return RSSM_ERR_INVALID_ARGUMENT;
  if (batch == 0) return RSSM_OK;
  if (tokens > 0) {
    st = delta_tokens(a.c, cache->dkey, q, k, v, q_stride, k_stride, v_stride, g, beta, scale, l2norm, out, &a.tk);
    if (st != RSSM_OK) return st;
  }
  if (!al(slot_idx, 4) || (accepted && !al(accepted, 4)) || (cu_seqlens && !al(cu_seqlens, 4)) || !al(scratch, 16))
    return RSSM_ERR_INVALID_ARGUMENT;
  if (scratch_bytes < kDeltaHead) return RSSM_ERR_SCRATCH_TOO_SMALL;
  a.slot_idx = slot_idx;
  a.accepted = accepted;
  a.cu = cu_seqlens;
  a.batch = batch;
  a.T = T;
  a.tokens = tokens;
  a.tiles = (a.c.dv + kStepRows - 1) / kStepRows;
  a.ticket = static_cast<unsigned*>(scratch);
  a.items = a.c.rep * a.tiles;
  // Items a block takes: all of a (row, key head)'s for as many whole waves of
  // blocks as there are -- what the items share is worth more than the spread
  // (64 rows of 16 key heads with 4 items, fp32: 82 us with 1 item a block, 61
  // with 4) -- and of the rest as few as give one more wave, so that it does not
  // take as long as a whole one (55 us).
  const long long wave = static_cast<long long>(step_blocks(a.c.dtype == RSSM_F32)) * num_sms(), units = static_cast<long long>(batch) * a.c.Hk;
  if (wave == 0) return RSSM_ERR_CUDA;
  if (units * a.items > 0x7fffffffll) return RSSM_ERR_UNSUPPORTED;
  a.whole = static_cast<int>(units / wave * wave);
  const long long rest = units - a.whole;
  const auto spread = [&](int per) { return rest * ((a.items + per - 1) / per); };
  a.per = 1;
  while (a.per < a.items && spread(a.per) > wave) a.per = a.per * 2 < a.items ? a.per * 2 : a.items;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(a.whole + spread(a.per));
  const bool f32 = a.c.dtype == RSSM_F32;
  const cudaError_t e = cache->dkey == 128 ? (f32 ? launch_step<128, true>(a, grid, cs) : launch_step<128, false>(a, grid, cs))
                                           : (f32 ? launch_step<64, true>(a, grid, cs) : launch_step<64, false>(a, grid, cs));
  return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}
