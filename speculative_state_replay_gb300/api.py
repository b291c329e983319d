"""Python binding of librssm: the C ABI entry points with torch tensors.

Every function marshals tensor pointers, sizes and the current CUDA stream
into the C call of the same name and raises on a non-OK status.  All work
runs in the library's CUDA kernels; nothing here computes any part of the op.
Layouts and semantics are those of include/rssm.h.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib

F32, BF16, F16, I8, E4M3, NVFP4 = 0, 1, 2, 3, 4, 5
NEAREST, STOCHASTIC = 0, 1
ERRBIT_PNAT, ERRBIT_SEQLEN, ERRBIT_ACCEPT, ERRBIT_TIMEOUT, ERRBIT_TOKEN = 1, 2, 4, 8, 16
DIM, DSTATE = 64, 128
STATE_TORCH = {F32: torch.float32, BF16: torch.int16, F16: torch.int16, I8: torch.int8, E4M3: torch.uint8,
               NVFP4: torch.uint8}


class RssmError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = _lib.load().rssm_status_string(status).decode()
        super().__init__(f"{fn} failed: {msg} (status {status})")
        self.status = status


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(fn, status):
    if status != 0:
        raise RssmError(fn, status)


def _check_tokens(fn, cache, slot_idx, T, cu_seqlens, **per_token):
    """Host-side size check of the per-token tensors (no device read).

    Without cu_seqlens the kernels address batch * T tokens in every per-token
    tensor (x, dt, B, C, z, out), so each must hold at least that many token
    rows of its row size; with cu_seqlens the token count lives on the device
    and the caller sizes the tensors (include/rssm.h)."""
    if cu_seqlens is not None:
        return
    need = slot_idx.numel() * T
    row = {"x": cache.H * DIM, "out": cache.H * DIM, "z": cache.H * DIM, "dt": cache.H,
           "B": cache.G * DSTATE, "C": cache.G * DSTATE}
    for name, t in per_token.items():
        if t is None or need == 0:
            continue
        if t.numel() < need * row[name]:
            raise ValueError(f"{fn}: {name} holds {t.numel()} elements, fewer than batch * T = {need} tokens of "
                             f"{row[name]} (pass cu_seqlens for variable-length rows)")


class RssmCache:
    """Cache of all slots on one device: checkpoints, rings, bookkeeping.

    Every tensor is 2-D [slot, slot_stride]; `slot_pad_bytes` adds padding
    after each slot's page.  bf16/f16 data is held as raw 16-bit words.
    `read_dtype` (I8 or E4M3) adds a separate 8-bit read checkpoint
    (`read_state`, `read_scale`) that the step's readout reads S0 from;
    NVFP4 adds an NVFP4 one (`read_state` codes two per byte, `read_sf` block
    scales, `read_gs` per-slot global scales).
    """

    def __init__(self, num_slots, nheads, ngroups, max_window, npredicted, state_dtype, rounding=NEAREST,
                 device="cuda", slot_pad_bytes=0, read_dtype=None):
        self.S, self.H, self.G = num_slots, nheads, ngroups
        self.W, self.Tmax = max_window, npredicted
        self.L = max_window + npredicted
        self.state_dtype, self.rounding = state_dtype, rounding
        dev = torch.device(device)
        sd = STATE_TORCH[state_dtype]
        esz = torch.empty(0, dtype=sd).element_size()

        def stride(n, itemsize):
            return n + slot_pad_bytes // itemsize

        z = lambda shape, dt: torch.zeros(shape, dtype=dt, device=dev)  # noqa: E731
        self.state = z((num_slots, stride(nheads * DIM * DSTATE, esz)), sd)
        self.scale = torch.ones((num_slots, stride(nheads * DIM, 4)), dtype=torch.float32, device=dev)
        self.x_cache = z((num_slots, stride(nheads * self.L * DIM, 2)), torch.int16)
        self.B_cache = z((num_slots, stride(ngroups * self.L * DSTATE, 2)), torch.int16)
        self.dt_cache = z((num_slots, stride(nheads * self.L, 4)), torch.float32)
        self.ring_start = z((num_slots,), torch.int32)
        self.flush_epoch = z((num_slots,), torch.int32)
        self.error_word = z((1,), torch.int32)
        self.read_dtype = read_dtype
        self.read_state = self.read_scale = self.read_sf = self.read_gs = None
        if read_dtype == NVFP4:
            self.read_state = z((num_slots, stride(nheads * DIM * DSTATE // 2, 1)), torch.uint8)
            self.read_sf = z((num_slots, stride(nheads * DIM * DSTATE // 16, 1)), torch.uint8)
            self.read_gs = torch.ones((num_slots,), dtype=torch.float32, device=dev)
        elif read_dtype is not None:
            self.read_state = z((num_slots, stride(nheads * DIM * DSTATE, 1)), STATE_TORCH[read_dtype])
            self.read_scale = torch.ones((num_slots, stride(nheads * DIM, 4)), dtype=torch.float32, device=dev)
        self._struct = None

    def struct(self):
        if self._struct is None:
            c = _lib.RssmCacheStruct()
            c.num_slots, c.nheads, c.ngroups = self.S, self.H, self.G
            c.dim, c.dstate = DIM, DSTATE
            c.max_window, c.npredicted = self.W, self.Tmax
            c.state_dtype, c.rounding = self.state_dtype, self.rounding
            c.state, c.state_slot_stride = self.state.data_ptr(), self.state.shape[1]
            c.scale, c.scale_slot_stride = self.scale.data_ptr(), self.scale.shape[1]
            c.x_cache, c.x_slot_stride = self.x_cache.data_ptr(), self.x_cache.shape[1]
            c.B_cache, c.B_slot_stride = self.B_cache.data_ptr(), self.B_cache.shape[1]
            c.dt_cache, c.dt_slot_stride = self.dt_cache.data_ptr(), self.dt_cache.shape[1]
            c.ring_start = self.ring_start.data_ptr()
            c.flush_epoch = self.flush_epoch.data_ptr()
            c.error_word = self.error_word.data_ptr()
            if self.read_state is not None:
                c.read_state, c.read_slot_stride = self.read_state.data_ptr(), self.read_state.shape[1]
                c.read_dtype = self.read_dtype
                if self.read_dtype == NVFP4:
                    c.read_sf, c.read_sf_slot_stride = self.read_sf.data_ptr(), self.read_sf.shape[1]
                    c.read_gs = self.read_gs.data_ptr()
                else:
                    c.read_scale, c.read_scale_slot_stride = self.read_scale.data_ptr(), self.read_scale.shape[1]
            self._struct = c
        return ctypes.byref(self._struct)

    # logical views (without the slot padding)
    def state_view(self):
        return self.state[:, : self.H * DIM * DSTATE].view(self.S, self.H, DIM, DSTATE)

    def scale_view(self):
        return self.scale[:, : self.H * DIM].view(self.S, self.H, DIM)

    def x_view(self):
        return self.x_cache[:, : self.H * self.L * DIM].view(self.S, self.H, self.L, DIM)

    def B_view(self):
        return self.B_cache[:, : self.G * self.L * DSTATE].view(self.S, self.G, self.L, DSTATE)

    def dt_view(self):
        return self.dt_cache[:, : self.H * self.L].view(self.S, self.H, self.L)


def rssm_scratch_bytes(cache: RssmCache, batch: int, T: int) -> int:
    return int(_lib.load().rssm_scratch_bytes(cache.struct(), batch, T))


def alloc_scratch(cache: RssmCache, batch: int, T: int) -> torch.Tensor:
    n = rssm_scratch_bytes(cache, batch, T)
    if n == 0:
        raise RssmError("rssm_scratch_bytes", 1)
    # zero-filled: rssm_flush keeps a counter in the first word, which must start
    # at zero (every call leaves it at zero)
    return torch.zeros(n, dtype=torch.uint8, device=cache.state.device)


def rssm_init_state(cache, states, slot_idx, seed=0, stream=None):
    _check("rssm_init_state", _lib.load().rssm_init_state(cache.struct(), _ptr(states), _ptr(slot_idx),
                                                          slot_idx.numel(), seed, _stream(stream)))


def rssm_flush(cache, A, slot_idx, pnat, T, scratch, cu_seqlens=None, force=0, seed=0, stream=None):
    _check("rssm_flush", _lib.load().rssm_flush(cache.struct(), _ptr(A), _ptr(slot_idx), _ptr(pnat),
                                                _ptr(cu_seqlens), slot_idx.numel(), T, force, seed,
                                                _ptr(scratch), scratch.numel(), _stream(stream)))


def rssm_accept_flush(cache, A, slot_idx, pnat, accepted, accept_T, T, scratch, accept_cu_seqlens=None,
                      cu_seqlens=None, force=0, seed=0, stream=None):
    """rssm_accept(accepted, accept_cu_seqlens, accept_T) then rssm_flush(...), one launch."""
    _check("rssm_accept_flush", _lib.load().rssm_accept_flush(
        cache.struct(), _ptr(A), _ptr(slot_idx), _ptr(pnat), _ptr(accepted), _ptr(accept_cu_seqlens), accept_T,
        _ptr(cu_seqlens), slot_idx.numel(), T, force, seed, _ptr(scratch), scratch.numel(), _stream(stream)))


def _step(fn, cache, x, dt, A, B, C, D, dt_bias, slot_idx, pnat, T, out, scratch, cu_seqlens, stream):
    _check_tokens(fn, cache, slot_idx, T, cu_seqlens, x=x, dt=dt, B=B, C=C, out=out)
    f = getattr(_lib.load(), fn)
    _check(fn, f(cache.struct(), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(dt_bias),
                 _ptr(slot_idx), _ptr(pnat), _ptr(cu_seqlens), slot_idx.numel(), T, _ptr(out), _ptr(scratch),
                 scratch.numel(), _stream(stream)))


def _step_gated(fn, cache, x, dt, A, B, C, D, dt_bias, slot_idx, pnat, T, z, out, scratch, cu_seqlens, stream):
    _check_tokens(fn, cache, slot_idx, T, cu_seqlens, x=x, dt=dt, B=B, C=C, z=z, out=out)
    f = getattr(_lib.load(), fn)
    _check(fn, f(cache.struct(), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(dt_bias),
                 _ptr(slot_idx), _ptr(pnat), _ptr(cu_seqlens), slot_idx.numel(), T, _ptr(z), _ptr(out),
                 _ptr(scratch), scratch.numel(), _stream(stream)))


def rssm_step(cache, x, dt, A, B, C, D, dt_bias, slot_idx, pnat, T, out, scratch, cu_seqlens=None, stream=None,
              z=None):
    """`z`: optional output gate (bf16 bits [tok][H][64]): y * silu(z)."""
    if z is None:
        _step("rssm_step", cache, x, dt, A, B, C, D, dt_bias, slot_idx, pnat, T, out, scratch, cu_seqlens, stream)
    else:
        _step_gated("rssm_step_gated", cache, x, dt, A, B, C, D, dt_bias, slot_idx, pnat, T, z, out, scratch,
                    cu_seqlens, stream)


def rssm_step_precompute(cache, x, dt, A, B, C, D, dt_bias, slot_idx, pnat, T, out, scratch, cu_seqlens=None,
                         stream=None):
    _step("rssm_step_precompute", cache, x, dt, A, B, C, D, dt_bias, slot_idx, pnat, T, out, scratch, cu_seqlens,
          stream)


def rssm_step_readout(cache, x, dt, A, B, C, D, dt_bias, slot_idx, pnat, T, out, scratch, cu_seqlens=None,
                      stream=None, z=None):
    if z is None:
        _step("rssm_step_readout", cache, x, dt, A, B, C, D, dt_bias, slot_idx, pnat, T, out, scratch, cu_seqlens,
              stream)
    else:
        _step_gated("rssm_step_readout_gated", cache, x, dt, A, B, C, D, dt_bias, slot_idx, pnat, T, z, out,
                    scratch, cu_seqlens, stream)


def _flush_step(fn, cache, x, dt, A, B, C, D, dt_bias, slot_idx, pnat, T, out, scratch, cu_seqlens, force, seed,
                stream):
    _check_tokens(fn, cache, slot_idx, T, cu_seqlens, x=x, dt=dt, B=B, C=C, out=out)
    f = getattr(_lib.load(), fn)
    _check(fn, f(cache.struct(), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(dt_bias),
                 _ptr(slot_idx), _ptr(pnat), _ptr(cu_seqlens), slot_idx.numel(), T, force, seed, _ptr(out),
                 _ptr(scratch), scratch.numel(), _stream(stream)))


def rssm_flush_step(cache, x, dt, A, B, C, D, dt_bias, slot_idx, pnat, T, out, scratch, cu_seqlens=None, force=0,
                    seed=0, stream=None):
    _flush_step("rssm_flush_step", cache, x, dt, A, B, C, D, dt_bias, slot_idx, pnat, T, out, scratch, cu_seqlens,
                force, seed, stream)


def rssm_flush_step_classify(cache, x, dt, A, B, C, D, dt_bias, slot_idx, pnat, T, out, scratch, cu_seqlens=None,
                               force=0, seed=0, stream=None):
    _flush_step("rssm_flush_step_classify", cache, x, dt, A, B, C, D, dt_bias, slot_idx, pnat, T, out, scratch,
                cu_seqlens, force, seed, stream)


def rssm_flush_step_main(cache, x, dt, A, B, C, D, dt_bias, slot_idx, pnat, T, out, scratch, cu_seqlens=None,
                            force=0, seed=0, stream=None):
    _flush_step("rssm_flush_step_main", cache, x, dt, A, B, C, D, dt_bias, slot_idx, pnat, T, out, scratch,
                cu_seqlens, force, seed, stream)


def rssm_accept(cache, slot_idx, pnat, accepted, T, cu_seqlens=None, stream=None):
    _check("rssm_accept", _lib.load().rssm_accept(cache.struct(), _ptr(slot_idx), _ptr(pnat), _ptr(accepted),
                                                  _ptr(cu_seqlens), slot_idx.numel(), T, _stream(stream)))


def rssm_eval_spec_math(x, out_exp=None, out_softplus=None, stream=None):
    _check("rssm_eval_spec_math", _lib.load().rssm_eval_spec_math(_ptr(x), _ptr(out_exp), _ptr(out_softplus),
                                                                  x.numel(), _stream(stream)))


def rssm_selftest_wait_timeout(error_word, wait_ms=50, stream=None):
    """Diagnostics: one bounded mbarrier wait that runs out (sets ERRBIT_TIMEOUT)."""
    _check("rssm_selftest_wait_timeout", _lib.load().rssm_selftest_wait_timeout(_ptr(error_word), wait_ms,
                                                                                _stream(stream)))


# --------------------------------------------------------------------------
# Operators of the layers next to the state update: the gated delta rule,
# verification of drafted tokens, and the norms around a block.  Activations
# are torch tensors of their own types here (bf16, f16, f32); the checks below
# read no device data.
# --------------------------------------------------------------------------
_DTYPE = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}


def _refuse(fn, text):
    raise ValueError(f"{fn}: {text}")


# (messages are made only when a check fails: a decode step's calls are short)
def _ids(fn, name, t, n):
    if t.dtype is not torch.int32 or t.numel() < n or not t.is_contiguous():
        _refuse(fn, f"{name} must be a contiguous int32 tensor of at least {n} values")


def _f32(fn, name, t, n):
    if t.dtype is not torch.float32 or t.numel() < n or not t.is_contiguous():
        _refuse(fn, f"{name} must be a contiguous float32 tensor of at least {n} values")


def _p(t):
    return None if t is None else t.data_ptr()


def _s(fn, stream, d):
    """The stream's handle: the current one of device d where none is given (torch.cuda.current_stream() costs a small
    call 3 us).  d: the device of all of a call's tensors, by _lib.fast().device(..).  A launch goes to the current
    device with the tensors' addresses, so all of them have to be there; an address of another device or of the host
    would fault the GPU."""
    if d < 0:
        _refuse(fn, "all tensors must be on one CUDA device")
    if (d != 0 or _devices() > 1) and d != torch._C._cuda_getDevice():
        _refuse(fn, f"the tensors' device, {d}, is not the current one")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(d)
    if getattr(stream, "device_index", d) != d:  # (any object with a handle is a stream)
        _refuse(fn, "the stream is another device's")
    return stream.cuda_stream


@functools.cache
def _devices():
    return torch.cuda.device_count()


def _scratch(fn, t):
    """Bytes of a scratch buffer."""
    if not t.is_contiguous():
        _refuse(fn, "scratch must be contiguous")
    return t.numel()


class DeltaCache:
    """The gated delta rule's cache (rssm_delta_cache): states [S][Hv][dv][dk] in f32 or bf16, and the drafts of every
    slot's last step (`pend_*`, two halves).  Tensors that a program already has can be given instead of new ones; a
    slot's part must be contiguous, slots may be further apart.
    """

    def __init__(self, num_slots, k_heads, v_heads, key_dim, value_dim, npredicted, state_dtype=F32, device="cuda",
                 state=None, pend_k=None, pend_w=None, pend_c=None, pend=None, error_word=None, pend_cl=None):
        fn = "DeltaCache"
        if state_dtype not in (F32, BF16):
            _refuse(fn, "state_dtype must be F32 or BF16")
        self.S, self.Hk, self.Hv, self.dk, self.dv, self.Tmax = num_slots, k_heads, v_heads, key_dim, value_dim, npredicted
        self.state_dtype = state_dtype
        dev = torch.device(device)

        def make(name, t, shape, dtype):
            if t is None:
                return torch.zeros(shape, dtype=dtype, device=dev)
            dense = [1] * len(shape)
            for i in range(len(shape) - 2, 0, -1):
                dense[i] = dense[i + 1] * shape[i + 1]
            fits = all(n == 1 or x == d for n, x, d in zip(shape[1:], t.stride()[1:], dense[1:]))
            if tuple(t.shape) != shape or t.dtype is not dtype or not fits:
                _refuse(fn, f"{name} must be {dtype} {list(shape)}, contiguous within a slot")
            return t

        self.state = make("state", state, (num_slots, v_heads, value_dim, key_dim),
                          torch.float32 if state_dtype == F32 else torch.bfloat16)
        self.pend_k = make("pend_k", pend_k, (num_slots, 2, k_heads, npredicted, key_dim), torch.bfloat16)
        self.pend_w = make("pend_w", pend_w, (num_slots, 2, v_heads, npredicted, value_dim), torch.float32)
        self.pend_c = make("pend_c", pend_c, (num_slots, 2, v_heads, npredicted), torch.float32)
        self.pend_cl = make("pend_cl", pend_cl, (num_slots, 2, v_heads, npredicted), torch.float32)
        self.pend = make("pend", pend, (num_slots, 2), torch.int32)
        if not self.pend.is_contiguous():
            _refuse(fn, "pend must be contiguous")
        self.error_word = make("error_word", error_word, (1,), torch.int32)
        if len({t.device for t in (self.state, self.pend_k, self.pend_w, self.pend_c, self.pend_cl, self.pend, self.error_word)}) > 1:
            _refuse(fn, "tensors on different devices")
        c = _lib.RssmDeltaCacheStruct()
        c.num_slots, c.nkheads, c.nvheads, c.dkey, c.dvalue = num_slots, k_heads, v_heads, key_dim, value_dim
        c.npredicted, c.state_dtype = npredicted, state_dtype
        for name in ("state", "pend_k", "pend_w", "pend_c", "pend_cl"):
            t = getattr(self, name)
            setattr(c, name, t.data_ptr())
            setattr(c, name + "_slot_stride", t.stride(0))
        c.pend, c.error_word = self.pend.data_ptr(), self.error_word.data_ptr()
        self._struct = c
        self._ref, self._addr = ctypes.byref(c), ctypes.addressof(c)

    def struct(self):
        return self._ref


def rssm_delta_scratch_bytes(cache: DeltaCache, batch: int, tokens: int) -> int:
    return int(_lib.load().rssm_delta_scratch_bytes(cache.struct(), batch, tokens))


def alloc_delta_scratch(cache: DeltaCache, batch: int, tokens: int) -> torch.Tensor:
    """Scratch for steps and prompts of up to `batch` rows and `tokens` tokens."""
    n = rssm_delta_scratch_bytes(cache, batch, tokens)
    if n == 0:
        raise RssmError("rssm_delta_scratch_bytes", 1)
    return torch.zeros(n, dtype=torch.uint8, device=cache.state.device)  # its counters start at zero


def _heads(fn, name, t, n, h, d):
    """Elements between the tokens of t [n, h, d]."""
    if t.dtype is torch.bfloat16 and t.shape == (n, h, d):
        st = t.stride()
        if n == 0 or ((d == 1 or st[2] == 1) and (h == 1 or st[1] == d)):
            return st[0] if n > 1 else h * d
    _refuse(fn, f"{name} must be bfloat16 [{n}, {h}, {d}] with contiguous heads")


def _delta_tokens(fn, cache, q, k, v, g, beta, out):
    n = q.shape[0]
    sq, sk = _heads(fn, "q", q, n, cache.Hk, cache.dk), _heads(fn, "k", k, n, cache.Hk, cache.dk)
    sv = _heads(fn, "v", v, n, cache.Hv, cache.dv)
    if out.dtype is not torch.bfloat16 or out.shape != v.shape or not out.is_contiguous():
        _refuse(fn, f"out must be contiguous bfloat16 {list(v.shape)}")
    _f32(fn, "g", g, n * cache.Hv)
    _f32(fn, "beta", beta, n * cache.Hv)
    return n, sq, sk, sv


def rssm_delta_step(cache, q, k, v, g, beta, slot_idx, accepted, T, out, scratch, cu_seqlens=None, scale=None,
                    l2norm=False, stream=None):
    """One decode step of the gated delta rule: commits the accepted drafts of the last step, then runs the new tokens.

    q, k [tok, k_heads, key_dim], v and out [tok, v_heads, value_dim] bf16 (q, k, v may be columns of one projection);
    g, beta [tok, v_heads] f32; `scale` defaults to key_dim ** -0.5."""
    fn = "rssm_delta_step"
    n, sq, sk, sv = _delta_tokens(fn, cache, q, k, v, g, beta, out)
    batch = slot_idx.numel()
    _ids(fn, "slot_idx", slot_idx, batch)
    if accepted is not None:
        _ids(fn, "accepted", accepted, batch)
    if cu_seqlens is not None:
        _ids(fn, "cu_seqlens", cu_seqlens, batch + 1)
    lib = _lib.fast()
    status = lib.rssm_delta_step(
        cache._addr, q.data_ptr(), sq, k.data_ptr(), sk, v.data_ptr(), sv, g.data_ptr(), beta.data_ptr(),
        cache.dk ** -0.5 if scale is None else scale, int(l2norm), slot_idx.data_ptr(), _p(accepted),
        _p(cu_seqlens), batch, T, n, out.data_ptr(), scratch.data_ptr(), _scratch(fn, scratch),
        _s(fn, stream, lib.device(q, k, v, g, beta, slot_idx, accepted, cu_seqlens, out, scratch, cache.state)))
    if status:
        raise RssmError(fn, status)


def rssm_delta_prefill(cache, q, k, v, g, beta, slot_idx, cu_seqlens, out, scratch, initial=None, scale=None,
                       l2norm=False, stream=None):
    """The gated delta rule over whole prompts (tensors as in rssm_delta_step): outputs, and each slot's state after
    its prompt.  initial [batch] int32: nonzero rows go on from their slot's state."""
    fn = "rssm_delta_prefill"
    n, sq, sk, sv = _delta_tokens(fn, cache, q, k, v, g, beta, out)
    batch = slot_idx.numel()
    _ids(fn, "slot_idx", slot_idx, batch)
    _ids(fn, "cu_seqlens", cu_seqlens, batch + 1)
    if initial is not None:
        _ids(fn, "initial", initial, batch)
    lib = _lib.fast()
    status = lib.rssm_delta_prefill(
        cache._addr, q.data_ptr(), sq, k.data_ptr(), sk, v.data_ptr(), sv, g.data_ptr(), beta.data_ptr(),
        cache.dk ** -0.5 if scale is None else scale, int(l2norm), slot_idx.data_ptr(), cu_seqlens.data_ptr(),
        _p(initial), batch, n, out.data_ptr(), scratch.data_ptr(), _scratch(fn, scratch),
        _s(fn, stream, lib.device(q, k, v, g, beta, slot_idx, cu_seqlens, initial, out, scratch, cache.state)))
    if status:
        raise RssmError(fn, status)


def _rows(fn, name, t, dtype, shape):
    """Elements between the rows of t."""
    if t.dtype is dtype and t.shape == shape:
        st = t.stride()
        if st[1] == 1 or shape[1] == 1:
            return st[0] if shape[0] > 1 else shape[1]
    _refuse(fn, f"{name} must be {dtype} {list(shape)} with contiguous rows")


def rssm_verify(target, tokens, u, u_next, T, accepted, next_token, draft=None, cu_seqlens=None, error_word=None,
                stream=None):
    """Accepted counts and next tokens of a speculative step; target (and draft) [tok, vocab] probabilities."""
    fn = "rssm_verify"
    ntok, vocab = target.shape
    batch = u_next.numel()
    dtype = target.dtype
    if dtype not in _DTYPE:
        _refuse(fn, "target must be f32, bf16 or f16")
    st = _rows(fn, "target", target, dtype, target.shape)
    sd = 0 if draft is None else _rows(fn, "draft", draft, dtype, target.shape)
    _ids(fn, "tokens", tokens, ntok)
    _f32(fn, "u", u, ntok)
    _f32(fn, "u_next", u_next, batch)
    _ids(fn, "accepted", accepted, batch)
    _ids(fn, "next_token", next_token, batch)
    if cu_seqlens is not None:
        _ids(fn, "cu_seqlens", cu_seqlens, batch + 1)
    if error_word is not None and (error_word.element_size() != 4 or error_word.numel() < 1):
        _refuse(fn, "error_word must be a tensor of one 32-bit word")
    lib = _lib.fast()
    status = lib.rssm_verify(
        target.data_ptr(), st, _p(draft), sd, _DTYPE[dtype], vocab, tokens.data_ptr(), u.data_ptr(), u_next.data_ptr(),
        _p(cu_seqlens), batch, T, ntok, accepted.data_ptr(), next_token.data_ptr(), _p(error_word),
        _s(fn, stream, lib.device(target, draft, tokens, u, u_next, cu_seqlens, accepted, next_token, error_word)))
    if status:
        raise RssmError(fn, status)


def rssm_gated_norm(x, z, weight, out, group=None, eps=1e-5, norm_first=False, stream=None):
    """RMS norm over groups of channels with the silu gate z, before the norm or (norm_first) after it; x, z, out
    [rows, dim], weight f32 [dim], or [group] for every group."""
    fn = "rssm_gated_norm"
    rows, dim = x.shape
    group = dim if group is None else group
    dtype, shape = x.dtype, x.shape
    if dtype not in _DTYPE:
        _refuse(fn, "x must be f32, bf16 or f16")
    sx, sz, so = _rows(fn, "x", x, dtype, shape), _rows(fn, "z", z, dtype, shape), _rows(fn, "out", out, dtype, shape)
    weights = weight.numel()
    if weights != dim and weights != group:
        _refuse(fn, f"weight must hold {dim} or {group} values")
    _f32(fn, "weight", weight, 1)
    lib = _lib.fast()
    status = lib.rssm_gated_norm(x.data_ptr(), sx, z.data_ptr(), sz, _DTYPE[dtype], weight.data_ptr(),
                                         int(weights != dim), rows, dim, group, eps, int(norm_first), out.data_ptr(), so,
                                         _s(fn, stream, lib.device(x, z, weight, out)))
    if status:
        raise RssmError(fn, status)


def rssm_residual_norm(x, residual, weight, out, residual_out, post_weight=None, scale=None, alpha=1.0, eps=1e-5,
                       stream=None):
    """residual_out = residual + alpha scale [norm](x), out = norm(residual_out) weight; [rows, dim] each, the
    residual in x's type or f32, weights f32 [dim]."""
    fn = "rssm_residual_norm"
    rows, dim = x.shape
    dtype, shape, rtype = x.dtype, x.shape, residual.dtype
    if dtype not in _DTYPE or (rtype is not torch.float32 and rtype is not dtype):
        _refuse(fn, "types must be f32, bf16 or f16, the residual's f32 or x's")
    sx, so = _rows(fn, "x", x, dtype, shape), _rows(fn, "out", out, dtype, shape)
    sr, sro = _rows(fn, "residual", residual, rtype, shape), _rows(fn, "residual_out", residual_out, rtype, shape)
    for name, t in (("weight", weight), ("post_weight", post_weight), ("scale", scale)):
        if t is not None and (t.numel() != dim or t.dtype is not torch.float32 or not t.is_contiguous()):
            _refuse(fn, f"{name} must hold {dim} contiguous float32 values")
    lib = _lib.fast()
    status = lib.rssm_residual_norm(
        x.data_ptr(), sx, residual.data_ptr(), sr, _DTYPE[dtype], _DTYPE[rtype], _p(post_weight), _p(scale), alpha,
        weight.data_ptr(), rows, dim, eps, residual_out.data_ptr(), sro, out.data_ptr(), so,
        _s(fn, stream, lib.device(x, residual, weight, out, residual_out, post_weight, scale)))
    if status:
        raise RssmError(fn, status)
