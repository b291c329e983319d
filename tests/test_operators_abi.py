"""Refusals of the added operators: a status before anything is launched, and the binding's own checks (no GPU)."""
import ctypes

import pytest
import torch

import __graft_entry__ as entry
from speculative_state_replay_gb300 import _lib, api

P = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 2)
NUL = None


@pytest.fixture(scope="module")
def lib():
    entry.build()
    return _lib.load()


def cache(**kw):
    c = _lib.RssmDeltaCacheStruct()
    d = dict(num_slots=4, nkheads=2, nvheads=4, dkey=128, dvalue=64, npredicted=4, state_dtype=api.F32)
    d.update(state=1 << 20, state_slot_stride=4 * 64 * 128, pend_k=1 << 20, pend_k_slot_stride=2 * 2 * 4 * 128, pend_w=1 << 20,
             pend_w_slot_stride=2 * 4 * 4 * 64, pend_c=1 << 20, pend_c_slot_stride=2 * 4 * 4, pend=1 << 20, error_word=1 << 20)
    d.update(kw)
    for n, v in d.items():
        setattr(c, n, v)
    return ctypes.byref(c)


BAD = [dict(num_slots=0), dict(nkheads=0), dict(nvheads=3), dict(dvalue=0), dict(npredicted=0), dict(state_dtype=api.F16),
       dict(state=0), dict(state=(1 << 20) + 8), dict(state_slot_stride=8), dict(pend_k_slot_stride=2 * 2 * 4 * 128 + 4),
       dict(pend_w=0), dict(pend_w_slot_stride=9), dict(pend_c_slot_stride=1), dict(pend=(1 << 20) + 4), dict(error_word=0)]
UNSUPPORTED = [dict(dkey=96), dict(dvalue=24), dict(dvalue=2048), dict(npredicted=9)]


def step(lib, c, q=P, qs=256, ks=256, vs=256, l2=1, slots=P, acc=P, cu=NUL, batch=2, T=4, tokens=8, out=P, scratch=P, nbytes=1 << 20):
    return lib.rssm_delta_step(c, q, qs, P, ks, P, vs, P, P, 1.0, l2, slots, acc, cu, batch, T, tokens, out, scratch, nbytes, NUL)


def prefill(lib, c, q=P, qs=256, vs=256, slots=P, cu=P, ini=NUL, batch=2, tokens=8, out=P, scratch=P, nbytes=1 << 24):
    return lib.rssm_delta_prefill(c, q, qs, P, 256, P, vs, P, P, 1.0, 1, slots, cu, ini, batch, tokens, out, scratch, nbytes, NUL)


def test_delta_refusals(lib):
    assert lib.rssm_delta_scratch_bytes(cache(), 4, 100) > 0
    for kw, want in [(b, 1) for b in BAD] + [(u, 2) for u in UNSUPPORTED]:
        assert lib.rssm_delta_scratch_bytes(cache(**kw), 4, 100) == 0, kw
        assert step(lib, cache(**kw)) == want, kw
        assert prefill(lib, cache(**kw)) == want, kw
    assert lib.rssm_delta_scratch_bytes(None, 4, 100) == 0 and step(lib, None) == 1
    assert lib.rssm_delta_scratch_bytes(cache(), -1, 100) == 0 and lib.rssm_delta_scratch_bytes(cache(), 1, -1) == 0
    c = cache()
    assert step(lib, c, q=NUL) == 1 and step(lib, c, q=ODD) == 1 and step(lib, c, qs=128) == 1 and step(lib, c, qs=260) == 1
    assert step(lib, c, vs=255) == 1 and step(lib, c, l2=2) == 1 and step(lib, c, slots=NUL) == 1 and step(lib, c, acc=ODD) == 1
    assert step(lib, c, batch=-1) == 1 and step(lib, c, T=0) == 1 and step(lib, c, T=5) == 2 and step(lib, c, tokens=7) == 1
    assert step(lib, c, out=NUL) == 1 and step(lib, c, scratch=NUL) == 1 and step(lib, c, nbytes=7) == 3
    assert step(lib, c, batch=0) == 0
    assert prefill(lib, c, q=ODD) == 1 and prefill(lib, c, qs=8) == 1 and prefill(lib, c, vs=8) == 1 and prefill(lib, c, cu=NUL) == 1
    assert prefill(lib, c, ini=ODD) == 1 and prefill(lib, c, tokens=-1) == 1 and prefill(lib, c, tokens=1 << 31) == 1
    assert prefill(lib, c, nbytes=8) == 3 and prefill(lib, c, batch=0) == 0


def test_verify_refusals(lib):
    def verify(target=P, ts=100, draft=P, ds=100, dt=api.F32, V=100, tok=P, u=P, un=P, cu=NUL, batch=2, T=4, ntok=8, acc=P, nxt=P, err=NUL):
        return lib.rssm_verify(target, ts, draft, ds, dt, V, tok, u, un, cu, batch, T, ntok, acc, nxt, err, NUL)

    assert verify(batch=-1) == 1 and verify(T=0) == 1 and verify(V=0) == 1 and verify(ntok=-1) == 1 and verify(dt=api.I8) == 1
    assert verify(T=33) == 2 and verify(batch=0) == 0
    assert verify(target=NUL) == 1 and verify(tok=NUL) == 1 and verify(u=NUL) == 1 and verify(un=ODD) == 1 and verify(acc=NUL) == 1
    assert verify(nxt=ODD) == 1 and verify(err=ODD) == 1 and verify(ts=99) == 1 and verify(ds=99) == 1 and verify(target=ODD) == 1
    assert verify(ntok=7) == 1 and verify(cu=ODD) == 1


def test_norm_refusals(lib):
    def gated(x=P, xs=64, z=P, zs=64, dt=api.F32, w=P, sh=0, rows=2, dim=64, group=32, eps=1e-5, first=0, out=P, os=64):
        return lib.rssm_gated_norm(x, xs, z, zs, dt, w, sh, rows, dim, group, eps, first, out, os, NUL)

    assert gated(rows=-1) == 1 and gated(dim=0) == 1 and gated(group=0) == 1 and gated(group=48) == 1 and gated(eps=-1.0) == 1
    assert gated(eps=float("nan")) == 1 and gated(dt=api.E4M3) == 1 and gated(sh=2) == 1 and gated(first=3) == 1 and gated(xs=63) == 1
    assert gated(zs=63) == 1 and gated(os=1) == 1 and gated(x=NUL) == 1 and gated(z=ODD) == 1 and gated(w=ODD) == 1
    assert gated(rows=0) == 0 and gated(rows=1 << 40) == 2

    def resid(x=P, xs=64, r=P, rs=64, dt=api.BF16, rdt=api.F32, post=NUL, scale=NUL, w=P, rows=2, dim=64, eps=1e-5, ro=P, ros=64, out=P, os=64):
        return lib.rssm_residual_norm(x, xs, r, rs, dt, rdt, post, scale, 1.0, w, rows, dim, eps, ro, ros, out, os, NUL)

    assert resid(rows=-1) == 1 and resid(dim=0) == 1 and resid(dt=api.I8) == 1 and resid(rdt=api.F16) == 1 and resid(xs=1) == 1
    assert resid(rs=1) == 1 and resid(ros=1) == 1 and resid(os=1) == 1 and resid(x=NUL) == 1 and resid(r=ODD) == 1 and resid(w=NUL) == 1
    assert resid(post=ODD) == 1 and resid(scale=ODD) == 1 and resid(ro=NUL) == 1 and resid(eps=-1.0) == 1
    assert resid(rows=0) == 0 and resid(rows=1 << 40) == 2


def test_binding_checks():
    """Wrong types and shapes are refused before the library is asked."""
    c = api.DeltaCache(3, 2, 4, 64, 32, 4, device="cpu")
    bf = torch.bfloat16
    q, v = torch.zeros(4, 2, 64, dtype=bf), torch.zeros(4, 4, 32, dtype=bf)
    g, ids, s = torch.zeros(4, 4), torch.zeros(1, dtype=torch.int32), torch.zeros(64, dtype=torch.uint8)
    for bad in (dict(q=q.float()), dict(q=q[:3]), dict(k=torch.zeros(4, 2, 128, dtype=bf)[..., ::2]), dict(v=v.transpose(1, 2)),
                dict(out=torch.zeros(4, 8, 32, dtype=bf)[:, ::2]), dict(g=g[:3]), dict(beta=g.double()), dict(slot_idx=ids.long()),
                dict(accepted=torch.zeros(0, dtype=torch.int32)), dict(cu_seqlens=ids)):
        kw = dict(q=q, k=q, v=v, g=g, beta=g, slot_idx=ids, accepted=ids, T=4, out=v.clone(), scratch=s)
        kw.update(bad)
        with pytest.raises(ValueError):
            api.rssm_delta_step(c, **kw)
    with pytest.raises(ValueError):
        api.rssm_delta_prefill(c, q, q, v, g, g, ids, ids, v, s)  # bounds too short
    with pytest.raises(ValueError):
        api.DeltaCache(3, 2, 4, 64, 32, 4, device="cpu", state=torch.zeros(3, 4, 64, 32).transpose(2, 3))
    with pytest.raises(ValueError):
        api.DeltaCache(3, 2, 4, 64, 32, 4, state_dtype=api.I8, device="cpu")
    t, i4 = torch.zeros(4, 10), torch.zeros(4, dtype=torch.int32)
    f4, i1, f1 = torch.zeros(4), torch.zeros(1, dtype=torch.int32), torch.zeros(1)
    for bad in (dict(target=t.double()), dict(tokens=i4[:3]), dict(u=f4.half()), dict(draft=t[:3]), dict(draft=t.half()), dict(accepted=f1),
                dict(next_token=i1.long()), dict(cu_seqlens=i1), dict(target=torch.zeros(10, 4).t())):
        kw = dict(target=t, tokens=i4, u=f4, u_next=f1, T=4, accepted=i1, next_token=i1)
        kw.update(bad)
        with pytest.raises(ValueError):
            api.rssm_verify(**kw)
    x, w = torch.zeros(3, 64), torch.ones(64)
    for bad in (dict(x=x.double()), dict(z=x.half()), dict(z=x[:2]), dict(weight=w[:31]), dict(weight=w.half()), dict(out=torch.zeros(64, 3).t())):
        kw = dict(x=x, z=x, weight=w, out=x, group=32)
        kw.update(bad)
        with pytest.raises(ValueError):
            api.rssm_gated_norm(**kw)
    for bad in (dict(residual=x.half()), dict(residual_out=x.bfloat16()), dict(weight=w[:5]), dict(post_weight=w.double()), dict(scale=w[:5])):
        kw = dict(x=x, residual=x, weight=w, out=x, residual_out=x)
        kw.update(bad)
        with pytest.raises(ValueError):
            api.rssm_residual_norm(**kw)


def test_fast_calls_are_the_abi_calls(lib):
    """The binding's C module makes the library's calls: the same statuses, and refuses what is no argument."""
    f, p, c = _lib.fast(), 1 << 20, cache()
    struct = c._obj
    addr = ctypes.addressof(struct)
    step_args = [addr, p, 256, p, 256, p, 256, p, p, 1.0, 1, p, p, None, 0, 4, 8, p, p, 1 << 20, 0]
    assert f.rssm_delta_step(*step_args) == 0  # empty batch
    step_args[14:16] = [2, 9]
    assert f.rssm_delta_step(*step_args) == 2
    step_args[14:16] = [2, 4]
    step_args[1] = p + 2
    assert f.rssm_delta_step(*step_args) == 1
    prefill_args = [addr, p, 256, p, 256, p, 256, p, p, 1.0, 1, p, p, None, 2, 8, p, p, 8, 0]
    assert f.rssm_delta_prefill(*prefill_args) == 3
    assert f.rssm_verify(p, 100, p, 100, 0, 100, p, p, p, None, 2, 33, 99, p, p, None, 0) == 2
    assert f.rssm_verify(p, 99, p, 100, 0, 100, p, p, p, None, 2, 3, 99, p, p, None, 0) == 1
    assert f.rssm_gated_norm(p, 64, p, 64, 0, p, 0, 0, 64, 32, 1e-5, 0, p, 64, 0) == 0
    assert f.rssm_gated_norm(p, 64, p, 64, 0, p, 0, 4, 64, 48, 1e-5, 0, p, 64, 0) == 1
    assert f.rssm_residual_norm(p, 64, p, 64, 1, 0, None, None, 1.0, p, 0, 64, 1e-5, p, 64, p, 64, 0) == 0
    assert f.rssm_residual_norm(p, 64, p, 64, 1, 2, None, None, 1.0, p, 4, 64, 1e-5, p, 64, p, 64, 0) == 1
    for bad in (step_args[:-1], ["x"] + step_args[1:], step_args[:14] + [1 << 40] + step_args[15:], step_args[:9] + [None] + step_args[10:]):
        with pytest.raises((TypeError, OverflowError)):
            f.rssm_delta_step(*bad)
