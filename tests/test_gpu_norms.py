"""The norms around a block against their definitions in 64 bits.

Tolerances: 2-byte outputs are rounded once, at most half a unit in the last
place (2^-9 bf16, 2^-12 f16 of the value, taken twice for values next to a
boundary), and fp32 arithmetic before it adds less than 2e-6 of the value: a
sum over n terms in fp32 is off by less than n 2^-24 at worst and about
sqrt(n) 2^-24 here, rsqrt and the gate's exp and division a few 2^-22.
"""
import pytest
import torch

from operators_plain import gated_norm, residual_norm
from speculative_state_replay_gb300 import api

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
ULP = {torch.float32: 0.0, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}


def close(x, ref, dtype):
    x = x.double()
    assert torch.isfinite(x).all()
    tiny = 2.0**-24 if dtype is torch.float16 else 1e-30  # f16's subnormal spacing
    bad = (x - ref).abs() > (ULP[dtype] + 4e-6) * ref.abs() + tiny
    assert not bad.any(), float(((x - ref).abs() / ref.abs().clamp(min=1e-30)).max())


def rnd(gen, *s):
    return torch.randn(s, generator=gen, device="cuda")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group,groups", [(1, 3), (2, 2), (7, 5), (64, 3), (128, 4), (129, 2), (512, 2), (1000, 3), (1024, 2),
                                          (4096, 1), (5000, 2), (16384, 1), (36864, 1), (9001, 1)])
def test_gated_norm(group, groups, dtype):
    gen = torch.Generator(device="cuda").manual_seed(group)
    D = group * groups
    for rows, first, shared in ((1, False, False), (9, True, True), (33, False, True), (5, True, False)):
        x, z = rnd(gen, rows, D).to(dtype), (2.0 * rnd(gen, rows, D)).to(dtype)
        w = 1.0 + 0.2 * rnd(gen, group if shared else D)
        out = torch.empty_like(x)
        api.rssm_gated_norm(x, z, w, out, group, eps=1e-5, norm_first=first)
        close(out, gated_norm(x, z, w, group, 1e-5, first), dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("dim", [1, 5, 64, 513, 1000, 4096, 5120, 12288, 33000, 40960])
def test_residual_norm(dim, f32, dtype):
    gen = torch.Generator(device="cuda").manual_seed(dim)
    for rows, has_post, has_scale in ((1, False, False), (6, True, False), (3, False, True), (17, True, True)):
        x = rnd(gen, rows, dim).to(dtype)
        res = (2.0 * rnd(gen, rows, dim)).to(torch.float32 if f32 else dtype)
        w = 1.0 + 0.2 * rnd(gen, dim)
        post = 1.0 + 0.2 * rnd(gen, dim) if has_post else None
        scale = 0.5 + 0.2 * rnd(gen, dim) if has_scale else None
        out, rout = torch.empty_like(x), torch.empty_like(res)
        api.rssm_residual_norm(x, res, w, out, rout, post_weight=post, scale=scale, alpha=0.7, eps=1e-5)
        h, o = residual_norm(x, res, w, post, scale, 0.7, 1e-5)
        # sums of two terms: an error relative to the terms
        size = res.double().abs() + (h - res.double()).abs()
        ulp = 0.0 if f32 else ULP[dtype]
        assert ((rout.double() - h).abs() <= ulp * h.abs() + 4e-6 * size + 2.0**-24 * (not f32)).all()
        rms = o.pow(2).mean(-1, keepdim=True).sqrt()
        assert ((out.double() - o).abs() <= ULP[dtype] * o.abs() + 1e-5 * (o.abs() + rms) + 2.0**-24).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_strides_alignment_in_place(dtype):
    gen = torch.Generator(device="cuda").manual_seed(2)
    R, D = 7, 768
    wide = rnd(gen, R, 3 * D + 5).to(dtype)
    for at in (0, 8, 3):
        x, z = wide[:, at : at + D].clone(), wide[:, at + D : at + 2 * D]
        w = (1.0 + 0.2 * rnd(gen, D + 1))[1:]  # not on 16 bytes
        ref = gated_norm(x, z, w, 96, 1e-6, False)
        out = torch.zeros(R, D + 8, dtype=dtype, device="cuda")
        api.rssm_gated_norm(x, z, w, out[:, :D], 96, eps=1e-6)
        close(out[:, :D], ref, dtype)
        assert (out[:, D:] == 0).all()
        w2 = w.clone()
        api.rssm_gated_norm(x, z, w2, x, 96, eps=1e-6)
        close(x, ref, dtype)
        x, res = wide[:, at : at + D].clone(), wide[:, at + D : at + 2 * D].float()
        h, o = residual_norm(x, res, w, None, None, 1.0, 1e-6)
        api.rssm_residual_norm(x, res, w2, x, res, eps=1e-6)
        assert ((res.double() - h).abs() <= 1e-6 * h.abs() + 1e-6).all()
        close(x, o, dtype)


def test_edges():
    z = torch.zeros(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    api.rssm_gated_norm(z, z, w, z)
    api.rssm_residual_norm(z, z, w, z, z)
    x = torch.zeros(2, 64, device="cuda")  # zero rows: zero, not NaN
    out = torch.full_like(x, 3.0)
    api.rssm_gated_norm(x, x, w, out)
    assert (out == 0).all()
    api.rssm_residual_norm(x, x, w, out, torch.empty_like(x), post_weight=w)
    assert (out == 0).all()
    big = torch.full((1, 64), -120.0, device="cuda")  # gates far below zero vanish
    api.rssm_gated_norm(torch.ones_like(big), big, w, out[:1], norm_first=True)
    assert (out[0].abs() < 1e-30).all()
    big = torch.full((3, 64), 1.0, device="cuda")
    big[1] = float("nan")  # a row's NaN stays in its row
    api.rssm_gated_norm(big, torch.ones_like(big), w, out := torch.empty_like(big), 32)
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[2]).all() and torch.isnan(out[1]).all()


def test_stream_and_graph():
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, z, w = rnd(gen, 50, 512).bfloat16(), rnd(gen, 50, 512).bfloat16(), rnd(gen, 512)
    out = [torch.empty_like(x) for _ in range(3)]
    api.rssm_gated_norm(x, z, w, out[0], 128)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        api.rssm_gated_norm(x, z, w, out[1], 128)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.rssm_gated_norm(x, z, w, out[2], 128)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [255, 1025, 2047, 4001, 4097, 2056, 8200, 32768, 32776])
def test_gated_norm_long_groups(group, dtype):
    """Lengths on both sides of what a thread's vectors hold, odd ones value by value."""
    gen = torch.Generator(device="cuda").manual_seed(group)
    for rows, first in ((1, False), (5, True)):
        x, z = rnd(gen, rows, 2 * group).to(dtype), (2.0 * rnd(gen, rows, 2 * group)).to(dtype)
        w = 1.0 + 0.2 * rnd(gen, group)
        out = torch.empty_like(x)
        api.rssm_gated_norm(x, z, w, out, group, eps=1e-5, norm_first=first)
        close(out, gated_norm(x, z, w, group, 1e-5, first), dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shift", [0, 4, 8, 1])
@pytest.mark.parametrize("dim", [1001, 2048, 4001, 8192, 16384, 16392])
def test_residual_norm_alignment(dim, shift, dtype):
    """fp32 residuals and weights on 32 bytes, on 16, and on neither, give the same rows."""
    gen = torch.Generator(device="cuda").manual_seed(dim)
    R = 3
    x = rnd(gen, R, dim).to(dtype)
    full = 2.0 * rnd(gen, R * (dim + 8))
    vec = [1.0 + 0.2 * rnd(gen, dim) for _ in range(3)]
    res = full[: R * dim].view(R, dim).contiguous()
    w, post, scale = vec
    want, rwant = torch.empty_like(x), torch.empty_like(res)
    api.rssm_residual_norm(x, res, w, want, rwant, post_weight=post, scale=scale, alpha=0.7, eps=1e-5)
    pad = torch.empty(R * dim + 16, device="cuda")
    moved = pad[shift : shift + R * dim].view(R, dim).copy_(res)
    wv = [torch.empty(dim + 16, device="cuda")[shift : shift + dim].copy_(v) for v in vec]
    out, rout = torch.empty_like(x), torch.empty(R * dim + 16, device="cuda")[shift : shift + R * dim].view(R, dim)
    api.rssm_residual_norm(x, moved, wv[0], out, rout, post_weight=wv[1], scale=wv[2], alpha=0.7, eps=1e-5)
    h, o = residual_norm(x, res, w, post, scale, 0.7, 1e-5)
    rms = o.pow(2).mean(-1, keepdim=True).sqrt()
    for a, r in ((want, rwant), (out, rout)):
        size = res.double().abs() + (h - res.double()).abs()
        assert ((r.double() - h).abs() <= 4e-6 * size).all()
        assert ((a.double() - o).abs() <= ULP[dtype] * o.abs() + 1e-5 * (o.abs() + rms) + 2.0**-24).all()
