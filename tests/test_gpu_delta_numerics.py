"""The gated delta rule where fp32 arithmetic shows: states that need all of their 24 bits, strong decays in mid-step,
decay factors by themselves, and a log decay that is NaN.

Every bound below is derived in its test from the operations that the rule needs in fp32: a sum of n products is off by
at most a few 2^-23 of the sum of their magnitudes (the tensor cores add 16 products at a time, four such sums one after
another), an exponential by 2 units in the last place.
"""
import math

import pytest
import torch

from operators_plain import delta_tokens
from speculative_state_replay_gb300 import api

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
SHAPES = [(1, 1, 64, 16), (2, 4, 128, 64), (1, 3, 128, 80), (2, 2, 64, 256), (4, 8, 128, 128)]


@pytest.fixture
def gen():
    return torch.Generator(device="cuda").manual_seed(20261207)


def ones(*shape, dtype=BF):
    return torch.ones(shape, dtype=dtype, device="cuda")


def rnd(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def off(x, ref):
    return float((x.double() - ref.double()).norm() / ref.double().norm())


@pytest.mark.parametrize("shape", SHAPES)
def test_step_takes_a_state_as_it_is(gen, shape):
    """Values of 1 + 2^-10 + 2^-18 that all add up: the last bit is 2^-18 of S k.  One token, so that u = v - S k, which
    is what is left of values that the state predicts.  S k is off by at most 5 2^-23 of sum |S k| (four sums of 16
    products, two more additions), v and the subtraction by 2^-24 each: 2^-20 of it."""
    hk, hv, dk, dv = shape
    B = 3
    cache = api.DeltaCache(B + 1, hk, hv, dk, dv, 1)
    sign = torch.where(rnd(gen, hv, dk) > 0, 1.0, -1.0)
    size = torch.exp2(torch.randint(-2, 3, (B + 1, hv, dv, 1), generator=gen, device="cuda").float())
    cache.state.copy_((1.0 + 2.0**-10 + 2.0**-18) * size * sign[:, None, :])
    k = (rnd(gen, B, hk, dk).abs() + 0.5).to(BF) * sign.view(hk, hv // hk, dk)[:, 0].to(BF)
    for h in range(hv):  # value heads of one key head share its signs
        cache.state[:, h] = cache.state[:, h].abs() * sign[h // (hv // hk) * (hv // hk)]
    S = cache.state[1:].double()
    kd = k.double().repeat_interleave(hv // hk, 1)
    Sk = torch.einsum("bhvk,bhk->bhv", S, kd)
    v = Sk.to(BF)
    g, beta = torch.zeros(B, hv, device="cuda"), torch.ones(B, hv, device="cuda")
    out = torch.empty(B, hv, dv, dtype=BF, device="cuda")
    slots = torch.arange(1, B + 1, dtype=torch.int32, device="cuda")
    api.rssm_delta_step(cache, k, k, v, g, beta, slots, None, 1, out, api.alloc_delta_scratch(cache, B, B))
    u = v.double() - Sk
    got = cache.pend_w[1:, 1, :, 0].double()
    size = torch.einsum("bhvk,bhk->bhv", S.abs(), kd.abs())
    assert ((got - u).abs() <= 2.0**-20 * size).all(), float(((got - u).abs() / size).max())


def many_resets(gen, n, hv):
    """Log decays with resets (-inf), near ones and ordinary ones in every order."""
    g = -0.5 * torch.rand(n, hv, generator=gen, device="cuda")
    kind = torch.rand(n, hv, generator=gen, device="cuda")
    g = torch.where(kind < 0.3, torch.full_like(g, -math.inf), g)
    return torch.where((kind >= 0.3) & (kind < 0.5), g - 60.0, g)


@pytest.mark.parametrize("T", [2, 5, 8])
def test_resets_in_mid_step(gen, T):
    """Resets and decays of -60 among a step's tokens, then a commit.  What a later token's factors need is a difference
    of running sums that is O(1), whatever the sums are: corrections, and the state after the commit, are fp32 sums of
    at most 136 terms with factors that are a few 2^-23 off: 1e-6 of their norm."""
    hk, hv, dk, dv, B = 2, 4, 128, 64, 12
    cache = api.DeltaCache(B + 1, hk, hv, dk, dv, T)
    cache.state.copy_(0.3 * rnd(gen, *cache.state.shape))
    scratch = api.alloc_delta_scratch(cache, B, B * T)
    slots = torch.arange(1, B + 1, dtype=torch.int32, device="cuda")
    before = cache.state.clone()
    q, k, v = rnd(gen, B * T, hk, dk).to(BF), rnd(gen, B * T, hk, dk).to(BF), rnd(gen, B * T, hv, dv).to(BF)
    g, beta = many_resets(gen, B * T, hv), torch.rand(B * T, hv, generator=gen, device="cuda")
    out = torch.empty(B * T, hv, dv, dtype=BF, device="cuda")
    api.rssm_delta_step(cache, q, k, v, g, beta, slots, None, T, out, scratch, l2norm=True)
    acc = torch.tensor([b % T + 1 for b in range(B)], dtype=torch.int32, device="cuda")
    want, us = [], []
    for b in range(B):
        part = slice(b * T, b * T + T)
        _, u, S = delta_tokens(before[b + 1], q[part], k[part], v[part], g[part], beta[part], dk**-0.5, True, keep=int(acc[b]))
        want.append(S)
        us.append(u * (k[part].double().pow(2).sum(-1) + 1e-6).rsqrt().repeat_interleave(hv // hk, 1)[..., None])
    assert off(cache.pend_w[1:, 1].transpose(1, 2), torch.stack(us)) <= 1e-6
    none = [x[:0] for x in (q, k, v, g, beta)]
    api.rssm_delta_step(cache, *none, slots, acc, T, out[:0], scratch, l2norm=True,
                        cu_seqlens=torch.zeros(B + 1, dtype=torch.int32, device="cuda"))
    for b in range(B):
        assert off(cache.state[b + 1], want[b]) <= 1e-6, b


@pytest.mark.parametrize("how", ["step", "prompt"])
def test_decay_of_a_state(gen, how):
    """Keys of zero: the state is multiplied by e^c and nothing else.  expf is at most 2 units (2^-22) off and the
    product half a one: 5 2^-24."""
    hk, hv, dk, dv, B = 4, 8, 64, 32, 8
    cache = api.DeltaCache(B + 1, hk, hv, dk, dv, 2)
    cache.state.copy_(rnd(gen, *cache.state.shape))
    before = cache.state[1:].double()
    c = -8.0 - 8.0 * torch.rand(B, hv, generator=gen, device="cuda")
    slots = torch.arange(1, B + 1, dtype=torch.int32, device="cuda")
    zero = torch.zeros(B, hk, dk, dtype=BF, device="cuda")
    v, beta = torch.zeros(B, hv, dv, dtype=BF, device="cuda"), torch.ones(B, hv, device="cuda")
    out = torch.empty_like(v)
    scratch = api.alloc_delta_scratch(cache, B, B)
    if how == "prompt":
        api.rssm_delta_prefill(cache, zero, zero, v, c, beta, slots, torch.arange(B + 1, dtype=torch.int32, device="cuda"), out,
                               scratch, initial=torch.ones(B, dtype=torch.int32, device="cuda"))
    else:
        api.rssm_delta_step(cache, zero, zero, v, c, beta, slots, None, 1, out, scratch)
        api.rssm_delta_step(cache, zero, zero, v, c, beta, slots, torch.ones(B, dtype=torch.int32, device="cuda"), 1, out, scratch)
    want = before * torch.exp(c.double())[..., None, None]
    worst = float(((cache.state[1:].double() - want).abs() / want.abs()).max())
    assert worst <= 5 * 2.0**-24, worst


def test_a_nan_decay_in_a_step(gen):
    """One head's log decay of token 2 is NaN: its outputs are NaN from there on, and so is its state once that token is
    accepted; earlier tokens and the other head do not know."""
    hk, hv, dk, dv, T, B = 1, 2, 64, 32, 5, 2
    cache = api.DeltaCache(B + 1, hk, hv, dk, dv, T)
    cache.state.copy_(0.3 * rnd(gen, *cache.state.shape))
    before = cache.state.clone()
    scratch = api.alloc_delta_scratch(cache, B, B * T)
    slots = torch.arange(1, B + 1, dtype=torch.int32, device="cuda")
    q, k, v = rnd(gen, B * T, hk, dk).to(BF), rnd(gen, B * T, hk, dk).to(BF), rnd(gen, B * T, hv, dv).to(BF)
    g, beta = -torch.rand(B * T, hv, generator=gen, device="cuda"), torch.rand(B * T, hv, generator=gen, device="cuda")
    g[[2, T + 2], 1] = math.nan
    out = torch.empty(B * T, hv, dv, dtype=BF, device="cuda")
    api.rssm_delta_step(cache, q, k, v, g, beta, slots, None, T, out, scratch, l2norm=True)
    clean = g.nan_to_num(nan=-0.1)
    ref = [delta_tokens(before[b + 1], *(x[b * T : b * T + T] for x in (q, k, v, clean, beta)), dk**-0.5, True, keep=[2, 4][b])
           for b in range(B)]
    for b in range(B):
        o = out[b * T : b * T + T]
        assert torch.isnan(o[2:, 1]).all()
        assert off(o[:, 0], ref[b][0][:, 0]) <= 2.0**-8 and off(o[:2, 1], ref[b][0][:2, 1]) <= 2.0**-8
        assert torch.isnan(cache.pend_c[b + 1, 1, 1, 2:]).all() and torch.isfinite(cache.pend_c[b + 1, 1, 1, :2]).all()
    api.rssm_delta_step(cache, q, k, v, clean, beta, slots, torch.tensor([2, 4], dtype=torch.int32, device="cuda"), T, out, scratch,
                        l2norm=True)
    assert off(cache.state[1], ref[0][2]) <= 1e-5 and off(cache.state[2, 0], ref[1][2][0]) <= 1e-5
    assert torch.isnan(cache.state[2, 1]).all()


def test_a_nan_decay_in_a_prompt(gen):
    """The head's outputs are NaN from the token on, its state too; the chunks before, the other head and the other
    prompt do not know."""
    hk, hv, dk, dv = 1, 2, 128, 64
    lens = [150, 90]
    tot = sum(lens)
    q, k, v = rnd(gen, tot, hk, dk).to(BF), rnd(gen, tot, hk, dk).to(BF), rnd(gen, tot, hv, dv).to(BF)
    g, beta = -torch.rand(tot, hv, generator=gen, device="cuda"), torch.rand(tot, hv, generator=gen, device="cuda")
    ref = [delta_tokens(torch.zeros(hv, dv, dk, device="cuda"), *(x[a : a + n] for x in (q, k, v, g, beta)), dk**-0.5, True)
           for a, n in ((0, 150), (150, 90))]
    g[100, 1] = math.nan
    cache = api.DeltaCache(3, hk, hv, dk, dv, 2)
    out = torch.empty(tot, hv, dv, dtype=BF, device="cuda")
    api.rssm_delta_prefill(cache, q, k, v, g, beta, torch.tensor([1, 2], dtype=torch.int32, device="cuda"),
                           torch.tensor([0, 150, 240], dtype=torch.int32, device="cuda"), out, api.alloc_delta_scratch(cache, 2, tot),
                           l2norm=True)
    assert torch.isnan(out[100:150, 1]).all() and torch.isnan(cache.state[1, 1]).all()
    assert off(out[:150, 0], ref[0][0][:, 0]) <= 2.0**-8 and off(out[:64, 1], ref[0][0][:64, 1]) <= 2.0**-8
    assert off(out[150:], ref[1][0]) <= 2.0**-8
    assert off(cache.state[1, 0], ref[0][2][0]) <= 1e-5 and off(cache.state[2], ref[1][2]) <= 1e-5


@pytest.mark.parametrize("n", [77, 300])
@pytest.mark.parametrize("corr", [0.7, 0.95])
def test_prompts_of_correlated_keys(gen, n, corr):
    """Prompts take fp32 factors in 16 significant bits (include/rssm.h): a factor is at most 2^-17 off, a product of two
    2^-16, and the solve multiplies that by its own size, about one where keys are normalised and rates below one.
    2^-15 of an fp32 state's norm; outputs do not show it (2^-8 as everywhere)."""
    hk, hv, dk, dv = 2, 4, 128, 64
    q, k = ((corr * rnd(gen, 1, hk, dk) + math.sqrt(1 - corr * corr) * rnd(gen, n, hk, dk)).to(BF) for _ in range(2))
    v = rnd(gen, n, hv, dv).to(BF)
    g, beta = -0.02 * torch.rand(n, hv, generator=gen, device="cuda"), 0.9 + 0.1 * torch.rand(n, hv, generator=gen, device="cuda")
    cache = api.DeltaCache(2, hk, hv, dk, dv, 2)
    out = torch.empty(n, hv, dv, dtype=BF, device="cuda")
    api.rssm_delta_prefill(cache, q, k, v, g, beta, torch.ones(1, dtype=torch.int32, device="cuda"),
                           torch.tensor([0, n], dtype=torch.int32, device="cuda"), out, api.alloc_delta_scratch(cache, 1, n), l2norm=True)
    o, _, S = delta_tokens(torch.zeros(hv, dv, dk, device="cuda"), q, k, v, g, beta, dk**-0.5, True)
    assert off(out, o) <= 2.0**-8 and off(cache.state[1], S) <= 2.0**-15


@pytest.mark.parametrize("corr", [0.0, 0.95])
def test_steps_of_correlated_keys(gen, corr):
    """The same tokens by steps of 8, all accepted, keep fp32: 136 terms a product and a decay a commit, each a few 2^-24
    off, over 19 commits: 2e-6."""
    hk, hv, dk, dv, n = 2, 4, 128, 64, 152
    q, k = ((corr * rnd(gen, 1, hk, dk) + math.sqrt(1 - corr * corr) * rnd(gen, n, hk, dk)).to(BF) for _ in range(2))
    v = rnd(gen, n, hv, dv).to(BF)
    g, beta = -0.02 * torch.rand(n, hv, generator=gen, device="cuda"), 0.9 + 0.1 * torch.rand(n, hv, generator=gen, device="cuda")
    cache = api.DeltaCache(2, hk, hv, dk, dv, 8)
    scratch, slot = api.alloc_delta_scratch(cache, 1, 8), torch.ones(1, dtype=torch.int32, device="cuda")
    out = torch.empty(n, hv, dv, dtype=BF, device="cuda")
    for at in range(0, n, 8):
        x = [t[at : at + 8] for t in (q, k, v, g, beta)]
        api.rssm_delta_step(cache, *x, slot, slot * (8 if at else 0), 8, out[at : at + 8], scratch, l2norm=True)
    none = [t[:0] for t in (q, k, v, g, beta)]
    api.rssm_delta_step(cache, *none, slot, slot * 8, 8, out[:0], scratch, l2norm=True,
                        cu_seqlens=torch.zeros(2, dtype=torch.int32, device="cuda"))
    o, _, S = delta_tokens(torch.zeros(hv, dv, dk, device="cuda"), q, k, v, g, beta, dk**-0.5, True)
    assert off(out, o) <= 2.0**-8 and off(cache.state[1], S) <= 2e-6
