"""rssm_logits against its definition in 64 bits, through the public call."""
import math
import random

import pytest
import torch

import attention_plain as P

pytestmark = pytest.mark.gpu
api = None
HALF = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}  # a rounding is off by that much at most


@pytest.fixture(scope="module", autouse=True)
def _api():
    global api
    from speculative_state_replay_gb300 import api as a

    api = a


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(V, lens, H, seed, tree=False, bias=0, mask=False, dtype=torch.float32, prompts=True):
    rng, gen = random.Random(seed), torch.Generator(device="cuda").manual_seed(seed)
    n, ntok = len(lens), sum(lens)
    few = [rng.randrange(V) for _ in range(30)]
    some = lambda m: [rng.choice(few) if rng.random() < 0.7 else rng.randrange(V) for _ in range(m)]  # noqa: E731
    c = dict(V=V, lens=lens, x=(3 * torch.randn(ntok, V, generator=gen, device="cuda")).to(dtype))
    c["history"] = [some(rng.randint(0, H)) for _ in range(n)]
    c["prompt"] = [rng.randint(0, len(h)) if prompts else 0 for h in c["history"]]
    c["tokens"] = some(ntok)
    c["parents"] = [-1 if t == 0 else rng.randint(-1, t - 1) for m in lens for t in range(m)] if tree else None
    u = lambda lo, hi: torch.rand(n, generator=gen, device="cuda") * (hi - lo) + lo  # noqa: E731
    c["repetition"], c["presence"], c["frequency"], c["temperature"] = u(0.8, 1.5), u(-0.2, 1.0), u(0.0, 0.4), u(0.3, 2.0)
    c["bias"] = [[(i, rng.gauss(0, 3)) for i in some(rng.randint(0, bias))] for _ in range(n)] if bias else None
    c["mask"] = [[rng.random() < 0.6 for _ in range(V)] for _ in range(ntok)] if mask else None
    return c


def packed(mask, V):
    words = (V + 31) // 32
    out = torch.zeros(len(mask), words, dtype=torch.int64)
    for r, row in enumerate(mask):
        for i, ok in enumerate(row):
            out[r, i // 32] |= ok << (i % 32)
    return torch.where(out >= 1 << 31, out - (1 << 32), out).int().cuda()


def call(c, out, **kw):
    H = max([len(h) for h in c["history"]] + [1])
    flat = [e for b in (c["bias"] or []) for e in b]
    starts = [0]
    for b in c["bias"] or []:
        starts.append(starts[-1] + len(b))
    cu = [0]
    for m in c["lens"]:
        cu.append(cu[-1] + m)
    args = dict(temperature=c["temperature"], repetition=c["repetition"], presence=c["presence"], frequency=c["frequency"],
                history=ints([h + [0] * (H - len(h)) for h in c["history"]]), history_len=ints([len(h) for h in c["history"]]),
                prompt_len=ints(c["prompt"]), tokens=ints(c["tokens"]), parents=None if c["parents"] is None else ints(c["parents"]),
                bias_start=ints(starts) if c["bias"] else None, bias_id=ints([e[0] for e in flat]) if c["bias"] else None,
                bias_value=torch.tensor([e[1] for e in flat], device="cuda") if c["bias"] else None,
                mask=None if c["mask"] is None else packed(c["mask"], c["V"]), cu_seqlens=ints(cu))
    args.update(kw)
    api.rssm_logits(c["x"], max(c["lens"]), out, **args)


def rows(c, probs=True):
    """What the definition gives, and the largest |x| / temperature that an exponent is formed from."""
    at, biases = 0, c["bias"] or [[] for _ in c["lens"]]
    f = lambda name, b: float(c[name][b])  # noqa: E731
    for b, m in enumerate(c["lens"]):
        for t in range(m):
            fed = [c["tokens"][at + j] for j in P.path(None if c["parents"] is None else c["parents"][at : at + m], t)]
            bias = [(i, float(torch.tensor(y))) for i, y in biases[b]]
            mask = None if c["mask"] is None else c["mask"][at + t]
            a = (c["x"][at + t].cpu().float(), c["history"][b], c["prompt"][b], fed, f("repetition", b), f("presence", b), f("frequency", b), bias, mask,
                 f("temperature", b))
            yield at + t, P.logits_row(*a, probs=probs), P.logits_row(*a, probs=False)
        at += m


def check(c, out, probs=True):
    got = out.cpu().double()
    for r, want, x in rows(c, probs):
        # the processed logit: at most 5 + (biases of an id) fp32 operations on values up to `big`; softmax: that and the
        # difference from the maximum in the exponent, expf 2 units in the last place, the sum and its reciprocal
        fine = x[x.isfinite()].abs()
        big = float(fine.max()) if len(fine) else 0.0
        few = 12 * 2.0**-24 * max(big, 1.0)
        if probs:
            tol = want * (HALF[out.dtype] + 2 * few + 16 * 2.0**-24) + (2.0**-25 if out.dtype == torch.float16 else 2.0**-134 if out.dtype == torch.bfloat16 else 2.0**-126)
        else:
            same = want == got[r]
            assert bool((same | want.isfinite()).all())
            want = torch.where(same, got[r], want)
            tol = want.abs() * HALF[out.dtype] + few
            tol = torch.where(same, torch.zeros_like(tol), tol)
        d = torch.where(want == got[r], torch.zeros_like(want), (got[r] - want).abs())
        assert bool((d <= tol).all()), (r, float((d - tol).max()))


@pytest.mark.parametrize("V,lens,H,tree,bias,mask,dtype,out", [
    (1, [1], 3, False, 0, False, torch.float32, torch.float32),
    (33, [2, 1], 40, False, 5, True, torch.bfloat16, torch.float32),
    (1000, [4, 0, 7, 1], 300, True, 40, True, torch.float16, torch.bfloat16),
    (4097, [3], 900, False, 700, False, torch.float32, torch.float16),
    (32000, [2], 100, False, 0, True, torch.bfloat16, torch.bfloat16),
    (70001, [1, 2], 2000, True, 60, False, torch.float16, torch.float32),
    (262144, [1], 5000, False, 3, False, torch.float32, torch.float32),
])
def test_logits(V, lens, H, tree, bias, mask, dtype, out):
    c = make(V, lens, H, V + H, tree, bias, mask, dtype)
    for probs in (True, False):
        y = torch.full((sum(lens) + 1, V), 9.0, dtype=out, device="cuda")[:-1]
        call(c, y, probs=probs)
        check(c, y, probs)
        assert bool((y._base[-1] == 9.0).all())


def test_many_rows_strides_and_in_place():
    """More rows than run at once (one block a row), rows of another alignment, and the result over the logits."""
    c = make(3001, [5] * 70, 50, 1, bias=4)
    wide = torch.zeros(350, 3011, device="cuda")
    wide[:, 3:3004] = c["x"]
    y = torch.zeros(350, 3001, device="cuda")
    call(c, y)
    check(c, y)
    c2 = dict(c, x=wide[:, 3:3004])
    z = torch.zeros(350, 3004, dtype=torch.float32, device="cuda")[:, 1:3002]
    call(c2, z)
    check(c, z)  # (how a row is cut goes by its alignment: each result is within its own roundings of the definition)
    call(c2, c2["x"])
    check(c, c2["x"])
    assert torch.equal(z, c2["x"]) and not wide[:, :3].any() and not wide[:, 3004:].any()


def test_edges():
    """Greedy rows and their ties, infinities, NaN, all masked, nothing given."""
    V = 5000
    x = torch.randn(6, V, device="cuda")
    x[0, 70] = x[0, 4999] = x[0, 4000] = 50.0
    x[1] = -math.inf
    x[2, 10] = x[2, 4500] = math.inf
    x[3, 5] = math.nan
    x[4, :] = 0.0
    x[4, 1::2] = -0.0
    out = torch.empty_like(x)
    t = torch.tensor([0.0, 1.0, 0.5, 0.0, 0.0, 1.0], device="cuda")
    api.rssm_logits(x, 1, out, temperature=t)
    want = torch.zeros(6, V, dtype=torch.float64)
    want[0, 70] = 1
    want[2, 10] = want[2, 4500] = 0.5
    y = x[3].cpu().clone()
    y[5] = -math.inf
    want[3, y.argmax()] = 1
    want[4, 0] = 1
    want[5] = torch.softmax(x[5].cpu().double(), 0)
    assert torch.equal(out[:5].cpu().double(), want[:5])
    assert float((out[5].cpu().double() - want[5]).abs().max()) < 1e-6 * float(want[5].max())
    # temperatures of any size
    x = torch.randn(4, V, device="cuda")
    mask = torch.full((4, (V + 31) // 32), -2, dtype=torch.int32, device="cuda")  # ids 0, 32, .. are out
    api.rssm_logits(x, 1, out[:4], temperature=torch.tensor([1e-42, math.inf, math.nan, -1.0], device="cuda"), mask=mask)
    allowed = torch.arange(V) % 32 != 0
    z = torch.where(allowed, x.cpu().double(), -math.inf)
    got = out[:4].cpu().double()
    assert torch.equal(got[0], torch.zeros(V, dtype=torch.float64).index_fill_(0, z[0].argmax(), 1.0))
    assert float((got[1] - allowed / allowed.sum()).abs().max()) < 1e-6 / V
    for r in (2, 3):
        w = torch.softmax(z[r], 0)
        assert float(((got[r] - w).abs() - 4e-6 * w).max()) <= 0
    mask.zero_()
    api.rssm_logits(x, 1, out[:4], mask=mask)
    assert not out[:4].any()


def test_same_bias_many_times_and_same_bits():
    """One id thousands of times among the biases: in order, the same bits every time."""
    V = 9000
    gen = torch.Generator(device="cuda").manual_seed(1)
    n = 3000
    ids = torch.randint(0, 3, (n,), generator=gen, device="cuda").int() * 4000
    ids[100:200] = torch.tensor([-1, V, 2**31 - 1, -(2**31)] * 25, dtype=torch.int32)
    val = torch.randn(n, generator=gen, device="cuda") * 10 ** torch.randint(-4, 4, (n,), generator=gen, device="cuda")
    x = torch.zeros(1, V, device="cuda")
    outs = [torch.empty_like(x) for _ in range(3)]
    for y in outs:
        api.rssm_logits(x, 1, y, bias_start=ints([0, n + 50]), bias_id=ids, bias_value=val, probs=False)  # past the last entry: left out
    want = torch.zeros(V)
    for i in (0, 4000, 8000):
        s = torch.zeros(())
        part = []
        on = [(k, float(v)) for k, v in zip(ids.tolist(), val.tolist())]
        for k, v in on:
            if k == i:
                part.append(v)
        want[i] = sum(part)
    assert all(torch.equal(outs[0], y) for y in outs)
    assert float((outs[0].cpu()[0] - want).abs().max()) <= n * 2.0**-24 * float(val.abs().sum())
    # in order: the same as adding them one after the other in fp32
    import numpy as np

    for i in (0, 4000, 8000):
        s = np.float32(0)
        for k, v in zip(ids.tolist(), val.cpu().numpy()):
            if k == i:
                s = np.float32(s + v)
        assert float(outs[0][0, i]) == float(s)


def test_bad_rows():
    c = make(300, [2, 2, 2], 20, 3, tree=True)
    good = torch.zeros(6, 300, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    call(c, good, error_word=word)
    assert int(word) == 0
    out = torch.full((6, 300), 4.0, device="cuda")
    call(c, out, error_word=word, cu_seqlens=ints([0, 2, 4, 7]))
    assert int(word) == api.ERRBIT_SEQLEN and torch.equal(out[:4], good[:4]) and bool((out[4:] == 4.0).all())
    word.zero_()
    p = list(c["parents"])
    p[3] = 1  # itself
    call(c, out, error_word=word, parents=ints(p))
    assert int(word) == api.ERRBIT_TREE and torch.equal(out[[0, 1, 4, 5]], good[[0, 1, 4, 5]])
    # lengths outside the history's are held to it, ids outside the vocabulary are not counted
    word.zero_()
    H = max(len(h) for h in c["history"])
    more = ints([h + [-5, 300, 2**31 - 1] + [-1] * (H - len(h)) for h in c["history"]])
    call(c, out, error_word=word, history=more, history_len=ints([2**31 - 1] * 3))
    assert int(word) == 0 and torch.equal(out, good)
    call(c, out, history_len=ints([-3] * 3), prompt_len=ints([99] * 3), cu_seqlens=None)
    c["history"] = [[] for _ in c["history"]]
    check(c, out)
