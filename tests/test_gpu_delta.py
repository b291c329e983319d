"""The gated delta rule's step and prefill against the rule itself in 64 bits.

Tolerances.  bf16 outputs: one rounding is at most 2^-9 of the value; products
may round their factors to bf16 once more, each term at most 2^-9 off and the
terms' errors independent, so an error of about 2^-9 of the outputs' own size
(their rms over the value columns) is expected and 2^-6 is over five of its
standard deviations; over a whole tensor the errors' norm is at most the sum
of the two, 2^-8.  fp32 states and corrections: factors carry at least 16
bits, at most 2^-17 off a term; 1e-5 of the tensor's norm.  bf16 states: one
rounding, 2^-9, against the norm, and the fp32 error.
"""
import math

import pytest
import torch

from operators_plain import delta_tokens
from speculative_state_replay_gb300 import api

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
SHAPES = [(1, 1, 64, 16), (2, 4, 128, 64), (1, 3, 128, 80), (2, 2, 64, 256), (4, 8, 128, 128), (2, 6, 64, 112)]


def close(x, ref):
    x, ref = x.double(), ref.double()
    assert torch.isfinite(x).all()
    if not x.numel():
        return
    rms = ref.pow(2).mean(-1, keepdim=True).sqrt()
    bad = (x - ref).abs() > 2.0**-8 * ref.abs() + 2.0**-6 * rms + 1e-30
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outputs off"
    assert (x - ref).norm() <= 2.0**-8 * ref.norm() + 1e-30


def near(x, ref, tol):
    x, ref = x.double(), ref.double()
    assert torch.isfinite(x).all()
    assert (x - ref).norm() <= tol * ref.norm() + 1e-30, float((x - ref).norm() / ref.norm())


def tokens(n, hk, hv, dk, dv, gen, pad=0, decay=0.3):
    dev = gen.device
    w = 2 * hk * dk + hv * dv + pad
    proj = torch.randn(n, w, generator=gen, device=dev).to(BF)
    q = proj[:, : hk * dk].unflatten(1, (hk, dk))
    k = proj[:, hk * dk : 2 * hk * dk].unflatten(1, (hk, dk))
    v = proj[:, 2 * hk * dk : 2 * hk * dk + hv * dv].unflatten(1, (hv, dv))
    g = -decay * torch.rand(n, hv, generator=gen, device=dev)
    beta = torch.rand(n, hv, generator=gen, device=dev)
    return q, k, v, g, beta


def small_keys(tk, l2norm, dk):
    """Without normalisation keys of norm about 1 keep the rule contracting."""
    q, k, v, g, beta = tk
    return tk if l2norm else (q, (k / math.sqrt(dk)).to(BF), v, g, beta)


def cu_of(lens, dev):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=dev)


@pytest.fixture
def gen():
    return torch.Generator(device="cuda").manual_seed(20261206)


@pytest.mark.parametrize("state", [api.F32, api.BF16])
@pytest.mark.parametrize("l2norm", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_prefill_lengths(gen, shape, l2norm, state):
    hk, hv, dk, dv = shape
    lens = [1, 64, 0, 7, 65, 130, 8, 63, 9, 191, 2]
    n, tot = len(lens), sum(lens)
    tk = small_keys(tokens(tot, hk, hv, dk, dv, gen, pad=8), l2norm, dk)
    cache = api.DeltaCache(n + 1, hk, hv, dk, dv, 4, state)
    start = 0.3 * torch.randn(cache.state.shape, generator=gen, device="cuda")
    cache.state.copy_(start)
    before = cache.state.clone()
    cache.pend.fill_(1)
    slots = (torch.randperm(n, generator=gen, device="cuda") + 1).int()
    initial = torch.tensor([i % 2 for i in range(n)], dtype=torch.int32, device="cuda")
    out = torch.full((tot, hv, dv), 7.0, dtype=BF, device="cuda")
    scratch = api.alloc_delta_scratch(cache, n, tot)
    cu = cu_of(lens, "cuda")
    api.rssm_delta_prefill(cache, *tk, slots, cu, out, scratch, initial=initial, l2norm=l2norm, scale=0.25)
    torch.cuda.synchronize()
    for b, m in enumerate(lens):
        at, s = int(cu[b]), int(slots[b])
        S0 = before[s] if b % 2 else torch.zeros_like(before[s])
        o, _, S = delta_tokens(S0, *(x[at : at + m] for x in tk), 0.25, l2norm)
        close(out[at : at + m], o)
        near(cache.state[s], S, 1e-5 if state == api.F32 else 2.0**-9 + 1e-5)
    assert torch.equal(cache.state[0], before[0])
    assert (cache.pend[1:] == 0).all() and (cache.pend[0] == 1).all()
    assert int(cache.error_word) == 0


@pytest.mark.parametrize("T", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("shape", SHAPES)
def test_steps_follow_the_accepted_tokens(gen, shape, T):
    """Several steps with random acceptances: outputs and, after a last commit, states are those of the rule over the
    accepted tokens alone; the rejected drafts (some of them NaN) leave nothing behind."""
    hk, hv, dk, dv = shape
    B, steps = 5, 4
    l2norm = T != 3
    cache = api.DeltaCache(B + 2, hk, hv, dk, dv, T, api.F32)
    cache.state.copy_(0.3 * torch.randn(cache.state.shape, generator=gen, device="cuda"))
    slots = torch.tensor([3, 1, 0, 6, 2], dtype=torch.int32, device="cuda")  # row 2 is padding
    ref = {b: cache.state[int(slots[b])].double() for b in range(B)}
    acc = torch.zeros(B, dtype=torch.int32, device="cuda")
    scratch = api.alloc_delta_scratch(cache, B, B * T)
    cpu = torch.Generator().manual_seed(T)
    for step in range(steps):
        lens = torch.randint(0, T + 1, (B,), generator=cpu).tolist() if step % 2 else [T] * B
        tot = sum(lens)
        tk = small_keys(tokens(tot, hk, hv, dk, dv, gen), l2norm, dk)
        nxt = [int(torch.randint(0, m + 1, (1,), generator=cpu)) for m in lens]
        cu = cu_of(lens, "cuda")
        for b, m in enumerate(lens):  # the last of the drafts that will be rejected
            if step == 2 and nxt[b] < m:
                tk[2][int(cu[b]) + m - 1] = float("nan")
        out = torch.empty(tot, hv, dv, dtype=BF, device="cuda")
        api.rssm_delta_step(cache, *tk, slots, acc, T, out, scratch, cu_seqlens=cu if step % 2 else None, l2norm=l2norm)
        for b, m in enumerate(lens):
            at = int(cu[b])
            if int(slots[b]) == 0:
                assert (out[at : at + m] == 0).all()
                continue
            live = m - (1 if step == 2 and nxt[b] < m else 0)
            o, u, S = delta_tokens(ref[b], *(x[at : at + m] for x in tk), dk**-0.5, l2norm, keep=nxt[b])
            close(out[at : at + live], o[:live])
            near(cache.state[int(slots[b])], ref[b], 1e-5)
            side, count = cache.pend[int(slots[b])].tolist()
            assert count == m
            r = tk[1][at : at + live].double().pow(2).sum(-1).add(1e-6).rsqrt() if l2norm else torch.ones(live, hk, device="cuda")
            near(cache.pend_w[int(slots[b]), side, :, :live].transpose(0, 1), u[:live] * r.repeat_interleave(hv // hk, 1)[..., None], 1e-5)
            ref[b] = S
        acc = torch.tensor(nxt, dtype=torch.int32, device="cuda")
    # a step of no tokens commits
    e = torch.empty(0, hv, dv, dtype=BF, device="cuda")
    none = tokens(0, hk, hv, dk, dv, gen)
    api.rssm_delta_step(cache, *none, slots, acc, T, e, scratch, cu_seqlens=torch.zeros(B + 1, dtype=torch.int32, device="cuda"),
                        l2norm=l2norm)
    for b in range(B):
        if int(slots[b]):
            near(cache.state[int(slots[b])], ref[b], 1e-5)
            assert cache.pend[int(slots[b]), 1] == 0
    assert int(cache.error_word) == 0 and (scratch[: 4 * B] == 0).all()


def test_step_bf16_state_and_padded_slots(gen):
    hk, hv, dk, dv, T, B = 2, 4, 128, 128, 4, 3
    big = torch.zeros(B + 1, hv * dv * dk + 64, dtype=BF, device="cuda")
    state = big[:, : hv * dv * dk].unflatten(1, (hv, dv, dk))
    state.copy_(0.3 * torch.randn(state.shape, generator=gen, device="cuda"))
    cache = api.DeltaCache(B + 1, hk, hv, dk, dv, T, api.BF16, state=state)
    before = state.clone()
    slots = torch.tensor([2, 3, 1], dtype=torch.int32, device="cuda")
    tk = tokens(B * T, hk, hv, dk, dv, gen)
    out = torch.empty(B * T, hv, dv, dtype=BF, device="cuda")
    scratch = api.alloc_delta_scratch(cache, B, B * T)
    api.rssm_delta_step(cache, *tk, slots, None, T, out, scratch, l2norm=True)
    assert torch.equal(cache.state, before)
    tk2 = tokens(B * T, hk, hv, dk, dv, gen)
    acc = torch.tensor([T, 0, 2], dtype=torch.int32, device="cuda")
    api.rssm_delta_step(cache, *tk2, slots, acc, T, out, scratch, l2norm=True)
    for b in range(B):
        part = slice(b * T, b * T + T)
        _, _, S = delta_tokens(before[int(slots[b])], *(x[part] for x in tk), dk**-0.5, True, keep=int(acc[b]))
        o, _, _ = delta_tokens(S, *(x[part] for x in tk2), dk**-0.5, True)
        close(out[part], o)
        near(cache.state[int(slots[b])], S, 2.0**-9 + 1e-5)
    assert torch.equal(cache.state[int(slots[1])], before[int(slots[1])])
    assert (big[:, hv * dv * dk :] == 0).all()


def test_step_refuses_on_the_device(gen):
    hk, hv, dk, dv, T, B = 1, 2, 64, 32, 4, 4
    cache = api.DeltaCache(B + 1, hk, hv, dk, dv, T)
    cache.state.copy_(torch.randn(cache.state.shape, generator=gen, device="cuda"))
    scratch = api.alloc_delta_scratch(cache, B, B * T)
    slots = torch.arange(1, B + 1, dtype=torch.int32, device="cuda")
    out = torch.full((B * T, hv, dv), 7.0, dtype=BF, device="cuda")
    tk = tokens(B * T, hk, hv, dk, dv, gen)
    before = cache.state.clone()
    api.rssm_delta_step(cache, *tk, slots, torch.tensor([0, 1, -1, 0], dtype=torch.int32, device="cuda"), T, out, scratch)
    assert int(cache.error_word) == api.ERRBIT_ACCEPT  # no draft waits yet
    assert (out[T : 3 * T] == 0).all() and (out[:T] != 0).any() and torch.equal(cache.state, before)
    assert cache.pend[:, 1].tolist() == [0, T, 0, 0, T]
    cache.error_word.zero_()
    out.fill_(7.0)
    bad = torch.tensor([0, 4, 9, 8, 17], dtype=torch.int32, device="cuda")  # rows of 4, 5 (> T), -1, and past the tokens
    api.rssm_delta_step(cache, *tk, slots, None, T, out, scratch, cu_seqlens=bad)
    assert int(cache.error_word) == api.ERRBIT_SEQLEN
    assert (out[:4] != 7.0).any() and (out[4:] == 7.0).all()
    cache.error_word.zero_()
    api.rssm_delta_prefill(cache, *tk, slots, bad, out, scratch)
    assert int(cache.error_word) == api.ERRBIT_SEQLEN


def test_strong_decays_and_neighbours(gen):
    """g of -inf resets a state; a NaN prompt leaves its neighbours alone."""
    hk, hv, dk, dv = 1, 2, 128, 64
    lens = [70, 40, 75]
    tot = sum(lens)
    q, k, v, g, beta = tokens(tot, hk, hv, dk, dv, gen)
    g[20] = -math.inf
    g[64] = -math.inf
    g[118:123] = -60.0
    for x in (q, k, v):
        x[70:110] = float("nan")
    beta[75] = float("inf")
    cache = api.DeltaCache(4, hk, hv, dk, dv, 4)
    cache.state.copy_(torch.randn(cache.state.shape, generator=gen, device="cuda"))
    before = cache.state.clone()
    slots = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    out = torch.empty(tot, hv, dv, dtype=BF, device="cuda")
    scratch = api.alloc_delta_scratch(cache, 3, tot)
    one = torch.ones(3, dtype=torch.int32, device="cuda")
    cu = cu_of(lens, "cuda")
    api.rssm_delta_prefill(cache, q, k, v, g, beta, slots, cu, out, scratch, initial=one, l2norm=True)
    for b in (0, 2):
        part = slice(int(cu[b]), int(cu[b + 1]))
        o, _, S = delta_tokens(before[b + 1], q[part], k[part], v[part], g[part], beta[part], dk**-0.5, True)
        close(out[part], o)
        near(cache.state[b + 1], S, 1e-4)  # running sums near 200 are held to 2^-17


def test_equal_keys(gen):
    """The hardest triangular system: one key for every token, rates near one, no decay."""
    hk, hv, dk, dv, n = 1, 1, 128, 32, 200
    q, k, v, g, beta = tokens(n, hk, hv, dk, dv, gen, decay=0.0)
    k[:] = k[:1]
    beta[:] = 1.0 - 0.01 * beta
    cache = api.DeltaCache(2, hk, hv, dk, dv, 4)
    out = torch.empty(n, hv, dv, dtype=BF, device="cuda")
    scratch = api.alloc_delta_scratch(cache, 1, n)
    slots = torch.ones(1, dtype=torch.int32, device="cuda")
    api.rssm_delta_prefill(cache, q, k, v, g, beta, slots, cu_of([n], "cuda"), out, scratch, l2norm=True)
    o, _, S = delta_tokens(torch.zeros(hv, dv, dk, device="cuda"), q, k, v, g, beta, dk**-0.5, True)
    close(out, o)
    near(cache.state[1], S, 2e-4)  # differences of neighbouring values, which lose two digits


def test_parts_of_a_prompt_equal_the_whole(gen):
    hk, hv, dk, dv, n = 2, 4, 128, 128, 300
    tk = tokens(n, hk, hv, dk, dv, gen)
    whole, parts = (api.DeltaCache(2, hk, hv, dk, dv, 8) for _ in range(2))
    scratch = api.alloc_delta_scratch(whole, 1, n)
    slots = torch.ones(1, dtype=torch.int32, device="cuda")
    out, out2 = (torch.empty(n, hv, dv, dtype=BF, device="cuda") for _ in range(2))
    api.rssm_delta_prefill(whole, *tk, slots, cu_of([n], "cuda"), out, scratch, l2norm=True)
    at = 0
    for m in (1, 100, 64, 131):
        x = [t[at : at + m] for t in tk]
        o = torch.empty(m, hv, dv, dtype=BF, device="cuda")
        api.rssm_delta_prefill(parts, *x, slots, cu_of([m], "cuda"), o, scratch, l2norm=True,
                               initial=torch.full((1,), int(at > 0), dtype=torch.int32, device="cuda"))
        out2[at : at + m] = o
        at += m
    x = [t[at:] for t in tk]  # the last 4 as a step, all accepted, then committed
    api.rssm_delta_step(parts, *x, slots, None, 4, out2[at:], scratch, l2norm=True)
    none = [t[:0] for t in tk]
    api.rssm_delta_step(parts, *none, slots, torch.full((1,), 4, dtype=torch.int32, device="cuda"), 4, out2[:0], scratch,
                        cu_seqlens=torch.zeros(2, dtype=torch.int32, device="cuda"), l2norm=True)
    close(out2, out.double())
    near(parts.state[1], whole.state[1], 1e-5)


def test_streams_graphs_and_determinism(gen):
    """The same bits on another stream, from a captured graph and twice in a row."""
    hk, hv, dk, dv, T, B = 2, 4, 128, 128, 3, 6
    lens = [90, 3, 128, 1, 64, 77]
    tot = sum(lens)
    tk, tk2 = tokens(tot, hk, hv, dk, dv, gen), tokens(B * T, hk, hv, dk, dv, gen)
    slots = torch.arange(1, B + 1, dtype=torch.int32, device="cuda")
    acc = torch.tensor([3, 0, 1, 2, 3, 3], dtype=torch.int32, device="cuda")
    cu = cu_of(lens, "cuda")

    def run(how):
        cache = api.DeltaCache(B + 1, hk, hv, dk, dv, T)
        scratch = api.alloc_delta_scratch(cache, B, tot)
        out, out2 = torch.empty(tot, hv, dv, dtype=BF, device="cuda"), torch.empty(B * T, hv, dv, dtype=BF, device="cuda")

        def calls():
            api.rssm_delta_prefill(cache, *tk, slots, cu, out, scratch, l2norm=True)
            api.rssm_delta_step(cache, *tk2, slots, None, T, out2, scratch, l2norm=True)
            api.rssm_delta_step(cache, *tk2, slots, acc, T, out2, scratch, l2norm=True)

        torch.cuda.synchronize()
        if how == "graph":
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                calls()
            g.replay()
        elif how == "stream":
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                calls()
            st.synchronize()
        else:
            calls()
        torch.cuda.synchronize()
        return out, out2, cache.state, cache.pend_w, cache.pend

    first = run("plain")
    for how in ("plain", "stream", "graph"):
        for x, y in zip(first, run(how)):
            assert torch.equal(x, y), how


def test_slots_past_32_bits(gen):
    """States whose element offsets pass 2^31."""
    hk, hv, dk, dv, T = 2, 32, 128, 128, 2
    S = (1 << 31) // (hv * dv * dk) + 9
    cache = api.DeltaCache(S, hk, hv, dk, dv, T, api.BF16)
    s = S - 1
    cache.state[s] = 0.3 * torch.randn(cache.state[s].shape, generator=gen, device="cuda")
    S0 = cache.state[s].clone()
    slots = torch.tensor([s], dtype=torch.int32, device="cuda")
    scratch = api.alloc_delta_scratch(cache, 1, 70)
    tk = tokens(70, hk, hv, dk, dv, gen)
    out = torch.empty(70, hv, dv, dtype=BF, device="cuda")
    api.rssm_delta_prefill(cache, *tk, slots, cu_of([70], "cuda"), out, scratch, l2norm=True,
                           initial=torch.ones(1, dtype=torch.int32, device="cuda"))
    o, _, St = delta_tokens(S0, *tk, dk**-0.5, True)
    close(out, o)
    near(cache.state[s], St, 2.0**-9 + 1e-5)
    tk = tokens(T, hk, hv, dk, dv, gen)
    S0, out = cache.state[s].clone(), out[:T]
    api.rssm_delta_step(cache, *tk, slots, None, T, out, scratch, l2norm=True)
    close(out, delta_tokens(S0, *tk, dk**-0.5, True)[0])
    assert (cache.state[: S - 1].view(torch.int16).amax() == 0) and int(cache.error_word) == 0


def test_scratch_is_shared_by_calls_of_other_sizes(gen):
    """A small prompt between the steps of a larger batch, on one buffer: the steps' counters stay at zero."""
    hk, hv, dk, dv, T, B = 1, 2, 64, 32, 2, 300
    cache = api.DeltaCache(B + 1, hk, hv, dk, dv, T)
    scratch = torch.zeros(max(api.rssm_delta_scratch_bytes(cache, B, B * T), api.rssm_delta_scratch_bytes(cache, 1, 500)),
                          dtype=torch.uint8, device="cuda")
    slots = torch.arange(1, B + 1, dtype=torch.int32, device="cuda")
    acc = torch.zeros(B, dtype=torch.int32, device="cuda")
    out = torch.empty(B * T, hv, dv, dtype=BF, device="cuda")
    for step in range(3):
        api.rssm_delta_step(cache, *tokens(B * T, hk, hv, dk, dv, gen), slots, acc, T, out, scratch, l2norm=True)
        assert cache.pend[1:].tolist() == [[(step + 1) % 2, T]] * B
        o = torch.empty(500, hv, dv, dtype=BF, device="cuda")
        other = api.DeltaCache(2, hk, hv, dk, dv, T)
        api.rssm_delta_prefill(other, *tokens(500, hk, hv, dk, dv, gen), slots[:1], cu_of([500], "cuda"), o, scratch, l2norm=True)
    assert int(cache.error_word) == 0 and (scratch[: 4 * 65536] == 0).all()
