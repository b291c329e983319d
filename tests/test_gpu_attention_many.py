"""Attention of many queries of a head where it can go wrong: what is not finite and not seen, bad rows, other layouts, captured
calls, two calls at once, pages far apart.  The tolerance is test_gpu_attention's: the output's rounding and each weight's."""
import math

import pytest
import torch

import attention_plain as P
import test_gpu_attention as A
from test_gpu_attention import _api, check_rows, make_cache, offsets, tree  # noqa: F401

pytestmark = pytest.mark.gpu


def tensors(gen, n, hq, h, d):
    return (torch.randn(n, x, d, generator=gen, device="cuda").bfloat16() for x in (hq, h, h))


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("fmt", ["BF16", "I8", "E4M3"])
@pytest.mark.parametrize("d,is_tree", [(64, True), (128, False), (128, True)])
def test_unseen_values_do_not_reach(fmt, d, is_tree):
    lengths, new, h, hq = [21, 300], [45, 64], 2, 8
    cache, table, gen = make_cache(getattr(A.api, fmt), d, h, 16, lengths, new)
    q, k, v = tensors(gen, sum(new), hq, h, d)
    parents = [tree(n, 5 + b) if is_tree else None for b, n in enumerate(new)]
    bad = [[7, 30], [2, 40, 41]]  # places in their rows
    ln, cu = ints(lengths), offsets(new)
    pt = ints(parents[0] + parents[1]) if is_tree else None
    kb, vb = k.clone(), v.clone()
    for b, places in enumerate(bad):
        for j, t in enumerate(places):
            (vb if j % 2 == 0 else kb)[b * new[0] + t, :, 3 + j] = (math.nan, math.inf, -math.inf)[j]
    scratch, out = A.api.alloc_attention_scratch(cache, hq), torch.zeros_like(q)
    A.api.rssm_kv_append(cache, kb, vb, table, ln, 64, cu_seqlens=cu)
    A.api.rssm_tree_attention(cache, q, table, ln, 64, out, scratch, parents=pt, cu_seqlens=cu)
    KB, VB = P.decoded(cache, "k"), P.decoded(cache, "v")
    A.api.rssm_kv_append(cache, k, v, table, ln, 64, cu_seqlens=cu)  # those who do not see them: as if they were others
    K, V = P.decoded(cache, "k"), P.decoded(cache, "v")
    weight = 2.0**-8 if fmt == "BF16" else 2.0**-11
    spared = 0
    for b, n in enumerate(new):
        kk, vv = (P.row_tokens(x, table[b].cpu(), 16, 0, lengths[b] + n) for x in (K, V))
        want, size = P.attention_row(kk, vv, q[b * new[0] :][:n].cpu(), parents[b], lengths[b], d**-0.5)
        shown, _ = P.attention_row(*(P.row_tokens(x, table[b].cpu(), 16, 0, lengths[b] + n) for x in (KB, VB)), q[b * new[0] :][:n].cpu(), parents[b],
                                   lengths[b], d**-0.5)
        for t in range(n):
            got = out[b * new[0] + t].cpu().double()
            if any(x in P.path(parents[b], t) for x in bad[b]):
                # as the formula has it: a key of inf is a score of inf, and then NaN, or of -inf, and then a weight of 0; 8-bit: NaN
                assert torch.equal(got.isfinite(), shown[t].isfinite())
            else:
                spared += 1
                assert ((got - want[t]).abs() - (2.0**-8 * want[t].abs() + (weight + 2.0**-12) * size[t])).max() <= 0
    assert spared >= 9
    assert int(cache.error_word) == 0


@pytest.mark.parametrize("fmt", ["BF16", "E4M3"])
def test_bad_rows(fmt):
    """Bad pages, tables, counts and parents set their bit; only their own rows are concerned."""
    api, d, h, hq, T = A.api, 128, 1, 2, 40
    lengths, new = [40, 200, 40, 150], [T] * 4
    cache, table, gen = make_cache(getattr(api, fmt), d, h, 16, lengths, new)
    q, k, v = tensors(gen, 4 * T, hq, h, d)
    ln, cu = ints(lengths), offsets(new)
    api.rssm_kv_append(cache, k, v, table, ln, T, cu_seqlens=cu)
    scratch = api.alloc_attention_scratch(cache, hq)
    K, V = P.decoded(cache, "k"), P.decoded(cache, "v")

    def again(bit, row, what, parents=None, pages=table, at=ln, bounds=cu):
        out = torch.full((4 * T, hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
        api.rssm_tree_attention(cache, q, pages, at, T, out, scratch, parents=None if parents is None else ints(parents), cu_seqlens=bounds)
        assert int(cache.error_word) == bit
        cache.error_word.zero_()
        for b in range(4):
            got = out[b * T : (b + 1) * T].cpu().double()
            if b == row and what is not None:
                assert bool((got == what).all())
                continue
            gone = 16 if b == row else 0  # the page that is none holds the first 16 tokens
            kk, vv = (P.row_tokens(x, table[b].cpu(), 16, gone, lengths[b] + T - gone) for x in (K, V))
            up = None if parents is None else parents[b * T : (b + 1) * T]
            want, size = P.attention_row(kk, vv, q[b * T : (b + 1) * T].cpu(), up, lengths[b] - gone, d**-0.5)
            weight = 2.0**-8 if fmt == "BF16" else 2.0**-11
            assert ((got - want).abs() - (2.0**-8 * want.abs() + (weight + 2.0**-12) * size)).max() <= 0

    again(0, -1, None)
    again(api.ERRBIT_PAGE, 1, 0.0, at=ints([40, 2**31 - 1, 40, 150]))
    again(0, 2, 0.0, at=ints([40, 200, -7, 150]))
    again(api.ERRBIT_SEQLEN, 3, 3.0, bounds=ints([0, T, 2 * T, 3 * T, 4 * T + 1]))
    chain = [-1] + list(range(T - 1))
    again(api.ERRBIT_TREE, 0, 0.0, parents=[-1, 1] + chain[2:] + 3 * chain)
    again(api.ERRBIT_TREE, 3, 0.0, parents=3 * chain + chain[:-1] + [-2])
    for page in (-1, cache.pages, 2**31 - 1):
        t = table.clone()
        t[1, 0] = page
        again(api.ERRBIT_PAGE, 1, None, pages=t)


@pytest.mark.parametrize("fmt,page,new,is_tree", [("BF16", 48, [64, 5, 33], True), ("I8", 80, [130, 1, 40], False), ("E4M3", 256, [64, 64, 2], True),
                                                  ("BF16", 256, [300, 40, 0], False)])
def test_pages_and_layers(fmt, page, new, is_tree):
    """Pages that end inside a step of tokens or hold several, keys and values side by side, and a layer that is not the first."""
    api, d, h, hq, lengths = A.api, 128, 2, 8, [0, 517, 200]
    f = getattr(api, fmt)
    B = 3
    need = [-(-(a + b) // page) for a, b in zip(lengths, new)]
    total = sum(need) + 1
    dtype = {"BF16": torch.bfloat16, "I8": torch.int8, "E4M3": torch.uint8}[fmt]
    both = torch.zeros(3, total, 2, h, page, d, dtype=dtype, device="cuda")
    scales = None if fmt == "BF16" else torch.full((3, total, 2, h, page), math.nan, device="cuda")
    own = {} if scales is None else dict(k_scale=scales[:, :, 0], v_scale=scales[:, :, 1])
    cache = api.KVCache(total, h, d, page, f, layers=3, k=both[:, :, 0], v=both[:, :, 1], **own)
    gen = torch.Generator(device="cuda").manual_seed(page)
    order = torch.randperm(total, generator=gen, device="cuda").int()
    table, at = torch.full((B, max(need)), -5, dtype=torch.int32, device="cuda"), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at : at + n]
        at += n
    for first, count in (([0] * B, lengths), (lengths, new)):
        _, k, v = tensors(gen, sum(count), 1, h, d)
        api.rssm_kv_append(cache, k, v, table, ints(first), max(count), cu_seqlens=offsets(count), layer=2)
    q = torch.randn(sum(new), hq, d, generator=gen, device="cuda").bfloat16()
    parents = sum((tree(n, b) for b, n in enumerate(new)), []) if is_tree else None
    out = torch.zeros_like(q)
    api.rssm_tree_attention(cache, q, table, ints(lengths), max(new), out, api.alloc_attention_scratch(cache, hq),
                            parents=None if parents is None else ints(parents), cu_seqlens=offsets(new), layer=2)
    own = {} if scales is None else dict(k_scale=scales[2:, :, 0], v_scale=scales[2:, :, 1])
    one = api.KVCache(total, h, d, page, f, k=both[2:, :, 0], v=both[2:, :, 1], **own)
    check_rows(one, table, lengths, new, q, parents, out, d**-0.5)
    assert int(cache.error_word) == 0 and not both[:2].any()


@pytest.mark.parametrize("fmt,T", [("BF16", 24), ("I8", 24), ("E4M3", 5)])
def test_captured_and_at_once(fmt, T):
    """A captured step replayed on other inputs and lengths, while another stream runs calls with scratch of their own."""
    api, d, h, hq, lengths, new = A.api, 128, 2, 8, [700, 3, 90], [T] * 3
    cache, table, gen = make_cache(getattr(api, fmt), d, h, 16, lengths, [T + 8] * 3)
    ln = ints(lengths)
    q, k, v = (torch.zeros(3 * T, x, d, dtype=torch.bfloat16, device="cuda") for x in (hq, h, h))
    out, scratch = torch.zeros_like(q), api.alloc_attention_scratch(cache, hq)

    def step():
        api.rssm_kv_append(cache, k, v, table, ln, T)
        api.rssm_tree_attention(cache, q, table, ln, T, out, scratch)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    other, table2, _ = make_cache(api.BF16, d, h, 32, [400, 400], [40, 40], seed=9)
    q2, k2, v2 = tensors(gen, 80, hq, h, d)
    ln2, scratch2 = ints([400, 400]), api.alloc_attention_scratch(other, hq)
    api.rssm_kv_append(other, k2, v2, table2, ln2, 40)
    alone, along = torch.zeros_like(q2), torch.zeros(20, *q2.shape, dtype=torch.bfloat16, device="cuda")
    api.rssm_tree_attention(other, q2, table2, ln2, 40, alone, scratch2)
    st = torch.cuda.Stream()
    for it in range(3):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
        torch.cuda.synchronize()
        along.zero_()
        st.wait_stream(torch.cuda.current_stream())
        for i in range(20):
            api.rssm_tree_attention(other, q2, table2, ln2, 40, along[i], scratch2, stream=st)
            if i == 5:
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, alone) for x in along)
        check_rows(cache, table, ln.tolist(), new, q, None, out, d**-0.5)
        ln += ints([3, 2, 0])
    assert int(cache.error_word) == 0 and int(other.error_word) == 0


@pytest.mark.parametrize("fmt,T", [("BF16", 3), ("BF16", 30), ("I8", 3), ("E4M3", 30)])
@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_scales(fmt, T, scale):
    """No scale, a negative one, and one that leaves most weights at nothing; heads of keys and values that are zero or tiny."""
    api, d, h, hq, lengths, new = A.api, 64, 2, 8, [150, 9], [T, T]
    cache, table, gen = make_cache(getattr(api, fmt), d, h, 16, lengths, new)
    q, k, v = tensors(gen, 2 * T, hq, h, d)
    k[0], v[1], k[2], v[2] = 0, 0, 2.0**-60, 2.0**-90
    cu, ln = offsets(new), ints(lengths)
    api.rssm_kv_append(cache, k, v, table, ln, T, cu_seqlens=cu)
    out = torch.zeros_like(q)
    api.rssm_tree_attention(cache, q, table, ln, T, out, api.alloc_attention_scratch(cache, hq), cu_seqlens=cu, scale=scale)
    # A weight of an 8-bit cache is fp16 times 2^11 or more, against a maximum that is the largest or below it: an error of up to
    # 2^-25 2^-11 of the largest p_j b_j (b: the values' scales, here at most 1), where the largest's value may be the zero one.
    # Times codes of at most 448 of each token: what the output may be off by, whatever the other values add up to.
    slack = 0.0 if fmt == "BF16" else 2.0**-36 * 448 * (max(lengths) + T)
    check_rows(cache, table, lengths, new, q, None, out, scale, slack)


@pytest.mark.parametrize("fmt", ["BF16", "I8"])
def test_far_pages(fmt):
    """Pages past 2^32 bytes: the same bits as near."""
    api, d, h, hq, page, T = A.api, 128, 1, 2, 64, 40
    big = 270000 if fmt == "BF16" else 530000
    far, near = (api.KVCache(n, h, d, page, getattr(api, fmt)) for n in (big, 80))
    gen = torch.Generator(device="cuda").manual_seed(5)
    n = 64 * 70 + 3
    q, _, _ = tensors(gen, T, hq, h, d)
    _, k, v = tensors(gen, n + T, hq, h, d)
    outs = []
    for c, first in ((far, big - 72), (near, 0)):
        table = torch.arange(first, first + 72, dtype=torch.int32, device="cuda").view(1, -1)
        api.rssm_kv_append(c, k, v, table, ints([0]), n + T)
        out = torch.zeros(T, hq, d, dtype=torch.bfloat16, device="cuda")
        api.rssm_tree_attention(c, q, table, ints([n]), T, out, api.alloc_attention_scratch(c, hq))
        outs.append(out)
    assert torch.equal(*outs)
    check_rows(near, table, [n], [T], q, None, outs[1], d**-0.5)
