"""rssm_tree_attention on rows and calls where its kernels can go wrong; both kernels, and both ways in which the one for many
queries cuts its work."""
import math

import pytest
import torch

from test_gpu_attention import check_rows, make_cache, offsets, tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _api():
    import test_gpu_attention as A
    from speculative_state_replay_gb300 import api

    A.api = api


def api():
    import test_gpu_attention as A

    return A.api


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def tensors(gen, n, hq, h, d):
    return (torch.randn(n, x, d, generator=gen, device="cuda").bfloat16() for x in (hq, h, h))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sms", [1, 5, None])
def test_many_short_pieces(monkeypatch, sms, d):
    """Rows of one to three steps of tokens, all of which some query does not see, by blocks that take many of them in turn."""
    if sms:
        monkeypatch.setenv("RSSM_SM_LIMIT", str(sms))
    h, hq, T, lengths = 2, 8, 40, [0, 90, 200, 128, 1, 300, 88, 87] * 8
    new = [T - b % 3 for b in range(len(lengths))]
    cache, table, gen = make_cache(api().BF16, d, h, 16, lengths, new)
    q, k, v = tensors(gen, sum(new), hq, h, d)
    ln, cu = ints(lengths), offsets(new)
    api().rssm_kv_append(cache, k, v, table, ln, T, cu_seqlens=cu)
    scratch, first = api().alloc_attention_scratch(cache, hq), torch.zeros_like(q)
    api().rssm_tree_attention(cache, q, table, ln, T, first, scratch, cu_seqlens=cu)
    out = torch.zeros_like(q)
    for _ in range(60):
        api().rssm_tree_attention(cache, q, table, ln, T, out, scratch, cu_seqlens=cu)
    assert int(cache.error_word) == 0 and torch.equal(out, first)
    check_rows(cache, table, lengths[:8], new[:8], q, None, out, d**-0.5)


def test_a_warp_that_gives_up_does_not_keep_its_partner():
    """Of two warps that meet in every step one's wait runs out, the other's does not: the kernel ends, and calls go on as before."""
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    for ms in (1, 20):
        api().rssm_selftest_wait_timeout(word, wait_ms=ms)
        torch.cuda.synchronize()
        assert int(word) == api().ERRBIT_TIMEOUT
    lengths, new, d, h, hq = [200, 3], [40, 40], 64, 2, 8
    cache, table, gen = make_cache(api().I8, d, h, 16, lengths, new)
    q, k, v = tensors(gen, 80, hq, h, d)
    api().rssm_kv_append(cache, k, v, table, ints(lengths), 40)
    out = torch.zeros_like(q)
    api().rssm_tree_attention(cache, q, table, ints(lengths), 40, out, api().alloc_attention_scratch(cache, hq))
    assert int(cache.error_word) == 0
    check_rows(cache, table, lengths, new, q, None, out, d**-0.5)


@pytest.mark.parametrize("T,sms", [(2, None), (40, None), (40, 1)])  # few queries; many; many, a segment a block
def test_any_negative_length_is_padding(monkeypatch, T, sms):
    if sms:
        monkeypatch.setenv("RSSM_SM_LIMIT", str(sms))
    d, h, hq, lengths = 64, 2, 4, [-2, 30, -1, -(2**31), 0, -3]
    new = [T] * len(lengths)
    cache, table, gen = make_cache(api().BF16, d, h, 16, lengths, new)
    q, k, v = tensors(gen, sum(new), hq, h, d)
    ln, cu = ints(lengths), offsets(new)
    api().rssm_kv_append(cache, k, v, table, ln, T, cu_seqlens=cu)
    out = torch.full_like(q, 7.0)
    api().rssm_tree_attention(cache, q, table, ln, T, out, api().alloc_attention_scratch(cache, hq), cu_seqlens=cu)
    assert int(cache.error_word) == 0
    check_rows(cache, table, lengths, new, q, None, out, d**-0.5)


@pytest.mark.parametrize("T", [2, 40])
def test_what_is_not_finite_beside_a_missing_page(T):
    """A row of three hundred tokens without its second page: NaN and infinities in the other pages reach all queries, which see them."""
    d, h, hq, lengths, new = 64, 2, 4, [300, 300], [T, T]
    cache, table, gen = make_cache(api().BF16, d, h, 16, lengths, new)
    q, k, v = tensors(gen, sum(new), hq, h, d)
    ln, cu = ints(lengths), offsets(new)
    api().rssm_kv_append(cache, k, v, table, ln, T, cu_seqlens=cu)
    cache.v[0, int(table[0, 3]), 0, 5, 11] = math.inf
    cache.v[0, int(table[0, 3]), 1, 7, 60] = math.nan
    holes = table.clone()
    holes[0, 1] = -1
    out = torch.zeros_like(q)
    api().rssm_tree_attention(cache, q, holes, ln, T, out, api().alloc_attention_scratch(cache, hq), cu_seqlens=cu)
    assert int(cache.error_word) == api().ERRBIT_PAGE
    got = out[:T].float().cpu().view(T, h, hq // h, d)
    assert bool((got[:, 0, :, 11] == math.inf).all()) and bool(got[:, 1, :, 60].isnan().all())
    got[:, 0, :, 11] = got[:, 1, :, 60] = 0.0
    assert bool(got.isfinite().all())
    check_rows(cache, table[1:], lengths[1:], new[1:], q[T:], None, out[T:], d**-0.5)


@pytest.mark.parametrize("fmt", ["I8", "E4M3"])
@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("power", [-96, 100, 118, 126])
def test_values_of_any_size(fmt, T, power):
    """Values up to the largest of bf16, whose scales pass 2^118, and as small as the cache's scales go."""
    d, h, hq, lengths, new = 64, 2, 8, [200, 9], [T, T]
    cache, table, gen = make_cache(getattr(api(), fmt), d, h, 16, lengths, new)
    q, k, _ = tensors(gen, 2 * T, hq, h, d)
    ln, cu = ints(lengths), offsets(new)
    draw = lambda n: ((torch.rand(n, h, d, generator=gen, device="cuda") * 2 - 1) * 2.0**power).bfloat16()  # noqa: E731
    old = draw(sum(lengths))
    kk = torch.randn(sum(lengths), h, d, generator=gen, device="cuda").bfloat16()
    api().rssm_kv_append(cache, kk, old, table, ints([0, 0]), max(lengths), cu_seqlens=offsets(lengths))
    api().rssm_kv_append(cache, k, draw(2 * T), table, ln, T, cu_seqlens=cu)
    out = torch.zeros_like(q)
    api().rssm_tree_attention(cache, q, table, ln, T, out, api().alloc_attention_scratch(cache, hq), cu_seqlens=cu)
    assert int(cache.error_word) == 0
    # check_rows has the output's rounding and the weights'; what a weight of an 8-bit cache is off by below the fp16 range (2^-36 of
    # the largest p_j b_j) times codes of at most 448.  Scales are at most 2^power / 127 (1 + 2^-8), and the tokens 240.  The inverse
    # of the largest scale, 2^119, has 14 bits left in the sum's unit: 2^-15 of a weight, within the 2^-12 that are counted.
    check_rows(cache, table, lengths, new, q, None, out, d**-0.5, 2.0**-36 * 448 * (max(lengths) + T) * 2.0**power / 126)


REPEAT = [
    # format, head_dim, query heads, lengths, new tokens, tree
    ("BF16", 128, 8, [3000, 5, 700, 0, -1, 1900], [4, 3, 1, 1, 2, 4], False),
    ("E4M3", 64, 4, [4000, 17], [5, 5], False),
    ("I8", 128, 8, [2500, 5, 700, 0], [64, 3, 33, 1], True),
    ("BF16", 128, 8, [2500, 130, 0, 90], [64, 40, 64, 9], True),
    ("E4M3", 64, 8, [2000, 17, 640], [70, 200, 129], False),
    ("BF16", 256, 4, [1500, 3], [12, 5], True),
]


@pytest.mark.parametrize("fmt,d,hq,lengths,new,is_tree", REPEAT)
@pytest.mark.parametrize("sms", [None, 2, 7])
def test_the_same_call_gives_the_same_bits(monkeypatch, sms, fmt, d, hq, lengths, new, is_tree):
    if sms:
        monkeypatch.setenv("RSSM_SM_LIMIT", str(sms))
    cache, table, gen = make_cache(getattr(api(), fmt), d, 2, 32, lengths, new)
    q, k, v = tensors(gen, sum(new), hq, 2, d)
    ln, cu = ints(lengths), offsets(new)
    api().rssm_kv_append(cache, k, v, table, ln, max(new), cu_seqlens=cu)
    parents = [p for b, m in enumerate(new) for p in tree(m, b)] if is_tree else None
    scratch = api().alloc_attention_scratch(cache, hq)
    outs = torch.full((12, *q.shape), 7.0, dtype=torch.bfloat16, device="cuda")
    for out in outs:
        api().rssm_tree_attention(cache, q, table, ln, max(new), out, scratch, parents=None if parents is None else ints(parents), cu_seqlens=cu)
    assert int(cache.error_word) == 0
    assert all(torch.equal(out.view(torch.int16), outs[0].view(torch.int16)) for out in outs[1:])
    check_rows(cache, table, lengths, new, q, parents, outs[0], d**-0.5)
