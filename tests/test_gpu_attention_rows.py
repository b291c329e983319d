"""rssm_tree_attention on rows and calls where its kernels can go wrong; both kernels, and both ways in which the one for many
queries cuts its work."""
import math

import pytest
import torch

from test_gpu_attention import check_rows, make_cache, offsets

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
