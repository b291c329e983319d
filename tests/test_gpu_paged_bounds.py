"""rssm_kv_append and rssm_kv_read on bounds that fall, are too far apart or pass the tokens: the bit is set, the rows that they
spoil are skipped, and every other row is served as if it were alone."""
import pytest
import torch

from test_gpu_attention import offsets

pytestmark = pytest.mark.gpu

H, D, PAGE = 2, 64, 16
BOUNDS = [
    # T, token rows, bounds
    (4, 6, [0, 4, 2, 6]),  # the second row falls; the third begins inside the first
    (5, 8, [0, 5, 3, 8]),
    (8, 8, [0, 8, 12]),  # a row behind the tokens
    (8, 8, [0, 8, 8, 12, 16]),
    (4, 4, [0, 9, 2, 4]),  # too long and past the tokens, then back
    (3, 9, [0, 3, 9, 9]),  # too long
    (4, 6, [-2, 2, 4, 6]),
    (4, 4, [6, 2, 4]),
    (3, 210, [3 * b for b in range(35)] + [90, 93, 96] + [3 * b for b in range(38, 71)]),
    (3, 210, [3 * b for b in range(40)] + [2**31 - 1] + [3 * b for b in range(41, 71)]),
]


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def sound(T, n, cu):
    return [(b, a, z) for b, (a, z) in enumerate(zip(cu, cu[1:])) if 0 <= z - a <= T and a >= 0 and z <= n]


@pytest.mark.parametrize("fmt", ["BF16", "I8", "E4M3"])
@pytest.mark.parametrize("T,n,cu", BOUNDS)
def test_bounds(fmt, T, n, cu):
    from speculative_state_replay_gb300 import api

    batch, good = len(cu) - 1, sound(T, n, cu)
    gen = torch.Generator(device="cuda").manual_seed(n)
    make = lambda: api.KVCache(2 * batch, H, D, PAGE, getattr(api, fmt), layers=2)  # noqa: E731
    cache, want = make(), make()
    table = torch.randperm(2 * batch, generator=gen, device="cuda").int().view(batch, 2)
    lengths = [5 * b % 17 for b in range(batch)]
    k, v = (torch.randn(n, H, D, generator=gen, device="cuda").bfloat16() for _ in range(2))
    api.rssm_kv_append(cache, k, v, table, ints(lengths), T, cu_seqlens=ints(cu), layer=1)
    assert int(cache.error_word) == api.ERRBIT_SEQLEN
    for b, a, z in good:
        if z > a:
            api.rssm_kv_append(want, k[a:z], v[a:z], table[b : b + 1], ints([lengths[b]]), z - a, layer=1)
    assert int(want.error_word) == 0
    for x, y in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), (want.k, want.v, want.k_scale, want.v_scale)):
        assert x is y or torch.equal(x, y)
    # back again; no row is too long to be read, and an output that lies in two rows is either's
    cache.error_word.zero_()
    good = sound(2**31, n, cu)
    ko, vo = (torch.full((n, H, D), 5.0, device="cuda") for _ in range(2))
    api.rssm_kv_read(cache, table, ints(cu), ko, vo, starts=ints(lengths), layer=1)
    past = any(lengths[b] + z - a > 2 * PAGE for b, a, z in good)  # tokens past the row's table
    assert int(cache.error_word) == (api.ERRBIT_SEQLEN if len(good) < batch else 0) | (api.ERRBIT_PAGE if past else 0)
    claims = {}
    for b, a, z in good:
        if z > a:
            one = [torch.empty(z - a, H, D, device="cuda") for _ in range(2)]
            api.rssm_kv_read(cache, table[b : b + 1], offsets([z - a]), *one, starts=ints([lengths[b]]), layer=1)
            for t in range(z - a):
                claims.setdefault(a + t, []).append([x[t] for x in one])
    for t in range(n):
        for i, got in enumerate((ko[t], vo[t])):
            if t not in claims:
                assert bool((got == 5.0).all())
            else:
                either = torch.stack([c[i] for c in claims[t]])
                assert bool((either == got).any(0).all())
