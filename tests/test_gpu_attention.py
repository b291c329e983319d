"""The paged cache and attention over it against their definitions in 64 bits, through the public calls."""
import math
import random

import pytest
import torch

import attention_plain as P

pytestmark = pytest.mark.gpu
api = None


@pytest.fixture(scope="module", autouse=True)
def _api():
    global api
    from speculative_state_replay_gb300 import api as a

    api = a


def offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def make_cache(fmt, d, h, page, lengths, new, layers=1, spare=2, columns=2, seed=0):
    """A cache with every row's committed tokens in it (pages in no order), its table, and the generator.  lengths < 0: padding."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-(max(a, 0) + b) // page) for a, b in zip(lengths, new)]
    total = sum(need) + spare
    order = torch.randperm(total, generator=gen, device="cuda").int().cpu()
    table = torch.full((len(lengths), max(need + [0]) + columns), 1 << 30, dtype=torch.int32)  # entries past a row's are not read
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at : at + n]
        at += n
    cache = api.KVCache(total, h, d, page, fmt, layers=layers)
    table = table.cuda()
    # what no row holds is rubbish
    if fmt == api.BF16:
        cache.k.fill_(math.nan)
        cache.v.fill_(math.inf)
    else:
        cache.k_scale.fill_(math.nan)
        cache.v_scale.fill_(math.inf)
    have = [max(a, 0) for a in lengths]
    n = sum(have)
    for layer in range(layers):
        k = torch.randn(n, h, d, generator=gen, device="cuda").bfloat16()
        v = torch.randn(n, h, d, generator=gen, device="cuda").bfloat16()
        zero = torch.tensor([0 if a >= 0 else -1 for a in lengths], dtype=torch.int32, device="cuda")
        api.rssm_kv_append(cache, k, v, table, zero, max(have + [1]), cu_seqlens=offsets(have), layer=layer)
    return cache, table, gen


def tree(n, seed):
    rng = random.Random(seed)
    return [-1 if t == 0 else rng.randint(max(-1, t - 9), t - 1) for t in range(n)]


def check_rows(cache, table, lengths, new, q, parents, out, scale, slack=0.0):
    K, V = P.decoded(cache, "k"), P.decoded(cache, "v")
    at = 0
    for b, (a, n) in enumerate(zip(lengths, new)):
        got = out[at : at + n].cpu().double()
        if a < 0:
            assert not got.any()
        elif n:
            k, v = (P.row_tokens(x, table[b].cpu(), cache.page_size, 0, a + n) for x in (K, V))
            want, size = P.attention_row(k, v, q[at : at + n].cpu(), None if parents is None else parents[at : at + n], a, scale)
            # the output's rounding; each weight's (bf16: 8 bits, fp16: 11); 2^-12 for scores, exponentials and sums in fp32
            weight = 2.0**-8 if cache.format == api.BF16 else 2.0**-11
            far = (got - want).abs() - (2.0**-8 * want.abs() + (weight + 2.0**-12) * size + slack)
            assert far.max() <= 0, (b, float(far.max()))
        at += n


CASES = [
    # format, head_dim, query heads, heads, page, lengths, new tokens, tree
    ("BF16", 128, 32, 8, 16, [500], [1], False),
    ("BF16", 128, 8, 8, 64, [0, 1, 15, 16, 17, 63, 64, 65], [1] * 8, False),
    ("E4M3", 128, 32, 8, 64, [300, 5, 0, 1023, -1, 64], [4, 4, 4, 4, 4, 4], False),
    ("I8", 128, 16, 2, 48, [100, 47, 48, 49, 2000], [3, 0, 8, 1, 5], False),
    ("I8", 64, 7, 1, 32, [1, 31, 33, 700], [2, 7, 1, 4], True),
    ("E4M3", 64, 8, 1, 16, [0, 129], [33, 64], True),
    ("BF16", 64, 14, 2, 16, [257, 0, 12], [40, 64, 1], True),
    ("BF16", 256, 8, 2, 32, [77, 400], [5, 17], True),
    ("E4M3", 256, 4, 1, 64, [1000, 3], [1, 8], False),
    ("I8", 256, 16, 2, 128, [130], [12], True),
    ("BF16", 128, 4, 2, 16, [0, 37], [200, 131], False),
    ("E4M3", 128, 12, 4, 64, [65, 0], [97, 150], False),
    ("I8", 64, 2, 2, 16, [3000], [65], False),
    ("BF16", 128, 8, 1, 64, [4000, -1, 90], [48, 3, 20], True),
    ("I8", 128, 32, 8, 16, [7 * b for b in range(40)], [9 - b % 3 for b in range(40)], True),
    ("BF16", 64, 20, 4, 32, [300, 0, -1, 129], [70, 300, 2, 0], False),
    ("E4M3", 128, 2, 2, 16, [120] * 3, [130, 127, 1], False),
    ("I8", 64, 8, 8, 16, [11 * b for b in range(20)], [300 if b == 3 else b for b in range(20)], False),
]


@pytest.mark.parametrize("fmt,d,hq,h,page,lengths,new,is_tree", CASES)
def test_attention(fmt, d, hq, h, page, lengths, new, is_tree):
    cache, table, gen = make_cache(getattr(api, fmt), d, h, page, lengths, new)
    n = sum(new)
    wide = torch.randn(n, (hq + 2 * h) * d + 8, generator=gen, device="cuda").bfloat16()  # columns of one projection
    q, k, v = (x.unflatten(1, (-1, d)) for x in (wide[:, : hq * d], wide[:, hq * d : (hq + h) * d], wide[:, (hq + h) * d : -8]))
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    cu = offsets(new)
    api.rssm_kv_append(cache, k, v, table, ln, max(new), cu_seqlens=cu)
    parents = None
    if is_tree:
        parents = [p for b, m in enumerate(new) for p in tree(m, b)]
    out = torch.full((n + 2, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    scratch = api.alloc_attention_scratch(cache, hq)
    pt = None if parents is None else torch.tensor(parents, dtype=torch.int32, device="cuda")
    for _ in range(2):  # the second call finds the counters as the first did
        api.rssm_tree_attention(cache, q, table, ln, max(new), out[:n], scratch, parents=pt, cu_seqlens=cu, scale=0.11)
        first = out.clone()
    assert torch.equal(first, out) and bool((out[n:] == 7.0).all())
    assert int(cache.error_word) == 0 and not scratch[:4096].any()
    check_rows(cache, table, lengths, new, q, parents, out, 0.11)


CUTS = [
    # segments of one and of two query tiles, rows without tokens, pieces of one tile: format, query heads, lengths, new tokens, tree
    ("I8", 8, [3000, 5, 700, 0, -1, 1900, 130], [64, 3, 33, 1, 2, 0, 48], True),
    ("BF16", 8, [128 * 7 - 40, 2500, 0, 1], [40, 64, 64, 9], True),
    ("E4M3", 8, [2000, 17, 640], [70, 200, 129], False),
    ("BF16", 4, [40 * b for b in range(30)], [8 - b % 5 for b in range(30)], False),
    ("E4M3", 2, [5000, 3], [5, 4], False),
]


@pytest.mark.parametrize("fmt,hq,lengths,new,is_tree", CUTS)
@pytest.mark.parametrize("sms", [1, 2, 7, 40])
def test_cuts(monkeypatch, sms, fmt, hq, lengths, new, is_tree):
    """Grids of few blocks: a block has many segments, and every block's first and last are shared."""
    monkeypatch.setenv("RSSM_SM_LIMIT", str(sms))
    test_attention(fmt, 64 if sms == 2 else 128, hq, 2, 32, lengths, new, is_tree)


@pytest.mark.parametrize("fmt", ["BF16", "I8", "E4M3"])
def test_append_and_read(fmt):
    """What is written is what the format's definition says, bit for bit; nothing else changes; it reads back as the values it stands for."""
    f = getattr(api, fmt)
    for d, h, page, lengths, new in ((128, 8, 16, [15, 0, -1, 40, 3], [2, 33, 4, 0, 1]), (64, 3, 48, [47, 100], [50, 1]), (256, 1, 32, [0], [70])):
        cache, table, gen = make_cache(f, d, h, page, lengths, new, layers=2)
        n = sum(new)
        k, v = (torch.randn(n + 1, h, d, generator=gen, device="cuda").bfloat16() * 10 ** random.Random(d + i).uniform(-3, 3) for i in (0, 1))
        k[0, 0] = 0.0
        v[1, 0, 5] = math.nan if fmt != "BF16" else 1.0
        v[1, h - 1, 0] = -math.inf if fmt != "BF16" else 1.0
        before = [None if x is None else x.clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
        ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        api.rssm_kv_append(cache, k, v, table, ln, max(new), cu_seqlens=offsets(new), layer=1)
        assert int(cache.error_word) == 0
        want = [None if x is None else x.cpu() for x in before]
        at = 0
        for b, m in enumerate(new):
            for t in range(m if lengths[b] >= 0 else 0):
                pg, slot = int(table[b, (lengths[b] + t) // page]), (lengths[b] + t) % page
                for i, x in enumerate((k, v)):
                    y = x[at + t].cpu()
                    if f == api.BF16:
                        want[i][1, pg, :, slot] = y
                    else:
                        want[i][1, pg, :, slot], want[2 + i][1, pg, :, slot] = P.quantised(y, f)
            at += m
        for got, y in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), want):
            if y is not None:
                got = got.cpu()
                same = (got == y) | (got.isnan() & y.isnan()) if got.is_floating_point() else got == y
                assert bool(same.all())
        # back again, from a place before the new tokens
        start = [max(0, a - 5) if a >= 0 else a for a in lengths]
        count = [a + m - s if a >= 0 else m for a, m, s in zip(lengths, new, start)]
        K, V = P.decoded(cache, "k", 1), P.decoded(cache, "v", 1)
        for dtype in (torch.float32, torch.bfloat16, torch.float16):
            ko = torch.full((sum(count) + 1, h, d + 8), 5.0, dtype=dtype, device="cuda")[:, :, :d] if h == 1 else \
                torch.full((sum(count) + 1, h, d), 5.0, dtype=dtype, device="cuda")
            vo = torch.full((sum(count) + 1, h, d), 5.0, dtype=dtype, device="cuda")
            api.rssm_kv_read(cache, table, offsets(count), ko, vo, starts=torch.tensor(start, dtype=torch.int32, device="cuda"), layer=1)
            assert bool((ko[-1] == 5.0).all()) and bool((vo[-1] == 5.0).all())
            at = 0
            for b, m in enumerate(count):
                for got, x in ((ko, K), (vo, V)):
                    got = got[at : at + m].cpu()
                    want_row = torch.zeros(m, h, d, dtype=torch.float64) if lengths[b] < 0 else P.row_tokens(x, table[b].cpu(), page, start[b], m)
                    # code * scale is exact in 64 bits; one rounding to fp32, one to the output's type
                    assert torch.equal(torch.nan_to_num(got.double(), nan=9e9), torch.nan_to_num(want_row.float().to(dtype).double(), nan=9e9))
                at += m


def test_unseen_values_do_not_reach():
    """NaN and infinities in tokens that a query does not see, and behind the row's end, leave it alone; those it sees reach it."""
    for fmt in ("BF16", "I8", "E4M3"):
        f = getattr(api, fmt)
        lengths, new, d, h, hq = [21, 70], [6, 6], 64, 2, 4
        parents = [-1, 0, 0, 1, 2, 2] * 2
        cache, table, gen = make_cache(f, d, h, 16, lengths, new)
        q, k, v = (torch.randn(12, x, d, generator=gen, device="cuda").bfloat16() for x in (hq, h, h))
        k[2, 1, 7], v[2, 0, 3], v[7, 1, 9] = math.inf, math.nan, math.inf  # token 2 of row 0; token 1 of row 1
        ln, cu = torch.tensor(lengths, dtype=torch.int32, device="cuda"), offsets(new)
        out = torch.zeros(12, hq, d, dtype=torch.bfloat16, device="cuda")
        scratch = api.alloc_attention_scratch(cache, hq)
        pt = torch.tensor(parents, dtype=torch.int32, device="cuda")
        api.rssm_kv_append(cache, k, v, table, ln, 6, cu_seqlens=cu)
        api.rssm_tree_attention(cache, q, table, ln, 6, out, scratch, parents=pt, cu_seqlens=cu)
        bad = out.cpu().float().isfinite().logical_not()
        sees = [any(j in P.path(parents[:6], t) for j in ((2,) if b == 0 else (1,))) for b in range(2) for t in range(6)]
        for i in range(12):
            heads = bad[i].any(-1).tolist()
            if not sees[i]:
                assert not any(heads), (fmt, i)
            elif i < 6:
                assert bool(bad[i, 0, 3]) and bool(bad[i, 1, 3])
            else:
                assert bool(bad[i, 2, 9]) and bool(bad[i, 3, 9]) and not any(heads[:2])
        # a chain: earlier tokens of the same tile do not see later ones
        api.rssm_tree_attention(cache, q, table, ln, 6, out, scratch, cu_seqlens=cu)
        bad = out.cpu().float().isfinite().logical_not().flatten(1).any(1).tolist()
        assert bad == [False, False, True, True, True, True, False, True, True, True, True, True]


def test_bad_rows():
    """Bad pages, tables, counts and parents set their bit; only their own rows are concerned."""
    d, h, hq = 64, 1, 2
    lengths, new = [40, 40, 40, 40], [2, 2, 2, 2]
    cache, table, gen = make_cache(api.BF16, d, h, 16, lengths, new)
    q, k, v = (torch.randn(8, x, d, generator=gen, device="cuda").bfloat16() for x in (hq, h, h))
    ln, cu = torch.tensor(lengths, dtype=torch.int32, device="cuda"), offsets(new)
    api.rssm_kv_append(cache, k, v, table, ln, 2, cu_seqlens=cu)
    scratch = api.alloc_attention_scratch(cache, hq)
    good = torch.zeros(8, hq, d, dtype=torch.bfloat16, device="cuda")
    api.rssm_tree_attention(cache, q, table, ln, 2, good, scratch, cu_seqlens=cu)
    assert int(cache.error_word) == 0

    def again(bit, row, zeros=True, **kw):
        a = dict(pages=table, lengths=ln, parents=None, cu_seqlens=cu, T=2)
        a.update(kw)
        out = torch.full((8, hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
        api.rssm_tree_attention(cache, q, a["pages"], a["lengths"], a["T"], out, scratch, parents=a["parents"], cu_seqlens=a["cu_seqlens"])
        assert int(cache.error_word) == bit
        cache.error_word.zero_()
        rest = [i for i in range(8) if i // 2 != row]
        assert torch.equal(out[rest], good[rest])
        if zeros is not None:
            assert bool((out[2 * row : 2 * row + 2] == (0.0 if zeros else 3.0)).all())

    again(api.ERRBIT_PAGE, 1, lengths=torch.tensor([40, 2**31 - 1, 40, 40], dtype=torch.int32, device="cuda"))
    again(0, 2, lengths=torch.tensor([40, 40, -7, 40], dtype=torch.int32, device="cuda"))
    again(api.ERRBIT_SEQLEN, 3, zeros=False, cu_seqlens=torch.tensor([0, 2, 4, 6, 9], dtype=torch.int32, device="cuda"))
    again(api.ERRBIT_TREE, 0, parents=torch.tensor([-1, 1] + [-1, 0] * 3, dtype=torch.int32, device="cuda"))
    again(api.ERRBIT_TREE, 3, parents=torch.tensor([-1, 0] * 3 + [-2, 0], dtype=torch.int32, device="cuda"))
    for page in (-1, cache.pages, 2**31 - 1):
        t = table.clone()
        t[2, 0] = page
        again(api.ERRBIT_PAGE, 2, zeros=None, pages=t)
        kc = cache.k.clone()
        t[2, 2] = page  # where the new tokens go
        api.rssm_kv_append(cache, -k, v, t, ln, 2, cu_seqlens=cu)
        assert int(cache.error_word) == api.ERRBIT_PAGE
        cache.error_word.zero_()
        pg = int(table[2, 2])
        assert torch.equal(cache.k[0, pg].view(torch.int16), kc[0, pg].view(torch.int16))
        api.rssm_kv_append(cache, k, v, table, ln, 2, cu_seqlens=cu)
        ko, vo = torch.ones(48, h, d, device="cuda"), torch.ones(48, h, d, device="cuda")
        api.rssm_kv_read(cache, t[2:3], offsets([48]), ko, vo)
        assert int(cache.error_word) == api.ERRBIT_PAGE
        cache.error_word.zero_()
        assert not ko[:16].any() and bool(ko[16:32].any()) and not ko[32:].any()


def test_accept():
    """The walk, and every layer's entries, codes and scales, where the accepted tokens go."""
    for fmt, d, page, layers, lens in (("BF16", 128, 16, 3, [8, 1, 64, 0, 30, 5]), ("I8", 64, 48, 2, [40, 64]), ("E4M3", 256, 16, 1, [17, 3, 12])):
        rng = random.Random(page + d)
        lengths = [rng.randint(0, 60) for _ in lens]
        lengths[-1] = -1 if len(lens) > 3 else lengths[-1]
        cache, table, gen = make_cache(getattr(api, fmt), d, 2, page, lengths, lens, layers=layers)
        n, cu, T = sum(lens), offsets(lens), max(lens)
        ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        for layer in range(layers):
            k, v = (torch.randn(n, 2, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
            api.rssm_kv_append(cache, k, v, table, ln, T, cu_seqlens=cu, layer=layer)
        rows = []
        for m in lens:
            up = [-1 if t == 0 else rng.randint(max(0, t - 4), t - 1) for t in range(m)]
            tok = [rng.randint(0, 5) for _ in range(m)]  # some drafts are alike
            below = [[t for t in range(m) if up[t] == i] for i in range(m)]
            rows.append((up, tok, [tok[rng.choice(x)] if x and rng.random() < 0.9 else 99 for x in below]))
        flat = [torch.tensor([x for r in rows for x in r[i]], dtype=torch.int32, device="cuda") for i in range(3)]
        want = [None if x is None else x.cpu().clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
        acc, nxt = torch.full((len(lens),), 55, dtype=torch.int32, device="cuda"), torch.full((len(lens),), 55, dtype=torch.int32, device="cuda")
        path = torch.full((len(lens), T), 55, dtype=torch.int32, device="cuda")
        api.rssm_tree_accept(cache, table, ln, flat[1], flat[0], flat[2], T, acc, nxt, path, cu_seqlens=cu)
        assert int(cache.error_word) == 0
        for b, (up, tok, drawn) in enumerate(rows):
            walk, last = P.accept_row(tok, up, drawn) if lengths[b] >= 0 else ([], -1)
            assert int(acc[b]) == len(walk) and int(nxt[b]) == last and path[b].tolist() == walk + [-1] * (T - len(walk))
            place = lambda p: (int(table[b, p // page]), p % page)  # noqa: E731
            old = [None if x is None else x.clone() for x in want]
            for j, t in enumerate(walk):
                (p0, s0), (p1, s1) = place(lengths[b] + t), place(lengths[b] + j)
                for x, y in zip(want, old):
                    if x is not None:
                        x[:, p1, :, s1] = y[:, p0, :, s0]
        for got, y in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), want):
            if y is not None:
                got = got.cpu()
                same = (got == y) | (got != got) & (y != y)
                assert bool(same.all())
        # without a cache: the walk alone; a chain
        acc2, nxt2, path2 = torch.empty_like(acc), torch.empty_like(nxt), torch.empty_like(path)
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        api.rssm_tree_accept(None, None, None, flat[1], None, flat[2], T, acc2, nxt2, path2, cu_seqlens=cu, error_word=word)
        for b, (_, tok, drawn) in enumerate(rows):
            walk, last = P.accept_row(tok, None, drawn)
            assert int(acc2[b]) == len(walk) and int(nxt2[b]) == last
        up = flat[0].clone()
        up[0] = 0
        api.rssm_tree_accept(None, None, None, flat[1], up, flat[2], T, acc2, nxt2, path2, cu_seqlens=cu, error_word=word)
        assert int(word) == api.ERRBIT_TREE and int(acc2[0]) == 0 and int(nxt2[0]) == -1 and path2[0].tolist() == [-1] * T


def test_accept_bad_page_moves_nothing():
    cache, table, gen = make_cache(api.BF16, 64, 1, 16, [15, 15], [4, 4], layers=2)
    ln = torch.tensor([15, 15], dtype=torch.int32, device="cuda")
    up, tok = torch.tensor([-1, 0, 0, 2] * 2, dtype=torch.int32, device="cuda"), torch.tensor([1, 2, 3, 4] * 2, dtype=torch.int32, device="cuda")
    drawn = torch.tensor([3, 0, 4, 9] * 2, dtype=torch.int32, device="cuda")
    k = torch.randn(8, 1, 64, generator=gen, device="cuda").bfloat16()
    for layer in (0, 1):
        api.rssm_kv_append(cache, k, k, table, ln, 4, layer=layer)
    t = table.clone()
    t[1, 1] = -3
    before = cache.k.clone()
    acc, nxt, path = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((2,), (2,), (2, 4)))
    api.rssm_tree_accept(cache, t, ln, tok, up, drawn, 4, acc, nxt, path)
    assert int(cache.error_word) == api.ERRBIT_PAGE and acc.tolist() == [3, 0] and nxt.tolist() == [9, -1]
    assert path.tolist() == [[0, 2, 3, -1], [-1] * 4]
    bits = lambda x: x.view(torch.int16)  # noqa: E731
    pg = [int(p) for p in table[1, :2]]
    assert torch.equal(bits(cache.k[:, pg]), bits(before[:, pg]))
    p0 = int(table[0, 1])
    assert torch.equal(cache.k[1, p0, 0, :2], k[2:4, 0]) and torch.equal(cache.k[0, p0, 0, :2], k[2:4, 0])


def test_strided_cache_and_captured_call():
    """Keys and values of a page beside each other (strides), more than one layer, a call captured and replayed on other inputs."""
    d, h, hq, page, layers = 64, 2, 8, 16, 2
    both = torch.zeros(layers, 12, 2, h, page, d, dtype=torch.bfloat16, device="cuda")
    cache = api.KVCache(12, h, d, page, api.BF16, layers=layers, k=both[:, :, 0], v=both[:, :, 1])
    table = torch.arange(11, -1, -1, dtype=torch.int32, device="cuda").view(2, 6)
    gen = torch.Generator(device="cuda").manual_seed(3)
    ln = torch.zeros(2, dtype=torch.int32, device="cuda")
    q, k, v = (torch.zeros(6, x, d, dtype=torch.bfloat16, device="cuda") for x in (hq, h, h))
    out = torch.zeros(6, hq, d, dtype=torch.bfloat16, device="cuda")
    scratch = api.alloc_attention_scratch(cache, hq)

    def step():
        api.rssm_kv_append(cache, k, v, table, ln, 3, layer=1)
        api.rssm_tree_attention(cache, q, table, ln, 3, out, scratch, layer=1)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for it in range(9):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        one = api.KVCache(12, h, d, page, api.BF16, k=both[1:2, :, 0], v=both[1:2, :, 1])
        check_rows(one, table, ln.tolist(), [3, 3], q, None, out, d**-0.5)
        ln += torch.tensor([3, 2], dtype=torch.int32, device="cuda")
    assert not both[0].any() and int(cache.error_word) == 0


def test_far_pages():
    """A cache whose pages lie past 2^32 bytes, and rows of many pieces: the same result as near."""
    d, h, hq, page = 128, 1, 2, 64
    big = 420000  # 6.9 GB of keys
    cache = api.KVCache(big, h, d, page, api.I8)
    near = api.KVCache(80, h, d, page, api.I8)
    gen = torch.Generator(device="cuda").manual_seed(5)
    n = 64 * 70 + 3
    k, v = (torch.randn(n + 1, h, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(1, hq, d, generator=gen, device="cuda").bfloat16()
    t_far = torch.arange(big - 72, big, dtype=torch.int32, device="cuda").view(1, -1)
    t_near = torch.arange(72, dtype=torch.int32, device="cuda").view(1, -1)
    ln, zero = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = []
    for c, t in ((cache, t_far), (near, t_near)):
        api.rssm_kv_append(c, k, v, t, zero, n + 1)
        out = torch.zeros(1, hq, d, dtype=torch.bfloat16, device="cuda")
        api.rssm_tree_attention(c, q, t, ln, 1, out, api.alloc_attention_scratch(c, hq))
        outs.append(out)
    assert torch.equal(*outs) and bool(outs[0].any())
    check_rows(near, t_near, [n], [1], q, None, outs[1], d**-0.5)
