"""Verification of drafted tokens: integers and single fp32 operations, so every result has to be equal."""
import pytest
import torch

from operators_plain import verify_row
from speculative_state_replay_gb300 import api

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def inputs(gen, lens, V, dtype, lookup=False):
    tot = sum(lens)
    dev = "cuda"
    logits = 2.0 * torch.randn(tot, V, generator=gen, device=dev)
    target = torch.softmax(logits, -1)
    q = torch.softmax(logits + 0.5 * torch.randn(tot, V, generator=gen, device=dev), -1)
    tokens = torch.multinomial(q, 1, generator=gen)[:, 0].int() if tot else torch.empty(0, dtype=torch.int32, device=dev)
    u = torch.rand(tot, generator=gen, device=dev)
    un = torch.rand(len(lens), generator=gen, device=dev)
    return target.to(dtype), None if lookup else q.to(dtype), tokens, u, un


def check(lens, T, target, draft, tokens, u, un, cu=None, err=0):
    B = len(un)
    accepted, nxt = (torch.full((B,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.rssm_verify(target, tokens, u, un, T, accepted, nxt, draft=draft, cu_seqlens=cu, error_word=word)
    t, d = target.float().cpu(), None if draft is None else draft.float().cpu()
    tok, u, un = tokens.cpu(), u.cpu(), un.cpu()
    at = 0
    for b, m in enumerate(lens):
        want = (0, -1) if m == 0 else verify_row(t[at : at + m], None if d is None else d[at : at + m], tok[at : at + m],
                                                 u[at : at + m], un[b])
        assert (int(accepted[b]), int(nxt[b])) == want, (b, m)
        at += m
    assert int(word) == err
    return accepted, nxt


@pytest.mark.parametrize("lookup", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [1, 2, 31, 1000, 4097, 50001])
def test_sizes(V, dtype, lookup):
    gen = torch.Generator(device="cuda").manual_seed(V)
    T = 5
    lens = [5, 1, 0, 3, 2, 5, 4]
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")
    check(lens, T, *inputs(gen, lens, V, dtype, lookup), cu=cu)
    for one in (1, 4):  # few rows: several blocks a row; without offsets
        check([T] * one, T, *inputs(gen, [T] * one, V, dtype, lookup))


def test_many_rows_and_32_tokens():
    gen = torch.Generator(device="cuda").manual_seed(3)
    check([2] * 400, 2, *inputs(gen, [2] * 400, 700, torch.float32))
    lens = [32] * 3
    target, draft, tokens, u, un = inputs(gen, lens, 300, torch.float32)
    check(lens, 32, target, target, tokens, u, un)  # the draft model is the target: all are accepted
    accepted, _ = check(lens, 32, target, target.clone(), tokens, u * 0.0, un)
    assert (accepted == 32).all()


@pytest.mark.parametrize("un", [0.0, 0.5, 1.0 - 2.0**-24])
def test_ends_of_the_distribution(un):
    """The first and the last token with mass, zeros around them; one token with all of it."""
    V = 20011
    t = torch.zeros(3, V, device="cuda")
    t[0, 7000:7003] = torch.tensor([0.25, 0.5, 0.25])
    t[1, V - 1] = 1.0
    t[2, 0] = 1.0
    z = torch.zeros(3, device="cuda")
    tok = torch.zeros(3, dtype=torch.int32, device="cuda")
    check([1, 1, 1], 1, t, None, tok, z, torch.full((3,), un, device="cuda"))


def test_nothing_left_and_odd_values():
    """A rejected draft with nothing of the target above the draft's row; NaN, negative, infinite and large entries; a
    row without mass; ids outside the vocabulary."""
    V = 1003
    gen = torch.Generator(device="cuda").manual_seed(5)
    target, draft, tokens, u, un = inputs(gen, [2] * 6, V, torch.float32)
    draft[1] = target[0]
    tokens[1] = 5
    draft[1, 5] = 2.0  # rejected at u = 0.9, and target - draft is nowhere positive
    u[1] = 0.9
    u[3::2] = 0.999999
    draft[3::2] += 1e-3
    target[2, ::7] = float("nan")
    target[4, ::5] = -1.0
    target[6, 3] = float("inf")
    target[8, 10:20] = 3.0
    draft[5, ::3] = float("nan")
    check([2] * 6, 2, target, draft, tokens, u, un)
    target[0] = 0.0
    check([2] * 6, 2, target, draft, tokens, u, un, err=api.ERRBIT_TOKEN)
    target, draft, tokens, u, un = inputs(gen, [2] * 6, V, torch.float32)
    tokens[1], tokens[5], tokens[0] = V, -1, V + 7  # a row's first token is not tested
    check([2] * 6, 2, target, draft, tokens, u, un, err=api.ERRBIT_TOKEN)
    check([2] * 6, 2, target, None, tokens, u, un, err=api.ERRBIT_TOKEN)


@pytest.mark.parametrize("left", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
def test_rows_of_two_alignments(dtype, left):
    """Long rows of the draft that start elsewhere in 16 bytes than the target's, with and without anything left above
    them."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    V, B = 20011, 3
    target, draft, tokens, u, un = inputs(gen, [2] * B, V, dtype)
    if not left:
        draft[1::2] = target[::2]
        tokens[1::2] = torch.tensor([0, 9999, V - 1], dtype=torch.int32, device="cuda")
        draft[1::2].scatter_(1, tokens[1::2, None].long(), 2.0)
    u[1::2] = 0.999999
    n = 16 // target.element_size()
    first = None
    for shift in range(n):
        wide = torch.full((2 * B, V + n + (-V) % n), 0.5, dtype=dtype, device="cuda")
        wide[:, shift : shift + V] = draft
        got = check([2] * B, 2, target, wide[:, shift : shift + V], tokens, u, un)
        first = first or got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


@pytest.mark.parametrize("rows", [1, 200])
@pytest.mark.parametrize("dtype", TYPES)
def test_certain_token_anywhere(dtype, rows):
    """A lookup's rejected token holds half of the target's mass, which is not drawn, wherever in the row it stands."""
    gen = torch.Generator(device="cuda").manual_seed(13)
    V = 17001
    places = [0, 1, 7, 8, 127, 128, 255, 256, 1023, 1024, 2047, 2048, 4100, 8191, 8192, 12345, V - 2, V - 1]
    base = torch.softmax(torch.randn(rows * 2, V, generator=gen, device="cuda"), -1) * 0.5
    tokens = torch.tensor([places[b // 2 % len(places)] for b in range(2 * rows)], dtype=torch.int32, device="cuda")
    un = torch.rand(rows, generator=gen, device="cuda")
    u = torch.full((2 * rows,), 0.999, device="cuda")
    for i in range(len(places) if rows == 1 else 1):
        if rows == 1:
            tokens[:] = places[i]
        target = base.clone()
        target.scatter_(1, tokens[:, None].long(), 0.5)
        accepted, nxt = check([2] * rows, 2, target.to(dtype), None, tokens, u, un)
        assert int(accepted.max()) == 1 and not (nxt == tokens[1::2]).any()


def test_strides_alignment_and_bounds():
    gen = torch.Generator(device="cuda").manual_seed(9)
    V = 5001
    lens = [3] * 4
    target, draft, tokens, u, un = inputs(gen, lens, V, torch.bfloat16)
    wide = torch.full((12, V + 13), 0.5, dtype=torch.bfloat16, device="cuda")
    wide[:, 1 : V + 1] = target
    a = check(lens, 3, wide[:, 1 : V + 1], draft, tokens, u, un)
    b = check(lens, 3, target.contiguous(), draft, tokens, u, un)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    cu = torch.tensor([0, 3, 1, 5, 13], dtype=torch.int32, device="cuda")  # -2 tokens, 4 > T, past the end
    accepted, nxt = (torch.empty(4, dtype=torch.int32, device="cuda") for _ in range(2))
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.rssm_verify(target, tokens, u, un, 3, accepted, nxt, draft=draft, cu_seqlens=cu, error_word=word)
    assert accepted.tolist()[1:] == [0, 0, 0] and nxt.tolist()[1:] == [-1, -1, -1] and int(accepted[0]) > 0
    assert int(word) == api.ERRBIT_SEQLEN


def test_rows_past_32_bits():
    """Row offsets that pass 2^31 elements."""
    V = 131072
    rows = (1 << 31) // V + 5
    target = torch.zeros(rows, V, dtype=torch.bfloat16, device="cuda")
    target[-1, 77777] = 0.5
    target[-2, 99] = 0.25
    target[-3, 123] = 1.0
    tokens = torch.full((rows,), 123, dtype=torch.int32, device="cuda")
    u = torch.full((rows,), 0.5, device="cuda")
    cu = torch.tensor([rows - 3, rows - 1, rows], dtype=torch.int32, device="cuda")
    accepted, nxt = (torch.empty(2, dtype=torch.int32, device="cuda") for _ in range(2))
    api.rssm_verify(target, tokens, u, torch.tensor([0.3, 0.3], device="cuda"), 2, accepted, nxt, cu_seqlens=cu)
    assert accepted.tolist() == [2, 1] and nxt.tolist() == [99, 77777]


def test_accepted_feeds_the_cache():
    """`accepted` is what the state's own calls take: T_b tokens at most."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    lens = [4] * 64
    accepted, _ = check(lens, 4, *inputs(gen, lens, 200, torch.float32))
    assert accepted.min() >= 1 and accepted.max() <= 4 and accepted.unique().numel() > 1
