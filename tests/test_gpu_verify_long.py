"""Verification with long runs, weights of one over the longest vocabulary, and certain drafts above one.

RSSM_SM_LIMIT makes the device small, so that a few rows have one block each and its runs are as long as those of
hundreds of rows on the whole device.
"""
import pytest
import torch

from operators_plain import verify_row
from speculative_state_replay_gb300 import api

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def verify(target, draft, tokens, u, un, T):
    B = len(un)
    accepted, nxt = (torch.full((B,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.rssm_verify(target, tokens, u, un, T, accepted, nxt, draft=draft, error_word=word)
    assert int(word) == 0
    return accepted.tolist(), nxt.tolist()


@pytest.mark.parametrize("lookup", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [100279, 131072])
def test_long_runs(monkeypatch, V, dtype, lookup):
    gen = torch.Generator(device="cuda").manual_seed(V)
    B, T = 6, 2
    logits = 2.0 * torch.randn(B * T, V, generator=gen, device="cuda")
    target = torch.softmax(logits, -1).to(dtype)
    q = torch.softmax(logits + 0.5 * torch.randn(B * T, V, generator=gen, device="cuda"), -1)
    tokens = torch.multinomial(q, 1, generator=gen)[:, 0].int()
    draft = None if lookup else q.to(dtype)
    u = torch.rand(B * T, generator=gen, device="cuda")
    u[1] = 0.0  # accepted
    u[3::4] = 0.999999
    t, d, tok, uc = target.float().cpu(), None if lookup else draft.float().cpu(), tokens.cpu(), u.cpu()
    for un in ([0.0, 0.1, 0.3, 0.5, 0.7, 1.0 - 2.0**-24], torch.rand(B, generator=gen, device="cuda").tolist()):
        un = torch.tensor(un, device="cuda")
        whole = verify(target, draft, tokens, u, un, T)
        monkeypatch.setenv("RSSM_SM_LIMIT", "1")
        one = verify(target, draft, tokens, u, un, T)
        monkeypatch.delenv("RSSM_SM_LIMIT")
        assert one == whole
        for b in range(B):
            part = slice(b * T, b * T + T)
            want = verify_row(t[part], None if lookup else d[part], tok[part], uc[part], un[b].cpu())
            assert (one[0][b], one[1][b]) == want, b


def test_weights_of_one(monkeypatch):
    """2^25 values of 1, the most a row can hold: W = 2^61, and the token is floor(2^25 u)."""
    monkeypatch.setenv("RSSM_SM_LIMIT", "1")  # one block a row, as hundreds of rows have
    V, B = 1 << 25, 3
    target = torch.ones(B, V, dtype=torch.bfloat16, device="cuda")
    un = [0.0, 0.37109375, 1.0 - 2.0**-24]
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    got = verify(target, None, zero, torch.zeros(B, device="cuda"), torch.tensor(un, device="cuda"), 1)
    assert got == ([1] * B, [int(x * V) for x in un])
    wide = torch.ones(B, V + 8, dtype=torch.bfloat16, device="cuda")[:, 5 : V + 5]  # rows that do not start on 16 bytes
    assert verify(wide, None, zero, torch.zeros(B, device="cuda"), torch.tensor(un, device="cuda"), 1) == got


@pytest.mark.parametrize("rows", [1, 200])
@pytest.mark.parametrize("dtype", TYPES)
def test_certain_draft_above_one(dtype, rows):
    """A rejected certain draft whose entry is 3: what is left of it is 2, a weight of one, wherever it stands."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    V = 17001
    places = [0, 7, 128, 1023, 4100, 8192, 12345, V - 1]
    for i in range(len(places) if rows == 1 else 1):
        tokens = torch.tensor([places[(b // 2 + i) % len(places)] for b in range(2 * rows)], dtype=torch.int32, device="cuda")
        target = torch.softmax(torch.randn(rows * 2, V, generator=gen, device="cuda"), -1)
        target.scatter_(1, tokens[:, None].long(), 3.0)
        target = target.to(dtype)
        un = torch.rand(rows, generator=gen, device="cuda")
        u = torch.full((2 * rows,), 4.0, device="cuda")
        accepted, nxt = verify(target, None, tokens, u, un, 2)
        t = target.float().cpu()
        for b in range(rows):
            want = verify_row(t[2 * b : 2 * b + 2], None, tokens[2 * b : 2 * b + 2].cpu(), u[:2].cpu(), un[b].cpu())
            assert (accepted[b], nxt[b]) == want, b
