"""rssm_logits: ids at the ends of their type, and parents that are looked at whatever the penalties."""
import random

import pytest
import torch

import test_gpu_logits as L
from test_gpu_logits import _api, check, ints, make  # noqa: F401

pytestmark = pytest.mark.gpu


ODD_IDS = [2**31 - 1 - i for i in range(9)] + [-(2**31), -(2**31) + 1, -1, -7, -8]


@pytest.mark.parametrize("V,dtype", [(100, torch.bfloat16), (4099, torch.float32), (40000, torch.float16)])
@pytest.mark.parametrize("off", [0, 1, 3, 7])
def test_ids_at_the_ends_of_their_type_are_not_counted(V, dtype, off):
    """Rows that begin up to seven values behind a 16-byte boundary: the id of a block's first word is then below 0."""
    c = make(V, [2, 1, 3], 30, off, tree=True, bias=20, dtype=dtype)
    odd = ODD_IDS + [V, V + 1]
    rng = random.Random(V)
    for h in c["history"]:
        h += odd
    for b in c["bias"]:
        b += [(i, 1e6) for i in odd]
    c["tokens"][1], c["tokens"][3], c["tokens"][5] = 2**31 - 1, -(2**31), rng.choice(odd)
    wide = torch.zeros(6, V + 9, dtype=dtype, device="cuda")
    wide[:, off : off + V] = c["x"]
    c["x"] = wide[:, off : off + V]
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    for probs in (True, False):
        out = torch.zeros(6, V, device="cuda")
        L.call(c, out, probs=probs, error_word=word)
        check(c, out, probs)
    assert int(word) == 0


@pytest.mark.parametrize("options", [{}, dict(temperature=None, repetition=None, presence=None, frequency=None)])
@pytest.mark.parametrize("with_tokens", [True, False])
def test_bad_parents_set_their_bit(options, with_tokens):
    c = make(300, [3, 4, 2], 20, 1, tree=True)
    c["parents"] = [-1, 0, 1, -1, 0, 2, 1, -1, 0]  # token 2 of the second row follows itself
    if options:
        n = len(c["lens"])
        for name, x in (("temperature", 1.0), ("repetition", 1.0), ("presence", 0.0), ("frequency", 0.0)):
            c[name] = torch.full((n,), x, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.zeros(9, 300, device="cuda")
    L.call(c, out, error_word=word, **options, **({} if with_tokens else dict(tokens=None)))
    assert int(word) == L.api.ERRBIT_TREE
    word.zero_()
    c["parents"][5] = 1
    L.call(c, out, error_word=word, **options, **({} if with_tokens else dict(tokens=None)))
    assert int(word) == 0
    if with_tokens:
        check(c, out)


def test_rows_behind_the_last_request_are_left():
    """Seven rows in requests of three tokens: two requests, and a row that belongs to none; the same with their number given."""
    x = torch.randn(7, 50, generator=torch.Generator(device="cuda").manual_seed(0), device="cuda")
    for kw, whole in ((dict(), 6), (dict(batch=1), 3), (dict(cu_seqlens=ints([0, 2, 5])), 5)):
        out = torch.full((7, 50), 9.0, device="cuda")
        L.api.rssm_logits(x, 3, out, **kw)
        assert bool((out[whole:] == 9.0).all())
        # expf of at most 12 off by 2^-23 (1 + 12), the sum of 50 and its reciprocal
        assert (out[:whole].double() - torch.softmax(x[:whole].double(), -1)).abs().max() <= 2.0**-23 * 13 + 52 * 2.0**-24
