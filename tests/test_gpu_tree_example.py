"""The tree example's serving loop: the cache that trees of drafts leave is the one that the committed tokens alone leave.

Tolerance: both runs see the same tokens, but their projections are matrix
products of other shapes, and the attention cuts its sums elsewhere, so bf16
results may round the other way now and then.  A key of the second layer is
behind some eight such roundings of 2^-8: 2^-5 of the norm.  An 8-bit code may
then be the neighbouring one, a step of 1/127 of the row's largest value, which
is about three times its root mean square: 2^-5 more.
"""
import os
import sys

import pytest
import torch

from speculative_state_replay_gb300 import api

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.gpu
@pytest.mark.parametrize("format,nodes", [("bf16", [10, 10, 10, 10]), ("int8", [10, 1, 4, 7]), ("bf16", [1, 1, 1, 1])])
def test_cache_is_that_of_the_committed_tokens(format, nodes):
    import tree_decode as ex

    lens, steps = [5, 40, 1, 130], 8
    B, most = len(lens), 130 + 9 * 10
    model = ex.TreeModel(B, most, ex.FORMATS[format], seed=3)
    prompts = torch.randint(0, ex.VOCAB, (sum(lens),), generator=model.gen, device="cuda", dtype=torch.int32)
    committed = ex.generate(model, lens, prompts, steps, nodes)
    deepest = [max(_depth(ex.PARENTS, t) for t in range(k)) + 1 for k in nodes]
    assert all(steps <= len(c) <= steps * d for c, d in zip(committed, deepest))
    if max(nodes) == 10:
        assert sum(len(c) for c in committed) > steps * B  # some drafts were taken
    else:
        assert all(len(c) == steps for c in committed)
    total = [n + len(c) for n, c in zip(lens, committed)]
    assert model.lengths.tolist() == total

    again = ex.TreeModel(B, most, ex.FORMATS[format], seed=3)
    whole, at = [], 0
    for n, c in zip(lens, committed):
        whole.append(torch.cat([prompts[at : at + n], torch.tensor(c, dtype=torch.int32, device="cuda")]))
        at += n
    again.prompts(total, torch.cat(whole))
    again.check()
    cu = torch.tensor([0] + list(torch.tensor(total).cumsum(0)), dtype=torch.int32, device="cuda")
    limit = 2.0**-5 if format == "bf16" else 2.0**-4
    for layer in range(ex.LAYERS):
        got, want = ([torch.empty(sum(total), ex.HKV, ex.DIM, device="cuda") for _ in range(2)] for _ in range(2))
        api.rssm_kv_read(model.cache, model.pages, cu, *got, layer=layer)
        api.rssm_kv_read(again.cache, again.pages, cu, *want, layer=layer)
        for x, y in zip(got, want):
            assert (x - y).norm() <= limit * y.norm()


def _depth(parents, t):
    return 0 if parents[t] < 0 else 1 + _depth(parents, parents[t])
