"""The example's serving loop: speculative decoding leaves the states that the committed tokens alone leave.

Tolerance: both runs see the same tokens, but their projections are matrix
products of other shapes, whose bf16 results may round the other way now and
then (2^-8 of a value); a state sums many such terms.  2^-6 of its norm.
"""
import os
import sys

import pytest
import torch

from speculative_state_replay_gb300 import api

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.gpu
@pytest.mark.parametrize("drafts", [0, 3, 7])
def test_states_are_those_of_the_committed_tokens(drafts):
    import hybrid_decode as ex

    lens = [5, 70, 1, 130]
    model = ex.HybridModel(len(lens), drafts + 1, seed=drafts)
    prompts = torch.randint(0, ex.VOCAB, (sum(lens),), generator=model.gen, device="cuda", dtype=torch.int32)
    committed, taken = ex.generate(model, lens, prompts, 6)
    assert all(6 <= len(c) <= 6 * (drafts + 1) for c in committed)
    assert taken == sum(len(c) for c in committed) - 6 * len(lens)
    if drafts:
        assert 0 < taken < 6 * drafts * len(lens)
    # commit the last step's drafts of the delta layer: a step of no tokens
    B = len(lens)
    none = torch.empty(0, ex.MODEL, dtype=torch.bfloat16, device="cuda")
    model.accepted = model.delta_accepted
    model.delta_layer(none, torch.zeros(B + 1, dtype=torch.int32, device="cuda"))

    again = ex.HybridModel(len(lens), drafts + 1, seed=drafts)
    whole, at = [], 0
    for b, n in enumerate(lens):
        whole.append(torch.cat([prompts[at : at + n], torch.tensor(committed[b], dtype=torch.int32, device="cuda")]))
        at += n
    all_lens = [len(w) for w in whole]
    again.prompts(all_lens, torch.cat(whole))
    for b in range(B):
        x, y = model.delta.state[b + 1].double(), again.delta.state[b + 1].double()
        assert (x - y).norm() <= 2.0**-6 * y.norm()
    # and the Mamba-2 layer's checkpoints, once both have folded all that is live
    for m in (model, again):
        api.rssm_accept_flush(m.ssm, m.A, m.slots, m.pnat, m.accepted, m.fed, m.T, m.ssm_scratch, accept_cu_seqlens=m.fed_cu, force=1)
        m.check()
        assert int(m.pnat.abs().sum()) == 0
    x, y = model.ssm.state_view()[1:].double(), again.ssm.state_view()[1:].double()
    assert (x - y).norm() <= 2.0**-6 * y.norm()
