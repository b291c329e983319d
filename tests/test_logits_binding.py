"""What the binding of rssm_logits takes and refuses, by its messages (no GPU: a call that passes its checks is refused for its device)."""
import pytest
import torch

import __graft_entry__ as entry
from speculative_state_replay_gb300 import api

DEVICE = "on one CUDA device"


def call(**kw):
    entry.build()
    x = torch.zeros(6, 20)
    a = dict(logits=x, T=3, out=x.clone()) | kw
    api.rssm_logits(**a)


def test_a_mask_of_one_column_is_taken_whatever_its_stride():
    words = torch.zeros(6, 4, dtype=torch.int32)
    for mask in (words[:, :1], torch.zeros(1, 6, dtype=torch.int32).t(), words[:, ::2][:, :1]):
        with pytest.raises(ValueError, match=DEVICE):
            call(mask=mask)
    with pytest.raises(ValueError, match="mask must be"):
        call(mask=words[:, ::2])


def test_a_message_names_the_argument_at_fault():
    history, length = torch.zeros(2, 9, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for bad in (history.long(), history[:1], history.t(), history[0]):
        with pytest.raises(ValueError, match=r"history must be int32 \[2, "):
            call(history=bad, history_len=length)
    with pytest.raises(ValueError, match=DEVICE):
        call(history=history, history_len=length)
