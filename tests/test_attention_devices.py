"""The calls of the paged cache and of the sampler refuse tensors that are not all on the current device before anything is
launched (no GPU: tensors that say where they are, and a library that only notes that it was called)."""
import pytest
import torch

import __graft_entry__ as entry
from speculative_state_replay_gb300 import _lib, api
from test_operators_devices import BF, I32, Handle, Library, Stream, on


@pytest.fixture
def library(monkeypatch):
    entry.build()
    lib = Library(_lib.fast().device)
    monkeypatch.setattr(_lib, "fast", lambda: lib)
    monkeypatch.setattr(_lib, "fast_kv", lambda: lib)
    monkeypatch.setattr(api, "_devices", lambda: 2)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    return lib


def calls():
    """(function, its tensors by name, its other arguments), all on device 0."""
    cache = api.KVCache(4, 2, 64, 16, device="cpu", k=on(0, 1, 4, 2, 16, 64, dtype=BF), v=on(0, 1, 4, 2, 16, 64, dtype=BF),
                        error_word=on(0, 1, dtype=I32))
    rows = dict(pages=on(0, 2, 2, dtype=I32), lengths=on(0, 2, dtype=I32))
    one = lambda n: on(0, n, dtype=I32)  # noqa: E731
    return [
        (api.rssm_kv_append, dict(rows, k=on(0, 6, 2, 64, dtype=BF), v=on(0, 6, 2, 64, dtype=BF), cu_seqlens=one(3)), dict(cache=cache, T=3)),
        (api.rssm_kv_read, dict(pages=rows["pages"], cu_seqlens=one(3), k_out=on(0, 6, 2, 64), v_out=on(0, 6, 2, 64), starts=one(2)), dict(cache=cache)),
        (api.rssm_tree_attention, dict(rows, q=on(0, 6, 4, 64, dtype=BF), out=on(0, 6, 4, 64, dtype=BF), scratch=on(0, 64, dtype=torch.uint8), parents=one(6),
                                       cu_seqlens=one(3)), dict(cache=cache, T=3)),
        (api.rssm_tree_accept, dict(rows, tokens=one(6), parents=one(6), drawn=one(6), accepted=one(2), next_token=one(2), path=on(0, 2, 3, dtype=I32),
                                    cu_seqlens=one(3)), dict(cache=cache, T=3)),
        (api.rssm_logits, dict(logits=on(0, 6, 40), out=on(0, 6, 40), temperature=on(0, 2), repetition=on(0, 2), presence=on(0, 2), frequency=on(0, 2),
                               history=on(0, 2, 9, dtype=I32), history_len=one(2), prompt_len=one(2), tokens=one(6), parents=one(6), bias_start=one(3),
                               bias_id=one(5), bias_value=on(0, 5), mask=on(0, 6, 2, dtype=I32), cu_seqlens=one(3), error_word=one(1)), dict(T=3)),
    ]


def test_devices(library):
    for i in range(5):
        f, good, rest = calls()[i]
        for extra in ({}, dict(stream=Stream(0)), dict(stream=Handle())):
            f(**good, **rest, **extra)
        assert library.calls == 3 * (i + 1)
    library.calls = 0
    for i in range(5):
        f, good, rest = calls()[i]
        for place in (-1, 1):  # the host, another device
            for name, t in good.items():
                bad = dict(good)
                bad[name] = on(place, *t.shape, dtype=t.dtype)
                with pytest.raises(ValueError):
                    f(**bad, **rest)
        with pytest.raises(ValueError):
            f(**good, **rest, stream=Stream(1))
        if "cache" in rest:
            rest["cache"].k.place = 1
            with pytest.raises(ValueError):
                f(**good, **rest)
    assert library.calls == 0
