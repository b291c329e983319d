"""A call whose tensors are not all on the current device is refused before anything is launched (no GPU: tensors that
say where they are, and a library that only notes that it was called)."""
import pytest
import torch

import __graft_entry__ as entry
from speculative_state_replay_gb300 import _lib, api

BF, I32 = torch.bfloat16, torch.int32


class Placed(torch.Tensor):
    def get_device(self):
        return self.place


def on(place, *shape, dtype=torch.float32):
    t = torch.zeros(shape, dtype=dtype).as_subclass(Placed)
    t.place = place
    return t


class Library:
    def __init__(self, device):
        self.device, self.calls = device, 0

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return 0

        return call


class Stream:
    cuda_stream = 0

    def __init__(self, device_index):
        self.device_index = device_index


def calls():
    """(function, its tensors by name, its other arguments), all on device 0."""
    c = api.DeltaCache(3, 2, 4, 64, 32, 4, device="cpu", **{
        n: on(0, *s, dtype=d) for n, s, d in (("state", (3, 4, 32, 64), torch.float32), ("pend_k", (3, 2, 2, 4, 64), BF),
                                              ("pend_w", (3, 2, 4, 4, 32), torch.float32), ("pend_c", (3, 2, 4, 4), torch.float32),
                                              ("pend", (3, 2), I32), ("error_word", (1,), I32))})
    tokens = dict(q=on(0, 4, 2, 64, dtype=BF), k=on(0, 4, 2, 64, dtype=BF), v=on(0, 4, 4, 32, dtype=BF), g=on(0, 4, 4), beta=on(0, 4, 4),
                  slot_idx=on(0, 1, dtype=I32), out=on(0, 4, 4, 32, dtype=BF), scratch=on(0, 64, dtype=torch.uint8))
    rows = dict(x=on(0, 3, 64), weight=on(0, 64), out=on(0, 3, 64))
    return [
        (api.rssm_delta_step, dict(tokens, accepted=on(0, 1, dtype=I32), cu_seqlens=on(0, 2, dtype=I32)), dict(cache=c, T=4)),
        (api.rssm_delta_prefill, dict(tokens, initial=on(0, 1, dtype=I32), cu_seqlens=on(0, 2, dtype=I32)), dict(cache=c)),
        (api.rssm_verify, dict(target=on(0, 4, 10), draft=on(0, 4, 10), tokens=on(0, 4, dtype=I32), u=on(0, 4), u_next=on(0, 1),
                               accepted=on(0, 1, dtype=I32), next_token=on(0, 1, dtype=I32), cu_seqlens=on(0, 2, dtype=I32),
                               error_word=on(0, 1, dtype=I32)), dict(T=4)),
        (api.rssm_gated_norm, dict(rows, z=on(0, 3, 64)), {}),
        (api.rssm_residual_norm, dict(rows, residual=on(0, 3, 64), residual_out=on(0, 3, 64), post_weight=on(0, 64), scale=on(0, 64)), {}),
    ]


@pytest.fixture
def library(monkeypatch):
    entry.build()
    lib = Library(_lib.fast().device)
    monkeypatch.setattr(_lib, "fast", lambda: lib)
    monkeypatch.setattr(api, "_devices", lambda: 2)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    return lib


def test_devices(library):
    for i in range(5):
        f, tensors, rest = calls()[i]
        f(**tensors, **rest)
        f(**tensors, **rest, stream=Stream(0))
        assert library.calls == 2 * (i + 1)
    library.calls = 0
    for i in range(5):
        f, tensors, rest = calls()[i]
        for place in (-1, 1):  # the host, another device
            for name in tensors:
                bad = dict(tensors)
                bad[name] = on(place, *tensors[name].shape, dtype=tensors[name].dtype)
                with pytest.raises(ValueError):
                    f(**bad, **rest)
            with pytest.raises(ValueError):  # all of them elsewhere
                f(**{n: on(place, *t.shape, dtype=t.dtype) for n, t in tensors.items()}, **rest)
        with pytest.raises(ValueError):
            f(**tensors, **rest, stream=Stream(1))
    assert library.calls == 0


def test_the_caches_device(library):
    f, tensors, rest = calls()[0]
    rest["cache"].state.place = 1
    with pytest.raises(ValueError):
        f(**tensors, **rest)
    with pytest.raises(ValueError):
        api.DeltaCache(3, 2, 4, 64, 32, 4, device="cpu", state=torch.zeros(3, 4, 32, 64, device="meta"))
    assert library.calls == 0


def test_scratch(library):
    """A view whose elements share bytes holds less than its size says."""
    f, tensors, rest = calls()[0]
    few = on(0, 1, dtype=torch.uint8)
    tensors["scratch"] = few.expand(1 << 20)
    tensors["scratch"].place = 0
    with pytest.raises(ValueError):
        f(**tensors, **rest)
    assert library.calls == 0


class Handle:
    cuda_stream = 0


def test_streams(library):
    """Any object with a handle is a stream, as for the other calls."""
    for i in range(5):
        f, tensors, rest = calls()[i]
        f(**tensors, **rest, stream=Handle())
    assert library.calls == 5


@pytest.mark.gpu
def test_a_given_stream():
    x = torch.randn(40, 512, device="cuda")
    w, out, here = torch.ones(512, device="cuda"), torch.empty_like(x), torch.empty_like(x)
    api.rssm_gated_norm(x, x, w, here)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    api.rssm_gated_norm(x, x, w, out, stream=st)
    st.synchronize()
    assert torch.equal(out, here)
    with pytest.raises(ValueError):
        api.rssm_gated_norm(x.cpu(), x, w, out)
    with pytest.raises(ValueError):
        api.rssm_gated_norm(x, x, w.cpu(), out)
