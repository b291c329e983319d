"""rssm_kv_read, rssm_logits and rssm_tree_accept captured into a graph and replayed on other inputs, while another stream runs calls
of its own: every result is bit for bit the one of an eager call on the same inputs."""
import random

import pytest
import torch

import test_gpu_attention as A
from test_gpu_attention import _api, make_cache, offsets  # noqa: F401

pytestmark = pytest.mark.gpu

B, T, V, H, D, PAGE, LAYERS = 5, 12, 5003, 2, 64, 16, 3


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Step:
    """Buffers of a step's three calls, and the calls."""

    def __init__(self, fmt, seed):
        self.rng, self.gen = random.Random(seed), torch.Generator(device="cuda").manual_seed(seed)
        self.cache, self.table, _ = make_cache(getattr(A.api, fmt), D, H, PAGE, [40, 3, 0, 90, 17], [T] * B, layers=LAYERS, seed=seed)
        for name in ("k", "v", "k_scale", "v_scale"):
            x = getattr(self.cache, name)
            if x is not None and x.is_floating_point():
                x.nan_to_num_(nan=1.0, posinf=1.0)  # bits can be compared
        n = B * T
        self.lengths, self.cu, self.starts = ints([0] * B), offsets([T] * B), ints([0] * B)
        self.tokens, self.parents, self.drawn = ints([0] * n), ints([0] * n), ints([0] * n)
        self.history, self.history_len = ints([[0] * 50] * B), ints([0] * B)
        self.logits = torch.zeros(n, V, device="cuda").bfloat16()
        self.penalty = torch.full((B,), 1.2, device="cuda")
        self.fill()
        self.out = dict(k=torch.zeros(n, H, D, device="cuda"), v=torch.zeros(n, H, D, device="cuda"), probs=torch.zeros(n, V, device="cuda"),
                        accepted=ints([0] * B), nxt=ints([0] * B), path=ints([[0] * T] * B))

    def fill(self):
        """Other inputs in the same buffers."""
        rng, n = self.rng, B * T
        few = [rng.randrange(V) for _ in range(4)]
        self.lengths.copy_(ints([40, 3, 0, rng.randint(60, 90), rng.choice([-1, 17])]))
        self.starts.copy_(ints([rng.randint(0, 3) for _ in range(B)]))
        self.parents.copy_(ints([-1 if t == 0 else rng.randint(max(0, t - 3), t - 1) for _ in range(B) for t in range(T)]))
        for x in (self.tokens, self.drawn):
            x.copy_(ints([rng.choice(few) for _ in range(n)]))
        self.history.copy_(ints([[rng.choice(few + [rng.randrange(V)]) for _ in range(50)] for _ in range(B)]))
        self.history_len.copy_(ints([rng.randint(0, 50) for _ in range(B)]))
        self.logits.copy_(3 * torch.randn(n, V, generator=self.gen, device="cuda"))

    def run(self, stream=None, out=None, cache=None):
        o, c, api = out or self.out, cache or self.cache, A.api
        api.rssm_kv_read(c, self.table, self.cu, o["k"], o["v"], starts=self.starts, layer=1, stream=stream)
        api.rssm_logits(self.logits, T, o["probs"], temperature=self.penalty, repetition=self.penalty, frequency=self.penalty, history=self.history,
                        history_len=self.history_len, tokens=self.tokens, parents=self.parents, cu_seqlens=self.cu, stream=stream)
        api.rssm_tree_accept(c, self.table, self.lengths, self.tokens, self.parents, self.drawn, T, o["accepted"], o["nxt"], o["path"],
                             cu_seqlens=self.cu, stream=stream)

    def copy(self):
        """The cache and the outputs once more, for an eager call."""
        c = self.cache
        kw = {name: getattr(c, name).clone() for name in ("k", "v", "k_scale", "v_scale") if getattr(c, name) is not None}
        return A.api.KVCache(c.pages, H, D, PAGE, c.format, layers=LAYERS, **kw), {name: torch.full_like(x, 3) for name, x in self.out.items()}


def same(out, cache, want, want_cache):
    assert all(torch.equal(out[name], want[name]) for name in out)
    for name in ("k", "v", "k_scale", "v_scale"):
        x, y = getattr(cache, name), getattr(want_cache, name)
        assert x is y or torch.equal(x, y)


@pytest.mark.parametrize("fmt", ["BF16", "I8"])
def test_captured_and_at_once(fmt):
    step, other = Step(fmt, 1), Step("E4M3", 2)
    step.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step.run()
    st, moved = torch.cuda.Stream(), 0
    for it in range(4):
        step.fill()
        other.fill()
        for x in step.out.values():
            x.fill_(7)
        cache, want = step.copy()
        step.run(out=want, cache=cache)
        caches, outs = zip(*(other.copy() for _ in range(6)))
        torch.cuda.synchronize()
        st.wait_stream(torch.cuda.current_stream())
        for i in range(6):
            other.run(stream=st, out=outs[i], cache=caches[i])
            if i == 1:
                g.replay()
        torch.cuda.synchronize()
        same(step.out, step.cache, want, cache)
        for i in range(1, 6):
            same(outs[i], caches[i], outs[0], caches[0])
        moved += int((step.out["accepted"] > 1).sum())
        assert int(step.cache.error_word) == 0 and all(int(c.error_word) == 0 for c in caches)
    assert moved > 0
