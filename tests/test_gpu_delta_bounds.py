"""Prompt bounds that are none: their rows are skipped, and the rows around them are what they are without them."""
import pytest
import torch

from speculative_state_replay_gb300 import api

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

# (bounds, valid rows): a row that falls, and then rows inside an earlier one, whose chunks would share its place in
# the scratch; bounds past the tokens and negative ones; the last row begins where the valid ones end
CASES = [([0, 200, 50, 120, 200, 260], [0, 4]),
         ([0, 64, 0, 64, 128, 260], [0, 3, 4]),
         ([10, 9999, 10, 70, -5, 70, 260], [2, 5]),
         ([130, 260, 0, 130, 129, 131], [0]),
         ([0, 3, 2**31 - 1, -2**31, 3, 260], [0, 4])]


@pytest.mark.parametrize("dv", [64, 96])
@pytest.mark.parametrize("bounds,valid", CASES)
def test_rows_of_malformed_bounds(bounds, valid, dv):
    gen = torch.Generator(device="cuda").manual_seed(len(bounds))
    hk, hv, dk, n, B = 1, 2, 128, 260, len(bounds) - 1
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    q, k, v = rnd(n, hk, dk).to(BF), rnd(n, hk, dk).to(BF), rnd(n, hv, dv).to(BF)
    g, beta = -torch.rand(n, hv, generator=gen, device="cuda"), torch.rand(n, hv, generator=gen, device="cuda")
    start = rnd(B + 1, hv, dv, dk)
    slots = torch.arange(1, B + 1, dtype=torch.int32, device="cuda")
    one = torch.ones(B, dtype=torch.int32, device="cuda")

    def run(cu, slots, want):
        cache = api.DeltaCache(B + 1, hk, hv, dk, dv, 4, state=start.clone())
        cache.pend.fill_(3)
        out = torch.full((n, hv, dv), 7.0, dtype=BF, device="cuda")
        scratch = api.alloc_delta_scratch(cache, len(slots), n)
        api.rssm_delta_prefill(cache, q, k, v, g, beta, slots, torch.tensor(cu, dtype=torch.int32, device="cuda"), out, scratch,
                               initial=one, l2norm=True)
        assert int(cache.error_word) == want
        return cache, out

    for _ in range(3):  # (a race would not show every time)
        cache, out = run(bounds, slots, api.ERRBIT_SEQLEN)
        untouched = torch.ones(n, dtype=torch.bool, device="cuda")
        for b in range(B):
            if b not in valid:
                assert torch.equal(cache.state[b + 1], start[b + 1]) and (cache.pend[b + 1] == 3).all()
                continue
            alone, o = run([bounds[b], bounds[b + 1]], slots[b : b + 1], 0)
            part = slice(bounds[b], bounds[b + 1])
            assert torch.equal(cache.state[b + 1], alone.state[b + 1]) and torch.equal(out[part], o[part])
            assert (cache.pend[b + 1] == 0).all()
            untouched[part] = False
        assert (out[untouched] == 7.0).all()
