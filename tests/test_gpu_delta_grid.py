"""The step's grid: blocks that take all items of a (row, key head), blocks that take a few, and rows split between both.

RSSM_SM_LIMIT makes the device small, so that few rows are many waves of blocks.  Outputs, states and corrections are
held to the rule in 64 bits (tolerances as in test_gpu_delta.py: 2^-8 of the outputs' norm, 1e-5 of fp32 tensors', 2^-9
more for bf16 states), and have the bits that the whole device's grid gives.
"""
import pytest
import torch

from operators_plain import delta_tokens
from speculative_state_replay_gb300 import api

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def near(x, ref, tol):
    x, ref = x.double(), ref.double()
    assert torch.isfinite(x).all()
    assert float((x - ref).norm()) <= tol * float(ref.norm()) + 1e-30, float((x - ref).norm() / ref.norm())


# (rows, key heads, value heads, dk, dv): units of several items (value heads x 64-row tiles), tiles whose last warps
# have no rows (80, 112), rows whose units are partly whole and partly spread
@pytest.mark.parametrize("state", [api.F32, api.BF16])
@pytest.mark.parametrize("B,hk,hv,dk,dv", [(5, 2, 8, 128, 128), (7, 1, 4, 128, 80), (3, 3, 6, 64, 256), (9, 2, 8, 64, 112), (2, 2, 4, 128, 16)])
@pytest.mark.parametrize("limit", ["1", "2"])
def test_items_and_waves(monkeypatch, B, hk, hv, dk, dv, state, limit):
    T = 4
    gen = torch.Generator(device="cuda").manual_seed(B * 1000 + dv)
    cpu = torch.Generator().manual_seed(B)
    lens = [torch.randint(0, T + 1, (B,), generator=cpu).tolist() for _ in range(3)]
    lens[1] = [T] * B
    acc = [None] + [torch.tensor([int(torch.randint(0, m + 1, (1,), generator=cpu)) for m in row], dtype=torch.int32, device="cuda")
                    for row in lens[:2]]

    def token(n):
        rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        return (rnd(n, hk, dk).to(BF), rnd(n, hk, dk).to(BF), rnd(n, hv, dv).to(BF), -0.3 * torch.rand(n, hv, generator=gen, device="cuda"),
                torch.rand(n, hv, generator=gen, device="cuda"))

    tk = [token(sum(row)) for row in lens]
    start = (0.3 * torch.randn(B + 1, hv, dv, dk, generator=gen, device="cuda")).to(torch.float32 if state == api.F32 else BF)
    slots = (torch.randperm(B, generator=gen, device="cuda") + 1).int()
    cus = [torch.tensor([0] + list(torch.tensor(row).cumsum(0)), dtype=torch.int32, device="cuda") for row in lens]

    def run():
        cache = api.DeltaCache(B + 1, hk, hv, dk, dv, T, state, state=start.clone())
        scratch = api.alloc_delta_scratch(cache, B, B * T)
        outs = []
        for row, x, a, cu in zip(lens, tk, acc, cus):
            out = torch.empty(sum(row), hv, dv, dtype=BF, device="cuda")
            api.rssm_delta_step(cache, *x, slots, a, T, out, scratch, cu_seqlens=cu, l2norm=True)
            outs.append(out)
        assert int(cache.error_word) == 0 and (scratch[: 4 * B] == 0).all()
        return cache, outs

    whole, outs = run()
    monkeypatch.setenv("RSSM_SM_LIMIT", limit)
    small, outs_s = run()
    monkeypatch.delenv("RSSM_SM_LIMIT")
    for x, y in zip(outs, outs_s):
        assert torch.equal(x, y)
    for name in ("state", "pend", "pend_k", "pend_w", "pend_c"):
        assert torch.equal(getattr(whole, name), getattr(small, name)), name
    tol = 1e-5 if state == api.F32 else 2.0**-9 + 1e-5
    for b in range(B):
        S = start[int(slots[b])]
        for i, row in enumerate(lens):
            at, n = int(cus[i][b]), row[b]
            o, u, _ = delta_tokens(S, *(x[at : at + n] for x in tk[i]), dk**-0.5, True)
            near(outs_s[i][at : at + n], o, 2.0**-8 + (tol if i else 0.0))
            if i < 2:
                _, _, S = delta_tokens(S, *(x[at : at + n] for x in tk[i]), dk**-0.5, True, keep=int(acc[i + 1][b]))
        near(small.state[int(slots[b])], S, 2 * tol)
        side, count = small.pend[int(slots[b])].tolist()
        assert count == lens[2][b]
        n = lens[2][b]
        r = (tk[2][1][int(cus[2][b]) : int(cus[2][b]) + n].double().pow(2).sum(-1) + 1e-6).rsqrt().repeat_interleave(hv // hk, 1)
        near(small.pend_w[int(slots[b]), side, :, :n].transpose(0, 1), u * r[..., None], 2 * tol)
