"""The gated norm with two groups a team of lanes, and fp32 gates far below zero."""
import pytest
import torch

from operators_plain import gated_norm
from speculative_state_replay_gb300 import api

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
ULP = {torch.float32: 0.0, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}  # as in test_gpu_norms.py


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [8, 24, 40, 128, 200, 480])
def test_two_groups_a_team(group, dtype):
    """Enough groups that a team of lanes takes two, and a last block that is not full: every row against the definition
    (tolerance as in test_gpu_norms.py: one rounding, and 4e-6)."""
    gen = torch.Generator(device="cuda").manual_seed(group)
    vec = 4 if dtype is torch.float32 else 8
    vecs = -(-group // vec)
    team = 8 if vecs <= 8 else 16 if vecs <= 16 else 32
    groups = 5
    rows = -(-(1 << 20) // team // groups) + 3
    x, z = (torch.randn(rows, groups * group, generator=gen, device="cuda").to(dtype) for _ in range(2))
    w = 1.0 + 0.2 * torch.randn(groups * group, generator=gen, device="cuda")
    wide = torch.full((rows, groups * group + 8), 7.0, dtype=dtype, device="cuda")
    out = wide[:, : groups * group]
    for first in (False, True):
        api.rssm_gated_norm(x, z, w, out, group, eps=1e-5, norm_first=first)
        for at in range(0, rows, 4096):
            part = slice(at, at + 4096)
            ref = gated_norm(x[part], z[part], w, group, 1e-5, first)
            tiny = 2.0**-24 if dtype is torch.float16 else 1e-30
            assert ((out[part].double() - ref).abs() <= (ULP[dtype] + 4e-6) * ref.abs() + tiny).all()
        assert (wide[:, groups * group :] == 7.0).all()


def test_gates_far_below_zero():
    """fp32: x of +-1, so that its norm is 1 / sqrt(1 + eps); expf and rsqrtf are at most 2 units in the last place off
    (2^-22 each), the sum, the division and three products half of one: 8e-7 of the value, down to z = -86, and below
    that, where e^z is no longer a normal number, 2^-149 / e^z more."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    z = torch.linspace(-86.0, 10.0, 1 << 16, device="cuda").view(-1, 64)
    x = torch.where(torch.rand(z.shape, generator=gen, device="cuda") < 0.5, -1.0, 1.0)
    w = torch.ones(64, device="cuda")
    out = torch.empty_like(x)
    api.rssm_gated_norm(x, z, w, out, norm_first=True, eps=1e-6)
    ref = gated_norm(x, z, w, 64, 1e-6, True)
    worst = ((out.double() - ref).abs() / ref.abs()).nan_to_num(nan=0.0)
    assert float(worst.max()) <= 8e-7, (float(worst.max()), float(z.flatten()[worst.argmax()]))
    z = torch.linspace(-92.0, -86.0, 64, device="cuda")[None]
    api.rssm_gated_norm(x[:1], z, w, out[:1], norm_first=True, eps=1e-6)
    ref = gated_norm(x[:1], z, w, 64, 1e-6, True)
    assert ((out[:1].double() - ref).abs() <= 8e-7 * ref.abs() + 2.0**-149 * 100).all()
