"""Speculative decoding of a small hybrid model: a gated-delta-rule layer and a Mamba-2 layer.

One request batch from prompts to tokens through the library's calls, in the
order a serving loop makes them:

    prompts   rssm_delta_prefill -> rssm_gated_norm -> rssm_residual_norm -> Mamba-2 layer -> first token
    a step    rssm_delta_step -> rssm_gated_norm -> rssm_residual_norm
              rssm_accept_flush -> rssm_step -> rssm_gated_norm -> rssm_residual_norm -> logits
              rssm_verify: `accepted` goes into the next step's rssm_delta_step and rssm_accept_flush

Weights are random (there is nothing to learn here), projections are plain
matrix products, drafts are drawn from the last step's distribution.

    python examples/hybrid_decode.py [--rows 8] [--steps 12] [--drafts 3]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from speculative_state_replay_gb300 import api  # noqa: E402

VOCAB, MODEL = 1000, 256
HK, HV, DK, DV = 2, 4, 128, 64  # the delta layer's heads
H, G = 8, 1                      # the Mamba-2 layer's heads (of 64) and groups
WINDOW = 16


class HybridModel:
    """The model and the state of `rows` requests, each in its own slot of the two layers' caches."""

    def __init__(self, rows: int, tokens_a_step: int, seed: int = 0, device: str = "cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.dev, self.gen, self.rows, self.T = device, gen, rows, tokens_a_step

        def weight(*shape):
            return (torch.randn(shape, generator=gen, device=device) / shape[0] ** 0.5).bfloat16()

        def ones(n):
            return torch.ones(n, device=device)

        self.embed = weight(VOCAB, MODEL) * VOCAB**0.5
        self.delta_in = weight(MODEL, 2 * HK * DK + 2 * HV * DV + 2 * HV)
        self.delta_out = weight(HV * DV, MODEL)
        self.delta_rate = torch.exp(torch.rand(HV, generator=gen, device=device))
        self.ssm_in = weight(MODEL, 2 * H * 64 + 2 * G * 128 + H)
        self.ssm_out = weight(H * 64, MODEL)
        self.A = -torch.exp(torch.rand(H, generator=gen, device=device))
        self.D, self.dt_bias = ones(H), torch.zeros(H, device=device)
        self.head = 0.3 * weight(MODEL, VOCAB)
        self.norms = [ones(MODEL) for _ in range(3)]
        self.post = [ones(MODEL) for _ in range(2)]
        self.delta_norm, self.ssm_norm = ones(DV), ones(H * 64)

        self.slots = torch.arange(1, rows + 1, dtype=torch.int32, device=device)
        self.delta = api.DeltaCache(rows + 1, HK, HV, DK, DV, tokens_a_step, api.F32, device=device)
        self.ssm = api.RssmCache(rows + 1, H, G, WINDOW, tokens_a_step, api.F32, device=device)
        api.rssm_init_state(self.ssm, torch.zeros(rows, H, 64, 128, device=device), self.slots)
        self.pnat = torch.zeros(rows, dtype=torch.int32, device=device)
        self.ssm_scratch = api.alloc_scratch(self.ssm, rows, tokens_a_step)
        self.delta_scratch = api.alloc_delta_scratch(self.delta, rows, rows * tokens_a_step)
        # what the last step's verification accepted, and that step's tokens a row
        self.accepted = torch.zeros(rows, dtype=torch.int32, device=device)
        self.fed, self.fed_cu = 0, None

    def check(self):
        words = int(self.delta.error_word), int(self.ssm.error_word)
        if words != (0, 0):
            raise RuntimeError(f"the device reported errors: {words}")

    # the layers, for packed tokens [n, MODEL]
    def delta_layer(self, x, cu=None, prompt=False):
        n = x.shape[0]
        p = x @ self.delta_in
        q, k, v, z, a, b = p.split((HK * DK, HK * DK, HV * DV, HV * DV, HV, HV), 1)
        g = (-self.delta_rate * torch.nn.functional.softplus(a.float() - 2.0)).contiguous()
        beta = torch.sigmoid(b.float()).contiguous()
        out = torch.empty(n, HV, DV, dtype=torch.bfloat16, device=self.dev)
        heads = (q.unflatten(1, (HK, DK)), k.unflatten(1, (HK, DK)), v.unflatten(1, (HV, DV)), g, beta)
        if prompt:
            scratch = api.alloc_delta_scratch(self.delta, self.rows, n)
            api.rssm_delta_prefill(self.delta, *heads, self.slots, cu, out, scratch, l2norm=True)
        else:
            api.rssm_delta_step(self.delta, *heads, self.slots, self.accepted, self.T, out, self.delta_scratch,
                                cu_seqlens=cu, l2norm=True)
        y = out.view(n, HV * DV)
        api.rssm_gated_norm(y, z, self.delta_norm, y, DV, norm_first=True)
        return y @ self.delta_out

    def ssm_layer(self, x, rows_cu=None, T=None):
        """One block of at most T tokens a row; the block before is committed by `self.accepted`."""
        n = x.shape[0]
        T = self.T if T is None else T
        p = x @ self.ssm_in
        xs, bs, cs, z, dt = p.split((H * 64, G * 128, G * 128, H * 64, H), 1)
        xs, bs, cs, dt = (t.contiguous() for t in (xs, bs, cs, dt.float()))
        out = torch.empty(n, H * 64, dtype=torch.bfloat16, device=self.dev)
        api.rssm_accept_flush(self.ssm, self.A, self.slots, self.pnat, self.accepted, self.fed, T, self.ssm_scratch,
                              accept_cu_seqlens=self.fed_cu, cu_seqlens=rows_cu)
        api.rssm_step(self.ssm, xs, dt, self.A, bs, cs, self.D, self.dt_bias, self.slots, self.pnat, T, out,
                      self.ssm_scratch, cu_seqlens=rows_cu)
        self.fed, self.fed_cu = T, rows_cu
        api.rssm_gated_norm(out, z, self.ssm_norm, out, H * 64 // G)
        return out @ self.ssm_out

    def between(self, x, residual, i, post=None):
        """Residual add and the norm before the next block; x becomes the normed stream."""
        out = torch.empty_like(x)
        api.rssm_residual_norm(x, residual, self.norms[i], out, residual, post_weight=post)
        return out

    def start(self, tokens):
        residual = torch.zeros(tokens.shape[0], MODEL, device=self.dev)
        return self.between(self.embed[tokens.long()], residual, 0), residual

    def prompts(self, lens, tokens):
        """Packed prompts through both layers; target probabilities after each prompt's last token."""
        cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=self.dev)
        x, residual = self.start(tokens)
        x = self.between(self.delta_layer(x, cu, prompt=True), residual, 1, self.post[0])
        # the Mamba-2 layer goes through the prompts in blocks of a step's tokens, all of them accepted
        y = torch.empty_like(x)
        for at in range(0, max(lens), self.T):
            now = [min(max(m - at, 0), self.T) for m in lens]
            where = torch.cat([int(cu[b]) + at + torch.arange(m) for b, m in enumerate(now)]).to(self.dev)
            rows_cu = torch.tensor([0] + list(torch.tensor(now).cumsum(0)), dtype=torch.int32, device=self.dev)
            y[where] = self.ssm_layer(x[where], rows_cu)
            self.accepted = torch.tensor(now, dtype=torch.int32, device=self.dev)
        x = self.between(y, residual, 2, self.post[1])
        p = torch.softmax((x[cu[1:].long() - 1] @ self.head).float(), -1)
        self.delta_accepted = torch.zeros_like(self.accepted)
        return p

    def step(self, tokens):
        """T tokens a row (the last sampled one and the drafts): target probabilities after each."""
        x, residual = self.start(tokens)
        ssm_accepted, self.accepted = self.accepted, self.delta_accepted
        x = self.between(self.delta_layer(x), residual, 1, self.post[0])
        self.accepted = ssm_accepted
        x = self.between(self.ssm_layer(x), residual, 2, self.post[1])
        return torch.softmax((x @ self.head).float(), -1)

    def commit(self, accepted):
        self.accepted = self.delta_accepted = accepted


def generate(model: HybridModel, lens, prompts, steps: int):
    """Speculative decoding: the tokens every row committed, and how many drafts were accepted."""
    B, T, dev, gen = model.rows, model.T, model.dev, model.gen
    p = model.prompts(lens, prompts)
    last = torch.multinomial(p, 1, generator=gen)[:, 0].int()
    committed = [[] for _ in range(B)]
    accepted = torch.empty(B, dtype=torch.int32, device=dev)
    nxt = torch.empty(B, dtype=torch.int32, device=dev)
    word = torch.zeros(1, dtype=torch.int32, device=dev)
    taken = 0
    for _ in range(steps):
        q = p[:, None, :].expand(B, T, VOCAB).reshape(B * T, VOCAB).contiguous()
        tokens = torch.multinomial(q, 1, generator=gen)[:, 0].int()
        tokens.view(B, T)[:, 0] = last
        target = model.step(tokens)
        u = torch.rand(B * T, generator=gen, device=dev)
        u_next = torch.rand(B, generator=gen, device=dev)
        api.rssm_verify(target, tokens, u, u_next, T, accepted, nxt, draft=q, error_word=word)
        model.commit(accepted.clone())
        n = accepted.tolist()
        for b in range(B):
            committed[b] += tokens.view(B, T)[b, : n[b]].tolist()
        taken += sum(n) - B
        last = nxt.clone()
        p = target.view(B, T, VOCAB)[torch.arange(B, device=dev), (accepted - 1).long()]
    model.check()
    if int(word):
        raise RuntimeError(f"rssm_verify reported {int(word)}")
    return committed, taken


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rows", type=int, default=8)
    ap.add_argument("--steps", type=int, default=12)
    ap.add_argument("--drafts", type=int, default=3)
    a = ap.parse_args()
    model = HybridModel(a.rows, a.drafts + 1)
    lens = [7 + 37 * i % 150 for i in range(a.rows)]
    prompts = torch.randint(0, VOCAB, (sum(lens),), generator=model.gen, device="cuda", dtype=torch.int32)
    committed, taken = generate(model, lens, prompts, a.steps)
    total = sum(len(c) for c in committed)
    print(f"{a.rows} rows, {a.steps} steps of 1 + {a.drafts} tokens: {total} tokens committed, "
          f"{taken} of {a.rows * a.steps * a.drafts} drafts accepted")


if __name__ == "__main__":
    main()
