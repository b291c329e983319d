"""Speculative decoding of a small attention model with trees of drafts over a paged cache.

One request batch from prompts to tokens through the library's calls, in the
order a serving loop makes them:

    a layer   rssm_kv_append -> rssm_tree_attention -> rssm_residual_norm
    prompts   the layers, every prompt a chain of new tokens, then rssm_logits
    a step    the layers for every row's tree (the last drawn token and drafts after it), rssm_logits with the penalties
              each token's own path earns, rssm_verify with a token a row (draws after every token), rssm_tree_accept:
              the path that the draws follow moves into place, and `lengths` grows by what it accepted

Weights are random (there is nothing to learn here), projections are plain
matrix products, drafts are what the head alone would have follow a token's embedding.

    python examples/tree_decode.py [--rows 8] [--steps 12] [--format bf16|int8|e4m3]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from speculative_state_replay_gb300 import api  # noqa: E402

VOCAB, MODEL, LAYERS = 500, 256, 2
HQ, HKV, DIM, PAGE = 8, 2, 64, 16
# a row's tree: the place that each token comes after (-1: the committed ones), and which of its parent's likeliest it is
PARENTS = [-1, 0, 0, 0, 1, 1, 2, 4, 4, 7]
CHOICE = [0, 0, 1, 2, 0, 1, 0, 0, 1, 0]
FORMATS = {"bf16": api.BF16, "int8": api.I8, "e4m3": api.E4M3}


class TreeModel:
    """The model, its cache, and `rows` requests with pages enough for `most` tokens each."""

    def __init__(self, rows: int, most: int, format: int, seed: int = 0, device: str = "cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.dev, self.gen, self.rows = device, gen, rows

        def weight(*shape):
            return (torch.randn(shape, generator=gen, device=device) / shape[0] ** 0.5).bfloat16()

        self.embed = weight(VOCAB, MODEL) * VOCAB**0.5
        self.qkv = [weight(MODEL, (HQ + 2 * HKV) * DIM) for _ in range(LAYERS)]
        self.out = [weight(HQ * DIM, MODEL) for _ in range(LAYERS)]
        self.head = 2 * weight(MODEL, VOCAB)
        self.follow = (self.embed @ self.head).topk(3, -1).indices.int()  # drafts of a token's successors
        self.norms = [torch.ones(MODEL, device=device) for _ in range(LAYERS + 1)]
        pages = (most + PAGE - 1) // PAGE
        self.cache = api.KVCache(rows * pages, HKV, DIM, PAGE, format, LAYERS, device=device)
        self.pages = torch.randperm(rows * pages, generator=gen, device=device).int().view(rows, pages)
        self.scratch = api.alloc_attention_scratch(self.cache, HQ)
        self.lengths = torch.zeros(rows, dtype=torch.int32, device=device)
        # what every request has seen, for the penalties
        self.history = torch.zeros(rows, most, dtype=torch.int32, device=device)
        self.temperature, self.repetition = (torch.full((rows,), x, device=device) for x in (0.7, 1.1))

    def turned(self, x, at):
        """Rotary positions."""
        a, b = x.float().chunk(2, -1)
        angle = at[:, None, None] * 10000.0 ** (-torch.arange(DIM // 2, device=self.dev) / (DIM // 2))
        c, s = angle.cos(), angle.sin()
        return torch.cat([a * c - b * s, a * s + b * c], -1).bfloat16()

    def layers(self, tokens, at, T, parents, cu):
        """New tokens [n] at positions `at`, at most T a row: the logits after each."""
        x, residual = torch.empty(len(tokens), MODEL, dtype=torch.bfloat16, device=self.dev), torch.zeros(len(tokens), MODEL, device=self.dev)
        api.rssm_residual_norm(self.embed[tokens.long()], residual, self.norms[0], x, residual)
        for i in range(LAYERS):
            q, k, v = (x @ self.qkv[i]).view(-1, HQ + 2 * HKV, DIM).split((HQ, HKV, HKV), 1)
            q, k, out = self.turned(q, at), self.turned(k, at), torch.empty(len(tokens), HQ, DIM, dtype=torch.bfloat16, device=self.dev)
            api.rssm_kv_append(self.cache, k, v, self.pages, self.lengths, T, cu, layer=i)
            api.rssm_tree_attention(self.cache, q, self.pages, self.lengths, T, out, self.scratch, parents, cu, layer=i)
            api.rssm_residual_norm(out.flatten(1) @ self.out[i], residual, self.norms[i + 1], x, residual)
        return x @ self.head

    def prompts(self, lens, tokens):
        """Packed prompts; the probabilities after each one's last token."""
        cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=self.dev)
        at = torch.cat([torch.arange(n) for n in lens]).to(self.dev)
        logits = self.layers(tokens, at, max(lens), None, cu)[cu[1:].long() - 1]
        for b, n in enumerate(lens):
            self.history[b, :n] = tokens[int(cu[b]) : int(cu[b]) + n]
        self.lengths += torch.tensor(lens, dtype=torch.int32, device=self.dev)
        probs = torch.empty(self.rows, VOCAB, device=self.dev)
        api.rssm_logits(logits, 1, probs, self.temperature, self.repetition, history=self.history, history_len=self.lengths)
        return probs

    def check(self):
        if int(self.cache.error_word):
            raise RuntimeError(f"the device reported errors: {int(self.cache.error_word)}")


def generate(model: TreeModel, lens, prompts, steps: int, nodes):
    """Tree decoding, row b with a tree of nodes[b] tokens: the tokens every row committed."""
    B, dev, gen, T = model.rows, model.dev, model.gen, max(nodes)
    p = model.prompts(lens, prompts)
    last = torch.multinomial(p, 1, generator=gen)[:, 0].int()
    n = sum(nodes)
    cu = torch.tensor([0] + list(torch.tensor(nodes).cumsum(0)), dtype=torch.int32, device=dev)
    row = torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(nodes, device=dev))
    parents = torch.tensor(sum((PARENTS[:k] for k in nodes), []), dtype=torch.int32, device=dev)
    choice = torch.tensor(sum((CHOICE[:k] for k in nodes), []), device=dev)
    depth = [0] * len(PARENTS)
    for t, up in enumerate(PARENTS):
        depth[t] = depth[up] + 1 if up >= 0 else 0
    depth = torch.tensor(sum((depth[:k] for k in nodes), []), device=dev)
    before = (cu[row] + parents.clamp(min=0)).long()  # the place that each token comes after, among all rows'
    drawn, ones = (torch.empty(n, dtype=torch.int32, device=dev) for _ in range(2))
    accepted, nxt = (torch.empty(B, dtype=torch.int32, device=dev) for _ in range(2))
    path = torch.empty(B, T, dtype=torch.int32, device=dev)
    probs = torch.empty(n, VOCAB, device=dev)
    word = torch.zeros(1, dtype=torch.int32, device=dev)
    committed = [[] for _ in range(B)]
    for _ in range(steps):
        tokens = last[row]
        for d in range(1, int(depth.max()) + 1):
            tokens = torch.where(depth == d, model.follow[tokens[before].long(), choice], tokens)
        logits = model.layers(tokens, model.lengths[row] + depth, T, parents, cu)
        api.rssm_logits(logits, T, probs, model.temperature, model.repetition, history=model.history, history_len=model.lengths,
                        tokens=tokens, parents=parents, cu_seqlens=cu, error_word=word)
        api.rssm_verify(probs, tokens, torch.rand(n, generator=gen, device=dev), torch.rand(n, generator=gen, device=dev), 1, ones, drawn,
                        error_word=word)
        api.rssm_tree_accept(model.cache, model.pages, model.lengths, tokens, parents, drawn, T, accepted, nxt, path, cu)
        for b, k in enumerate(accepted.tolist()):
            took = tokens[cu[b] + path[b, :k]]
            model.history[b, model.lengths[b] : model.lengths[b] + k] = took
            committed[b] += took.tolist()
        model.lengths += accepted
        last = nxt.clone()
    model.check()
    if int(word):
        raise RuntimeError(f"the device reported errors: {int(word)}")
    return committed


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rows", type=int, default=8)
    ap.add_argument("--steps", type=int, default=12)
    ap.add_argument("--format", choices=FORMATS, default="int8")
    a = ap.parse_args()
    lens = [7 + 37 * i % 150 for i in range(a.rows)]
    nodes = [len(PARENTS)] * a.rows
    model = TreeModel(a.rows, max(lens) + (a.steps + 1) * len(PARENTS), FORMATS[a.format])
    prompts = torch.randint(0, VOCAB, (sum(lens),), generator=model.gen, device="cuda", dtype=torch.int32)
    committed = generate(model, lens, prompts, a.steps, nodes)
    total = sum(len(c) for c in committed)
    print(f"{a.rows} rows, {a.steps} steps of trees of {len(PARENTS)} tokens: {total} tokens committed, "
          f"{total - a.rows * a.steps} of them drafts")


if __name__ == "__main__":
    main()
