"""The operators of attention layers and of the sampler from their definitions, in 64 bits, token by token (tests only)."""
import math

import torch

QMAX = {3: 127.0, 4: 448.0}  # api.I8, api.E4M3


def decoded(cache, name, layer=0):
    """A layer's keys or values in 64 bits: [page, head, place, dim]."""
    x = getattr(cache, name)[layer].cpu()
    if cache.format == 1:
        return x.double()
    x = x.view(torch.float8_e4m3fn).float().double() if cache.format == 4 else x.double()
    return x * getattr(cache, name + "_scale")[layer].cpu().double()[..., None]


def quantised(x, fmt):
    """Codes and scales of bf16 rows [.., dim], in the fp32 operations of the format's definition."""
    x = x.float()
    most = x.abs().amax(-1)
    scale = torch.where(most < 2.0**-100, torch.ones_like(most), most * torch.tensor(1.0 / QMAX[fmt], dtype=torch.float32))
    y = x * (1.0 / scale)[..., None]
    codes = y.round().clamp(-127, 127).to(torch.int8) if fmt == 3 else y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    fine = most.isfinite()
    return torch.where(fine[..., None], codes, torch.zeros_like(codes)), torch.where(fine, scale, math.nan)


def row_tokens(x, table, page, first, count):
    """[page, head, place, dim] -> [count, head, dim] of a row's positions first .. ."""
    out = x.new_zeros(count, x.shape[1], x.shape[3])
    for i in range(count):
        p = first + i
        out[i] = x[int(table[p // page]), :, p % page]
    return out


def path(parents, t):
    """Places in the row of the tokens that t comes after, itself included, root first; parents None: a chain."""
    if parents is None:
        return list(range(t + 1))
    up = [t]
    while parents[up[-1]] >= 0:
        up.append(int(parents[up[-1]]))
    return up[::-1]


def attention_row(k, v, q, parents, length, scale):
    """Row of new tokens q [n, hq, d] over k, v [length + n, h, d]: the output, and sum p |v| beside it."""
    n, hq, d = q.shape
    rep = hq // k.shape[1]
    out, size = torch.zeros(n, hq, d, dtype=torch.float64), torch.zeros(n, hq, d, dtype=torch.float64)
    for t in range(n):
        seen = torch.tensor(list(range(length)) + [length + j for j in path(parents, t)])
        kk, vv = k[seen].repeat_interleave(rep, 1), v[seen].repeat_interleave(rep, 1)
        p = torch.softmax(torch.einsum("hd,shd->hs", q[t].double(), kk) * scale, -1)
        out[t], size[t] = torch.einsum("hs,shd->hd", p, vv), torch.einsum("hs,shd->hd", p, vv.abs())
    return out, size


def accept_row(tokens, parents, drawn):
    """(path, what was drawn after its last token) of one row's lists."""
    if not tokens:
        return [], -1
    up = list(range(-1, len(tokens) - 1)) if parents is None else parents
    walk = [0]
    while True:
        nxt = drawn[walk[-1]]
        on = [t for t in range(len(tokens)) if up[t] == walk[-1] and tokens[t] == nxt] if nxt >= 0 else []
        if not on:
            return walk, nxt
        walk.append(on[0])


def logits_row(x, history, prompt, fed, repetition, presence, frequency, bias, mask, temperature, probs=True):
    """One row x [V]: history and fed are lists of ids, bias a list of (id, value), mask a list of truth values or None."""
    x = x.double().clone()
    V = x.numel()
    count, seen = torch.zeros(V, dtype=torch.float64), torch.zeros(V, dtype=torch.bool)
    for i, tok in enumerate(history):
        if 0 <= tok < V:
            seen[tok] = True
            if i >= prompt:
                count[tok] += 1
    for tok in fed:
        if 0 <= tok < V:
            seen[tok] = True
            count[tok] += 1
    x = torch.where(seen, torch.where(x > 0, x / repetition, x * repetition), x)
    x = torch.where(count > 0, x - (presence + frequency * count), x)
    for i, y in bias:
        if 0 <= i < V:
            x[i] += y
    if mask is not None:
        x[~torch.tensor(mask)] = -math.inf
    x[x.isnan()] = -math.inf
    if not probs:
        return x / temperature if temperature > 0 else x
    top = x.max()
    if top == -math.inf:
        return torch.zeros_like(x)
    if temperature == 0:
        return torch.zeros_like(x).index_fill_(0, (x == top).nonzero()[0], 1.0)
    if top == math.inf:
        return (x == top).double() / (x == top).sum()
    return torch.softmax(x / temperature, 0)
