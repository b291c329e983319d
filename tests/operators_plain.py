"""The added operators from their definitions, in 64 bits, token by token and row by row (tests only)."""
import math

import torch


def unit(x):
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6)


def delta_tokens(S, q, k, v, g, beta, scale, l2norm, keep=None):
    """Tokens [n, H, d] through the rule from S [Hv, dv, dk]; returns (outputs, corrections u, S after `keep` tokens)."""
    S, q, k, v, g, beta = (x.double() for x in (S, q, k, v, g, beta))
    if l2norm:
        q, k = unit(q), unit(k)
    rep = v.shape[1] // k.shape[1]
    q, k = q.repeat_interleave(rep, 1) * scale, k.repeat_interleave(rep, 1)
    g = g.clamp(min=-100.0)
    S, out, us, kept = S.clone(), [], [], S.clone()
    for t in range(v.shape[0]):
        S = S * torch.exp(g[t])[:, None, None]
        u = beta[t][:, None] * (v[t] - torch.einsum("hvk,hk->hv", S, k[t]))
        S = S + u[:, :, None] * k[t][:, None, :]
        out.append(torch.einsum("hvk,hk->hv", S, q[t]))
        us.append(u)
        if keep is None or t < keep:
            kept = S
    z = v.new_zeros((0,) + tuple(v.shape[1:]))
    return (torch.stack(out) if out else z), (torch.stack(us) if us else z), kept


def verify_row(target, draft, tokens, u, u_next):
    """One row: probabilities as float32 tensors [n, V] (draft None: certain drafts); integers by Python's own."""
    n, V = target.shape
    one = torch.ones(())
    t = 0
    while t + 1 < n:
        tok = int(tokens[t + 1])
        if not 0 <= tok < V:
            break
        q = draft[t + 1, tok] if draft is not None else one
        if not bool(u[t + 1] * q < target[t, tok]):
            break
        t += 1
    r = target[t]
    if t + 1 < n:
        if draft is not None:
            r = r - draft[t + 1]
        elif 0 <= int(tokens[t + 1]) < V:
            r = r.clone()
            r[int(tokens[t + 1])] -= 1.0

    def fixed(x):
        return [int(math.floor(min(y, 1.0) * 2.0**36)) if y > 0 else 0 for y in x.tolist()]

    w = fixed(r)
    if sum(w) == 0 and t + 1 < n:
        w = fixed(target[t])
    total = sum(w)
    if total == 0:
        return t + 1, -1
    aim = (total * int(math.floor(float(u_next) * 2.0**24))) >> 24
    run = 0
    for i, x in enumerate(w):
        run += x
        if run > aim:
            return t + 1, i
    raise AssertionError("unreachable")


def gated_norm(x, z, w, group, eps, norm_first):
    x, z, w = x.double(), z.double(), w.double()
    gate = z * torch.sigmoid(z)
    y = (x if norm_first else x * gate).reshape(x.shape[0], -1, group)
    y = y / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + eps)
    y = (y * (w if w.numel() == group else w.reshape(-1, group))).reshape(x.shape)
    return y * gate if norm_first else y


def residual_norm(x, residual, w, post, scale, alpha, eps):
    m, residual, w = x.double(), residual.double(), w.double()
    if post is not None:
        m = m / torch.sqrt(m.pow(2).mean(-1, keepdim=True) + eps) * post.double()
    if scale is not None:
        m = m * scale.double()
    h = residual + alpha * m
    return h, h / torch.sqrt(h.pow(2).mean(-1, keepdim=True) + eps) * w
