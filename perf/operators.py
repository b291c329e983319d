"""Workloads of the layers around the state update of a decode step: what is
timed, the inputs, and the operators' plain forms.

Five operators that a hybrid model's serving loop runs next to the selective
state update:

  delta_step      gated delta rule, a decode step of 1..8 drafted tokens a row
                  that first commits the drafts accepted after the last step
  delta_prefill   gated delta rule over whole prompts, in chunks
  verify          verification of drafted tokens from given random numbers
  gated_norm      the mixer's output norm with its silu gate, per head or group
  residual_norm   norm after a block, residual scale and add, norm before the next

`run` computes them in plain torch operations in 32 bits (`own` false) or by
the library's calls (`own` true); both work on the same inputs and leave the
same buffers updated.
"""
import math
import random

import torch

own = False

DK = 128  # key width of the delta rule's heads in every case
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
FIXED = 36  # fraction bits of the sampling weights


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one request, one token a step: the latency of a chat's next token
        dict(name="step one token", op="delta_step", batch=1, T=1, ragged=False, hk=16, hv=32, dv=128, state="f32", lens=1),
        # a decode batch with four drafts a row (the Mamba-2 decode workload's batch)
        dict(name="step 64 rows", op="delta_step", batch=64, T=4, ragged=False, hk=16, hv=32, dv=128, state="f32", lens=2),
        # the sweep's largest batch: 1..5 drafts a row, packed, 2-byte states
        dict(name="step 1024 rows", op="delta_step", batch=1024, T=5, ragged=True, hk=16, hv=32, dv=128, state="bf16", lens=3),
        # a short prompt, not a multiple of any tile
        dict(name="prompt of 77", op="delta_prefill", seqs=1, tokens=77, hk=16, hv=32, dv=128, state="f32", lens=4),
        # sixteen prompts of very different lengths in one call, some of them one token
        dict(name="prompts ragged", op="delta_prefill", seqs=16, tokens=12001, hk=16, hv=32, dv=128, state="bf16", lens=5),
        # one long document
        dict(name="prompt of 16384", op="delta_prefill", seqs=1, tokens=16384, hk=16, hv=32, dv=128, state="f32", lens=6),
        # one request with four tokens fed, three of them drafts
        dict(name="verify one", op="verify", batch=1, T=4, ragged=False, vocab=32768, probs="f32", draft=True, lens=7),
        # the decode batch at seven tokens a row, 2-byte probabilities
        dict(name="verify 64 rows", op="verify", batch=64, T=7, ragged=False, vocab=131072, probs="bf16", draft=True, lens=8),
        # drafts from a lookup (no draft probabilities), 1..5 tokens a row, an odd vocabulary
        dict(name="verify 512 lookup", op="verify", batch=512, T=5, ragged=True, vocab=100279, probs="f32", draft=False, lens=9),
        # the Mamba-2 decode layer's output: 128 heads of 64 in 8 norm groups, gate first; 64 rows of 4 tokens
        dict(name="gated norm 256", op="gated_norm", rows=256, dim=8192, group=1024, dtype="bf16", norm_first=False, shared=False),
        # a long prompt's delta-rule output: norm per head, then the gate, one weight for all heads
        dict(name="gated norm 16384", op="gated_norm", rows=16384, dim=4096, group=128, dtype="bf16", norm_first=True, shared=True),
        # between two blocks of a prompt: both norms, per-channel residual scale, the residual stream in 32 bits
        dict(name="residual norm 8192", op="residual_norm", rows=8192, dim=5120, dtype="bf16", residual="f32", post=True, scale=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["delta_step", "delta_prefill", "verify", "gated_norm", "residual_norm"])
    seed = rng.randrange(1 << 30)
    if op == "delta_step":
        hk, T = rng.choice([2, 4, 8, 16]), rng.randint(1, 8)
        hv, dv = hk * rng.choice([1, 2, 4]), rng.choice([64, 128, 256])
        most = int(3e9 / (hv * dv * DK * 5 * T))  # rows that cost no more than the largest listed case
        return dict(op=op, batch=_log(rng, 1, min(512, most)), T=T, ragged=rng.random() < 0.5, hk=hk, hv=hv, dv=dv,
                    state=rng.choice(["f32", "bf16"]), lens=seed)
    if op == "delta_prefill":
        hk = rng.choice([4, 8, 16])
        tokens = _log(rng, 1, 16384)
        return dict(op=op, seqs=min(tokens, rng.choice([1, 2, 5, 16, 33])), tokens=tokens, hk=hk, hv=hk * rng.choice([1, 2]),
                    dv=rng.choice([64, 128]), state=rng.choice(["f32", "bf16"]), lens=seed)
    if op == "verify":
        return dict(op=op, batch=_log(rng, 1, 256), T=rng.randint(1, 8), ragged=rng.random() < 0.5, vocab=_log(rng, 1000, 131072),
                    probs=rng.choice(["f32", "bf16", "f16"]), draft=rng.random() < 0.7, lens=seed)
    if op == "gated_norm":
        group = rng.choice([64, 80, 128, 256, 1000, 1024, 2048])
        groups = rng.choice([1, 2, 8, 31, 32])
        return dict(op=op, rows=max(1, min(_log(rng, 1, 16384), 100_000_000 // (group * groups))), dim=group * groups, group=group,
                    dtype=rng.choice(["f32", "bf16", "f16"]), norm_first=rng.random() < 0.5, shared=rng.random() < 0.5)
    dim = rng.choice([513, 1000, 2048, 4096, 5120, 6144, 8192, 12288])
    return dict(op=op, rows=max(1, min(_log(rng, 1, 16384), 60_000_000 // dim)), dim=dim, dtype=rng.choice(["f32", "bf16", "f16"]),
                residual=rng.choice(["f32", "same"]), post=rng.random() < 0.5, scale=rng.random() < 0.5)


def _lengths(case):
    """Tokens per row of a step (and how many of each row's are accepted), or the prompts' lengths: plain lists."""
    rng = random.Random(case["lens"])
    if case["op"] == "delta_prefill":
        n, left = case["seqs"], case["tokens"] - case["seqs"]
        share = [rng.expovariate(1.0) ** 2 for _ in range(n)]  # a few long prompts and many short ones
        lens = [1 + int(left * s / sum(share)) for s in share]
        lens[share.index(max(share))] += case["tokens"] - sum(lens)
        return lens, None
    T = case["T"]
    lens = [rng.randint(1, T) if case["ragged"] else T for _ in range(case["batch"])]
    return lens, [rng.randint(0, t) for t in lens]


def _offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _delta_inputs(case, gen, ntok, dev):
    hk, hv, dv = case["hk"], case["hv"], case["dv"]
    rnd = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    # q, k and v are columns of one projection, as a layer has them
    qkv = rnd(ntok, 2 * hk * DK + hv * dv + 64).bfloat16()  # the last 64: what g and beta are made from
    q = qkv[:, : hk * DK].unflatten(1, (hk, DK))
    k = qkv[:, hk * DK : 2 * hk * DK].unflatten(1, (hk, DK))
    v = qkv[:, 2 * hk * DK : 2 * hk * DK + hv * dv].unflatten(1, (hv, dv))
    rate = torch.exp(torch.rand(hv, generator=gen, device=dev) * math.log(16.0))
    g = -rate * torch.nn.functional.softplus(rnd(ntok, hv) - 3.0)  # log decay, about -0.05..-1
    beta = torch.sigmoid(rnd(ntok, hv))
    return q, k, v, g, beta


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    s = dict(case=case)
    op = case["op"]
    if op in ("delta_step", "delta_prefill"):
        lens, accepted = _lengths(case)
        n, ntok = len(lens), sum(lens)
        hk, hv, dv = case["hk"], case["hv"], case["dv"]
        s["q"], s["k"], s["v"], s["g"], s["beta"] = _delta_inputs(case, gen, ntok, dev)
        s["lens"] = lens  # the scheduler knows them
        s["out"] = torch.empty(ntok, hv, dv, dtype=torch.bfloat16, device=dev)
        s["slots"] = (torch.randperm(n, generator=gen, device=dev) + 1).int()
        s["cu"] = torch.tensor(_offsets(lens), dtype=torch.int32, device=dev)
        np_ = case["T"] if op == "delta_step" else 4
        s["state"] = (0.1 * rnd(n + 1, hv, dv, DK)).to(DTYPES[case["state"]])
        # the drafts of the step before, waiting for their verification
        s["pend_k"] = rnd(n + 1, 2, hk, np_, DK).bfloat16()
        s["pend_w"] = rnd(n + 1, 2, hv, np_, dv) / math.sqrt(DK)
        s["pend_c"] = -0.1 * torch.rand(n + 1, 2, hv, np_, generator=gen, device=dev).cumsum(-1)
        s["pend"] = torch.zeros(n + 1, 2, dtype=torch.int32, device=dev)
        if op == "delta_step":
            s["accepted"] = torch.tensor(accepted, dtype=torch.int32, device=dev)
            s["pend"][s["slots"].long(), 1] = torch.tensor(lens, dtype=torch.int32, device=dev)
        else:
            # a prompt is new, or goes on where an earlier part of it ended
            s["initial"] = torch.randint(0, 2, (n,), generator=gen, device=dev, dtype=torch.int32)
        if own:  # the handle and the workspace that a program keeps
            from speculative_state_replay_gb300 import api

            s["cache"] = api.DeltaCache(n + 1, hk, hv, DK, dv, np_, api.F32 if case["state"] == "f32" else api.BF16, device=dev,
                                        state=s["state"], pend_k=s["pend_k"], pend_w=s["pend_w"], pend_c=s["pend_c"], pend=s["pend"])
            s["scratch"] = api.alloc_delta_scratch(s["cache"], n, ntok)
    elif op == "verify":
        lens, accepted = _lengths(case)
        n, ntok, V = len(lens), sum(lens), case["vocab"]
        s["cu"] = torch.tensor(_offsets(lens), dtype=torch.int32, device=dev) if case["ragged"] else None
        logits = 3.0 * rnd(ntok, V)
        if case["draft"]:
            q = torch.softmax(logits + 0.7 * rnd(ntok, V), -1)
            s["draft"] = q.to(DTYPES[case["probs"]])
            s["tokens"] = (q / -torch.log1p(-torch.rand(ntok, V, generator=gen, device=dev))).argmax(-1).int()
            del q
        else:
            s["draft"] = None
            s["tokens"] = (logits + 2.0 * rnd(ntok, V)).argmax(-1).int()
        s["target"] = torch.softmax(logits, -1).to(DTYPES[case["probs"]])
        s["u"] = torch.rand(ntok, generator=gen, device=dev)
        s["u_next"] = torch.rand(n, generator=gen, device=dev)
        s["accepted"] = torch.empty(n, dtype=torch.int32, device=dev)
        s["next"] = torch.empty(n, dtype=torch.int32, device=dev)
    elif op == "gated_norm":
        R, D = case["rows"], case["dim"]
        dt = DTYPES[case["dtype"]]
        s["x"] = rnd(R, D).to(dt)
        s["z"] = rnd(R, 2 * D).to(dt)[:, D:]  # the gate is part of the input projection
        s["w"] = 1.0 + 0.1 * rnd(case["group"] if case["shared"] else D)
        s["out"] = torch.empty(R, D, dtype=dt, device=dev)
    else:
        R, D = case["rows"], case["dim"]
        dt = DTYPES[case["dtype"]]
        s["x"] = rnd(R, D).to(dt)
        s["residual"] = (3.0 * rnd(R, D)).to(torch.float32 if case["residual"] == "f32" else dt)
        s["w"] = 1.0 + 0.1 * rnd(D)
        s["post"] = 1.0 + 0.1 * rnd(D) if case["post"] else None
        s["scale"] = 0.5 + 0.1 * rnd(D) if case["scale"] else None
        s["alpha"] = 0.7
        s["out"] = torch.empty(R, D, dtype=dt, device=dev)
        s["residual_out"] = torch.empty_like(s["residual"])
    if own:
        from speculative_state_replay_gb300 import api

        s["api"] = api
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _unit(x):
    return x * torch.rsqrt(x.square().sum(-1, keepdim=True) + 1e-6)


def _inverse(A):
    """(I + A)^-1 of strictly lower triangular [..., n, n] blocks, n a power of two: the inverses of the diagonal blocks joined, from 1 x 1 up."""
    n = A.shape[-1]
    inv = torch.ones_like(A[..., 0]).reshape(*A.shape[:-2], n, 1, 1)
    m = 1
    while m < n:
        i = torch.arange(0, n, 2 * m, device=A.device)[:, None]
        r = torch.arange(m, device=A.device)
        low = A[..., (i + m + r)[:, :, None], (i + r)[:, None, :]]  # the block below the diagonal of each pair
        a, b = inv[..., 0::2, :, :], inv[..., 1::2, :, :]
        top = torch.cat([a, torch.zeros_like(a)], -1)
        inv = torch.cat([top, torch.cat([-(b @ low @ a), b], -1)], -2)
        m *= 2
    return inv[..., 0, :, :]


def _parts(q, k, v, g, beta):
    """What does not depend on the state, for chunks [..., C, d]: the rows to solve for (W, U), the scores, cumulative decays."""
    C = q.shape[-2]
    c = g.cumsum(-1)
    low = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    decay = torch.exp(torch.where(low, c[..., :, None] - c[..., None, :], -math.inf))
    A = (beta[..., None] * (k @ k.mT) * decay).tril(-1)
    inv = _inverse(A)
    W = inv @ (k * (beta * torch.exp(c))[..., None])
    U = inv @ (v * beta[..., None])
    return W, U, (q @ k.mT) * decay, c


def _heads(x, hv):
    return x.float().repeat_interleave(hv // x.shape[1], 1)


def _padded(x, lens, at, C):
    """[tok, H, d] -> [rows, H, C, d], zeros past a row's tokens."""
    i = torch.arange(C, device=x.device)
    live = i < lens[:, None]
    rows = x[torch.where(live, at[:, None] + i, 0)] * live[..., None, None]
    return rows.transpose(1, 2), live


def _plain_step(s):
    case = s["case"]
    hv, T = case["hv"], case["T"]
    C = 1 << (T - 1).bit_length()
    slots = s["slots"].long()
    cu = s["cu"].long()
    lens = cu[1:] - cu[:-1]
    side = s["pend"][slots, 0].long()
    a = s["accepted"].long()
    # the accepted drafts of the step before enter the state
    c = s["pend_c"][slots, side]
    live = torch.arange(T, device=c.device) < a[:, None]
    end = torch.where(a[:, None] > 0, c.gather(-1, (a - 1).clamp(min=0)[:, None, None].expand(-1, hv, 1))[..., 0], 0.0)
    wt = torch.where(live[:, None], torch.exp(end[..., None] - c), 0.0)
    S = s["state"][slots].float() * torch.exp(end)[..., None, None]
    S = S + (s["pend_w"][slots, side] * wt[..., None]).mT @ s["pend_k"][slots, side].float().repeat_interleave(hv // case["hk"], 1)
    s["state"][slots] = torch.where((a > 0)[:, None, None, None], S, s["state"][slots].float()).to(s["state"].dtype)
    # the drafts of this step
    norm = torch.rsqrt(s["k"].float().square().sum(-1) + 1e-6)
    q, _ = _padded(_heads(_unit(s["q"].float()), hv) / math.sqrt(DK), lens, cu[:-1], C)
    k, _ = _padded(_heads(_unit(s["k"].float()), hv), lens, cu[:-1], C)
    r, _ = _padded(norm.repeat_interleave(hv // case["hk"], 1)[..., None], lens, cu[:-1], C)
    v, _ = _padded(s["v"].float(), lens, cu[:-1], C)
    gb, live = _padded(torch.stack([s["g"], s["beta"]], -1), lens, cu[:-1], C)
    W, U, P, c = _parts(q, k, v, gb[..., 0], gb[..., 1])
    u = U - W @ S.mT
    o = torch.exp(c)[..., None] * (q @ S.mT) + P @ u
    s["out"].copy_(o.transpose(1, 2)[live])
    # they wait for their verification in the other half
    b, t = live[:, :T].nonzero(as_tuple=True)
    to = (slots[b], 1 - side[b], slice(None), t)
    s["pend_k"][to] = s["k"]
    s["pend_w"][to] = (u * r)[b, :, t]
    s["pend_c"][to] = c[b, :, t]
    s["pend"][slots] = torch.stack([1 - side, lens], -1).int()
    return {"out": s["out"], "state": s["state"], "pend_k": s["pend_k"], "pend_w": s["pend_w"], "pend_c": s["pend_c"], "pend": s["pend"]}


def _plain_prefill(s):
    case = s["case"]
    hv, C = case["hv"], 64
    cu = s["cu"].long()
    lens, slots = cu[1:] - cu[:-1], s["slots"].long()
    n = len(lens)
    chunks = -(-(lens) // C)
    first = chunks.cumsum(0) - chunks
    total, most = (f(-(-m // C) for m in s["lens"]) for f in (sum, max))
    row = torch.repeat_interleave(torch.arange(n, device=cu.device), chunks, output_size=total)
    i = torch.arange(total, device=cu.device) - first[row]
    clen, at = (lens[row] - C * i).clamp(max=C), cu[row] + C * i
    q, live = _padded(_heads(_unit(s["q"].float()), hv) / math.sqrt(DK), clen, at, C)
    k, _ = _padded(_heads(_unit(s["k"].float()), hv), clen, at, C)
    v, _ = _padded(s["v"].float(), clen, at, C)
    gb, _ = _padded(torch.stack([s["g"], s["beta"]], -1), clen, at, C)
    W, U, P, c = _parts(q, k, v, gb[..., 0], gb[..., 1])
    qd, kd = q * torch.exp(c)[..., None], k * torch.exp(c[..., -1:] - c)[..., None]
    S = torch.where((s["initial"] > 0)[:, None, None, None], s["state"][slots].float(), 0.0)
    o = torch.empty_like(v)
    for j in range(most):  # a chunk needs the state that the one before it leaves
        if n == 1:  # one prompt: views instead of gathers
            on, x = slice(None), slice(j, j + 1)
        else:
            on = (chunks > j).nonzero()[:, 0]
            x = first[on] + j
        St = S[on].mT
        u = U[x] - W[x] @ St
        o[x] = qd[x] @ St + P[x] @ u
        S[on] = S[on] * torch.exp(c[x][..., -1])[..., None, None] + u.mT @ kd[x]
    s["out"].copy_(o.transpose(1, 2)[live])
    s["state"][slots] = S.to(s["state"].dtype)
    s["pend"][slots] = 0  # no drafts wait
    return {"out": s["out"], "state": s["state"], "pend": s["pend"]}


def _weights(p):
    """Sampling weights in fixed point: sums of them do not depend on their order."""
    return torch.where(p > 0, p.clamp(max=1.0), 0.0).mul(2.0**FIXED).to(torch.int64)


def _plain_verify(s):
    case = s["case"]
    n, T = case["batch"], case["T"]
    dev = s["u"].device
    cu = torch.arange(n + 1, device=dev) * T if s["cu"] is None else s["cu"].long()
    lens = cu[1:] - cu[:-1]
    token = s["tokens"].long()
    # draft t of a row is tested against the target's probabilities after token t - 1
    i = torch.arange(len(token), device=dev)
    p_at = s["target"][(i - 1).clamp(min=0), token].float()
    q_at = s["draft"][i, token].float() if s["draft"] is not None else torch.ones_like(p_at)
    ok = s["u"] * q_at < p_at
    t = torch.arange(T, device=dev)
    at = cu[:-1, None] + t
    inside = t < lens[:, None]
    ok = (ok[torch.where(inside, at, 0)] | (t == 0)) & inside
    count = ok.int().cumprod(-1).sum(-1)  # the fed token and the leading drafts that pass
    last = cu[:-1] + count - 1
    p = s["target"][last].float()
    more = count < lens
    nxt = torch.where(more, last + 1, last)
    if s["draft"] is not None:
        q = torch.where(more[:, None], s["draft"][nxt].float(), 0.0)
    else:
        q = torch.zeros_like(p).scatter_(1, token[nxt][:, None], more[:, None].float())
    w = _weights(p - q)
    total = w.sum(-1)
    w = torch.where((total > 0)[:, None], w, _weights(p))
    cum = w.cumsum(-1)
    total = cum[:, -1]
    u = (s["u_next"] * 2.0**24).to(torch.int64)
    aim = (total >> 24) * u + (((total & 0xFFFFFF) * u) >> 24)
    s["accepted"].copy_(count)
    s["next"].copy_((cum <= aim[:, None]).sum(-1))
    return {"accepted": s["accepted"], "next": s["next"]}


def _plain_gated_norm(s):
    case = s["case"]
    R, D, G = case["rows"], case["dim"], case["group"]
    x, z, w = s["x"].float(), s["z"].float(), s["w"]
    gate = z / (1.0 + torch.exp(-z))
    if not case["norm_first"]:
        x = x * gate
    y = x.reshape(R, D // G, G)
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-5)
    y = y.reshape(R, D) * (w.repeat(D // G) if case["shared"] else w)
    if case["norm_first"]:
        y = y * gate
    s["out"].copy_(y)
    return {"out": s["out"]}


def _plain_residual_norm(s):
    x = s["x"].float()
    if s["post"] is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5) * s["post"]
    if s["scale"] is not None:
        x = x * s["scale"]
    h = s["residual"].float() + s["alpha"] * x
    s["residual_out"].copy_(h)
    s["out"].copy_(h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-5) * s["w"])
    return {"out": s["out"], "residual": s["residual_out"]}


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"delta_step": _plain_step, "delta_prefill": _plain_prefill, "verify": _plain_verify,
                "gated_norm": _plain_gated_norm, "residual_norm": _plain_residual_norm}[op](s)
    api = s["api"]
    if op == "delta_step":
        api.rssm_delta_step(s["cache"], s["q"], s["k"], s["v"], s["g"], s["beta"], s["slots"], s["accepted"], case["T"], s["out"],
                            s["scratch"], cu_seqlens=s["cu"] if case["ragged"] else None, l2norm=True)
        return {"out": s["out"], "state": s["state"], "pend_k": s["pend_k"], "pend_w": s["pend_w"], "pend_c": s["pend_c"], "pend": s["pend"]}
    if op == "delta_prefill":
        api.rssm_delta_prefill(s["cache"], s["q"], s["k"], s["v"], s["g"], s["beta"], s["slots"], s["cu"], s["out"], s["scratch"],
                               initial=s["initial"], l2norm=True)
        return {"out": s["out"], "state": s["state"], "pend": s["pend"]}
    if op == "verify":
        api.rssm_verify(s["target"], s["tokens"], s["u"], s["u_next"], case["T"], s["accepted"], s["next"], draft=s["draft"],
                        cu_seqlens=s["cu"])
        return {"accepted": s["accepted"], "next": s["next"]}
    if op == "gated_norm":
        api.rssm_gated_norm(s["x"], s["z"], s["w"], s["out"], case["group"], eps=1e-5, norm_first=case["norm_first"])
        return {"out": s["out"]}
    api.rssm_residual_norm(s["x"], s["residual"], s["w"], s["out"], s["residual_out"], post_weight=s["post"], scale=s["scale"],
                           alpha=s["alpha"], eps=1e-5)
    return {"out": s["out"], "residual": s["residual_out"]}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("delta_step", "delta_prefill"):
        lens, accepted = _lengths(case)
        hk, hv, dv = case["hk"], case["hv"], case["dv"]
        ntok, sb = sum(lens), BYTES[case["state"]]
        b = ntok * (4 * hk * DK + 4 * hv * dv + 8 * hv)  # q, k, v, out, g, beta
        if op == "delta_step":
            a, some = sum(accepted), sum(x > 0 for x in accepted)
            b += (case["batch"] + some) * hv * dv * DK * sb  # every state is read, those that change are written
            b += (a + ntok) * (2 * hk * DK + 4 * hv * dv + 4 * hv)  # waiting drafts in, new ones out
            f = 2 * hv * dv * DK * (a + 2 * ntok)
        else:
            b += 2 * case["seqs"] * hv * dv * DK * sb
            f = 6 * hv * dv * DK * ntok  # state times key, state times query, the state's update
        return {"bytes": b, "flops": f}
    if op == "verify":
        lens, _ = _lengths(case)
        # one row of each side for the next token, and single values for the tests
        return {"bytes": case["batch"] * case["vocab"] * BYTES[case["probs"]] * (2 if case["draft"] else 1) + 24 * sum(lens),
                "flops": 3 * case["batch"] * case["vocab"]}
    n = case["rows"] * case["dim"]
    e = BYTES[case["dtype"]]
    if op == "gated_norm":
        return {"bytes": 3 * n * e + 4 * (case["group"] if case["shared"] else case["dim"]), "flops": 8 * n}
    r = 4 if case["residual"] == "f32" else e
    return {"bytes": n * (2 * e + 2 * r) + 4 * case["dim"] * (1 + case["post"] + case["scale"]), "flops": 10 * n}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    op = case["op"]
    if op == "verify":
        return None  # whole numbers
    s = prepare(case, seed)
    f = lambda x: x.double()  # noqa: E731
    if op == "gated_norm":
        R, D, G = case["rows"], case["dim"], case["group"]
        gate = f(s["z"]) * torch.sigmoid(f(s["z"]))
        y = f(s["x"]) if case["norm_first"] else f(s["x"]) * gate
        y = y.view(R, -1, G)
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / G + 1e-5)
        y = (y * f(s["w"]) if case["shared"] else y * f(s["w"]).view(-1, G)).reshape(R, D)
        return {"out": y * gate if case["norm_first"] else y}
    if op == "residual_norm":
        m = f(s["x"])
        D = case["dim"]
        if s["post"] is not None:
            m = m / torch.sqrt((m * m).sum(-1, keepdim=True) / D + 1e-5) * f(s["post"])
        h = f(s["residual"]) + s["alpha"] * (m if s["scale"] is None else f(s["scale"]) * m)
        return {"out": h / torch.sqrt((h * h).sum(-1, keepdim=True) / D + 1e-5) * f(s["w"]), "residual": h}
    # the delta rule token by token: S <- e^g S, u = beta (v - S k), S <- S + u k', o = S q
    lens, accepted = _lengths(case)
    cu, rep, slots = _offsets(lens), case["hv"] // case["hk"], s["slots"].long()
    q = f(s["q"]) / torch.sqrt(f(s["q"]).pow(2).sum(-1, keepdim=True) + 1e-6) / math.sqrt(DK)
    r = 1.0 / torch.sqrt(f(s["k"]).pow(2).sum(-1) + 1e-6)
    k = f(s["k"]) * r[..., None]
    q, k, r = (x.repeat_interleave(rep, 1) for x in (q, k, r))
    v, g, beta = f(s["v"]), f(s["g"]), f(s["beta"])
    state = f(s["state"])
    o = torch.empty(v.shape, dtype=torch.float64, device=v.device)
    w, csum = torch.empty_like(o), torch.empty_like(g)
    if op == "delta_step":
        for b, a in enumerate(accepted if case["batch"] <= 64 else []):
            i = slots[b]
            for j in range(a):
                c = f(s["pend_c"][i, 0])
                d = torch.exp(c[:, j] - (c[:, j - 1] if j else 0.0))
                state[i] = d[:, None, None] * state[i] + f(s["pend_w"][i, 0, :, j])[:, :, None] * \
                    f(s["pend_k"][i, 0, :, j]).repeat_interleave(rep, 0)[:, None, :]
        if case["batch"] > 64:  # rows with as many accepted drafts together
            for a in range(1, case["T"] + 1):
                on = torch.tensor([b for b, x in enumerate(accepted) if x >= a], dtype=torch.long, device=v.device)
                if not len(on):
                    break
                i = slots[on]
                c = f(s["pend_c"][i, 0])
                d = torch.exp(c[..., a - 1] - (c[..., a - 2] if a > 1 else 0.0))
                state[i] = d[..., None, None] * state[i] + f(s["pend_w"][i, 0, :, a - 1])[..., None] * \
                    f(s["pend_k"][i, 0, :, a - 1]).repeat_interleave(rep, 1)[:, :, None, :]
        S = state[slots]
    else:
        S = state[slots] * (s["initial"] > 0)[:, None, None, None]
    order = sorted(range(len(lens)), key=lambda b: -lens[b])  # the rows still running come first
    S = S[torch.tensor(order, device=v.device)]
    base = torch.tensor([cu[b] for b in order], device=v.device)
    run_c = torch.zeros(len(lens), case["hv"], dtype=torch.float64, device=v.device)
    for t in range(max(lens)):
        n = sum(lens[b] > t for b in order) if len(lens) > 1 else 1
        x = base[:n] + t
        Sn = S[:n]
        Sn *= torch.exp(g[x])[..., None, None]
        kt = k[x][..., None]
        u = beta[x][..., None] * (v[x] - (Sn @ kt)[..., 0])
        Sn += u[..., None] * kt.mT
        o[x] = (Sn @ q[x][..., None])[..., 0]
        if op == "delta_step":
            run_c[:n] += g[x]
            w[x], csum[x] = u * r[x][..., None], run_c[:n]
    if op == "delta_prefill":
        state[slots[torch.tensor(order, device=v.device)]] = S
        return {"out": o, "state": state, "pend": None}
    pw, pc = f(s["pend_w"]), f(s["pend_c"])
    for t in range(case["T"]):
        on = torch.tensor([b for b in range(len(lens)) if lens[b] > t], dtype=torch.long, device=v.device)
        if len(on):
            x = torch.tensor([cu[b] for b in on.tolist()], device=v.device) + t
            pw[slots[on], 1, :, t], pc[slots[on], 1, :, t] = w[x], csum[x]
    return {"out": o, "state": state, "pend_k": None, "pend_w": pw, "pend_c": pc, "pend": None}
