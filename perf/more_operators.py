"""Workloads of a hybrid model's attention layers and of its sampler: what is
timed, the inputs, and the operators' plain forms.

Five operators that a serving loop runs next to the state updates when some of
the model's layers are attention:

  append    writes the keys and values of new tokens into a paged cache, as they
            are or in 8 bits with a scale for each token and head
  read      reads tokens back out of the cache, as the values they stand for
  attend    attention of a row's new tokens -- one token, a chain or a tree of
            drafts, a part of a prompt -- over the row's cached tokens
  accept    walks a tree of drafts along the target's draws and moves the
            accepted tokens' cache entries into place, in all layers
  logits    penalties for repeated tokens, biases, grammar masks and temperature
            on logits, and the probabilities that the verification takes

`run` computes them in plain torch operations in 32 bits (`own` false) or by
the library's calls (`own` true); both work on the same inputs and leave the
same buffers updated.
"""
import math
import random

import torch

own = False

QMAX = {"i8": 127.0, "e4m3": 448.0}
CODES = {"bf16": torch.bfloat16, "i8": torch.int8, "e4m3": torch.uint8}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "i8": 1, "e4m3": 1}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
LAYERS = 4  # attention layers of the hybrid model whose caches an acceptance moves


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # the decode batch's new tokens (64 rows of 4), into an 8-bit cache
        dict(name="append 64 rows", op="append", batch=64, T=4, ragged=False, context=4096, hkv=8, d=128, page=64, fmt="e4m3", lens=1),
        # sixteen prompts of very different lengths written at once
        dict(name="append prompts", op="append", batch=16, T=16384, ragged=True, tokens=16411, context=0, hkv=8, d=128, page=64, fmt="i8", lens=2),
        # one row's short context, for a prompt that goes on
        dict(name="read one row", op="read", batch=1, context=301, hkv=8, d=128, page=16, fmt="bf16", lens=3),
        # sixteen rows' contexts out of an 8-bit cache
        dict(name="read 16 rows", op="read", batch=16, context=8192, hkv=8, d=128, page=64, fmt="e4m3", lens=4),
        # a chat's next token
        dict(name="attend one token", op="attend", batch=1, T=1, ragged=False, tree=False, context=500, hq=32, hkv=8, d=128, page=16, fmt="bf16", lens=5),
        # the decode batch with four tokens a row, contexts of very different lengths, 8-bit cache
        dict(name="attend 64 rows", op="attend", batch=64, T=4, ragged=False, tree=False, context=16384, hq=32, hkv=8, d=128, page=64, fmt="e4m3", lens=6),
        # trees of up to 48 drafted tokens
        dict(name="attend trees", op="attend", batch=16, T=48, ragged=True, tree=True, context=16384, hq=32, hkv=8, d=128, page=64, fmt="i8", lens=7),
        # the second half of a prompt of 8192
        dict(name="attend prompt", op="attend", batch=1, T=4096, ragged=False, tree=False, context=4096, hq=32, hkv=8, d=128, page=64, fmt="bf16", lens=8),
        # one tree of eight tokens
        dict(name="accept one", op="accept", batch=1, T=8, ragged=False, context=1000, hkv=8, d=128, page=16, fmt="bf16", lens=9),
        # a batch's trees of up to 48 tokens
        dict(name="accept 64 rows", op="accept", batch=64, T=48, ragged=True, context=4096, hkv=8, d=128, page=64, fmt="bf16", lens=10),
        # one row of four tokens
        dict(name="logits one", op="logits", batch=1, T=4, ragged=False, tree=False, vocab=32768, history=200, bias=8, mask=True, dtype="bf16", probs="f32", lens=11),
        # the decode batch at seven tokens a row, long histories, an odd vocabulary
        dict(name="logits 64 rows", op="logits", batch=64, T=7, ragged=True, tree=True, vocab=131073, history=8192, bias=100, mask=True, dtype="bf16", probs="bf16", lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "accept", "logits"])
    seed = rng.randrange(1 << 30)
    if op == "logits":
        vocab = _log(rng, 1000, 200000)
        batch = _log(rng, 1, 64)
        T = rng.randint(1, max(1, min(32, 50_000_000 // (vocab * batch))))
        return dict(op=op, batch=batch, T=T, ragged=rng.random() < 0.5, tree=rng.random() < 0.5, vocab=vocab, history=_log(rng, 1, 8192),
                    bias=rng.choice([0, 1, 30, 300]), mask=rng.random() < 0.5, dtype=rng.choice(["f32", "bf16", "f16"]),
                    probs=rng.choice(["f32", "bf16", "f16"]), lens=seed)
    hkv, d, page = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256]), rng.choice([16, 32, 48, 64, 128])
    fmt = rng.choice(["bf16", "i8", "e4m3"])
    if op == "append":
        tokens = _log(rng, 1, 16384)
        batch = min(tokens, rng.choice([1, 2, 7, 33, 64]))
        return dict(op=op, batch=batch, T=tokens, ragged=True, tokens=tokens, context=rng.choice([0, 1000]), hkv=hkv, d=d, page=page, fmt=fmt, lens=seed)
    if op == "read":
        batch = _log(rng, 1, 64)
        return dict(op=op, batch=batch, context=_log(rng, 1, min(32768, 131072 // batch)), hkv=hkv, d=d, page=page, fmt=fmt, lens=seed)
    if op == "accept":
        return dict(op=op, batch=_log(rng, 1, 64), T=rng.randint(1, 64), ragged=rng.random() < 0.5, context=_log(rng, 1, 2048), hkv=hkv, d=d, page=page,
                    fmt=fmt, lens=seed)
    hq = hkv * rng.choice([1, 4, 7, 8])
    kind = rng.choice(["token", "chain", "tree", "prompt"])
    if kind == "prompt":
        batch, T = rng.choice([1, 1, 3]), _log(rng, 65, 2048)
        return dict(op=op, batch=batch, T=T, ragged=batch > 1, tree=False, context=_log(rng, 1, 4096), hq=hq, hkv=hkv, d=d, page=page, fmt=fmt, lens=seed)
    T = {"token": 1, "chain": rng.randint(2, 8), "tree": rng.randint(4, 64)}[kind]
    batch = _log(rng, 1, 128 if kind != "tree" else 16)
    context = _log(rng, 1, max(2, min(65536, 500_000_000 // (batch * hkv * d * (1 + T * hq // hkv // 128)))))
    return dict(op=op, batch=batch, T=T, ragged=rng.random() < 0.5, tree=kind == "tree", context=context, hq=hq, hkv=hkv, d=d, page=page, fmt=fmt, lens=seed)


def _lengths(case):
    """New tokens of each row, and its cached ones before them: plain lists."""
    rng = random.Random(case["lens"])
    n = case["batch"]
    if case["op"] == "read":  # tokens read, and where they begin
        lens = [case["context"] if n == 1 else max(1, int(case["context"] * rng.random())) for _ in range(n)]
        return lens, [rng.randint(0, 40) for _ in range(n)]
    if case["op"] == "append" and case["ragged"]:  # prompts: a few long ones and many short ones
        left = case["tokens"] - n
        share = [rng.expovariate(1.0) ** 2 for _ in range(n)]
        lens = [1 + int(left * s / sum(share)) for s in share]
        lens[share.index(max(share))] += case["tokens"] - sum(lens)
    else:
        lens = [rng.randint(1, case["T"]) if case["ragged"] else case["T"] for _ in range(n)]
    context = case.get("context", 0)
    if n == 1:
        return lens, [context]
    return lens, [int(context * rng.random() ** 2) for _ in range(n)]  # many short contexts, a few long ones


def _offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _tree(case, lens):
    """Each new token's parent within its row: the first token is the root, later ones hang on one of the few before."""
    rng = random.Random(case["lens"] + 1)
    return [-1 if t == 0 else rng.randint(max(0, t - 9), t - 1) for n in lens for t in range(n)]


def _columns(case):
    """Pages of a row's table."""
    lens, context = _lengths(case)
    return max(-(-(a + b) // case["page"]) for a, b in zip(lens, context)) + 1


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _cache(s, case, gen, layers):
    """A cache that has been written by such a model, and each row's pages in no order."""
    dev, fmt = "cuda", case["fmt"]
    n, columns = case["batch"], _columns(case)
    lens, context = _lengths(case)
    need = [-(-(a + b) // case["page"]) for a, b in zip(lens, context)]
    total = sum(need) + 3
    order = torch.randperm(total, generator=gen, device=dev).int()
    at = torch.tensor(_offsets(need)[:-1], device=dev)[:, None] + torch.arange(columns, device=dev)
    used = torch.arange(columns, device=dev) < torch.tensor(need, device=dev)[:, None]
    s["pages"] = torch.where(used, order[torch.where(used, at, 0)], 0).contiguous()
    shape = (layers, total, case["hkv"], case["page"], case["d"])
    for name, spread in (("k", 1.0), ("v", 0.7)):
        if fmt == "bf16":
            s[name + "_cache"] = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16).mul_(spread)
            s[name + "_scale"] = None
        else:
            s[name + "_scale"] = spread * (2.0 + 1.5 * torch.rand(shape[:-1], generator=gen, device=dev)) / QMAX[fmt]
            if fmt == "i8":
                s[name + "_cache"] = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16).mul_(45.0).clamp_(-127.0, 127.0).round_().to(torch.int8)
            else:
                codes = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16).mul_(160.0).clamp_(-448.0, 448.0)
                s[name + "_cache"] = codes.to(torch.float8_e4m3fn).view(torch.uint8)
    if own:  # the handle that a program keeps
        from speculative_state_replay_gb300 import api

        s["cache"] = api.KVCache(total, case["hkv"], case["d"], case["page"], {"bf16": api.BF16, "i8": api.I8, "e4m3": api.E4M3}[fmt], layers=layers,
                                 device=dev, k=s["k_cache"], v=s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    rnd = lambda *shape: torch.randn(shape, generator=gen, device=dev)  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    s = dict(case=case)
    op = case["op"]
    lens, context = _lengths(case)
    n, ntok = len(lens), sum(lens)
    s["lens"], s["context"] = lens, context  # the scheduler knows them
    s["cu"] = ints(_offsets(lens))
    s["lengths"] = ints(context)
    if op != "logits":
        hkv, d = case["hkv"], case["d"]
        _cache(s, case, gen, LAYERS if op == "accept" else 1)
    if op in ("append", "attend"):
        # q, k and v are columns of one projection, as a layer has them
        hq = case.get("hq", hkv)
        qkv = torch.randn((ntok, (hq + 2 * hkv) * d), generator=gen, device=dev, dtype=torch.bfloat16)
        s["q"] = qkv[:, : hq * d].unflatten(1, (hq, d))
        s["k"] = qkv[:, hq * d : (hq + hkv) * d].unflatten(1, (hkv, d))
        s["v"] = qkv[:, (hq + hkv) * d :].unflatten(1, (hkv, d))
    if op == "attend":
        s["parents"] = ints(_tree(case, lens)) if case["tree"] else None
        s["out"] = torch.empty(ntok, hq, d, dtype=torch.bfloat16, device=dev)
    if op == "read":
        s["k_out"] = torch.empty(ntok, hkv, d, dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.empty_like(s["k_out"])
    if op == "accept":
        parents = _tree(case, lens)
        cu = _offsets(lens)
        s["parents"] = ints(parents)
        s["tokens"] = torch.randint(0, 30000, (ntok,), generator=gen, device=dev, dtype=torch.int32)
        # the target's draw after a token is mostly one of the drafts that hang on it
        rng = random.Random(case["lens"] * 7 + seed)
        drawn = s["tokens"].clone()
        pick = []
        for b, m in enumerate(lens):
            below = [[] for _ in range(m)]
            for t in range(1, m):
                below[parents[cu[b] + t]].append(cu[b] + t)
            pick += [rng.choice(x) if x and rng.random() < 0.85 else -1 for x in below]
        pick = torch.tensor(pick, device=dev)
        s["drawn"] = torch.where(pick >= 0, s["tokens"][pick.clamp(min=0)], 30000 + drawn).int()
        s["accepted"] = torch.empty(n, dtype=torch.int32, device=dev)
        s["next"] = torch.empty(n, dtype=torch.int32, device=dev)
        s["path"] = torch.empty(n, case["T"], dtype=torch.int32, device=dev)
    if op == "logits":
        V, H = case["vocab"], case["history"]
        s["logits"] = rnd(ntok, V).mul_(2.5).to(DTYPES[case["dtype"]])
        s["parents"] = ints(_tree(case, lens)) if case["tree"] else None
        # a text's tokens: a few are frequent
        zipf = lambda *shape: (V * torch.rand(shape, generator=gen, device=dev) ** 4).int().clamp(max=V - 1)  # noqa: E731
        s["tokens"] = zipf(ntok)
        s["history"] = zipf(n, H)
        rng = random.Random(case["lens"] + 2)
        s["history_len"] = ints([H if n == 1 else rng.randint(0, H) for _ in range(n)])
        s["prompt_len"] = (s["history_len"] * torch.rand(n, generator=gen, device=dev)).int()
        u = lambda lo, hi: lo + (hi - lo) * torch.rand(n, generator=gen, device=dev)  # noqa: E731
        s["repetition"], s["presence"], s["frequency"] = u(1.0, 1.3), u(0.0, 0.6), u(0.0, 0.3)
        s["temperature"] = u(0.4, 1.2)
        if case["bias"]:
            m = [rng.randint(0, case["bias"]) for _ in range(n)]
            s["bias_start"] = ints(_offsets(m))
            s["bias_id"] = torch.randint(0, V, (max(1, sum(m)),), generator=gen, device=dev, dtype=torch.int32)
            s["bias_value"] = rnd(max(1, sum(m)))
        else:
            s["bias_start"] = s["bias_id"] = s["bias_value"] = None
        s["mask"] = None
        if case["mask"]:  # a bit for each id of the vocabulary, 1: the grammar allows it
            words = -(-V // 32)
            r = lambda: torch.randint(0, 1 << 32, (ntok, words), generator=gen, device=dev)  # noqa: E731
            bits = r() | r()
            s["mask"] = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).int()
        s["out"] = torch.empty(ntok, V, dtype=DTYPES[case["probs"]], device=dev)
    if own:
        from speculative_state_replay_gb300 import api

        s["api"] = api
        if op == "attend":
            s["scratch"] = api.alloc_attention_scratch(s["cache"], case["hq"])
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _rows(s):
    """Row and place of every new token."""
    cu = s["cu"].long()
    lens = cu[1:] - cu[:-1]
    row = torch.repeat_interleave(torch.arange(len(lens), device=cu.device), lens, output_size=sum(s["lens"]))
    return row, torch.arange(len(row), device=cu.device) - cu[row]


def _place(s, row, pos):
    """Page and place in it of positions of rows."""
    page = s["case"]["page"]
    return s["pages"][row, pos // page].long(), pos % page


def _values(s, name, pages, at):
    """Cached values [.., heads, d] of layer 0 in fp32."""
    x = s[name + "_cache"][0][pages, :, at]
    if s["case"]["fmt"] == "bf16":
        return x.float()
    x = x.view(torch.float8_e4m3fn).float() if s["case"]["fmt"] == "e4m3" else x.float()
    return x * s[name + "_scale"][0][pages, :, at][..., None]


def _held(s, name):
    """A cache's buffer as the numbers that it holds."""
    x = s[name + "_cache"]
    return x.view(torch.float8_e4m3fn) if s["case"]["fmt"] == "e4m3" else x


def _cache_out(s):
    out = {name: _held(s, name) for name in ("k", "v")}
    if s["case"]["fmt"] != "bf16":
        out |= {"k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    return out


def _plain_append(s):
    fmt = s["case"]["fmt"]
    row, t = _rows(s)
    pages, at = _place(s, row, s["lengths"].long()[row] + t)
    for name in ("k", "v"):
        x = s[name].float()
        if fmt != "bf16":
            most = x.abs().amax(-1)
            scale = torch.where(most < 2.0**-100, 1.0, most / QMAX[fmt])
            x = x * (1.0 / scale)[..., None]
            s[name + "_scale"][0][pages, :, at] = scale
        if fmt == "i8":
            x = x.round().clamp(-127.0, 127.0).to(torch.int8)
        elif fmt == "e4m3":
            x = x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            x = s[name]
        s[name + "_cache"][0][pages, :, at] = x
    return _cache_out(s)


def _plain_read(s):
    row, t = _rows(s)
    pages, at = _place(s, row, s["lengths"].long()[row] + t)
    s["k_out"].copy_(_values(s, "k", pages, at))
    s["v_out"].copy_(_values(s, "v", pages, at))
    return {"k": s["k_out"], "v": s["v_out"]}


def _ancestors(parents, row, t, n, T):
    """[row, t, j]: whether token j is on the path from the root to t, itself included."""
    below = torch.eye(T, device=parents.device).repeat(n, 1, 1)
    p = parents.long()
    below[row, t, p.clamp(min=0)] += (p >= 0).float()
    for _ in range(max(1, (T - 1).bit_length())):
        below = (below @ below).clamp(max=1.0)
    return below > 0


def _plain_attend(s):
    case = s["case"]
    n, hq, hkv, d = case["batch"], case["hq"], case["hkv"], case["d"]
    T, S = max(s["lens"]), max(a + b for a, b in zip(s["lens"], s["context"]))
    row, t = _rows(s)
    dev = row.device
    lengths = s["lengths"].long()
    pos = torch.arange(S, device=dev)
    live = pos < (lengths + (s["cu"][1:] - s["cu"][:-1]))[:, None]
    pages, at = _place(s, torch.arange(n, device=dev)[:, None], torch.where(live, pos, 0))
    q = torch.zeros(n, T, hq, d, device=dev)
    q[row, t] = s["q"].float()
    q = q.unflatten(2, (hkv, -1)).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)  # heads of a group, then tokens
    new = pos - lengths[:, None]  # [n, S]: which new token lies there
    if s["parents"] is None:
        seen = new[:, None, :] <= torch.arange(T, device=dev)[None, :, None]
    else:
        up = _ancestors(s["parents"], row, t, n, T)
        seen = up.gather(2, new.clamp(0, T - 1)[:, None, :].expand(-1, T, -1))
        seen = (new[:, None, :] < 0) | seen
    seen = (seen & live[:, None, :])[:, None, None]
    w = (q @ _values(s, "k", pages, at).permute(0, 2, 3, 1)).mul_(d**-0.5).unflatten(2, (-1, T))
    w = torch.where(seen, w, -math.inf)
    w = torch.exp_(w.sub_(w.amax(-1, keepdim=True).clamp(min=-1e30)))
    total = w.sum(-1, keepdim=True)
    v = torch.where(live[..., None, None], _values(s, "v", pages, at), 0.0)
    o = w.flatten(2, 3) @ v.transpose(1, 2)
    o = o.unflatten(2, (-1, T)) / torch.where(total > 0, total, 1.0)
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).flatten(2, 3)[row, t])
    return {"out": s["out"]}


def _plain_accept(s):
    case = s["case"]
    n, T = case["batch"], case["T"]
    row, t = _rows(s)
    dev = row.device
    parent = torch.full((n, T), -2, dtype=torch.long, device=dev)
    token, drawn = torch.full_like(parent, -1), torch.full_like(parent, -1)
    parent[row, t], token[row, t], drawn[row, t] = s["parents"].long(), s["tokens"].long(), s["drawn"].long()
    b = torch.arange(n, device=dev)
    path = torch.full((n, T), -1, dtype=torch.long, device=dev)
    cur = torch.where(torch.tensor([x > 0 for x in s["lens"]], device=dev), 0, -1)
    last = cur
    for j in range(T):  # a step down the trees
        path[:, j] = cur
        last = torch.where(cur >= 0, cur, last)
        hit = (parent == cur[:, None]) & (token == drawn[b, cur.clamp(min=0)][:, None]) & (cur >= 0)[:, None]
        cur = torch.where(hit.any(1), hit.int().argmax(1), -1)
    s["path"].copy_(path)
    s["accepted"].copy_((path >= 0).sum(1))
    s["next"].copy_(torch.where(last >= 0, drawn[b, last.clamp(min=0)], -1))
    # the accepted tokens' entries follow the committed ones
    on = path >= 0
    b, j = on.nonzero(as_tuple=True)
    at = s["lengths"].long()[b]
    (p0, a0), (p1, a1) = _place(s, b, at + path[b, j]), _place(s, b, at + j)
    for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
        if s[name] is not None:
            s[name][:, p1, :, a1] = s[name][:, p0, :, a0]
    return {"accepted": s["accepted"], "next": s["next"], "path": s["path"]} | _cache_out(s)


def _plain_logits(s):
    case = s["case"]
    n, V, T = case["batch"], case["vocab"], max(s["lens"])
    row, t = _rows(s)
    dev = row.device
    x = s["logits"].float()
    # how often each id is in a row's text: the prompt's only count as seen
    H = torch.arange(case["history"], device=dev)
    live = H < s["history_len"][:, None]
    out = live & (H >= s["prompt_len"][:, None])
    ids = s["history"].long()
    seen = torch.zeros(n, V, device=dev).scatter_add_(1, ids, live.float())
    count = torch.zeros(n, V, device=dev).scatter_add_(1, ids, out.float())
    seen, count = seen[row], count[row]
    # the fed tokens up to each one count too
    fed = torch.zeros(n, T, dtype=torch.long, device=dev)
    fed[row, t] = s["tokens"].long()
    if s["parents"] is None:
        up = (torch.arange(T, device=dev) <= t[:, None]).float()
    else:
        up = _ancestors(s["parents"], row, t, n, T)[row, t].float()
    count.scatter_add_(1, fed[row], up)
    seen = (seen + count) > 0
    r = s["repetition"][row][:, None]
    x = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
    x = torch.where(count > 0, x - (s["presence"][row][:, None] + s["frequency"][row][:, None] * count), x)
    if s["bias_id"] is not None:
        start = s["bias_start"].long()
        k = torch.arange(case["bias"], device=dev)
        on = k < (start[1:] - start[:-1])[:, None]
        e = torch.where(on, start[:-1, None] + k, 0)
        bias = torch.zeros(n, V, device=dev).scatter_add_(1, s["bias_id"].long()[e], torch.where(on, s["bias_value"][e], 0.0))
        x = x + bias[row]
    if s["mask"] is not None:
        bit = torch.arange(32, device=dev, dtype=torch.int32)
        allowed = ((s["mask"][:, :, None] >> bit) & 1).flatten(1)[:, :V]
        x = torch.where(allowed > 0, x, -math.inf)
    x = x / s["temperature"][row][:, None]
    x = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e30))
    total = x.sum(-1, keepdim=True)
    s["out"].copy_(x / torch.where(total > 0, total, 1.0))
    return {"out": s["out"]}


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"append": _plain_append, "read": _plain_read, "attend": _plain_attend, "accept": _plain_accept, "logits": _plain_logits}[op](s)
    api = s["api"]
    cu = s["cu"] if case.get("ragged", True) else None
    if op == "append":
        api.rssm_kv_append(s["cache"], s["k"], s["v"], s["pages"], s["lengths"], case["T"], cu_seqlens=cu)
        return _cache_out(s)
    if op == "read":
        api.rssm_kv_read(s["cache"], s["pages"], s["cu"], s["k_out"], s["v_out"], starts=s["lengths"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if op == "attend":
        api.rssm_tree_attention(s["cache"], s["q"], s["pages"], s["lengths"], case["T"], s["out"], s["scratch"], parents=s["parents"], cu_seqlens=cu)
        return {"out": s["out"]}
    if op == "accept":
        api.rssm_tree_accept(s["cache"], s["pages"], s["lengths"], s["tokens"], s["parents"], s["drawn"], case["T"], s["accepted"], s["next"], s["path"],
                             cu_seqlens=cu)
        return {"accepted": s["accepted"], "next": s["next"], "path": s["path"]} | _cache_out(s)
    api.rssm_logits(s["logits"], case["T"], s["out"], temperature=s["temperature"], repetition=s["repetition"], presence=s["presence"],
                    frequency=s["frequency"], history=s["history"], history_len=s["history_len"], prompt_len=s["prompt_len"], tokens=s["tokens"],
                    parents=s["parents"], bias_start=s["bias_start"], bias_id=s["bias_id"], bias_value=s["bias_value"], mask=s["mask"], cu_seqlens=cu)
    return {"out": s["out"]}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op = case["op"]
    lens, context = _lengths(case)
    ntok = sum(lens)
    if op == "logits":
        b = ntok * case["vocab"] * (BYTES[case["dtype"]] + BYTES[case["probs"]] + (0.125 if case["mask"] else 0.0))
        return {"bytes": b + 4 * case["batch"] * case["history"], "flops": 5 * ntok * case["vocab"]}
    hkv, d = case["hkv"], case["d"]
    held = 2 * hkv * (d * BYTES[case["fmt"]] + (0 if case["fmt"] == "bf16" else 4))  # a token's keys and values in the cache
    if op == "append":
        return {"bytes": ntok * (held + 4 * hkv * d), "flops": 4 * ntok * hkv * d}
    if op == "read":
        return {"bytes": ntok * (held + 4 * hkv * d), "flops": 2 * ntok * hkv * d}
    if op == "accept":  # a path's tokens, most of them moved: about twice the logarithm of the tree
        moved = sum(min(m - 1, 2 * math.log2(m)) for m in lens)
        return {"bytes": 16 * ntok + 4 * case["batch"] * case["T"] + LAYERS * 2 * moved * held, "flops": ntok}
    hq = case["hq"]
    if case["tree"]:
        parents, cu = _tree(case, lens), _offsets(lens)
        depth = []
        for b, m in enumerate(lens):
            for t in range(m):
                p = parents[cu[b] + t]
                depth.append(1 + (depth[cu[b] + p] if p >= 0 else 0))
        pairs = sum(m * c for m, c in zip(lens, context)) + sum(depth)
    else:
        pairs = sum(m * c + m * (m + 1) // 2 for m, c in zip(lens, context))
    return {"bytes": sum(m + c for m, c in zip(lens, context)) * held + 4 * ntok * hq * d, "flops": 4 * d * hq * pairs}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    lens, context = s["lens"], s["context"]
    cu = _offsets(lens)
    f = lambda x: x.double()  # noqa: E731
    fmt, page = case.get("fmt"), case.get("page")

    def cached(name, b, first, count):
        """Tokens first .. of row b in layer 0: [count, heads, d]."""
        at = torch.arange(first, first + count, device="cuda")
        pg = s["pages"][b].long()[at // page]
        x = s[name + "_cache"][0].transpose(1, 2)[pg, at % page]
        if fmt == "bf16":
            return f(x)
        x = f(x.view(torch.float8_e4m3fn).float()) if fmt == "e4m3" else f(x)
        return x * f(s[name + "_scale"][0].transpose(1, 2)[pg, at % page])[..., None]

    def path(b, t):
        """The new tokens of row b that t comes after, itself included."""
        if s["parents"] is None:
            return list(range(t + 1))
        up = [t]
        while parents[cu[b] + up[-1]] >= 0:
            up.append(parents[cu[b] + up[-1]])
        return up

    parents = s["parents"].tolist() if s.get("parents") is not None else None
    if op == "append":
        out = {"k": None, "v": None}  # kept as they are, or rounded onto a grid whose borders 64 bits do not share
        if fmt != "bf16":
            for name in ("k", "v"):
                scale = f(s[name + "_scale"])
                for b in range(len(lens)):
                    at = torch.arange(context[b], context[b] + lens[b], device="cuda")
                    x = f(s[name][cu[b] : cu[b + 1]])
                    scale[0].transpose(1, 2)[s["pages"][b].long()[at // page], at % page] = x.abs().amax(-1) / QMAX[fmt]
                out[name + "_scale"] = scale
        return out
    if op == "read":
        return {name: torch.cat([cached(name, b, context[b], lens[b]) for b in range(len(lens))]) for name in ("k", "v")}
    if op == "accept":
        return None  # whole numbers, and entries moved as they are
    if op == "attend":
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        out = torch.empty(cu[-1], hq, d, dtype=torch.float64, device="cuda")
        for b, m in enumerate(lens):
            S = context[b] + m
            k, v = cached("k", b, 0, S), cached("v", b, 0, S)
            hide = torch.ones(m, S, dtype=torch.bool, device="cuda")
            if parents is None:
                hide = torch.arange(S, device="cuda") > context[b] + torch.arange(m, device="cuda")[:, None]
            else:
                hide[:, : context[b]] = False
                for t in range(m):
                    hide[t, context[b] + torch.tensor(path(b, t), device="cuda")] = False
            for h in range(hkv):
                for g in range(hq // hkv):
                    i = h * (hq // hkv) + g
                    w = (f(s["q"][cu[b] : cu[b + 1], i]) @ k[:, h].T / math.sqrt(d)).masked_fill(hide, -math.inf)
                    out[cu[b] : cu[b + 1], i] = torch.softmax(w, -1) @ v[:, h]
        return {"out": out}
    V = case["vocab"]
    out = torch.empty(cu[-1], V, dtype=torch.float64, device="cuda")
    hist, hlen, plen, tokens = s["history"].long(), s["history_len"].tolist(), s["prompt_len"].tolist(), s["tokens"].long()
    for b, m in enumerate(lens):
        for t in range(m):
            x = f(s["logits"][cu[b] + t])
            fed = tokens[torch.tensor(path(b, t), device="cuda") + cu[b]]
            count = torch.bincount(torch.cat([hist[b, plen[b] : hlen[b]], fed]), minlength=V)
            seen = (torch.bincount(hist[b, : plen[b]], minlength=V) + count) > 0
            r = f(s["repetition"][b])
            x = torch.where(seen, torch.minimum(x * r, x / r), x)  # r >= 1
            x = x - f(s["presence"][b]) * (count > 0) - f(s["frequency"][b]) * count
            if s["bias_id"] is not None:
                e = slice(int(s["bias_start"][b]), int(s["bias_start"][b + 1]))
                x.index_add_(0, s["bias_id"][e].long(), f(s["bias_value"][e]))
            if s["mask"] is not None:
                i = torch.arange(V, device="cuda")
                x[(s["mask"][cu[b] + t].long()[i // 32] >> (i % 32)) & 1 == 0] = -math.inf
            out[cu[b] + t] = torch.softmax(x / f(s["temperature"][b]), -1)
    return {"out": out}
