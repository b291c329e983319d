"""Refusals of the calls for attention layers and the sampler: a status before anything is launched, and the binding's own checks (no GPU)."""
import ctypes

import pytest
import torch

import __graft_entry__ as entry
from speculative_state_replay_gb300 import _lib, api

AT = 1 << 20
P, ODD, NUL = ctypes.c_void_p(AT), ctypes.c_void_p(AT + 2), None


@pytest.fixture(scope="module")
def lib():
    entry.build()
    return _lib.load()


def cache(**kw):
    c = _lib.RssmKvCacheStruct()
    d = dict(num_pages=9, nlayers=2, nheads=2, head_dim=128, page_size=16, format=api.I8)
    page = 2 * 16 * 128
    for n in ("k", "v"):
        d |= {n: AT, n + "_layer_stride": 9 * page, n + "_page_stride": page, n + "_scale": AT, n + "_scale_layer_stride": 9 * 32,
              n + "_scale_page_stride": 32}
    d |= dict(error_word=AT) | kw
    for n, v in d.items():
        setattr(c, n, v)
    return ctypes.byref(c)


BAD = [dict(num_pages=0), dict(nlayers=0), dict(nheads=0), dict(page_size=0), dict(format=api.F32), dict(format=api.F16), dict(format=7),
       dict(k=0), dict(v=0), dict(k=AT + 8), dict(v=AT + 1), dict(k_scale=0), dict(v_scale=0), dict(v_scale=AT + 4), dict(error_word=0),
       dict(error_word=AT + 2), dict(k_page_stride=2 * 16 * 128 - 16), dict(v_page_stride=2 * 16 * 128 + 8), dict(k_layer_stride=100),
       dict(v_layer_stride=9 * 2 * 16 * 128 + 1), dict(k_scale_page_stride=31), dict(v_scale_page_stride=33), dict(k_scale_layer_stride=6)]
UNSUPPORTED = [dict(head_dim=96), dict(head_dim=512), dict(page_size=24), dict(page_size=1 << 17), dict(nheads=2048)]


def append(lib, c, layer=0, k=P, ks=256, v=P, vs=256, pages=P, ps=4, mp=4, ln=P, cu=NUL, batch=2, T=4, tokens=8):
    return lib.rssm_kv_append(c, layer, k, ks, v, vs, pages, ps, mp, ln, cu, batch, T, tokens, NUL)


def read(lib, c, layer=0, pages=P, ps=4, mp=4, starts=NUL, cu=P, batch=2, tokens=8, dt=api.BF16, k=P, ks=256, v=P, vs=256):
    return lib.rssm_kv_read(c, layer, pages, ps, mp, starts, cu, batch, tokens, dt, k, ks, v, vs, NUL)


def attend(lib, c, layer=0, q=P, qs=512, hq=4, scale=0.1, pages=P, ps=4, mp=4, ln=P, up=NUL, cu=NUL, batch=2, T=4, tokens=8, out=P, os=512,
           scratch=P, nbytes=1 << 30):
    return lib.rssm_tree_attention(c, layer, q, qs, hq, scale, pages, ps, mp, ln, up, cu, batch, T, tokens, out, os, scratch, nbytes, NUL)


def accept(lib, c, pages=P, ps=4, mp=4, ln=P, tok=P, up=NUL, drawn=P, cu=NUL, batch=2, T=4, ntok=8, acc=P, nxt=P, path=P, err=NUL):
    return lib.rssm_tree_accept(c, pages, ps, mp, ln, tok, up, drawn, cu, batch, T, ntok, acc, nxt, path, err, NUL)


def test_cache_refusals(lib):
    assert lib.rssm_attention_scratch_bytes(cache(), 4) > 0
    assert lib.rssm_attention_scratch_bytes(None, 4) == 0
    assert lib.rssm_attention_scratch_bytes(cache(), 0) == 0 and lib.rssm_attention_scratch_bytes(cache(), 3) == 0
    for kw, want in [(b, 1) for b in BAD] + [(u, 2) for u in UNSUPPORTED]:
        assert lib.rssm_attention_scratch_bytes(cache(**kw), 4) == 0, kw
        for call in (append, read, attend, accept):
            assert call(lib, cache(**kw)) == want, (call.__name__, kw)
    for call in (append, read, attend):
        assert call(lib, None) == 1 and call(lib, cache(), layer=2) == 1 and call(lib, cache(), layer=-1) == 1
    # a bf16 cache needs no scales, one layer no stride between layers
    bf = dict(format=api.BF16, k_scale=0, v_scale=0, k_scale_page_stride=0)
    assert append(lib, cache(**bf), batch=0) == 0 and append(lib, cache(nlayers=1, k_layer_stride=0, v_layer_stride=0), batch=0) == 0


def test_rows_refusals(lib):
    c = cache()
    for call in (append, read, attend, accept):
        n = "ntok" if call is accept else "tokens"
        assert call(lib, c, batch=-1) == 1 and call(lib, c, **{n: -1}) == 1 and call(lib, c, **{n: 1 << 31}) == 2 and call(lib, c, mp=-1) == 1
        assert call(lib, c, pages=NUL) == 1 and call(lib, c, pages=ODD) == 1 and call(lib, c, ps=3) == 1 and call(lib, c, cu=ODD) == 1
        assert call(lib, c, batch=1 << 25, cu=P) == 2 and call(lib, c, batch=0) == 0
    for call in (append, attend, accept):
        n = "ntok" if call is accept else "tokens"
        assert call(lib, c, T=0) == 1 and call(lib, c, **{n: 7}) == 1 and call(lib, c, ln=NUL) == 1 and call(lib, c, ln=ODD) == 1


def test_call_refusals(lib):
    c = cache()
    for kw in (dict(k=NUL), dict(v=NUL), dict(k=ODD), dict(ks=255), dict(ks=260), dict(vs=8), dict(v=ODD)):
        assert append(lib, c, **kw) == 1, kw
        assert read(lib, c, **kw) == 1, kw
    assert append(lib, c, tokens=0, batch=2, cu=P) == 0 and read(lib, c, tokens=0) == 0
    assert read(lib, c, cu=NUL) == 1 and read(lib, c, starts=ODD) == 1 and read(lib, c, dt=api.I8) == 1 and read(lib, c, dt=api.F32, ks=258) == 1
    for kw in (dict(q=NUL), dict(out=NUL), dict(q=ODD), dict(out=ODD), dict(qs=511), dict(qs=516), dict(os=511), dict(os=516), dict(hq=0), dict(hq=5),
               dict(up=ODD), dict(scratch=ODD), dict(scale=float("nan"))):
        assert attend(lib, c, **kw) == 1, kw
    assert attend(lib, c, up=P, T=65, tokens=130) == 2 and attend(lib, c, T=1 << 30, cu=P, tokens=1 << 30) == 2
    assert attend(lib, c, tokens=0, cu=P, q=NUL, out=NUL) == 0
    for kw in (dict(tok=NUL), dict(drawn=NUL), dict(tok=ODD), dict(up=ODD), dict(drawn=ODD), dict(acc=NUL), dict(nxt=NUL), dict(path=NUL), dict(acc=ODD),
               dict(nxt=ODD), dict(path=ODD), dict(err=ODD)):
        assert accept(lib, c, **kw) == 1, kw
        assert accept(lib, None, **kw) == 1, kw
    assert accept(lib, c, T=65, ntok=130) == 2 and accept(lib, None, T=65, ntok=130) == 2
    assert accept(lib, None, batch=0, pages=NUL, ln=NUL) == 0


def test_logits_refusals(lib):
    def logits(**kw):
        a = _lib.RssmLogitsArgs()
        d = dict(logits=AT, logits_stride=100, logits_dtype=api.BF16, out=AT, out_stride=100, out_dtype=api.F32, vocab=100, batch=2, T=4, probs=1, ntok=8)
        for n, v in (d | kw).items():
            setattr(a, n, v)
        return lib.rssm_logits(ctypes.byref(a), NUL)

    assert lib.rssm_logits(NUL, NUL) == 1
    for kw in (dict(batch=-1), dict(T=0), dict(vocab=0), dict(ntok=-1), dict(logits_dtype=api.I8), dict(out_dtype=9), dict(probs=2), dict(logits=AT + 1),
               dict(out=AT + 2), dict(logits=0), dict(out=0), dict(logits_stride=99), dict(out_stride=99), dict(ntok=7), dict(cu_seqlens=AT + 2),
               dict(temperature=AT + 1), dict(repetition=AT + 1), dict(presence=AT + 2), dict(frequency=AT + 2), dict(history=AT),
               dict(history=AT, history_len=AT, history_max=9, history_stride=8), dict(history=AT, history_len=AT, history_max=-1), dict(tokens=AT + 2),
               dict(parents=AT + 1), dict(bias_id=AT), dict(bias_id=AT, bias_start=AT), dict(bias_id=AT, bias_start=AT, bias_value=AT, biases=-1),
               dict(mask=AT, mask_stride=3), dict(mask=AT + 2, mask_stride=4), dict(error_word=AT + 2)):
        assert logits(**kw) == 1, kw
    assert logits(vocab=(1 << 18) + 1, logits_stride=1 << 19, out_stride=1 << 19) == 2 and logits(T=65, ntok=130) == 2
    assert logits(batch=1 << 24, T=64, cu_seqlens=AT) == 2 and logits(ntok=1 << 31) == 2
    assert logits(batch=0) == 0 and logits(ntok=0, cu_seqlens=AT, logits=0) == 0


def test_binding_checks():
    """Wrong types, shapes and devices are refused before the library is asked."""
    entry.build()
    bf, i32 = torch.bfloat16, torch.int32
    c = api.KVCache(4, 2, 64, 16, api.I8, layers=2, device="cpu")
    k, q = torch.zeros(6, 2, 64, dtype=bf), torch.zeros(6, 4, 64, dtype=bf)
    table, ln, cu = torch.zeros(2, 2, dtype=i32), torch.zeros(2, dtype=i32), torch.tensor([0, 3, 6], dtype=i32)
    ids, s = torch.zeros(6, dtype=i32), torch.zeros(64, dtype=torch.uint8)

    def refused(f, good, *bad):
        for b in bad:
            with pytest.raises(ValueError):
                f(**(good | b))
        with pytest.raises(ValueError):  # nothing of it is on a GPU
            f(**good)

    refused(lambda **a: api.rssm_kv_append(c, **a), dict(k=k, v=k, pages=table, lengths=ln, T=3),
            dict(k=k.float()), dict(k=k[:5]), dict(v=k[..., ::2]), dict(v=k.transpose(0, 1)), dict(pages=table[:1]), dict(pages=table.long()),
            dict(pages=table.t()), dict(lengths=ln.long()), dict(cu_seqlens=cu[:2]))
    refused(lambda **a: api.rssm_kv_read(c, **a), dict(pages=table, cu_seqlens=cu, k_out=k, v_out=k.clone()),
            dict(k_out=k.double()), dict(v_out=k.float()), dict(v_out=k[:5]), dict(starts=ln[:1]), dict(cu_seqlens=cu[:0]), dict(pages=table[0]))
    refused(lambda **a: api.rssm_tree_attention(c, **a), dict(q=q, pages=table, lengths=ln, T=3, out=q.clone(), scratch=s),
            dict(q=q.half()), dict(out=q[:, :3]), dict(out=q.float()), dict(parents=ids[:5]), dict(parents=ids.long()), dict(cu_seqlens=cu.long()),
            dict(scratch=s[::2]), dict(lengths=ln.float()))
    two, path = torch.zeros(2, dtype=i32), torch.zeros(2, 3, dtype=i32)
    refused(lambda **a: api.rssm_tree_accept(**a), dict(cache=c, pages=table, lengths=ln, tokens=ids, parents=None, drawn=ids, T=3, accepted=two, next_token=two,
                                                        path=path),
            dict(pages=None), dict(lengths=None), dict(tokens=ids.long()), dict(drawn=ids[:5]), dict(path=path[:1]), dict(path=path.t()), dict(next_token=two[:1]),
            dict(parents=ids[:3]), dict(cu_seqlens=two), dict(cache=None, error_word=torch.zeros(1, dtype=torch.int64)))
    x = torch.zeros(6, 50)
    h, hl = torch.zeros(2, 9, dtype=i32), two
    refused(lambda **a: api.rssm_logits(**a), dict(logits=x, T=3, out=x.clone()),
            dict(logits=x.double()), dict(out=x[:5]), dict(out=torch.zeros(50, 6).t()), dict(temperature=two), dict(repetition=x[0, :1]), dict(history=h),
            dict(history=h[:1], history_len=hl), dict(history=h.long(), history_len=hl), dict(history=h, history_len=hl[:1]), dict(tokens=ids[:5]),
            dict(parents=ids.long()), dict(bias_id=ids), dict(bias_id=ids, bias_start=two, bias_value=x[0]), dict(bias_id=ids, bias_start=cu, bias_value=x[0, :5]),
            dict(mask=torch.zeros(6, 1, dtype=i32)), dict(mask=torch.zeros(5, 2, dtype=i32)), dict(mask=torch.zeros(6, 2)), dict(cu_seqlens=cu[::2]),
            dict(error_word=torch.zeros(1, dtype=torch.int64)))
    for bad in (dict(format=api.F16), dict(k=torch.zeros(2, 4, 2, 16, 64)), dict(k_scale=torch.zeros(2, 4, 2, 15)), dict(v=torch.zeros(2, 4, 16, 2, 64, dtype=torch.int8).transpose(2, 3)),
                dict(format=api.BF16, k_scale=torch.zeros(2, 4, 2, 16)), dict(error_word=torch.zeros(1, dtype=torch.int64))):
        with pytest.raises(ValueError):
            api.KVCache(**(dict(num_pages=4, kv_heads=2, head_dim=64, page_size=16, format=api.I8, layers=2, device="cpu") | bad))


def test_fast_calls_are_the_abi_calls(lib):
    """The binding's C module makes the library's calls: the same statuses, and refuses what is no argument."""
    f, ref = _lib.fast_kv(), cache()
    struct = ref._obj
    at = ctypes.addressof(struct)
    a = [at, 0, AT, 256, AT, 256, AT, 4, 4, AT, None, 0, 4, 8, 0]
    r = [at, 0, AT, 4, 4, None, AT, 0, 8, api.BF16, AT, 256, AT, 256, 0]
    t = [at, 0, AT, 512, 4, 0.1, AT, 4, 4, AT, None, None, 0, 4, 8, AT, 512, AT, 1 << 30, 0]
    c = [at, AT, 4, 4, AT, AT, None, AT, None, 0, 4, 8, AT, AT, AT, None, 0]
    g = [AT, 100, 1, AT, 100, 0, 100, 0, 4, 1, 8] + [None] * 6 + [0, 0] + [None] * 7 + [0, None, 0, None, 0]
    for fn, args, i, v, want in ((f.rssm_kv_append, a, 11, -1, 1), (f.rssm_kv_read, r, 9, 3, 1), (f.rssm_tree_attention, t, 4, 3, 1),
                                 (f.rssm_tree_accept, c, 10, 65, 2), (f.rssm_logits, g, 8, 65, 2)):
        assert fn(*args) == 0  # an empty batch
        bad = list(args)
        bad[i] = v
        assert fn(*bad) == want
        for wrong in (args[:-1], ["x"] + args[1:], args[:i] + [1 << 40] + args[i + 1 :]):
            with pytest.raises((TypeError, OverflowError)):
                fn(*wrong)


def test_scratch_follows_the_cache(lib):
    """Scratch does not depend on the batch; a call with less is refused."""
    c = api.KVCache(4, 2, 64, 16, api.E4M3, device="cpu")
    n = api.rssm_attention_scratch_bytes(c, 8)
    assert api.alloc_attention_scratch(c, 8).numel() == n > 4096
    with pytest.raises(api.RssmError):
        api.alloc_attention_scratch(c, 7)
