"""Argument checks of the operators around the layer (norms, cache append,
shared-prefix attention): answered on the host, before anything is launched,
so no GPU is needed."""
import ctypes

import pytest
import torch

import dispatch_combine_gb300 as moe
from dispatch_combine_gb300 import _lib
from dispatch_combine_gb300 import build as build_mod

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = ctypes.c_void_p(4096)   # never dereferenced: every call below is refused
P2 = ctypes.c_void_p(8192)
P3 = ctypes.c_void_p(12288)
ODD = ctypes.c_void_p(4096 + 2)


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return _lib.lib()


def norm(**kw):
    base = dict(T=4, d=64, kind=0, dtype=0, eps=1e-6, weight_offset=0.0)
    base.update(kw)
    return _lib.MoeNorm(**base)


def norm_in(lib, n, x=P, xs=64, w=P3, b=None, out=P2, os_=64):
    return lib.moe_norm_in(ctypes.byref(n) if n is not None else None, x, xs, w, b, out, os_, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(d=0), dict(d=12), dict(d=16392), dict(kind=2), dict(dtype=2), dict(dtype=-1),
    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(weight_offset=float("nan")),
])
def test_norm_descriptor_refused(lib, bad):
    assert norm_in(lib, norm(**bad)) == INVALID


def test_norm_in_arguments(lib):
    assert norm_in(lib, None) == INVALID
    assert norm_in(lib, norm(T=0), x=None, out=None) == OK
    assert norm_in(lib, norm(), x=None) == INVALID
    assert norm_in(lib, norm(), out=None) == INVALID
    assert norm_in(lib, norm(), x=ODD) == INVALID
    assert norm_in(lib, norm(), w=ODD) == INVALID
    assert norm_in(lib, norm(), b=ODD) == INVALID
    assert norm_in(lib, norm(), xs=56) == INVALID       # rows overlap
    assert norm_in(lib, norm(), xs=0) == INVALID
    assert norm_in(lib, norm(), os_=68) == INVALID      # rows not 16-byte aligned
    assert norm_in(lib, norm(), x=P, out=P, xs=64, os_=128) == INVALID


def norm_out(lib, n, f=P, fs=64, x=P2, xs=64, post=1, pw=P3, pb=None, gk=0, g=None, gs=0,
             scale=1.0, nw=P3, nb=None, xo=P2, xos=64, no=P, nos=64):
    return lib.moe_norm_out(ctypes.byref(n), f, fs, x, xs, post, pw, pb, gk, g, gs, scale, nw, nb,
                            xo, xos, no, nos, None)


@pytest.mark.parametrize("bad", [
    dict(f=None), dict(x=None), dict(xo=None), dict(f=ODD), dict(fs=32), dict(xs=60), dict(nos=8),
    dict(post=0),                       # a post weight without the post norm
    dict(no=None),                      # a next weight without the next norm
    dict(gk=4), dict(gk=-1), dict(gk=1), dict(g=P3), dict(gk=1, g=ODD),
    dict(gk=3, g=P3, gs=32), dict(gk=3, g=P3, gs=68),
    dict(scale=float("nan")), dict(scale=float("inf")),
    dict(xo=P), dict(no=P2, xo=P3), dict(xo=P3, no=P3),  # outputs over the other input, or each other
    dict(xos=128), dict(nos=128),       # in place with another stride
])
def test_norm_out_refused(lib, bad):
    assert norm_out(lib, norm(), **bad) == INVALID


def kv(**kw):
    base = dict(num_q_heads=8, num_kv_heads=2, head_dim=64, page_size=16, num_pages=10, dtype=0)
    base.update(kw)
    return _lib.MoeKv(**base)


def append(lib, k_, T=3, q=P, qs=512, k=P, ks=128, v=P, vs=128, pos=P, slots=P, freq=P, rot=64,
           style=0, kc=P, vc=P2, qo=P3, qos=512, ws=None, n=0):
    return lib.moe_kv_append(ctypes.byref(k_) if k_ is not None else None, T, q, qs, k, ks, v, vs,
                             pos, slots, freq, rot, style, kc, vc, qo, qos, ws, n, None)


KV_BAD = [
    (dict(num_q_heads=7), INVALID), (dict(num_q_heads=0), INVALID), (dict(num_kv_heads=0), INVALID),
    (dict(num_pages=-1), INVALID), (dict(dtype=5), INVALID), (dict(head_dim=96), UNSUPPORTED),
    (dict(head_dim=256), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=48), UNSUPPORTED), (dict(page_size=512), UNSUPPORTED),
    (dict(num_q_heads=258), UNSUPPORTED),
    (dict(num_pages=1 << 27, page_size=16), INVALID),            # 2^31 slots
    (dict(num_pages=1 << 26, page_size=16), INVALID),            # 2^31 rows with two heads
]


@pytest.mark.parametrize("bad,want", KV_BAD)
def test_kv_descriptor_refused(lib, bad, want):
    assert append(lib, kv(**bad), qs=1 << 20, qos=1 << 20) == want
    assert attend(lib, kv(**bad), qs=1 << 20, os_=1 << 20)[0] == want
    out = ctypes.c_size_t(0)
    assert lib.moe_prefix_attention_workspace_size(ctypes.byref(kv(**bad)), 3, 3, 1, 20,
                                                   ctypes.byref(out)) == want


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(rot=-16), dict(rot=80), dict(rot=24), dict(style=2), dict(k=None), dict(v=None),
    dict(slots=None), dict(kc=None), dict(vc=None), dict(vc=P), dict(kc=ODD), dict(q=None),
    dict(qo=None), dict(q=ODD), dict(qs=504), dict(ks=64), dict(vs=132), dict(pos=None),
    dict(freq=None), dict(q=P3, qs=1024),
])
def test_append_refused(lib, bad):
    assert append(lib, kv(), **bad) == INVALID


def test_append_workspace_and_empty(lib):
    assert append(lib, None) == INVALID
    assert append(lib, kv(), T=0, q=None, k=None, v=None, slots=None) == OK
    assert append(lib, kv(), ws=P, n=128) == WORKSPACE
    assert append(lib, kv(), ws=ctypes.c_void_p(4096 + 16), n=4096) == WORKSPACE


def attend(lib, k_, T=3, B=3, mq=1, q=P, qs=512, off=None, kc=P, vc=P2, pp=P, plen=20, pt=P,
           mp=4, lens=P, scale=0.125, o=P3, os_=512, lse=None, ws=P, n=None):
    need = ctypes.c_size_t(0)
    st = lib.moe_prefix_attention_workspace_size(
        ctypes.byref(k_) if k_ is not None else None, T, B, mq, plen, ctypes.byref(need))
    if n is None:
        n = 0                            # too small, so that a call that passes its checks stops there
    return lib.moe_prefix_attention(ctypes.byref(k_) if k_ is not None else None, T, B, mq, q, qs,
                                    off, kc, vc, pp, plen, pt, mp, lens, scale, o, os_, lse, ws, n,
                                    None), st, need.value


@pytest.mark.parametrize("bad,want", [
    (dict(T=-1), INVALID), (dict(B=-1), INVALID), (dict(mq=0), INVALID), (dict(plen=-1), INVALID),
    (dict(mp=-1), INVALID), (dict(mp=1 << 27), INVALID), (dict(q=None), INVALID),
    (dict(q=ODD), INVALID), (dict(qs=504), INVALID), (dict(o=None), INVALID), (dict(o=P), INVALID),
    (dict(os_=516), INVALID), (dict(kc=None), INVALID), (dict(vc=ODD), INVALID),
    (dict(pp=None), INVALID), (dict(pt=None), INVALID), (dict(lens=None), INVALID),
    (dict(B=4), INVALID),                # one token each, but T != num_seqs
    (dict(B=4097, T=4097), UNSUPPORTED), (dict(T=1 << 28, B=5, off=P), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID),
    (dict(), WORKSPACE), (dict(ws=None), WORKSPACE), (dict(ws=ODD, n=1 << 40), WORKSPACE),
])
def test_attention_refused(lib, bad, want):
    assert attend(lib, kv(), **bad)[0] == want


def test_attention_empty_and_workspace_size(lib):
    assert attend(lib, None)[0] == INVALID
    assert attend(lib, kv(), T=0, B=0, q=None, o=None, ws=None)[0] == OK
    sizes = []
    for T in (1, 64, 1024):
        st, got = attend(lib, kv(), T=T, B=1, off=P, mq=T)[1:]
        assert st == OK and got >= 256
        sizes.append(got)
    assert sizes == sorted(sizes)
    assert lib.moe_prefix_attention_workspace_size(ctypes.byref(kv()), 3, 3, 1, 20, None) == INVALID


def test_binding_refuses_on_the_host():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.moe_norm_in(x)                                   # not on a CUDA device
    with pytest.raises(TypeError):
        moe.moe_norm_in(x.float())
    with pytest.raises(ValueError):
        moe.moe_norm_in(x[0])
    with pytest.raises(ValueError):
        moe.moe_norm_out(x, x, gate=torch.zeros(5, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        moe.kv_struct(8, 2, 64, 16, 10, dtype=torch.float32)
    k_ = moe.kv_struct(8, 2, 64, 16, 10)
    q, k = torch.zeros(3, 8, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(10, 2, 16, 64, dtype=torch.bfloat16)
    i32 = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        moe.moe_kv_append(k_, q, k, k, i32, i32, None, cache, cache)
    with pytest.raises(ValueError):
        moe.moe_prefix_attention(k_, q[:, :4], cache, cache, i32, 0, None, i32, None)


def test_a_strided_token_gate_lives_until_the_call(monkeypatch):
    """Its dense copy must not be freed before the outputs are allocated: they
    could get its memory."""
    import weakref

    from dispatch_combine_gb300 import _lib

    seen = {}

    def dense(t, dtype, shape, name):
        if t is not None and name == "gate":
            assert t.is_contiguous()
            seen["gate"] = weakref.ref(t)
        return None if t is None else t.data_ptr()

    def call(*args):
        seen["alive"] = seen["gate"]() is not None
        return 0

    monkeypatch.setattr(_lib, "_dense", dense)
    monkeypatch.setattr(_lib, "_rows", lambda t, dtype, shape, name: (t.data_ptr(), t.stride(0)))
    monkeypatch.setattr(_lib, "_fn", lambda name: call)
    monkeypatch.setattr(_lib, "_stream", lambda s: 0)
    f = torch.zeros(32, 8, dtype=torch.bfloat16)
    _lib.moe_norm_out(f, f, gate=torch.zeros(32, 4, dtype=torch.bfloat16)[:, 1])
    assert seen["alive"]
