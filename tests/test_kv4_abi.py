"""Argument checks of the 4-bit cache's calls and of the drafts' verification:
answered on the host, before anything is launched, so no GPU is needed."""
import ctypes

import pytest
import torch

import dispatch_combine_gb300 as moe
from dispatch_combine_gb300 import _lib
from dispatch_combine_gb300 import build as build_mod
from tests.test_block_abi import KV_BAD, ODD, P, P2, P3, kv
from tests.test_block_streams import trace  # noqa: F401

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P4 = ctypes.c_void_p(16384)


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return _lib.lib()


def ref(k_):
    return ctypes.byref(k_) if k_ is not None else None


def append(lib, k_, T=3, q=P, qs=512, k=P, ks=128, v=P, vs=128, pos=P, slots=P, freq=P, rot=64, style=0, kc=P, vc=P2,
           qo=P3, qos=512, ws=None, n=0):
    return lib.moe_kv4_append(ref(k_), T, q, qs, k, ks, v, vs, pos, slots, freq, rot, style, kc, vc, qo, qos, ws, n, None)


def read(lib, k_, n=3, slots=P, kc=P, vc=P2, dst=None, pages=0, ko=P3, ks=128, vo=P4, vs=128, ws=None, nb=0):
    return lib.moe_kv4_read(ref(k_), n, slots, kc, vc, dst, pages, ko, ks, vo, vs, ws, nb, None)


def size(lib, k_, T=3, B=3, mq=1):
    out = ctypes.c_size_t(0)
    return lib.moe_kv4_attention_workspace_size(ref(k_), T, B, mq, ctypes.byref(out)), out.value


def attend(lib, k_, T=3, B=3, mq=1, q=P, qs=512, off=None, kc=P, vc=P2, pt=P, mp=4, lens=P, scale=0.125, o=P3, os_=512,
           lse=None, ws=P, n=0):
    return lib.moe_kv4_attention(ref(k_), T, B, mq, q, qs, off, kc, vc, pt, mp, lens, scale, o, os_, lse, ws, n, None)


def verify(lib, T=4, B=2, V=100, dtype=2, p=P, ps=100, q=P2, qs=100, tok=P, u=P, off=P, acc=P3, out=P4, ws=None, n=0):
    return lib.moe_verify_drafts(T, B, V, dtype, p, ps, q, qs, tok, u, off, acc, out, ws, n, None)


@pytest.mark.parametrize("bad,want", KV_BAD)
def test_kv_descriptor_refused(lib, bad, want):
    assert append(lib, kv(**bad), qs=1 << 20, qos=1 << 20) == want
    assert read(lib, kv(**bad), ks=1 << 20, vs=1 << 20) == want
    assert attend(lib, kv(**bad), qs=1 << 20, os_=1 << 20) == want
    assert size(lib, kv(**bad))[0] == want
    assert lib.moe_kv4_page_bytes(ctypes.byref(kv(**bad))) == 0


def test_page_bytes(lib):
    assert lib.moe_kv4_page_bytes(None) == 0
    for page in (16, 64, 256):
        for D in (64, 128):
            # half a byte an element, and two for each 32
            assert lib.moe_kv4_page_bytes(ctypes.byref(kv(page_size=page, head_dim=D))) == page * D * 9 // 16


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(rot=-16), dict(rot=80), dict(rot=24), dict(style=2), dict(k=None), dict(v=None), dict(slots=None),
    dict(kc=None), dict(vc=None), dict(vc=P), dict(kc=ODD), dict(q=None), dict(qo=None), dict(q=ODD), dict(qs=504),
    dict(ks=64), dict(vs=132), dict(pos=None), dict(freq=None), dict(q=P3, qs=1024), dict(slots=ctypes.c_void_p(4097)),
])
def test_append_refused(lib, bad):
    assert append(lib, kv(), **bad) == INVALID


def test_append_workspace_and_empty(lib):
    assert append(lib, None) == INVALID
    assert append(lib, kv(), T=0, q=None, k=None, v=None, slots=None) == OK
    assert append(lib, kv(), ws=P, n=128) == WORKSPACE
    assert append(lib, kv(), ws=ctypes.c_void_p(4096 + 16), n=4096) == WORKSPACE


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(slots=None), dict(slots=ctypes.c_void_p(4098)), dict(kc=None), dict(vc=None), dict(kc=ODD), dict(vc=ODD),
    dict(ko=None), dict(vo=None), dict(ko=ODD), dict(vo=P3), dict(ks=64), dict(vs=132), dict(vs=0),
    dict(dst=ODD, pages=3), dict(dst=P, pages=-1), dict(dst=P, pages=1 << 27), dict(dst=P, pages=3, ko=None),
    dict(dst=P, pages=3, vo=ODD),
])
def test_read_refused(lib, bad):
    assert read(lib, kv(), **bad) == INVALID


def test_read_workspace_and_empty(lib):
    assert read(lib, None) == INVALID
    assert read(lib, kv(), n=0, slots=None, ko=None, vo=None) == OK
    assert read(lib, kv(), ws=P, nb=128) == WORKSPACE
    assert read(lib, kv(), ws=ODD, nb=4096) == WORKSPACE


@pytest.mark.parametrize("bad,want", [
    (dict(T=-1), INVALID), (dict(B=-1), INVALID), (dict(mq=0), INVALID), (dict(mp=-1), INVALID), (dict(mp=1 << 27), INVALID),
    (dict(q=None), INVALID), (dict(q=ODD), INVALID), (dict(qs=504), INVALID), (dict(o=None), INVALID), (dict(o=P), INVALID),
    (dict(os_=516), INVALID), (dict(kc=None), INVALID), (dict(vc=ODD), INVALID), (dict(pt=None), INVALID),
    (dict(lens=None), INVALID), (dict(lens=ODD), INVALID), (dict(off=ODD), INVALID), (dict(lse=ODD), INVALID),
    (dict(B=4), INVALID),                # one token each, but T != num_seqs
    (dict(B=4097, T=4097), UNSUPPORTED), (dict(T=1 << 28, B=5, off=P), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(), WORKSPACE), (dict(ws=None), WORKSPACE), (dict(ws=ODD, n=1 << 40), WORKSPACE),
])
def test_attention_refused(lib, bad, want):
    assert attend(lib, kv(), **bad) == want


def test_attention_empty_and_workspace_size(lib):
    assert attend(lib, None) == INVALID
    assert attend(lib, kv(), T=0, B=0, q=None, o=None, ws=None) == OK
    assert lib.moe_kv4_attention_workspace_size(ctypes.byref(kv()), 3, 3, 1, None) == INVALID
    # no smaller call needs more
    for shape in (dict(), dict(num_q_heads=40), dict(num_q_heads=10, head_dim=128), dict(num_q_heads=14)):
        most, before = 0, None
        for mq in range(1, 45):
            got = [size(lib, kv(**shape), T, 7, mq) for T in (1, 5, 30, 44, 300)]
            assert all(st == OK for st, _ in got)
            row = [n for _, n in got]
            assert row == sorted(row) and row[0] >= 256
            if before:
                assert all(a <= b for a, b in zip(before, row))
            before = row
            most = max(most, row[-1])
        assert size(lib, kv(**shape), 300, 9, 300)[1] >= most


@pytest.mark.parametrize("bad,want", [
    (dict(T=-1), INVALID), (dict(B=-1), INVALID), (dict(V=0), INVALID), (dict(V=(1 << 30) + 1, ps=1 << 31, qs=1 << 31), INVALID),
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(p=None), INVALID), (dict(p=ODD), INVALID), (dict(q=ODD), INVALID),
    (dict(p=ctypes.c_void_p(4097), dtype=0), INVALID), (dict(ps=99), INVALID), (dict(qs=99), INVALID), (dict(tok=None), INVALID),
    (dict(tok=ODD), INVALID), (dict(u=None), INVALID), (dict(u=ODD), INVALID), (dict(off=None), INVALID), (dict(off=ODD), INVALID),
    (dict(acc=None), INVALID), (dict(acc=ODD), INVALID), (dict(out=None), INVALID), (dict(out=ODD), INVALID), (dict(out=P), INVALID),
    (dict(acc=P), INVALID), (dict(acc=P4), INVALID), (dict(B=(1 << 27) + 1), UNSUPPORTED), (dict(ws=P, n=100), WORKSPACE),
    (dict(ws=ODD, n=4096), WORKSPACE),
])
def test_verify_refused(lib, bad, want):
    assert verify(lib, **bad) == want


def test_verify_empty(lib):
    assert verify(lib, B=0, p=None, tok=None, u=None, off=None, acc=None, out=None) == OK


def test_binding_refuses_on_the_host():
    k_ = moe.kv_struct(8, 2, 64, 16, 10)
    q, k = torch.zeros(3, 8, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(10, 2, moe.moe_kv4_page_bytes(k_), dtype=torch.uint8)
    i32 = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        moe.moe_kv4_append(k_, q, k, k, i32, i32, None, cache, cache)         # not on a CUDA device
    with pytest.raises(ValueError):
        moe.moe_kv4_read(k_, i32, cache, cache, k_out=k, v_out=k)
    with pytest.raises(ValueError):
        moe.moe_kv4_read(k_, i32, cache, cache, dst_slots=i32)
    with pytest.raises(ValueError):
        moe.moe_kv4_attention(k_, q[:, :4], cache, cache, None, i32, None)
    with pytest.raises(moe.MoEError):
        moe.moe_kv4_page_bytes(moe.kv_struct(8, 2, 96, 16, 10))
    with pytest.raises(moe.MoEError):
        moe.moe_kv4_attention_workspace_size(k_, 3, 3, 0)
    p = torch.zeros(4, 10)
    with pytest.raises(TypeError):
        moe.moe_verify_drafts(p.double(), i32, p[0], i32)
    with pytest.raises(ValueError):
        moe.moe_verify_drafts(p[0], i32, p[0], i32)
    with pytest.raises(ValueError):
        moe.moe_verify_drafts(p, i32, p[0], i32)


def test_tensors_of_another_device_are_refused(monkeypatch):
    class Elsewhere:
        is_cuda = True

        def get_device(self):
            return 1

    monkeypatch.setattr(_lib, "_one_device", lambda: False)
    monkeypatch.setattr(_lib, "_current_device", lambda: 0)
    with pytest.raises(ValueError):
        _lib._here(None, torch.zeros(1), Elsewhere())
    monkeypatch.setattr(_lib, "_current_device", lambda: 1)
    _lib._here(None, torch.zeros(1), Elsewhere())


@pytest.mark.parametrize("name,allocations", [("append", 1), ("read", 2), ("attention", 2), ("verify", 2)])
def test_memory_of_a_call_belongs_to_its_stream(trace, name, allocations):  # noqa: F811
    k_ = _lib.kv_struct(4, 2, 64, 16, 4)
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    cache, i32, p = torch.zeros(4, 2, 576, dtype=torch.uint8), torch.zeros(3, dtype=torch.int32), torch.zeros(3, 10)

    class Space:
        ptr, nbytes = 0, 0

    for stream in (1234, None):
        run = {"append": lambda: _lib.moe_kv4_append(k_, q, k, k, i32, i32, None, cache, cache, stream=stream),
               "read": lambda: _lib.moe_kv4_read(k_, i32, cache, cache, stream=stream),
               "attention": lambda: _lib.moe_kv4_attention(k_, q, cache, cache, None, i32, Space(), want_lse=True,
                                                           stream=stream),
               "verify": lambda: _lib.moe_verify_drafts(p, i32, p[0], i32, stream=stream)}[name]
        del trace[:]
        run()
        where = "current" if stream is None else ("stream", 1234)
        kept = [] if stream is None else [("kept for", "current")] * allocations
        assert sorted(trace, key=str) == sorted([("empty", where)] * allocations + kept, key=str)
