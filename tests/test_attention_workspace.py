"""The attention's workspace, sized once for the largest batch, serves every
smaller one: the size never falls as tokens, sequences, queries or the prefix
grow, whichever kernel would do the work.  Answered on the host."""
import ctypes

import pytest

from dispatch_combine_gb300 import _lib
from dispatch_combine_gb300 import build as build_mod


@pytest.fixture(scope="module")
def size():
    build_mod.build()
    lib = _lib.lib()

    def ask(kv, T, B, max_q, prefix):
        out = ctypes.c_size_t(0)
        assert lib.moe_prefix_attention_workspace_size(ctypes.byref(kv), T, B, max_q, prefix,
                                                       ctypes.byref(out)) == 0
        return out.value

    return ask


HEADS = [(hkv, G) for hkv in (1, 2, 8) for G in (1, 2, 3, 4, 7, 8, 16, 17, 31, 32, 33, 64, 100, 128)]


def heads(hkv, G, D=128):
    return _lib.kv_struct(hkv * G, hkv, D, 64, 1000)


def around(*values):
    return sorted({v + i for v in values for i in (-1, 0, 1) if v + i >= 1})


@pytest.mark.parametrize("hkv,G", HEADS)
def test_more_tokens_never_need_less(size, hkv, G):
    kv, tpt = heads(hkv, G), 128 // G
    Ts = around(1, 16 // G, 32 // G, 64 // G, tpt, 2 * tpt, 3 * tpt, 32 * tpt, 33 * tpt, 700, 5000)
    for B in (0, 1, 3, 300):
        for max_q in (1, 5, 5000):
            for prefix in (0, 8192):
                sizes = [size(kv, T, B, max_q, prefix) for T in Ts]
                assert sizes == sorted(sizes), (B, max_q, prefix)


@pytest.mark.parametrize("hkv,G", HEADS)
def test_more_queries_or_sequences_never_need_less(size, hkv, G):
    kv, tpt = heads(hkv, G), 128 // G
    qs = around(1, 16 // G, 32 // G, 64 // G, tpt, 2 * tpt, 4 * tpt, 1000)
    Bs = [0, 1, 2, 5, 64, 300, 4096]
    for T in (1, 7, 64, 333, 5000):
        for prefix in (0, 1, 8192):
            table = [[size(kv, T, B, q, prefix) for q in qs] for B in Bs]
            for row in table:
                assert row == sorted(row), (T, prefix)
            for column in zip(*table):
                assert list(column) == sorted(column), (T, prefix)


@pytest.mark.parametrize("hkv,G", HEADS)
def test_a_longer_prefix_never_needs_less(size, hkv, G):
    for T in (1, 4, 40, 700):
        sizes = [size(heads(hkv, G), T, 4, 3, p) for p in (0, 1, 100, 4096, 1 << 20)]
        assert sizes == sorted(sizes)


def test_a_server_that_drains(size):
    # 64 + 8 heads behind a prefix of 8192: sized for 8 sequences, used for fewer
    kv = heads(8, 8)
    sizes = [size(kv, T, T, 1, 8192) for T in range(1, 300)]
    assert sizes == sorted(sizes)
    # and queries for one kernel or the other
    assert size(kv, 64, 8, 8, 8192) <= size(kv, 64, 8, 9, 8192)
