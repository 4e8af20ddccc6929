"""Pointers to 32-bit and 16-bit values that are not aligned to them are refused
on the host: the kernels read them as such."""
import ctypes

import pytest

from tests.test_block_abi import INVALID, P, P3, append, attend, kv, lib, norm, norm_out  # noqa: F401

HALF = ctypes.c_void_p(4096 + 2)    # aligned to 16 bits only
BYTE = ctypes.c_void_p(4096 + 1)


@pytest.mark.parametrize("name", ["pos", "slots", "freq"])
@pytest.mark.parametrize("p", [HALF, BYTE])
def test_append(lib, name, p):  # noqa: F811
    assert append(lib, kv(), **{name: p}) == INVALID


@pytest.mark.parametrize("name", ["off", "pp", "pt", "lens", "lse"])
@pytest.mark.parametrize("p", [HALF, BYTE])
def test_attention(lib, name, p):  # noqa: F811
    assert attend(lib, kv(), **{name: p})[0] == INVALID


def test_token_gate(lib):  # noqa: F811
    assert norm_out(lib, norm(), gk=2, g=BYTE) == INVALID
