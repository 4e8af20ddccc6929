"""Lengths at the end of int: refused on the host, where the kernels' key numbers
could not hold them."""
import ctypes

import pytest

from tests.test_block_abi import INVALID, OK, WORKSPACE, attend, kv, lib  # noqa: F401

MOST = 2 ** 31 - 1024


@pytest.mark.parametrize("prefix", [2 ** 31 - 1, 2 ** 31 - 15, 2 ** 31 - 128, MOST + 1])
def test_prefix_too_long(lib, prefix):  # noqa: F811
    got, size, _ = attend(lib, kv(), plen=prefix)
    assert got == INVALID and size == INVALID


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_table_too_wide(lib, page):  # noqa: F811
    most = MOST // page
    assert attend(lib, kv(page_size=page), mp=most + 1)[0] == INVALID
    assert attend(lib, kv(page_size=page), mp=2 ** 31 // page - 1)[0] == INVALID
    assert attend(lib, kv(page_size=page), mp=most)[0] == WORKSPACE      # passes its checks


def test_the_longest_are_taken(lib):  # noqa: F811
    got, size, need = attend(lib, kv(), plen=MOST)
    assert got == WORKSPACE and size == OK and 256 <= need < 1 << 32
