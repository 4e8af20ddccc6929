"""Numbers of the norms given as tensors or arrays of one element: a call takes
their value at the call, whatever the same object held at an earlier one."""
import ctypes

import numpy as np
import pytest
import torch

from dispatch_combine_gb300 import _lib


@pytest.fixture
def seen(monkeypatch):
    out = []

    def call(n, *args):
        d = ctypes.cast(n, ctypes.POINTER(_lib.MoeNorm)).contents
        out.append((d.T, d.d, d.kind, d.eps, d.weight_offset))
        return 0

    monkeypatch.setattr(_lib, "_rows", lambda t, *a: (t.data_ptr(), t.stride(0)))
    monkeypatch.setattr(_lib, "_fn", lambda name: call)
    monkeypatch.setattr(_lib, "_stream", lambda s: 0)
    return out


@pytest.mark.parametrize("number", [torch.tensor, lambda v: torch.nn.Parameter(torch.tensor(v), requires_grad=False),
                                    lambda v: np.array(v)])
def test_a_number_that_changes_in_place(seen, number):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    eps, off, kind = number(0.5), number(0.0), number(0)
    for e, o, k in ((0.5, 0.0, 0), (0.25, 1.0, 1), (0.125, -0.5, 0)):
        eps[...], off[...], kind[...] = e, o, k
        _lib.moe_norm_in(x, eps=eps, weight_offset=off, kind=kind)
        _lib.moe_norm_out(x, x, eps=eps, weight_offset=off, kind=kind)
        assert seen[-1] == seen[-2] == (4, 64, k, e, o)
