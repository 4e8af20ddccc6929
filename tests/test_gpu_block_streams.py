"""The block operators on a stream that is not the current one: the strided
token gate of moe_norm_out, and results that the current stream reads."""
import pytest
import torch

import dispatch_combine_gb300 as moe
from tests.gpu_common import ensure_lib

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _lib():
    ensure_lib()


@pytest.mark.parametrize("as_handle", [False, True])
def test_strided_token_gate_on_a_side_stream(as_handle):
    T, d = 4096, 1024
    f, x = (torch.randn(T, d, device="cuda").to(BF16) for _ in range(2))
    values = torch.rand(T, device="cuda").to(BF16)
    want = moe.moe_norm_out(f, x, gate=values, next_norm=True)
    wide = torch.zeros(T, 4, dtype=BF16, device="cuda")
    big = torch.randn(4096, 4096, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.current_stream().synchronize()
    for _ in range(4):
        with torch.cuda.stream(s):
            wide.zero_()
            for _ in range(8):               # the gate comes late on its stream
                big = big @ big * 1e-4
            wide[:, 1] = values
        got = moe.moe_norm_out(f, x, gate=wide[:, 1], next_norm=True,
                               stream=s.cuda_stream if as_handle else s)
        # what the current stream allocates meanwhile is not the gate's copy
        junk = [torch.full((T,), 7.0, dtype=BF16, device="cuda") for _ in range(8)]
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        del junk
