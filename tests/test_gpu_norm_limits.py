"""The norms at the largest number of rows."""
import pytest
import torch

import dispatch_combine_gb300 as moe
from tests.gpu_common import ensure_lib
from tests.test_gpu_norm import check, ref_norm

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib():
    ensure_lib()


@pytest.mark.parametrize("T", [2 ** 31 - 8, 2 ** 31 - 7, 2 ** 31 - 1])
def test_as_many_rows_as_int_holds(T):
    # 34 GB, normalised in place; rows of zeros stay zeros
    x = torch.zeros(T, 8, dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, 7, 8, 12345678, 2 ** 30 + 3, T - 8, T - 2, T - 1]
    x[rows] = torch.randn(len(rows), 8, device="cuda").to(torch.bfloat16)
    want = ref_norm(x[rows], None, None, moe.MOE_NORM_RMS)
    moe.moe_norm_in(x, out=x)
    check(x[rows], want)
    assert torch.count_nonzero(x[2:7]) == 0 and torch.count_nonzero(x[T - 7:T - 2]) == 0
