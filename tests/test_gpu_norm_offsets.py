"""A norm without a weight is not scaled, whatever the weight offset is."""
import pytest
import torch

import dispatch_combine_gb300 as moe
from tests.gpu_common import ensure_lib
from tests.test_gpu_norm import check, rand, ref_norm

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib():
    ensure_lib()


@pytest.mark.parametrize("T,d", [(5, 256), (3, 1032)])
@pytest.mark.parametrize("kind", [moe.MOE_NORM_RMS, moe.MOE_NORM_LAYER])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_no_weight_with_an_offset(T, d, kind, dtype):
    x, f, w = (rand(T, d, dtype=dtype, seed=1), rand(T, d, dtype=dtype, seed=2),
               rand(d, dtype=dtype, seed=3, std=0.2))
    b = rand(d, dtype=dtype, seed=4)
    for off in (1.0, -0.75):
        assert torch.equal(moe.moe_norm_in(x, None, b, kind=kind, weight_offset=off),
                           moe.moe_norm_in(x, None, b, kind=kind))
        check(moe.moe_norm_in(x, None, b, kind=kind, weight_offset=off), ref_norm(x, None, b, kind))
        # one of two weights given: the offset is added to that one alone
        for post, nxt in ((w, None), (None, w)):
            _, got = moe.moe_norm_out(f, x, post, post_norm=True, next_weight=nxt, next_norm=True,
                                      kind=kind, weight_offset=off)
            r = x.double() + ref_norm(f, post, None, kind, off)
            check(got, ref_norm(r, nxt, None, kind, off))
