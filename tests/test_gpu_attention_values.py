"""moe_prefix_attention with values at the ends of their ranges: queries that
are not finite, scales and scores that fp32 can just hold, through each of the
kernels that can do the work."""
import math

import pytest
import torch

import dispatch_combine_gb300 as moe
from tests.gpu_common import ensure_lib
from tests.test_gpu_prefix_attention import BF16, FP16, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib():
    ensure_lib()


# (new tokens, own rows, prefix, query heads, key heads): few rows go to one
# kernel, many to the other, which takes 128 rows of a unit at a time or two
# times 128
ROUTES = {
    "rows": ([1, 2], [40, 317], 500, 4, 2),
    "rows beside tiles": ([1] * 40, [1 + 9 * b for b in range(40)], 300, 16, 2),
    "narrow tiles": ([10, 3], [333, 30], 0, 8, 1),
    "wide tiles": ([40, 1], [300, 9], 600, 16, 2),
}
FORMS = [(D, dtype) for D in (64, 128) for dtype in (BF16, FP16)]


def route(name, D, dtype, **kw):
    qs, lens, prefix, hq, hkv = ROUTES[name]
    return Case(qs, lens, prefix, hq=hq, hkv=hkv, D=D, dtype=dtype, **kw)


@pytest.mark.parametrize("name", ROUTES)
@pytest.mark.parametrize("D,dtype", FORMS)
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_a_query_that_is_not_finite_gives_nan(name, D, dtype, value):
    c = route(name, D, dtype)
    c.k[..., 5] = c.k[..., 5].abs()       # an infinite element here: every score is infinite
    ro, ra, rl = c.reference()
    t, h = c.T - 1, c.hq - 1
    bad = c.q.clone()
    bad[t, h, 5] = value
    bad[0, 1, 9] = value                  # here: of either sign
    o, lse = c.run(q=bad)
    rows = torch.zeros(c.T, c.hq, dtype=torch.bool, device="cuda")
    rows[t, h] = rows[0, 1] = True
    assert torch.isnan(o[rows]).all() and torch.isnan(lse[rows]).all()
    # the others are as right as ever
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    bound = half * ro.abs() + (half + 2e-4) * 1.01 * ra + tiny
    assert ((o.double() - ro).abs() <= bound)[~rows].all()
    assert ((lse.double() - rl).abs() <= 1e-4 + 2.0 ** -23 * rl.abs())[~rows].all()
    assert moe.moe_get_device_status(c.ws) == 0


@pytest.mark.parametrize("name", ROUTES)
@pytest.mark.parametrize("D,dtype", FORMS)
@pytest.mark.parametrize("scale", [1e-44, 1e-38, 2e-36, 1e-20])
def test_scales_near_the_smallest(name, D, dtype, scale):
    # every score is as good as zero: the mean of the values, the log of their number
    c = route(name, D, dtype)
    c.check(got=c.run(scale=scale), scale=scale)
