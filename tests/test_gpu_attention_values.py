"""moe_prefix_attention with values at the ends of their ranges: queries that
are not finite, scales and scores that fp32 can just hold, through each of the
kernels that can do the work."""
import math

import pytest
import torch

import dispatch_combine_gb300 as moe
from tests.gpu_common import ensure_lib
from tests.test_gpu_attention_tiles import LONG, long_case
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


def far_scores(name, D, dtype):
    """Queries of +-2^15 in one element (negative in every third head), keys that
    there hold distinct numbers of eight bits from 128 to 2^15: products of two
    such are exact in fp32 and 2^15 or more apart."""
    c = route(name, D, dtype)
    numbers = (torch.randperm(1024, generator=c.g, device="cuda") + 0x4300).to(torch.int16)
    numbers = numbers.view(BF16).to(dtype)
    c.q.zero_()
    c.q[..., 3] = 2.0 ** 15
    c.q[:, ::3, 3] = -2.0 ** 15
    for at, pages, n in [(0, c.prefix_pages, c.prefix)] + [(c.prefix, c.table[b], m)
                                                          for b, m in enumerate(c.lens_list)]:
        for i in range(-(-n // c.page)):
            m = min(c.page, n - i * c.page)
            c.k[pages[i].long(), :, :m, 3] = numbers[at + i * c.page:at + i * c.page + m]
    return c


@pytest.mark.parametrize("name", ROUTES)
@pytest.mark.parametrize("D,dtype", FORMS)
def test_scores_far_from_zero(name, D, dtype):
    """The largest scores that a type holds, and some 2^9 times smaller ones: 2^8
    or more apart, so the best key's probability is 1 to all bits.  The result is
    that key's value, off by the rounding of its probability to the type (2 to a
    broken power, since the offset is rounded) and by its own.  The log-sum-exp is
    the score after at most eight roundings of half a step of fp32 (log2 e and
    ln 2, the products with them and with the scale, the offset taken off and the
    logarithm of the sum)."""
    half = torch.finfo(dtype).eps / 2
    c = far_scores(name, D, dtype)
    for scale in (2.0 ** -7, 2.0 ** -7 if dtype is FP16 else 0.5):
        o, lse = c.run(scale=scale)
        ro, ra, rl = c.reference(scale)
        assert ((o.double() - ro).abs() <= half * ro.abs() + (half + 2e-4) * 1.01 * ra).all()
        assert ((lse.double() - rl).abs() <= 2.0 ** -21 * rl.abs()).all()
        assert moe.moe_get_device_status(c.ws) == 0


@pytest.mark.parametrize("name", ROUTES)
@pytest.mark.parametrize("D,dtype", FORMS)
@pytest.mark.parametrize("scale", [4.0, 16.0, 2.0 ** 64, 2.0 ** 127])
def test_scores_past_the_range_give_nan(name, D, dtype, scale):
    c = far_scores(name, D, dtype)
    o, lse = c.run(scale=scale)
    best = (c.reference(1.0)[2] > 2.0 ** 28)    # of a positive query: its largest score
    assert best.any() and torch.isnan(o[best]).all() and torch.isnan(lse[best]).all()


@pytest.mark.parametrize("D,dtype", FORMS)
@pytest.mark.parametrize("G,T,n", [(4, 2, 256), (64, 3, 512)])      # few rows; two times 128
def test_large_scores_that_rise_a_little(D, dtype, G, T, n):
    """Scores of 2^22, and 6 more for the last key, exact in fp32: the sum over the
    others is rescaled and stays over a third of the whole.  What it is rescaled by
    must fit what the exponentials were taken of, whose offset is rounded to 1/2.
    With a key head for every worker each row is one part (a part's log-sum-exp is
    rounded to 1/2 too).  Probabilities are then good to the exponentials' 2^-21
    and the halving of their rounding to the type."""
    workers = torch.cuda.get_device_properties(0).multi_processor_count * (8 if G == 4 else 1)
    c = Case([1] * T, [0] * T, n, hq=G * workers, hkv=workers, D=D, dtype=dtype)
    c.table = None
    c.q.zero_()
    c.q[..., 1], c.q[..., 2] = 2048.0, 1.0
    rows = torch.zeros(n, D, device="cuda")
    rows[:, 1], rows[-1, 2] = 2048.0, 6.0
    for at, pg in enumerate(c.prefix_pages.tolist()):
        c.k[pg] = rows[at * c.page:(at + 1) * c.page].to(dtype)
    o, lse = c.run(scale=1.0)
    v = c.v[c.prefix_pages.long()].transpose(0, 1).reshape(workers, n, D).double()
    p = torch.softmax((torch.arange(n, device="cuda") == n - 1) * 6.0, 0, dtype=torch.float64)
    ro, ra = (torch.einsum("k,hkd->hd", p, x).repeat_interleave(G, 0) for x in (v, v.abs()))
    half = torch.finfo(dtype).eps / 2
    assert ((o.double() - ro).abs() <= half * ro.abs() + (half + 2e-4) * 1.01 * ra).all()
    want = 2.0 ** 22 + math.log(n - 1 + math.exp(6.0))
    assert ((lse.double() - want).abs() <= 2.0 ** -21 * want).all()


@pytest.mark.parametrize("name", list(ROUTES) + list(LONG))
@pytest.mark.parametrize("D,dtype", FORMS)
@pytest.mark.parametrize("scale", [2.0 ** -8, 4.0, 2.0 ** 60])
@pytest.mark.parametrize("where", ["first", "prefix"])
def test_keys_far_below_the_others_weigh_nothing(name, D, dtype, scale, where):
    # scores of -2^30 * scale for the first third of the keys, or all of the
    # prefix's; of the others' as usual
    c = route(name, D, dtype) if name in ROUTES else long_case(name, D, dtype)
    if where == "prefix" and (not c.prefix or min(c.lens_list) == 0):
        pytest.skip("no token sees other keys")
    c.q = (c.q.double() * (D ** -0.5 / scale)).to(torch.float32)
    c.q = c.q.clamp(-2.0, 2.0).to(dtype)
    c.q[..., 3] = 2.0 ** 15
    for i, (pages, n) in enumerate([(c.prefix_pages, c.prefix)] + list(zip(c.table, c.lens_list))):
        far = n // 3 if where == "first" else n if i == 0 else 0
        for j in range(-(-n // c.page)):
            m = min(c.page, n - j * c.page)
            low = (torch.arange(m, device="cuda") + j * c.page < far).to(dtype)
            c.k[pages[j].long(), :, :m, 3] = low * -2.0 ** 15
    c.check(got=c.run(scale=scale), scale=scale)
