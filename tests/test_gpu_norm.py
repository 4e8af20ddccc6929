"""moe_norm_in and moe_norm_out against the formulas in 64 bits.

Bounds.  Each output is rounded once: half a step, finfo.eps / 2 relative
(plus half the smallest subnormal).  Before that everything is fp32: a row sum
of up to 16384 terms, each lane's part at most 64 additions and the tree 10
more, is good to 74 * 2^-24 < 5e-6 relative of the sum of magnitudes, which
moves a row's scale by half of that and, for the centred form, a value by 5e-6
of the row's mean magnitude (here below its root mean square); 1e-5 of the
row's largest result covers both norms of moe_norm_out in a row.
"""
import itertools

import pytest
import torch

import dispatch_combine_gb300 as moe
from tests.gpu_common import ensure_lib

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16
EPS = 1e-6


@pytest.fixture(autouse=True)
def _lib():
    ensure_lib()


def rand(*shape, dtype, seed, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


def ref_norm(v, w, b, kind, off=0.0, eps=EPS):
    v = v.double()
    if kind == moe.MOE_NORM_LAYER:
        v = v - v.mean(-1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    if w is not None:
        v = v * (w.double() + off)
    return v if b is None else v + b.double()


def check(got, ref):
    t = got.dtype
    row = ref.abs().amax(-1, keepdim=True)
    tiny = torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2
    bound = torch.finfo(t).eps / 2 * (ref.abs() + 1e-5 * row) + 1e-5 * row + tiny
    over = (got.double() - ref).abs() - bound
    assert torch.isfinite(got).all()
    assert over.max().item() <= 0, over.max().item()


# a row per warp (d <= 512) and per CTA; odd rows; the limits of d
SHAPES = [(1, 8), (3, 136), (17, 256), (9, 264), (33, 512), (5, 520), (64, 1032), (1, 7168),
          (130, 7168), (7, 4104), (2, 16384), (1, 16376)]


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("kind", [moe.MOE_NORM_RMS, moe.MOE_NORM_LAYER])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_norm_in(T, d, kind, dtype):
    x = rand(T, d, dtype=dtype, seed=T + d, mean=0.5)
    w, b = rand(d, dtype=dtype, seed=1, mean=1.0, std=0.2), rand(d, dtype=dtype, seed=2)
    check(moe.moe_norm_in(x, w, b, kind=kind), ref_norm(x, w, b, kind))
    check(moe.moe_norm_in(x, w, kind=kind, weight_offset=1.0), ref_norm(x, w, None, kind, 1.0))
    check(moe.moe_norm_in(x, None, b, kind=kind, eps=0.01), ref_norm(x, None, b, kind, eps=0.01))
    out = x.clone()
    moe.moe_norm_in(out, w, kind=kind, out=out)     # in place
    assert torch.equal(out, moe.moe_norm_in(x, w, kind=kind))


GATES = ["none", "channel", "token", "full"]


@pytest.mark.parametrize("T,d", [(1, 8), (6, 264), (1, 520), (37, 1032), (3, 7168), (2, 16384)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("kind", [moe.MOE_NORM_RMS, moe.MOE_NORM_LAYER])
def test_norm_out(T, d, dtype, kind):
    x, f = rand(T, d, dtype=dtype, seed=5, std=3.0), rand(T, d, dtype=dtype, seed=6, mean=0.2)
    pw, pb = rand(d, dtype=dtype, seed=1, mean=1.0, std=0.2), rand(d, dtype=dtype, seed=2, std=0.1)
    nw, nb = rand(d, dtype=dtype, seed=3, mean=1.0, std=0.2), rand(d, dtype=dtype, seed=4, std=0.1)
    gates = {"none": None, "channel": rand(d, dtype=dtype, seed=7),
             "token": rand(T, 1, dtype=dtype, seed=8), "full": rand(T, d, dtype=dtype, seed=9)}
    for gate, post, nxt, scale in itertools.product(GATES, (False, True), (False, True), (1.0, -0.37)):
        g = gates[gate]
        v = ref_norm(f, pw, pb, kind) if post else f.double()
        r = scale * x.double() + (v if g is None else g.double() * v)
        xo, no = moe.moe_norm_out(f, x, pw if post else None, pb if post else None, gate=g,
                                  residual_scale=scale, next_weight=nw if nxt else None,
                                  next_bias=nb if nxt else None, kind=kind)
        # r is a difference of terms: its fp32 error goes by their size
        size = scale * x.double().abs() + (v.abs() if g is None else (g.double() * v).abs())
        t = dtype
        bound = torch.finfo(t).eps / 2 * r.abs() + 1.01e-5 * size.abs().amax(-1, keepdim=True)
        assert ((xo.double() - r).abs() <= bound + torch.finfo(t).smallest_normal * torch.finfo(t).eps).all()
        if nxt:
            check(no, ref_norm(r, nw, nb, kind))
        else:
            assert no is None


def test_norm_out_without_weights_and_in_place():
    T, d = 11, 1024
    x, f = rand(T, d, dtype=BF16, seed=1), rand(T, d, dtype=BF16, seed=2)
    xo, no = moe.moe_norm_out(f, x, post_norm=True, next_norm=True)
    r = x.double() + ref_norm(f, None, None, 0)
    check(no, ref_norm(r, None, None, 0))
    x2, f2 = x.clone(), f.clone()
    moe.moe_norm_out(f2, x2, post_norm=True, x_out=x2, next_out=f2)
    assert torch.equal(x2, xo) and torch.equal(f2, no)


def test_strided_rows_and_guard_values():
    # rows inside a wider tensor: what lies between the rows is not touched
    T, d, wide = 19, 520, 1040
    big = rand(T, wide, dtype=BF16, seed=3)
    fbig, gbig = rand(T, wide, dtype=BF16, seed=4), rand(T, wide, dtype=BF16, seed=5)
    w = rand(d, dtype=BF16, seed=6)
    out = torch.full((T, wide), 7.0, dtype=BF16, device="cuda")
    nxt = torch.full((T, wide), 7.0, dtype=BF16, device="cuda")
    moe.moe_norm_in(big[:, 8:8 + d], w, out=out[:, 16:16 + d])
    check(out[:, 16:16 + d], ref_norm(big[:, 8:8 + d], w, None, 0))
    assert (out[:, :16] == 7).all() and (out[:, 16 + d:] == 7).all()
    out.fill_(7.0)
    moe.moe_norm_out(fbig[:, :d], big[:, 8:8 + d], w, gate=gbig[:, 24:24 + d], next_weight=w,
                     x_out=out[:, 16:16 + d], next_out=nxt[:, 32:32 + d])
    a = moe.moe_norm_out(fbig[:, :d].contiguous(), big[:, 8:8 + d].contiguous(), w,
                         gate=gbig[:, 24:24 + d].contiguous(), next_weight=w)
    assert torch.equal(out[:, 16:16 + d], a[0]) and torch.equal(nxt[:, 32:32 + d], a[1])
    assert (out[:, :16] == 7).all() and (nxt[:, 32 + d:] == 7).all()


def test_zero_rows_and_zero_values():
    assert moe.moe_norm_in(torch.empty(0, 64, dtype=BF16, device="cuda")).shape == (0, 64)
    z = torch.zeros(3, 1024, dtype=FP16, device="cuda")
    b = rand(1024, dtype=FP16, seed=1)
    for kind in (0, 1):
        assert torch.equal(moe.moe_norm_in(z, b, b, kind=kind), b.expand(3, -1))
    c = torch.full((3, 1024), 5.0, dtype=FP16, device="cuda")
    assert torch.equal(moe.moe_norm_in(c, None, b, kind=1), b.expand(3, -1))  # variance zero


def test_a_bad_row_stays_in_its_row():
    for d in (256, 7168):
        x = rand(6, d, dtype=BF16, seed=9)
        want = moe.moe_norm_in(x)
        x[2, 5], x[4, 7] = float("nan"), float("inf")
        got = moe.moe_norm_in(x)
        keep = [0, 1, 3, 5]
        assert torch.equal(got[keep], want[keep])
        assert torch.isnan(got[2]).all()


def test_large_values_and_another_stream():
    # squares of 1e15 sum to far below the fp32 limit; fp16's own limit does not matter
    x = rand(4, 4096, dtype=BF16, seed=11, std=1e15)
    check(moe.moe_norm_in(x), ref_norm(x, None, None, 0))
    h = (rand(4, 4096, dtype=FP16, seed=12) * 2000)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = moe.moe_norm_in(h)
    s.synchronize()
    check(got, ref_norm(h, None, None, 0))
