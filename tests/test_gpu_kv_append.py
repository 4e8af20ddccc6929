"""moe_kv_append against the rotation in 64 bits.

Bounds: one rounding of each result (finfo.eps / 2 relative, and half the
smallest subnormal), and before it a fp32 rotation: cosine and sine of a
reduced angle are good to 2^-22, the angle's fraction of a turn to 2^-25 (2
pi times that is 2e-7), and the two products and their sum round three times,
so a pair's error is below 1e-6 of the pair's length.
"""
import math

import pytest
import torch

import dispatch_combine_gb300 as moe
from tests.gpu_common import ensure_lib

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _lib():
    ensure_lib()


def rand(*shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def freqs(rot):
    return 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float32) / max(rot, 1))


def rotated(v, positions, inv_freq, style):
    """(rotated values, length of the pair each belongs to), 64 bits."""
    v = v.double().clone()
    if inv_freq is None:
        return v, v.abs() * 0
    n = inv_freq.numel()
    at = torch.arange(n, device="cuda")
    i, j = (at, at + n) if style == moe.MOE_ROPE_HALF else (2 * at, 2 * at + 1)
    t = (positions.double()[:, None] * inv_freq.double())[:, None]
    a, b = v[..., i], v[..., j]
    size = torch.zeros_like(v)
    size[..., i] = size[..., j] = torch.hypot(a, b)
    v[..., i], v[..., j] = a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()
    return v, size


def check(got, ref, size):
    t = torch.finfo(got.dtype)
    bound = t.eps / 2 * (ref.abs() + 1e-6 * size) + 1e-6 * size + t.smallest_normal * t.eps / 2
    assert ((got.double() - ref).abs() <= bound).all()


def run_case(T, hq, hkv, D, page, rot, style, dtype, far, pad=0, seed=0, status=0):
    pages = -(-T // page) + 2
    kv = moe.kv_struct(hq, hkv, D, page, pages, dtype)
    qkv = rand(T, (hq + 2 * hkv) * D + 8, dtype=dtype, seed=seed)[:, 8:]   # a strided slice
    q = qkv[:, :hq * D].unflatten(1, (hq, D))
    k = qkv[:, hq * D:(hq + hkv) * D].unflatten(1, (hkv, D))
    v = qkv[:, (hq + hkv) * D:].unflatten(1, (hkv, D))
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    pos = torch.randint(0, far, (T,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = far - 1
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].to(torch.int32)
    if pad:
        slots[-pad:] = -1
    kc, vc = rand(pages, hkv, page, D, dtype=dtype, seed=7), rand(pages, hkv, page, D, dtype=dtype, seed=8)
    want_k, want_v = kc.clone(), vc.clone()
    freq = freqs(rot) if rot else None
    ws = moe.Workspace(256)
    out = moe.moe_kv_append(kv, q, k, v, pos, slots, freq, kc, vc, ws, style=style)
    check(out, *rotated(q, pos, freq, style))
    ref, size = rotated(k, pos, freq, style)
    keep = slots >= 0
    at = slots[keep].long()
    check(kc[at // page, :, at % page], ref[keep], size[keep])
    assert torch.equal(vc[at // page, :, at % page], v[keep])
    # everything else of the cache is as it was
    kc[at // page, :, at % page] = want_k[at // page, :, at % page]
    vc[at // page, :, at % page] = want_v[at // page, :, at % page]
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)
    assert moe.moe_get_device_status(ws) == status


@pytest.mark.parametrize("T,hq,hkv,D,page,rot", [
    (1, 1, 1, 64, 16, 64), (1, 64, 8, 128, 64, 128), (5, 28, 4, 128, 32, 64), (130, 8, 8, 64, 128, 32),
    (33, 14, 2, 64, 256, 16), (17, 128, 1, 128, 16, 128), (7, 4, 2, 128, 16, 0), (300, 16, 4, 64, 64, 48),
])
@pytest.mark.parametrize("style", [moe.MOE_ROPE_HALF, moe.MOE_ROPE_PAIRS])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_append(T, hq, hkv, D, page, rot, style, dtype):
    run_case(T, hq, hkv, D, page, rot, style, dtype, far=4096, pad=min(2, T - 1))


@pytest.mark.parametrize("far", [1, 1 << 20, (1 << 31) - 1])
def test_far_positions(far):
    run_case(40, 4, 2, 128, 16, 128, moe.MOE_ROPE_HALF, FP16, far=far, seed=3)


def test_keys_only_and_in_place():
    kv = moe.kv_struct(4, 2, 64, 16, 3)
    T = 9
    q, k, v = (rand(T, h, 64, dtype=BF16, seed=s) for h, s in ((4, 1), (2, 2), (2, 3)))
    pos = torch.arange(100, 100 + T, device="cuda", dtype=torch.int32)
    slots = torch.arange(20, 20 + T, device="cuda", dtype=torch.int32)
    caches = [torch.zeros(3, 2, 16, 64, dtype=BF16, device="cuda") for _ in range(4)]
    q1 = moe.moe_kv_append(kv, q, k, v, pos, slots, freqs(64), caches[0], caches[1])
    assert moe.moe_kv_append(kv, None, k, v, pos, slots, freqs(64), caches[2], caches[3]) is None
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    q2 = q.clone()
    assert moe.moe_kv_append(kv, q2, k, v, pos, slots, freqs(64), caches[2], caches[3],
                             q_out=q2) is q2
    assert torch.equal(q1, q2)


def test_no_tokens_and_all_padding():
    kv = moe.kv_struct(4, 2, 64, 16, 2)
    kc, vc = (rand(2, 2, 16, 64, dtype=BF16, seed=s) for s in (1, 2))
    before = kc.clone(), vc.clone()
    i32 = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    k = rand(3, 2, 64, dtype=BF16, seed=3)
    moe.moe_kv_append(kv, None, k[:0], k[:0], i32[:0], i32[:0], freqs(64), kc, vc)
    moe.moe_kv_append(kv, None, k, k, i32, i32, freqs(64), kc, vc)
    assert torch.equal(kc, before[0]) and torch.equal(vc, before[1])


def test_slots_outside_the_cache_are_reported_and_skipped():
    kv = moe.kv_struct(2, 2, 64, 16, 2)
    # the caches are the middle of larger buffers, whose rest must not change
    buf = torch.full((2, 6, 2, 16, 64), 3.0, dtype=BF16, device="cuda")
    kc, vc = buf[0, 2:4], buf[1, 2:4]
    k = rand(4, 2, 64, dtype=BF16, seed=3)
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    slots = torch.tensor([32, -2, 31, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    ws = moe.Workspace(256)
    moe.moe_kv_append(kv, None, k, k, pos, slots, freqs(64), kc, vc, ws)
    assert moe.moe_get_device_status(ws) == 1
    assert torch.equal(vc[1, :, 15], k[2])
    vc[1, :, 15] = 3.0
    kc[1, :, 15] = 3.0
    assert (buf == 3.0).all()
    moe.moe_kv_append(kv, None, k, k, pos, slots, freqs(64), kc, vc)   # nobody to report to


def test_cache_past_32_bit_offsets():
    # 2^31 + elements per cache: the last page lies past a 32-bit element offset
    D, hkv, page = 128, 1, 256
    pages = (1 << 31) // (D * page) + 2
    kv = moe.kv_struct(1, hkv, D, page, pages)
    kc = torch.empty(pages, hkv, page, D, dtype=BF16, device="cuda")
    vc = torch.empty(pages, hkv, page, D, dtype=BF16, device="cuda")
    k, v = rand(2, 1, D, dtype=BF16, seed=1), rand(2, 1, D, dtype=BF16, seed=2)
    slots = torch.tensor([pages * page - 1, 3], dtype=torch.int32, device="cuda")
    kc[-1, 0, -2], vc[-1, 0, -2] = 1.0, 1.0
    moe.moe_kv_append(kv, None, k, v, slots, slots, None, kc, vc)
    assert torch.equal(vc[-1, 0, -1], v[0, 0]) and torch.equal(vc[0, 0, 3], v[1, 0])
    assert torch.equal(kc[-1, 0, -1], k[0, 0]) and torch.equal(kc[0, 0, 3], k[1, 0])
    assert (vc[-1, 0, -2] == 1).all() and (kc[-1, 0, -2] == 1).all()
