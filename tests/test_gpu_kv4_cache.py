"""moe_kv4_append and moe_kv4_read against the 4-bit form in 64 bits.

Bounds.  Rows that do not turn are quantised from 16-bit values: max|v| / 7 and
the quotients v / s of 8 to 11-bit numbers lie on a border between two codes or
further from it than a fp32 division's rounding, so codes and scales are those of
64 bits, and what is read back is their product rounded once: equal to the 64-bit
product rounded.  Rows that turn have an error of at most e = 4 * 2^-24 of the
pair's length (cosine and sine, two products and a sum, half a step each, and
1e-9 of the angle) before they are quantised: an element may change its code only
where v / s lies within 2 e / s of a border (its own error, and the scale's as
seen through a code of up to 7), and then by one; the scale may be the next fp16
number.
"""
import pytest
import torch

import dispatch_combine_gb300 as moe
from tests.gpu_common import ensure_lib
from tests.kv4_common import GROUP, held

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _lib():
    ensure_lib()


def rand(*shape, dtype=BF16, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def caches(kv, fill=0):
    return [torch.full((kv.num_pages, kv.num_kv_heads, moe.moe_kv4_page_bytes(kv)), fill, dtype=torch.uint8,
                       device="cuda") for _ in range(2)]


def i32(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def freqs(rot):
    return 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float32) / max(rot, 1))


def turned(v, positions, inv_freq, style):
    """(rotated, pair lengths) in 64 bits."""
    v, size = v.double().clone(), torch.zeros(v.shape, dtype=torch.float64, device=v.device)
    n = inv_freq.numel()
    at = torch.arange(n, device="cuda")
    i, j = (at, at + n) if style == moe.MOE_ROPE_HALF else (2 * at, 2 * at + 1)
    t = (positions.double()[:, None] * inv_freq.double())[:, None]
    a, b = v[..., i], v[..., j]
    size[..., i] = size[..., j] = torch.hypot(a, b)
    v[..., i], v[..., j] = a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()
    return v, size


@pytest.mark.parametrize("T,hq,hkv,D,page", [
    (1, 1, 1, 64, 16), (1, 64, 8, 128, 64), (5, 28, 4, 128, 32), (130, 8, 8, 64, 128), (33, 14, 2, 64, 256),
    (17, 128, 1, 128, 16), (3, 3, 3, 64, 16), (700, 16, 4, 64, 64),
])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_rows_come_back_as_they_are_held(T, hq, hkv, D, page, dtype):
    pages = -(-T // page) + 2
    kv = moe.kv_struct(hq, hkv, D, page, pages, dtype)
    wide = rand(T, (hq + 2 * hkv) * D + 8, dtype=dtype, seed=T)[:, 8:]     # a strided slice
    q, k, v = (wide[:, a * D:(a + n) * D].unflatten(1, (n, D)) for a, n in ((0, hq), (hq, hkv), (hq + hkv, hkv)))
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(T))[:T].to("cuda", torch.int32)
    kc, vc = caches(kv, fill=0xA5)
    before = kc.clone(), vc.clone()
    ws = moe.Workspace(256)
    out = moe.moe_kv4_append(kv, q, k, v, None, slots, None, kc, vc, ws)
    assert torch.equal(out, q)
    k2, v2 = moe.moe_kv4_read(kv, slots, kc, vc, ws)
    assert torch.equal(k2, held(k)[0].to(dtype)) and torch.equal(v2, held(v)[0].to(dtype))
    # nothing but these rows has changed: their bytes differ at most
    touched = T * hkv * (D // 2 + D // 16)
    assert (kc != before[0]).sum() <= touched and (vc != before[1]).sum() <= touched
    # and nothing at all when the tokens are padding
    again = kc.clone(), vc.clone()
    moe.moe_kv4_append(kv, q, rand(T, hkv, D, dtype=dtype, seed=9), v, None, torch.full_like(slots, -1), None, kc, vc, ws)
    assert torch.equal(kc, again[0]) and torch.equal(vc, again[1])
    assert moe.moe_get_device_status(ws) == 0


@pytest.mark.parametrize("D,rot", [(64, 64), (64, 32), (64, 48), (128, 128), (128, 64), (128, 16), (128, 112)])
@pytest.mark.parametrize("style", [moe.MOE_ROPE_HALF, moe.MOE_ROPE_PAIRS])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_rotation(D, rot, style, dtype):
    T, hq, hkv, page = 77, 6, 3, 32
    kv = moe.kv_struct(hq, hkv, D, page, 4, dtype)
    q, k, v = (rand(T, h, D, dtype=dtype, seed=s) for h, s in ((hq, 1), (hkv, 2), (hkv, 3)))
    pos = torch.randint(0, 100000, (T,), generator=torch.Generator().manual_seed(rot)).to("cuda", torch.int32)
    slots = torch.arange(T, device="cuda", dtype=torch.int32) + 20
    kc, vc = caches(kv)
    freq = freqs(rot)
    out = moe.moe_kv4_append(kv, q, k, v, pos, slots, freq, kc, vc, style=style)
    e = 4 * 2.0 ** -24
    want, size = turned(q, pos, freq, style)
    t = torch.finfo(dtype)
    assert ((out.double() - want).abs() <= t.eps / 2 * (want.abs() + e * size) + e * size + t.tiny * t.eps / 2).all()
    k2, v2 = moe.moe_kv4_read(kv, slots, kc, vc)
    assert torch.equal(v2, held(v)[0].to(dtype))
    want, size = turned(k, pos, freq, style)
    ref, scale = held(want)
    spread = size.unflatten(-1, (-1, GROUP)).amax(-1, keepdim=True).expand(-1, -1, -1, GROUP).flatten(-2)
    off = (k2.double() - ref).abs()
    # same code: the scale's next fp16 number (2^-10 relative), and the rounding of the result
    near = off <= (2.0 ** -10 + t.eps / 2) * ref.abs() + 1e-7
    share = want / scale
    border = ((share.abs() - 0.5) - torch.round(share.abs() - 0.5)).abs()
    at_border = (border <= 2 * e * spread / scale) & (off <= 1.01 * scale + t.eps / 2 * ref.abs())
    # a scale that is its neighbour moves the borders by up to 7 * 2^-10 of a code
    groups = lambda x: x.unflatten(-1, (-1, GROUP))  # noqa: E731
    exact = groups(want).abs().amax(-1) / 7
    rounds = exact.to(torch.float16).double()
    step = torch.finfo(FP16).eps * 2.0 ** torch.floor(torch.log2(rounds))
    unsure = ((exact - rounds).abs() >= step / 2 - 2 * e * groups(spread)[..., 0])[..., None].expand_as(groups(want)).flatten(-2)
    at_moved = unsure & (border <= 7 * 2.0 ** -10) & (off <= 1.01 * scale + t.eps / 2 * ref.abs())
    assert (near | at_border | at_moved).all()
    assert (~near).sum() <= 8       # chances of 1e-6 an element


@pytest.mark.parametrize("T", [700, 1300, 2605])
@pytest.mark.parametrize("D,style,dtype", [(128, moe.MOE_ROPE_HALF, BF16), (64, moe.MOE_ROPE_PAIRS, FP16)])
def test_a_token_is_the_same_among_many(T, D, style, dtype):
    """Bits do not depend on how many tokens a call has (and so on the warps that a token gets)."""
    hq, hkv, page = 6, 3, 64
    kv = moe.kv_struct(hq, hkv, D, page, -(-T // page), dtype)
    q, k, v = (rand(T, h, D, dtype=dtype, seed=s) for h, s in ((hq, 1), (hkv, 2), (hkv, 3)))
    pos = torch.randint(0, 2 ** 31 - 1, (T,), generator=torch.Generator().manual_seed(T)).to("cuda", torch.int32)
    slots = torch.randperm(T, generator=torch.Generator().manual_seed(1)).to("cuda", torch.int32)
    kc, vc = caches(kv)
    out = moe.moe_kv4_append(kv, q, k, v, pos, slots, freqs(D), kc, vc, style=style)
    few_k, few_v = caches(kv)
    few = torch.cat([moe.moe_kv4_append(kv, q[i:i + 90], k[i:i + 90], v[i:i + 90], pos[i:i + 90], slots[i:i + 90],
                                        freqs(D), few_k, few_v, style=style) for i in range(0, T, 90)])
    assert torch.equal(out, few) and torch.equal(kc, few_k) and torch.equal(vc, few_v)


def test_values_near_the_ends():
    """Groups of zeros, of one large element, of the smallest and largest numbers; NaN and infinities
    make their group of 32 NaN and no other."""
    kv = moe.kv_struct(2, 2, 64, 16, 1, BF16)
    k = rand(16, 2, 64, seed=5)
    k[0] = 0.0
    k[1, 0, 3] = 1000.0
    k[2] *= 1e-7                     # scales of a few fp16 subnormals
    k[3] *= 1e-9                     # scales of zero
    k[4] *= 1e4
    k[5, 0, 7] = 4.5e5               # the scale is just inside fp16
    k[6, 1, 40] = 6e5                # and past it
    k[7, 0, 0] = float("nan")
    k[8, 1, 63] = float("inf")
    k[9, 0, 33] = -float("inf")
    k[10] = -0.0
    k[11] = 1.0
    v = k.flip(0).contiguous()
    kc, vc = caches(kv)
    slots = torch.arange(16, device="cuda", dtype=torch.int32)
    moe.moe_kv4_append(kv, None, k, v, None, slots, None, kc, vc)
    k2, v2 = moe.moe_kv4_read(kv, slots, kc, vc)
    want = held(k)[0]
    for row, head, group in ((6, 1, 1), (7, 0, 0), (8, 1, 1), (9, 0, 1)):
        want[row, head, 32 * group:32 * group + 32] = float("nan")
    want = want.to(BF16)
    assert torch.equal(k2.isnan(), want.isnan()) and torch.equal(k2.nan_to_num(7.0), want.nan_to_num(7.0))
    assert torch.equal(v2.nan_to_num(7.0), want.flip(0).nan_to_num(7.0))


@pytest.mark.parametrize("D,page,hkv", [(64, 16, 3), (128, 64, 8), (64, 256, 1), (128, 16, 2)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_read_into_a_16_bit_cache(D, page, hkv, dtype):
    n = 3 * page + 5
    kv = moe.kv_struct(hkv, hkv, D, page, 6, dtype)
    k, v = rand(n, hkv, D, dtype=dtype, seed=1), rand(n, hkv, D, dtype=dtype, seed=2)
    g = torch.Generator().manual_seed(3)
    slots = torch.randperm(6 * page, generator=g)[:n].to("cuda", torch.int32)
    kc, vc = caches(kv)
    moe.moe_kv4_append(kv, None, k, v, None, slots, None, kc, vc)
    to = torch.randperm(5 * page, generator=g)[:n].to("cuda", torch.int32)
    to[4] = -1
    slots[7] = -1
    ko, vo = (torch.full((5, hkv, page, D), 3.0, dtype=dtype, device="cuda") for _ in range(2))
    ws = moe.Workspace(256)
    a, b = moe.moe_kv4_read(kv, slots, kc, vc, ws, k_out=ko, v_out=vo, dst_slots=to)
    assert a is ko and b is vo
    wk, wv = (torch.full((5, hkv, page, D), 3.0, dtype=dtype, device="cuda") for _ in range(2))
    for i in range(n):
        if i not in (4, 7):
            p, r = divmod(int(to[i]), page)
            wk[p, :, r], wv[p, :, r] = held(k[i])[0].to(dtype), held(v[i])[0].to(dtype)
    assert torch.equal(ko, wk) and torch.equal(vo, wv)
    assert moe.moe_get_device_status(ws) == 0
    # strided token rows; padding rows stay
    wide = torch.full((n, 2 * hkv * D + 8), 5.0, dtype=dtype, device="cuda")
    ko, vo = (wide[:, x:x + hkv * D].unflatten(1, (hkv, D)) for x in (0, hkv * D))
    moe.moe_kv4_read(kv, slots, kc, vc, ws, k_out=ko, v_out=vo)
    want = held(k)[0].to(dtype)
    want[7] = 5.0
    assert torch.equal(ko, want) and (wide[:, 2 * hkv * D:] == 5.0).all()


def test_slots_outside_are_reported_and_skipped():
    kv = moe.kv_struct(2, 2, 64, 16, 2, BF16)
    n = moe.moe_kv4_page_bytes(kv)
    # the caches are the middle of larger buffers, whose rest must not change
    buf = torch.full((2, 6, 2, n), 7, dtype=torch.uint8, device="cuda")
    kc, vc = buf[0, 2:4], buf[1, 2:4]
    k = rand(4, 2, 64, seed=3)
    ws = moe.Workspace(256)
    slots = i32(32, -2, 31, 2 ** 31 - 1)
    moe.moe_kv4_append(kv, None, k, k, None, slots, None, kc, vc, ws)
    assert moe.moe_get_device_status(ws) == 1
    assert (buf[:, :2] == 7).all() and (buf[:, 4:] == 7).all()
    assert (buf[:, 2:4] != 7).sum() <= 2 * 2 * (32 + 4)
    ko, vo = (torch.full((4, 2, 64), 3.0, dtype=BF16, device="cuda") for _ in range(2))
    moe.moe_kv4_read(kv, slots, kc, vc, ws, k_out=ko, v_out=vo)
    assert moe.moe_get_device_status(ws) == 1
    assert torch.equal(ko[2], held(k[2])[0].to(BF16)) and (ko[[0, 1, 3]] == 3.0).all() and (vo[[0, 1, 3]] == 3.0).all()
    big = torch.full((3, 2, 16, 64), 3.0, dtype=BF16, device="cuda")
    big2 = big.clone()
    moe.moe_kv4_read(kv, i32(31, 31, 31, 31), kc, vc, ws, k_out=big[1:2], v_out=big2[1:2], dst_slots=i32(16, -2, 3, 2 ** 31 - 1))
    assert moe.moe_get_device_status(ws) == 1
    assert torch.equal(big[1, :, 3], held(k[2])[0].to(BF16))
    big[1, :, 3] = 3.0
    assert (big == 3.0).all()
    moe.moe_kv4_append(kv, None, k, k, None, slots, None, kc, vc)          # nobody to report to
    moe.moe_kv4_read(kv, slots, kc, vc, k_out=ko, v_out=vo)


def test_no_tokens():
    kv = moe.kv_struct(4, 2, 64, 16, 2)
    kc, vc = caches(kv, 9)
    k = rand(3, 2, 64, seed=3)
    moe.moe_kv4_append(kv, None, k[:0], k[:0], None, i32(), None, kc, vc)
    a, b = moe.moe_kv4_read(kv, i32(), kc, vc)
    assert a.shape == b.shape == (0, 2, 64) and (kc == 9).all() and (vc == 9).all()
    a, b = moe.moe_kv4_read(kv, i32(-1, -1), kc, vc)
    assert (a == 0).all() and (b == 0).all()


def test_queries_turn_in_place():
    kv = moe.kv_struct(4, 2, 128, 16, 3)
    T = 9
    q, k, v = (rand(T, h, 128, seed=s) for h, s in ((4, 1), (2, 2), (2, 3)))
    pos = torch.arange(100, 100 + T, device="cuda", dtype=torch.int32)
    slots = torch.arange(20, 20 + T, device="cuda", dtype=torch.int32)
    one, two = caches(kv), caches(kv)
    q1 = moe.moe_kv4_append(kv, q, k, v, pos, slots, freqs(128), *one)
    q2 = q.clone()
    assert moe.moe_kv4_append(kv, q2, k, v, pos, slots, freqs(128), *two, q_out=q2) is q2
    assert torch.equal(q1, q2) and torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


def test_cache_past_32_bit_offsets():
    # 2^32 + bytes per cache: the last page lies past a 32-bit offset
    D, hkv, page = 128, 1, 256
    kv = moe.kv_struct(1, hkv, D, page, 1)
    pages = (1 << 32) // moe.moe_kv4_page_bytes(kv) + 2
    kv = moe.kv_struct(1, hkv, D, page, pages)
    kc, vc = (torch.empty(pages, hkv, moe.moe_kv4_page_bytes(kv), dtype=torch.uint8, device="cuda") for _ in range(2))
    k, v = rand(2, 1, D, seed=1), rand(2, 1, D, seed=2)
    slots = i32(pages * page - 1, 3)
    moe.moe_kv4_append(kv, None, k, v, None, slots, None, kc, vc)
    k2, v2 = moe.moe_kv4_read(kv, slots, kc, vc)
    assert torch.equal(k2, held(k)[0].to(BF16)) and torch.equal(v2, held(v)[0].to(BF16))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("style", [moe.MOE_ROPE_HALF, moe.MOE_ROPE_PAIRS])
def test_far_and_negative_positions(D, style):
    """Queries, whose rotation shows the angles: up to 2^31 positions the angle is good to 1.5 * 2^-53 of
    its turns (the frequency in 53 bits), 2e-7 of a turn at a frequency of 1, and at 10^6 to 3e-11."""
    pos = i32(0, 1, 999983, -999983, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 7, 12345678)
    kv = moe.kv_struct(2, 2, D, 16, 1, FP16)
    q, k = rand(8, 2, D, dtype=FP16, seed=1), rand(8, 2, D, dtype=FP16, seed=2)
    kc, vc = caches(kv)
    freq = freqs(D)
    freq[3] = -freq[3]
    out = moe.moe_kv4_append(kv, q, k, k, pos, torch.arange(8, device="cuda", dtype=torch.int32), freq, kc, vc, style=style)
    want, size = turned(q, pos, freq, style)
    turns = (pos.double().abs()[:, None] * freq.double().abs().max() / 6.283185307179586)[..., None]
    e = 4 * 2.0 ** -24 + 2 * 6.3 * 1.5 * 2.0 ** -53 * turns       # both sides' angles
    t = torch.finfo(FP16)
    assert ((out.double() - want).abs() <= t.eps / 2 * (want.abs() + e * size) + e * size + t.tiny * t.eps / 2).all()


def test_many_tokens_take_two_warps_each():
    """Past eight tokens an SM the kernel has several in a CTA: the last of them short."""
    T, hq, hkv, D, page = 2051, 6, 2, 128, 64
    kv = moe.kv_struct(hq, hkv, D, page, -(-T // page), BF16)
    q, k, v = (rand(T, h, D, seed=s) for h, s in ((hq, 1), (hkv, 2), (hkv, 3)))
    pos = torch.arange(T, device="cuda", dtype=torch.int32) + 5000
    slots = torch.randperm(kv.num_pages * page, generator=torch.Generator().manual_seed(1))[:T].to("cuda", torch.int32)
    slots[7] = -1
    many, few = caches(kv), caches(kv)
    a = moe.moe_kv4_append(kv, q, k, v, pos, slots, freqs(D), *many)
    b = torch.empty_like(a)
    for t in range(0, T, 200):      # the same tokens in calls of fewer
        s = slice(t, min(T, t + 200))
        moe.moe_kv4_append(kv, q[s], k[s], v[s], pos[s], slots[s], freqs(D), *few, q_out=b[s])
    assert torch.equal(a, b) and torch.equal(many[0], few[0]) and torch.equal(many[1], few[1])
    rows = [moe.moe_kv4_read(kv, slots, *many) for _ in range(2)]
    assert torch.equal(rows[0][0], rows[1][0]) and torch.equal(rows[0][1], held(v)[0].to(BF16) * (slots >= 0)[:, None, None])


def test_a_frequency_that_is_not_finite():
    kv = moe.kv_struct(1, 1, 64, 16, 1, BF16)
    freq = freqs(64)
    freq[5] = float("inf")
    freq[9] = float("nan")
    kc, vc = caches(kv)
    q = rand(1, 1, 64, seed=1)
    out = moe.moe_kv4_append(kv, q, q, q, i32(3), i32(0), freq, kc, vc)
    bad = torch.zeros(64, dtype=torch.bool, device="cuda")
    bad[[5, 9, 37, 41]] = True
    assert out[0, 0][bad].isnan().all() and not out[0, 0][~bad].isnan().any()
    k2, _ = moe.moe_kv4_read(kv, i32(0), kc, vc)
    assert k2.isnan().all()         # both groups hold one


def test_capture_and_replay():
    """The calls of a step in one graph, slots and positions changing between replays."""
    kv = moe.kv_struct(4, 2, 64, 16, 4, FP16)
    q, k, v = (rand(5, h, 64, dtype=FP16, seed=s) for h, s in ((4, 1), (2, 2), (2, 3)))
    pos, slots = i32(1, 2, 3, 4, 5), i32(0, 1, 2, 3, 4)
    kc, vc = caches(kv)
    qo, ko, vo = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)

    def step():
        moe.moe_kv4_append(kv, q, k, v, pos, slots, freqs_, kc, vc, q_out=qo)
        moe.moe_kv4_read(kv, slots, kc, vc, k_out=ko, v_out=vo)

    freqs_ = freqs(64)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        slots.copy_(torch.tensor([63, 5 + i, 17, 33, 50], dtype=torch.int32))
        pos.copy_(torch.arange(5) * (i + 7))
        graph.replay()
        got = qo.clone(), ko.clone(), vo.clone()
        kc2, vc2 = caches(kv)
        a = moe.moe_kv4_append(kv, q, k, v, pos, slots, freqs_, kc2, vc2)
        b = moe.moe_kv4_read(kv, slots, kc2, vc2)
        assert torch.equal(got[0], a) and torch.equal(got[1], b[0]) and torch.equal(got[2], b[1])
