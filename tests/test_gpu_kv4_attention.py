"""moe_kv4_attention against attention in 64 bits over what the cache holds.

Bounds.  The cache's numbers enter exactly, a query row's elements lose at most
2^-25 * 2^-14 of 2^15, its largest, so 2^-38 relative to it.  A score is a sum over
groups of fp32 sums of at most 32 products of up to 15 * |q| (the codes stand
from 1 to 15 there, and the offset of 8 is the sum's start): each of its D / 16
instructions and D / 32 more operations may round at 2^-22 of the magnitudes that
meet (tensor cores cut off instead of rounding), so its error is below
  d = 2^-20 * scale * sum_b s_b 15 sum |q|.
A probability has that error, 2^-21 from the exponential, and two roundings to
fp16, half a step each: relative e = 2 * 2^-11 + 2^-21 + d (plus 2^-25 of the type's
lowest step, kept 2^9 up: 2^-33 of the largest).  The output is a weighted mean,
each weight off by e against the unrounded sum: |o - ref| <= sum_j p_j e (|v_j| + 8
s_j) + d |ref| and the output's own rounding; the codes' offset again makes 15 s of
7 s at most.  lse: d, and 2^-20 from sums and logarithms.
"""
import math

import pytest
import torch

import dispatch_combine_gb300 as moe
from tests.gpu_common import ensure_lib
from tests.kv4_common import held

pytestmark = pytest.mark.gpu
BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _lib():
    ensure_lib()


def rand(*shape, dtype=BF16, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


class Batch:
    """Sequences with lengths `lens` and `qs` new tokens; their rows in pages in any order."""

    def __init__(self, lens, qs, hq, hkv, D, page, dtype=BF16, seed=0, spare=3, q_std=1.5, k_std=1.0, v_std=1.0):
        self.lens, self.qs, self.hq, self.hkv, self.D, self.page, self.dtype = lens, qs, hq, hkv, D, page, dtype
        each = [-(-n // page) for n in lens]
        pages = sum(each) + spare
        self.kv = moe.kv_struct(hq, hkv, D, page, pages, dtype)
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
        table = torch.full((len(lens), max(each + [1])), -7, dtype=torch.int32)   # never looked at past a length
        self.k, self.v, slots = [], [], []
        for b, n in enumerate(each):
            mine, order = order[:n], order[n:]
            table[b, :n] = torch.tensor(mine, dtype=torch.int32)
            slots += [mine[i // page] * page + i % page for i in range(lens[b])]
            self.k.append(rand(lens[b], hkv, D, dtype=dtype, seed=seed + 10 * b + 1, std=k_std))
            self.v.append(rand(lens[b], hkv, D, dtype=dtype, seed=seed + 10 * b + 2, std=v_std))
        # what nobody wrote: every byte 0xFF, so scales that are NaN
        self.kc, self.vc = (torch.full((pages, hkv, moe.moe_kv4_page_bytes(self.kv)), 0xFF, dtype=torch.uint8,
                                       device="cuda") for _ in range(2))
        if slots:
            moe.moe_kv4_append(self.kv, None, torch.cat(self.k), torch.cat(self.v), None,
                               torch.tensor(slots, dtype=torch.int32, device="cuda"), None, self.kc, self.vc)
        self.table = table.cuda()
        self.T = sum(qs)
        self.q = rand(self.T, hq, D, dtype=dtype, seed=seed + 5, std=q_std)
        self.kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.offsets = torch.tensor([sum(qs[:b]) for b in range(len(qs) + 1)], dtype=torch.int32, device="cuda")
        self.max_q = max(qs + [1])
        self.ws = moe.Workspace(moe.moe_kv4_attention_workspace_size(self.kv, self.T, len(lens), self.max_q))

    def run(self, **kw):
        kw = {"q_offsets": self.offsets, "max_q": self.max_q, "want_lse": True, **kw}
        return moe.moe_kv4_attention(self.kv, self.q, self.kc, self.vc, self.table, self.kv_lens, self.ws, **kw)

    def check(self, o, lse, scale=None, rows=None):
        G, D = self.hq // self.hkv, self.D
        scale = D ** -0.5 if scale is None else scale
        t = torch.finfo(self.dtype)
        at = 0
        for b, (n, m) in enumerate(zip(self.lens, self.qs)):
            kh, ks = held(self.k[b])
            vh, vs = held(self.v[b])
            for h in range(self.hkv):
                heads = slice(h * G, (h + 1) * G)
                for i in range(m):
                    sees = n - m + i + 1
                    if rows is not None and at + i not in rows:
                        continue
                    got, got_lse = o[at + i, heads].double(), lse[at + i, heads].double()
                    if sees <= 0:
                        assert (got == 0).all() and (got_lse == -math.inf).all()
                        continue
                    q, k, v = self.q[at + i, heads].double(), kh[:sees, h], vh[:sees, h]
                    # a query past fp16 is an infinity, and its head NaN
                    fine = q.isfinite().all(-1)
                    assert got[~fine].isnan().all() and got_lse[~fine].isnan().all()
                    q, got, got_lse = q[fine], got[fine], got_lse[fine]
                    z = scale * (q @ k.T)
                    ref_lse = torch.logsumexp(z, -1)
                    p = torch.exp(z - ref_lse[:, None])
                    ref = p @ v
                    d = 2.0 ** -20 * scale * 15 * (q.abs() @ ks[:sees, h].T)
                    dm = d.amax(-1, keepdim=True)
                    e = 2 * 2.0 ** -11 + 2.0 ** -21 + d + dm
                    peak = p.amax(-1, keepdim=True)
                    bound = (p * e + 2.0 ** -33 * peak) @ (v.abs() + 8 * vs[:sees, h]) + dm * ref.abs()
                    bound = bound + t.eps / 2 * (ref.abs() + bound) + t.tiny * t.eps / 2
                    assert ((got - ref).abs() <= bound).all(), (b, h, i, ((got - ref).abs() / bound).max())
                    assert ((got_lse - ref_lse).abs() <= dm[:, 0] + 2.0 ** -20 * (1 + ref_lse.abs())).all(), (b, h, i)
            at += m
        assert moe.moe_get_device_status(self.ws) == 0


@pytest.mark.parametrize("hq,hkv,D,page", [
    (8, 1, 128, 64), (64, 8, 128, 64), (28, 4, 64, 16), (1, 1, 64, 16), (5, 1, 128, 32), (12, 4, 64, 128),
    (16, 1, 128, 256), (20, 1, 128, 16), (24, 1, 64, 32), (32, 1, 64, 64), (128, 1, 128, 64), (34, 1, 128, 16),
    (74, 2, 64, 16),
])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_one_token_each(hq, hkv, D, page, dtype):
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 64, 65, 257, 500]
    b = Batch(lens, [1] * len(lens), hq, hkv, D, page, dtype, seed=hq)
    o, lse = b.run()
    b.check(o, lse)
    # without offsets it is the same call
    o2, lse2 = b.run(q_offsets=None)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("hq,hkv,D,page", [(8, 2, 128, 16), (28, 4, 64, 16), (8, 1, 64, 64), (64, 8, 128, 64), (40, 1, 128, 32)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_drafts(hq, hkv, D, page, dtype):
    lens, qs = [3, 40, 7, 100, 0, 33, 5, 130], [3, 1, 7, 0, 0, 6, 7, 2]
    b = Batch(lens, qs, hq, hkv, D, page, dtype, seed=hq + page)
    b.check(*b.run())


def test_more_new_tokens_than_rows():
    """A sequence whose first tokens see nothing."""
    b = Batch([2, 0, 20], [5, 3, 1], 8, 2, 64, 16)
    o, lse = b.run()
    b.check(o, lse)
    assert (o[:3] == 0).all() and (lse[5:8] == -math.inf).all()
    # and with scores too small to be anything: their mean
    o, lse = b.run(scale=1e-38)
    b.check(o, lse, scale=1e-38)


@pytest.mark.parametrize("D", [64, 128])
def test_long_and_uneven(D):
    b = Batch([5000, 1, 77, 2049, 16], [1, 1, 1, 1, 1], 8, 2, D, 64, seed=3)
    b.check(*b.run())
    b = Batch([20011], [4], 4, 1, D, 16, FP16, seed=4)
    b.check(*b.run())


def test_a_chunk_of_many_tokens():
    b = Batch([300, 70], [200, 70], 8, 2, 128, 32, seed=6)
    b.check(*b.run(), rows={0, 1, 63, 150, 199, 200, 231, 269})


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("v_std", [1e-4, 0.02, 20.0, 3000.0])
def test_sizes_of_values(D, v_std):
    """Value scales from fp16's subnormals to past 2, where the exponent moves."""
    b = Batch([200, 45], [1, 2], 8, 1, D, 16, BF16, seed=int(v_std), v_std=v_std)
    b.check(*b.run())


def test_value_scales_that_grow():
    b = Batch([400], [1], 8, 1, 128, 16, BF16, seed=2)
    b.v[0] = (b.v[0].float() * torch.exp2(torch.arange(400, device="cuda") / 40.0)[:, None, None]).to(BF16)
    slots = torch.cat([b.table[0, :25].long() * 16 + i for i in range(16)]).reshape(16, 25).T.reshape(-1)
    moe.moe_kv4_append(b.kv, None, b.k[0], b.v[0], None, slots.to(torch.int32), None, b.kc, b.vc)
    b.check(*b.run())


@pytest.mark.parametrize("q_std,k_std,scale", [(100.0, 1.0, None), (1e-6, 1.0, None), (1.0, 1.0, 1e-6), (1.0, 30.0, None),
                                               (3e4, 1e-3, 0.02), (1.0, 1e-3, 8.0)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_sizes_of_scores(q_std, k_std, scale, dtype):
    b = Batch([150, 33], [1, 3], 8, 1, 64, 16, dtype, seed=11, q_std=q_std, k_std=k_std)
    b.check(*b.run(scale=scale), scale=scale)


def test_heads_of_different_sizes():
    """A head's row is scaled by itself: a huge one takes nothing off the others."""
    b = Batch([100], [1], 8, 1, 128, 64, seed=1)
    b.q[0, 2] *= 1e20
    b.q[0, 5] *= 1e-12
    b.q[0, 6] = 0.0
    o, lse = b.run()
    assert o[0, 2].isnan().all() and lse[0, 2].isnan()
    keep = [0, 1, 3, 4, 5, 6, 7]
    part = Batch([100], [1], 8, 1, 128, 64, seed=1)
    part.q[0] = b.q[0]
    part.q[0, 2] = 1.0
    o2, lse2 = part.run()
    part.check(o2, lse2)
    assert torch.equal(o[0, keep], o2[0, keep]) and torch.equal(lse[0, keep], lse2[0, keep])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_query_that_is_not_finite(bad):
    b = Batch([90, 20], [1, 2], 8, 2, 64, 16, seed=1)
    b.q[1, 3, 17] = bad
    o, lse = b.run()
    assert o[1, 3].isnan().all() and lse[1, 3].isnan()
    o[1, 3], lse[1, 3] = 0.0, 0.0
    assert not o.isnan().any() and not lse.isnan().any()


def test_keys_that_stand_for_nan():
    """A NaN in a row that is seen shows; one behind the length does not."""
    b = Batch([50, 50], [1, 1], 4, 1, 64, 64, seed=1)
    k = b.k[0][:1].clone()
    k[0, 0, 3] = float("nan")
    slot = (b.table[0, :1] * 64 + 20).to(torch.int32)
    moe.moe_kv4_append(b.kv, None, k, k, None, slot, None, b.kc, b.vc)
    behind = (b.table[1, :1] * 64 + 50).to(torch.int32)
    moe.moe_kv4_append(b.kv, None, k, k, None, behind, None, b.kc, b.vc)
    o, lse = b.run()
    assert o[0].isnan().all() and lse[0].isnan().all() and not o[1].isnan().any()
    b.check(o, lse, rows={1})


@pytest.mark.parametrize("hq,hkv,D,dtype", [(8, 2, 128, BF16), (8, 2, 64, FP16), (28, 4, 64, BF16), (6, 3, 128, FP16)])
@pytest.mark.parametrize("what", ["k", "v", "both"])
def test_drafts_that_stand_for_nan(hq, hkv, D, dtype, what):
    """The rows of drafts that are not seen touch nothing: neither tokens before them nor other heads."""
    lens, qs = [70, 64, 6, 300, 129], [6, 5, 6, 1, 4]
    b = Batch(lens, qs, hq, hkv, D, 16, dtype, seed=9)
    clean, _ = b.run()
    bad = {0: 67, 1: 63, 2: 1, 4: 127}          # sequence: its row with a NaN in head 1, group 1
    for seq, r in bad.items():
        if what != "v":
            b.k[seq][r, 1, 40] = float("nan")
        if what != "k":
            b.v[seq][r, 1, 40] = float("nan")
        slot = (b.table[seq, r // 16] * 16 + r % 16).to(torch.int32)[None]
        moe.moe_kv4_append(b.kv, None, b.k[seq][r:r + 1], b.v[seq][r:r + 1], None, slot, None, b.kc, b.vc)
    o, lse = b.run()
    G, at, blind = hq // hkv, 0, set()
    for seq, (n, m) in enumerate(zip(lens, qs)):
        for i in range(m):
            if seq in bad and n - m + i >= bad[seq]:
                hit = o[at + i, G:2 * G]
                assert hit[:, 32:64].isnan().all()
                assert torch.equal(o[at + i, :G], clean[at + i, :G]) and torch.equal(o[at + i, 2 * G:], clean[at + i, 2 * G:])
            else:
                blind.add(at + i)
        at += m
    assert len(blind) == 3 + 4 + 1 + 1 + 2
    b.check(o, lse, rows=blind)


def test_strided_queries_and_outputs():
    b = Batch([40, 70], [2, 1], 8, 2, 64, 16, seed=1)
    want = b.run()
    wide = torch.full((b.T, 3 * 8 * 64 + 8), 2.0, dtype=BF16, device="cuda")
    wide[:, 8:8 + 512] = b.q.flatten(1)
    b.q = wide[:, 8:8 + 512].unflatten(1, (8, 64))
    out = wide[:, 520:520 + 512].unflatten(1, (8, 64))
    o, lse = b.run(out=out)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert (wide[:, :8] == 2.0).all() and (wide[:, 520 + 512:] == 2.0).all()
    assert b.run(want_lse=False)[1] is None


def test_bad_pages_lengths_and_offsets_are_reported():
    b = Batch([40, 70], [1, 1], 8, 2, 64, 16, seed=1)
    good, _ = b.run()
    table = b.table.clone()
    b.table[0, 1] = b.kv.num_pages
    o, _ = b.run()
    assert moe.moe_get_device_status(b.ws) == 1 and torch.equal(o[1], good[1])
    b.table[0, 1] = -1
    b.run()
    assert moe.moe_get_device_status(b.ws) == 1
    b.table = table
    for n in (-1, 16 * table.shape[1] + 1):
        b.kv_lens[0] = n
        o, _ = b.run()
        assert moe.moe_get_device_status(b.ws) == 1 and torch.equal(o[1], good[1])
    b.kv_lens[0] = 40
    for off in ([0, 2, 1], [-1, 1, 2], [0, 1, 3]):
        b.run(q_offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
        assert moe.moe_get_device_status(b.ws) == 1
    b.run(q_offsets=torch.tensor([0, 2, 2], dtype=torch.int32, device="cuda"))    # two tokens, max_q 1
    assert moe.moe_get_device_status(b.ws) == 1
    assert torch.equal(b.run()[0], good)
    assert moe.moe_get_device_status(b.ws) == 0


def test_nothing_to_attend():
    b = Batch([0, 0], [1, 2], 8, 2, 64, 16, seed=1)
    o, lse = b.run()
    assert (o == 0).all() and (lse == -math.inf).all()
    kv = moe.kv_struct(8, 2, 64, 16, 0)
    ws = moe.Workspace(moe.moe_kv4_attention_workspace_size(kv, 3, 0, 1))
    none = torch.empty(0, 2, moe.moe_kv4_page_bytes(kv), dtype=torch.uint8, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    o, lse = moe.moe_kv4_attention(kv, b.q, none, none, None, i32(), ws, q_offsets=i32(0), want_lse=True)
    assert (o == 0).all() and (lse == -math.inf).all() and moe.moe_get_device_status(ws) == 0


def test_the_same_call_gives_the_same_bits_and_replays():
    b = Batch([900, 33, 4000, 1], [2, 1, 3, 1], 28, 4, 64, 16, FP16, seed=8)
    first = b.run()
    again = b.run()
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    out, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
    b.run(out=out, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run(out=out, lse=lse)
    for lens in ([900, 33, 4000, 1], [500, 30, 77, 1]):
        b.kv_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        out.zero_()
        graph.replay()
        want = b.run()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_two_calls_side_by_side():
    """Two streams, a workspace each."""
    a, b = Batch([700] * 6, [1] * 6, 16, 2, 128, 64, seed=1), Batch([3000, 5], [4, 1], 16, 2, 128, 64, seed=2)
    want = a.run(), b.run()
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        got = a.run(stream=streams[0]), b.run(stream=streams[1])
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_a_workspace_serves_every_smaller_call():
    b = Batch([90] * 5, [7, 1, 3, 2, 7], 20, 4, 64, 16, seed=8)
    want = b.run()
    kv = b.kv
    ws = moe.Workspace(moe.moe_kv4_attention_workspace_size(kv, 64, 9, 40))
    b.ws = ws
    got = b.run()
    assert torch.equal(got[0], want[0])


@pytest.mark.parametrize("byte", [0xFF, 0x7F, 0x01])
@pytest.mark.parametrize("lens", [[1, 2, 65, 257, 500], [9000], [40] * 300])
def test_what_a_workspace_held_before_is_nothing(byte, lens):
    b = Batch(lens, [1] * len(lens), 14, 2, 64, 16, seed=4)
    o, lse = b.run()
    b.ws.buf[b.ws.offset + 256:b.ws.offset + b.ws.nbytes] = byte
    o2, lse2 = b.run()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    b.check(o, lse)


@pytest.mark.parametrize("lens,qs,hq,hkv,D", [
    ([3000, 0, 1, 2500, 70], [3, 2, 1, 5, 0], 16, 2, 128), ([1900, 2300], [1, 2], 34, 1, 128), ([6000], [7], 28, 4, 64),
    ([1345, 1400, 64, 65], [1, 1, 1, 1], 64, 16, 64), ([40000], [1], 1, 1, 64),
])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_few_units_of_many_parts(lens, qs, hq, hkv, D, dtype):
    b = Batch(lens, qs, hq, hkv, D, 16, dtype, seed=len(lens))
    o, lse = b.run()
    b.check(o, lse)
    # offsets that are refused leave nothing behind for the next call
    bad = b.offsets.clone()
    bad[-1] = b.T + 1
    b.run(q_offsets=bad)
    assert moe.moe_get_device_status(b.ws) != 0
    b.ws = moe.Workspace(b.ws.nbytes)
    o2, lse2 = b.run()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # and a larger batch, whose units are joined in the other way, agrees
    more = Batch(lens + [1] * 70, qs + [1] * 70, hq, hkv, D, 16, dtype, seed=len(lens))
    more.check(*more.run())


@pytest.mark.parametrize("hq,hkv,D", [(8, 1, 128), (14, 2, 64)])
def test_a_graph_follows_the_lengths(hq, hkv, D):
    """Few units in many parts, in one, in none: what a call left in the workspace is nothing to the next."""
    b = Batch([4000, 2000], [1, 1], hq, hkv, D, 16, seed=2)
    full = b.kv_lens.clone()
    b.run()
    out = torch.full((2, hq, D), 9.0, dtype=BF16, device="cuda")
    lse = torch.full((2, hq), 9.0, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run(out=out, lse=lse)
    for lens in ([4000, 2000], [1, 1], [0, 2000], [3999, 64], [65, 0], [0, 0], [4000, 2000]):
        b.kv_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        k, v, n = b.k, b.v, b.lens
        b.k, b.v, b.lens = [x[:m] for x, m in zip(k, lens)], [x[:m] for x, m in zip(v, lens)], lens
        b.check(out, lse)
        b.k, b.v, b.lens = k, v, n
    assert torch.equal(b.kv_lens, full)


def test_cache_past_32_bit_offsets():
    D, page = 128, 256
    kv = moe.kv_struct(8, 1, D, page, 1)
    pages = (1 << 32) // moe.moe_kv4_page_bytes(kv) + 3
    kv = moe.kv_struct(8, 1, D, page, pages)
    kc, vc = (torch.empty(pages, 1, moe.moe_kv4_page_bytes(kv), dtype=torch.uint8, device="cuda") for _ in range(2))
    small = Batch([600], [1], 8, 1, D, page, seed=1)
    mine = torch.tensor([pages - 1, 0, pages - 2], dtype=torch.int32, device="cuda")
    kc[mine.long()], vc[mine.long()] = small.kc[small.table[0].long()], small.vc[small.table[0].long()]
    want = small.run()
    got = moe.moe_kv4_attention(kv, small.q, kc, vc, mine[None], small.kv_lens, small.ws, want_lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_tokens_of_no_sequence():
    """A batch padded in front and behind: its tokens without a sequence see nothing."""
    b = Batch([40, 0, 70], [2, 1, 1], 8, 2, 64, 16, seed=1)
    want = b.run()
    q = torch.full((9, 8, 64), 3.0, dtype=BF16, device="cuda")
    q[2:6] = b.q
    off = torch.tensor([2, 4, 5, 6], dtype=torch.int32, device="cuda")
    ws = moe.Workspace(moe.moe_kv4_attention_workspace_size(b.kv, 9, 3, 2))
    out, lse = torch.full_like(q, 7.0), torch.full((9, 8), 7.0, device="cuda")
    moe.moe_kv4_attention(b.kv, q, b.kc, b.vc, b.table, b.kv_lens, ws, q_offsets=off, max_q=2, out=out, lse=lse)
    assert torch.equal(out[2:6], want[0]) and torch.equal(lse[2:6], want[1])
    rest = [0, 1, 6, 7, 8]
    assert (out[rest] == 0).all() and (lse[rest] == -math.inf).all()
    assert moe.moe_get_device_status(ws) == 0


@pytest.mark.parametrize("n,hq,hkv,D", [(1500, 2, 1, 64), (700, 6, 3, 128), (4096, 1, 1, 64)])
def test_many_short_sequences(n, hq, hkv, D):
    """Several units of a worker, several sequences of a thread of the scan, and none among them."""
    g = torch.Generator().manual_seed(n)
    lens = torch.randint(0, 80, (n,), generator=g).tolist()
    qs = torch.randint(0, 3, (n,), generator=g).tolist()
    b = Batch(lens, qs, hq, hkv, D, 16, BF16, seed=5)
    o, lse = b.run()
    rows = set(torch.randint(0, b.T, (40,), generator=g).tolist())
    b.check(o, lse, rows=rows)
    # the rest against the same sequences in calls of their own kind: nothing is left out
    assert not o.isnan().any()
    seen = torch.tensor([i for m, k in zip(lens, qs) for i in [m - k + j + 1 for j in range(k)]], device="cuda") > 0
    assert torch.equal(lse > -math.inf, seen[:, None].expand_as(lse))


def test_one_head_over_all_workers():
    b = Batch([70001], [1], 3, 1, 128, 64, BF16, seed=9)
    b.check(*b.run())
