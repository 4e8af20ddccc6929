"""moe_prefix_attention against softmax(scale q K^T) V in 64 bits.

Bounds.  Scores are fp32 sums of D exact products: an error of at most
(D/16 + 16) * 2^-23 of the sum of their magnitudes, which for the inputs here
is below 25, so 24 * 2^-23 * 25 < 8e-5; a probability moves by that, relative,
and so does their sum: 1.6e-4 together.  Each probability is rounded to the
cache's type, half a step relative.  Against A = sum_j p_j |v_j| / sum_j p_j
the result is off by at most (finfo.eps / 2 + 2e-4) * A, and the output's own
rounding adds half a step of it.  The log-sum-exp is off by at most the
scores' 8e-5 and its own fp32 rounding: 1e-4 + 2^-23 * |lse|.
Rows of the cache that no token may see hold NaN throughout.
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


class Case:
    """A batch with its pages scattered over a cache that is NaN elsewhere.
    qs, lens: new tokens and own rows of each sequence."""

    def __init__(self, qs, lens, prefix, hq=8, hkv=2, D=64, page=16, dtype=BF16, seed=0, spare=2,
                 loud=1.0, extra_table=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g, self.qs, self.lens_list, self.prefix = g, qs, lens, prefix
        self.hq, self.hkv, self.D, self.page, self.dtype = hq, hkv, D, page, dtype
        B, self.T = len(qs), sum(qs)
        npre = -(-prefix // page)
        mp = max([-(-n // page) for n in lens] + [0]) + extra_table
        pages = npre + B * mp + spare
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        self.prefix_pages = order[:npre].contiguous()
        self.table = order[npre:npre + B * mp].reshape(B, mp).contiguous()
        self.kv = moe.kv_struct(hq, hkv, D, page, pages, dtype)
        shape = (pages, hkv, page, D)
        self.k = torch.full(shape, float("nan"), dtype=dtype, device="cuda")
        self.v = torch.full(shape, float("nan"), dtype=dtype, device="cuda")
        for pg, n in [(self.prefix_pages, prefix)] + [(self.table[b], lens[b]) for b in range(B)]:
            for i in range(-(-n // page)):
                m = min(page, n - i * page)
                self.k[pg[i].long(), :, :m] = self.rand(hkv, m, D)
                self.v[pg[i].long(), :, :m] = self.rand(hkv, m, D)
        self.q = self.rand(self.T, hq, D, std=loud)
        self.off = torch.tensor([sum(qs[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.max_q = max(qs + [1])

    def rand(self, *shape, std=1.0):
        return (torch.randn(*shape, generator=self.g, device="cuda") * std).to(self.dtype)

    def workspace(self):
        return moe.Workspace(moe.moe_prefix_attention_workspace_size(
            self.kv, self.T, len(self.qs), self.max_q, self.prefix))

    def run(self, ws=None, **kw):
        self.ws = ws or self.workspace()
        a = dict(q_offsets=self.off, max_q=self.max_q, want_lse=True)
        a.update(kw)
        return moe.moe_prefix_attention(self.kv, a.pop("q", self.q), self.k, self.v, self.prefix_pages,
                                        self.prefix, self.table, self.lens, self.ws, **a)

    def rows(self, cache, pages, n, h):
        used = pages[:-(-n // self.page)].long()   # what lies past them may be no page at all
        return cache[used, h].reshape(-1, self.D)[:n].double()

    def reference(self, scale=None):
        scale = self.D ** -0.5 if scale is None else scale
        G = self.hq // self.hkv
        o = torch.zeros(self.T, self.hq, self.D, dtype=torch.float64, device="cuda")
        a = torch.zeros_like(o)
        lse = torch.full((self.T, self.hq), -math.inf, dtype=torch.float64, device="cuda")
        for h in range(self.hkv):
            pk, pv = (self.rows(c, self.prefix_pages, self.prefix, h) for c in (self.k, self.v))
            t = 0
            for b, (n, m) in enumerate(zip(self.qs, self.lens_list)):
                k = torch.cat([pk, self.rows(self.k, self.table[b], m, h)])
                v = torch.cat([pv, self.rows(self.v, self.table[b], m, h)])
                for i in range(n):
                    end = self.prefix + max(0, m - n + i + 1)
                    hs = slice(h * G, (h + 1) * G)
                    if end:
                        z = self.q[t, hs].double() @ k[:end].T * scale
                        p = torch.softmax(z, -1)
                        o[t, hs], a[t, hs] = p @ v[:end], p @ v[:end].abs()
                        lse[t, hs] = torch.logsumexp(z, -1)
                    t += 1
        return o, a, lse

    def check(self, got=None, scale=None, **kw):
        o, lse = got or self.run(**kw)
        ro, ra, rl = self.reference(scale)
        half = torch.finfo(self.dtype).eps / 2
        tiny = torch.finfo(self.dtype).smallest_normal * torch.finfo(self.dtype).eps
        over = (o.double() - ro).abs() - (half * ro.abs() + (half + 2e-4) * 1.01 * ra + tiny)
        assert torch.isfinite(o).all()
        assert over.max().item() <= 0, over.max().item()
        if lse is not None:
            seen = torch.isfinite(rl)
            assert torch.equal(seen, torch.isfinite(lse)) and (lse[~seen] == -math.inf).all()
            assert ((lse.double() - rl).abs()[seen] <= 1e-4 + 2.0 ** -23 * rl.abs()[seen]).all()
        assert moe.moe_get_device_status(self.ws) == 0
        return o, lse


# prefix and own lengths at the borders of a 16-row page and a 128-row tile
LENGTHS = [(0, 1), (1, 1), (15, 2), (16, 16), (17, 127), (127, 128), (128, 129), (129, 17), (255, 1),
           (300, 300), (1000, 64)]


@pytest.mark.parametrize("prefix,own", LENGTHS)
@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, BF16), (64, FP16), (128, FP16)])
def test_one_token_of_one_sequence(prefix, own, D, dtype):
    Case([1], [own], prefix, D=D, dtype=dtype).check()


@pytest.mark.parametrize("G,hkv", [(1, 1), (1, 3), (3, 2), (4, 1), (5, 2), (7, 1), (16, 2), (20, 1), (33, 1),
                                   (64, 1), (100, 1), (128, 1)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_head_layouts_and_pages(G, hkv, page):
    Case([1, 1, 1, 1, 1], [3, 140, 16, 257, 90], 333, hq=G * hkv, hkv=hkv, D=128, page=page).check()


@pytest.mark.parametrize("G", [1, 2, 7, 8, 40])
@pytest.mark.parametrize("prefix", [0, 130, 513])
def test_ragged_queries(G, prefix):
    # from no query to many: one tile of rows, several, tiles that end inside a sequence
    qs = [1, 0, 17, 5, 64, 2, 100]
    lens = [50, 10, 17, 300, 64, 129, 260]
    Case(qs, lens, prefix, hq=2 * G, hkv=2, D=64, dtype=FP16).check()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B", [31, 64, 200])
def test_many_sequences(B, D):
    lens = [1 + (37 * b) % 190 for b in range(B)]
    Case([1] * B, lens, 700, hq=16, hkv=2, D=D, page=32).check(q_offsets=None)


@pytest.mark.parametrize("prefix", [0, 5000, 20011])
def test_long_axis_is_split_and_joined(prefix):
    Case([1, 2], [6001, 130], prefix, hq=8, hkv=1, D=128, page=64).check()


def test_rows_that_see_nothing():
    # fewer own rows than queries: the first queries see only the prefix
    c = Case([4, 3, 1, 0, 2], [2, 0, 0, 0, 2], 0)
    o, lse = c.check()
    assert (o[:2] == 0).all() and (lse[:2] == -math.inf).all() and torch.isfinite(lse[2:4]).all()
    assert (o[4:8] == 0).all()
    Case([4, 3, 1, 0, 2], [2, 0, 0, 0, 2], 77).check()
    # and a batch that has no rows at all, with and without a table
    c = Case([1, 1], [0, 0], 0, extra_table=1)
    o, lse = c.check()
    assert (o == 0).all()
    c.table = None
    o, lse = c.run()
    assert (o == 0).all() and (lse == -math.inf).all()


def test_loud_scores_and_scale():
    # scores of several hundred: the running maximum moves through many tiles
    c = Case([1, 3], [400, 700], 900, D=64, dtype=FP16, loud=6.0)
    c.k *= 2
    # score magnitudes sum to under 64 * 3.3 * 6 * 2: the bound grows with them
    o, lse = c.run(scale=0.5)
    ro, ra, rl = c.reference(0.5)
    err = 24 * 2.0 ** -23 * 0.5 * 64 * 6 * 2
    assert ((o.double() - ro).abs() <= 2.0 ** -11 * ro.abs() + (2.0 ** -11 + 4 * err) * ra + 1e-6).all()
    assert ((lse.double() - rl).abs() <= err + 1e-4 + 2.0 ** -23 * rl.abs()).all()


def test_rising_scores_rescale_the_sum():
    # every tile's scores top the last one's, so each tile moves the maximum
    c = Case([1], [1], 2000, hq=4, hkv=1, D=64, page=16)
    c.q.fill_(1.0)
    ramp = torch.arange(2000, device="cuda") / 2000.0 * 8
    flat = (ramp[:, None] + 0 * torch.zeros(2000, 64, device="cuda")).to(BF16)
    for i, pg in enumerate(c.prefix_pages.tolist()):
        c.k[pg, 0] = flat[16 * i:16 * i + 16]
    err = 24 * 2.0 ** -23 * 64
    o, lse = c.run()
    ro, ra, rl = c.reference()
    assert ((o.double() - ro).abs() <= 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 4 * err) * 1.01 * ra).all()
    assert ((lse.double() - rl).abs() <= err + 1e-4).all()


def test_strides_streams_and_reused_workspace():
    big = Case([1] * 40, [200] * 40, 1500, hq=16, hkv=4, D=128, page=64, seed=1)
    ws = big.workspace()
    big.check(ws=ws)
    # smaller calls of other shapes in the same workspace, then the first again
    for c in (Case([3, 1], [70, 5], 40, hq=16, hkv=4, D=128, seed=2),
              Case([1], [9], 0, hq=8, hkv=8, D=64, seed=3)):
        need = moe.moe_prefix_attention_workspace_size(c.kv, c.T, len(c.qs), c.max_q, c.prefix)
        if need <= ws.nbytes:
            c.check(ws=ws)
        c.check()
    first = big.run(ws=ws)
    # queries and outputs inside wider tensors, on a stream of their own
    wide = torch.full((big.T, 40, 128), 5.0, dtype=BF16, device="cuda")
    wide[:, 8:24] = big.q
    out = torch.full((big.T, 20, 128), 5.0, dtype=BF16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = big.run(ws=ws, q=wide[:, 8:24], out=out[:, 2:18])
    s.synchronize()
    assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
    assert (out[:, :2] == 5).all() and (out[:, 18:] == 5).all()
    # without lse
    assert torch.equal(big.run(ws=ws, want_lse=False)[0], first[0])


def test_captured_graph_follows_the_lengths():
    c = Case([1] * 6, [140] * 6, 300, hq=8, hkv=2, D=64)
    ws = c.workspace()
    out, lse = torch.empty_like(c.q), torch.empty(c.T, c.hq, device="cuda")
    c.run(ws=ws, out=out, lse=lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(ws=ws, out=out, lse=lse)
    for lens in ([1, 2, 3, 139, 17, 16], [140] * 6, [128, 0, 1, 127, 129, 64]):
        c.lens_list = lens
        c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        for _ in range(2):
            out.fill_(float("nan"))
            graph.replay()
            c.check(got=(out, lse))


def test_the_same_call_gives_the_same_bits():
    c = Case([1] * 50 + [9], [1 + 13 * b for b in range(51)], 4000, hq=32, hkv=4, D=128, page=64)
    a, b = c.run(), c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_cache_past_32_bit_offsets():
    D, page, hkv = 128, 256, 1
    pages = (1 << 31) // (D * page) + 4
    kv = moe.kv_struct(4, hkv, D, page, pages, BF16)
    k = torch.empty(pages, hkv, page, D, dtype=BF16, device="cuda")
    v = torch.empty(pages, hkv, page, D, dtype=BF16, device="cuda")
    small = Case([1], [200], 500, hq=4, hkv=1, D=D, page=page, spare=0)
    n = small.kv.num_pages
    k[-n:], v[-n:] = small.k, small.v
    shift = pages - n
    ws = moe.Workspace(moe.moe_prefix_attention_workspace_size(kv, 1, 1, 1, 500))
    o, lse = moe.moe_prefix_attention(kv, small.q, k, v, small.prefix_pages + shift, 500,
                                      small.table + shift, small.lens, ws, want_lse=True)
    small.ws = ws
    small.check(got=(o, lse))


def test_bad_pages_and_lengths_are_reported():
    # every value is clamped on the device: the status says so and nothing
    # outside the output is written
    def run(change, **kw):
        c = Case([1, 2], [100, 40], 50, hq=8, hkv=2)
        c.k.nan_to_num_()
        c.v.nan_to_num_()
        change(c)
        out = torch.full((c.T + 2, c.hq, c.D), 5.0, dtype=BF16, device="cuda")
        c.run(out=out[1:-1], **kw)
        torch.cuda.synchronize()
        assert (out[0] == 5).all() and (out[-1] == 5).all()
        return moe.moe_get_device_status(c.ws)

    def at(name, index, value):
        def change(c):
            getattr(c, name)[index] = value
        return change

    assert run(lambda c: None) == 0
    assert run(at("prefix_pages", 1, 1 << 20)) == 1
    assert run(at("prefix_pages", 0, -1)) == 1
    assert run(at("table", (1, 0), 2 ** 31 - 1)) == 1
    assert run(at("lens", 0, -5)) == 1
    assert run(at("lens", 0, 100000)) == 1
    assert run(at("off", 1, 3000)) == 1
    assert run(at("off", 2, 3000)) == 1
    assert run(at("off", 1, -7)) == 1
    assert run(lambda c: None, max_q=1) == 1


def test_pages_past_the_end_are_not_looked_at():
    c = Case([1, 1], [20, 3], 10, extra_table=3)
    c.table[0, 2:] = -1
    c.table[1, 1:] = 1 << 25
    c.check()


@pytest.mark.parametrize("D,dtype", [(64, FP16), (128, BF16)])
@pytest.mark.parametrize("B,prefix,own", [(1, 130, 2000), (3, 128, 5000), (128, 1000, 40), (129, 40, 190),
                                          (300, 257, 20), (700, 129, 33)])
def test_prefix_tiles_beside_own_rows(B, prefix, own, D, dtype):
    # few and many sequences, either part the longer one: 32 heads a key head, so
    # that the prefix's rows are many and a sequence's few
    qs = [1 + (b % 7 == 3) for b in range(B)]
    lens = [max(q, own - (11 * b) % (own // 2 + 1)) for b, q in enumerate(qs)]
    lens[B // 2] = 0
    Case(qs, lens, prefix, hq=32, hkv=1, D=D, dtype=dtype, page=16).check()


def test_calls_in_a_row_see_their_own_lengths():
    # nothing waits on the host between the calls and the changes of their inputs
    c = Case([1] * 40, [400] * 40, 300, hq=16, hkv=2, D=128, page=16)
    ws = c.workspace()
    sets = [torch.tensor([1 + (i * s + 13 * s) % 400 for i in range(40)], dtype=torch.int32, device="cuda")
            for s in range(1, 9)]
    want = []
    for s in sets:
        c.lens.copy_(s)
        want.append(c.run(ws=ws)[0])
        torch.cuda.synchronize()
    q = c.q.clone()
    got = []
    for _ in range(3):
        for s in sets:
            c.lens.copy_(s)
            c.q.copy_(q)
            got.append(c.run(ws=ws)[0])
            c.q.zero_()
            c.lens.zero_()
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % len(sets)])
    assert moe.moe_get_device_status(ws) == 0
