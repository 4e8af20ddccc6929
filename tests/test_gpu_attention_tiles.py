"""moe_prefix_attention where there are many query rows and each worker has
several tiles of keys: running maxima that move from tile to tile, and masks
that differ from token to token.  The bounds are those of
test_gpu_prefix_attention, with the scores' error by the scores' size: fp32 sums
of D exact products are good to (D/16 + 16) * 2^-23 of the sum of magnitudes."""
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


FORMS = [(D, dtype) for D in (64, 128) for dtype in (BF16, FP16)]
# (new tokens, own rows, prefix, query heads, key heads): 512 tiles and more, so
# three or more for each worker, of units of 128 rows and of two times 128, in the
# prefix and in the sequences' own rows
LONG = {
    "narrow prefix": ([1, 1, 1], [0, 0, 5], 4100, 640, 16),
    "wide prefix": ([1] * 36, [0] * 35 + [9], 4100, 128, 16),
    "narrow own": ([14, 9], [2200, 2100], 0, 128, 16),
    "wide own": ([40, 33], [2200, 2100], 100, 128, 16),
}


def long_case(name, D, dtype, **kw):
    qs, lens, prefix, hq, hkv = LONG[name]
    return Case(qs, lens, prefix, hq=hq, hkv=hkv, D=D, dtype=dtype, page=64, **kw)


def check(c, size, scale):
    """size: a bound of scale * sum |q_i k_i| over all pairs of a query and a key."""
    o, lse = c.run(scale=scale)
    ro, ra, rl = c.reference(scale)
    err = 24 * 2.0 ** -23 * size
    half = torch.finfo(c.dtype).eps / 2
    assert ((o.double() - ro).abs() <= half * ro.abs() + (half + 2e-4 + 2 * err) * 1.01 * ra + 1e-7).all()
    assert ((lse.double() - rl).abs() <= err + 1e-4 + 2.0 ** -23 * rl.abs()).all()
    assert moe.moe_get_device_status(c.ws) == 0


@pytest.mark.parametrize("name", LONG)
@pytest.mark.parametrize("D,dtype", FORMS)
def test_loud_scores_move_the_maximum(name, D, dtype):
    # a standard deviation of 24 (34): the maximum moves now and then all along
    c = long_case(name, D, dtype, loud=6.0)
    c.k *= 2
    size = (c.q.double().norm(dim=-1).max() * c.k.nan_to_num().double().norm(dim=-1).max()).item()
    check(c, 0.25 * size, 0.25)


@pytest.mark.parametrize("name", LONG)
@pytest.mark.parametrize("D,dtype", FORMS)
def test_rising_scores_move_the_maximum_in_every_tile(name, D, dtype):
    # 10 powers of two from a tile of 128 keys to the next
    c = long_case(name, D, dtype)
    c.q.fill_(1.0)
    step = 10 * math.log(2) / 128
    top = 0
    for pages, first, n in [(c.prefix_pages, 0, c.prefix)] + [(c.table[b], c.prefix, m)
                                                              for b, m in enumerate(c.lens_list)]:
        score = (first + torch.arange(n, device="cuda")) * step
        for i in range(-(-n // c.page)):
            part = score[i * c.page:(i + 1) * c.page]
            c.k[pages[i].long(), :, :len(part)] = (part * D ** -0.5).to(dtype)[:, None]
        top = max(top, (first + n) * step)
    check(c, 1.01 * top, D ** -0.5)


@pytest.mark.parametrize("G", [2, 7, 8, 40])
@pytest.mark.parametrize("prefix", [0, 130, 513])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_ragged_queries_at_head_size_128(G, prefix, dtype):
    # from no query to many: tiles of rows that end inside a sequence, masked
    # token by token across the borders of 128 keys
    qs = [1, 0, 17, 5, 64, 2, 100]
    lens = [50, 10, 17, 300, 64, 129, 260]
    Case(qs, lens, prefix, hq=2 * G, hkv=2, D=128, dtype=dtype).check()


@pytest.mark.parametrize("D,dtype", FORMS)
@pytest.mark.parametrize("n,own", [(129, 129), (300, 300), (257, 700), (200, 120)])
def test_a_prompt_over_its_own_rows(n, own, D, dtype):
    # one sequence and its causal triangle; with rows before it; with tokens that see nothing
    Case([n], [own], 0, hq=16, hkv=2, D=D, dtype=dtype, page=32).check()


@pytest.mark.parametrize("D,dtype", FORMS)
@pytest.mark.parametrize("n,G", [(15, 1), (16, 1), (17, 1), (8, 2), (9, 2), (31, 1), (32, 1), (33, 1), (1, 16),
                                 (1, 17), (1, 32), (1, 33), (4, 8), (5, 8)])
@pytest.mark.parametrize("prefix", [0, 200, 4096, 4097])
def test_row_counts_where_the_kernel_changes(n, G, D, dtype, prefix):
    # of the sequence, and of the batch over the prefix
    Case([n], [max(n, 150)], prefix, hq=2 * G, hkv=2, D=D, dtype=dtype, page=64).check()
    Case([1] * n, [20 + 9 * b for b in range(n)], prefix, hq=G, hkv=1, D=D, dtype=dtype, page=64).check()


@pytest.mark.parametrize("D,dtype", [(64, FP16), (128, BF16)])
@pytest.mark.parametrize("B,prefix,own", [(3, 128, 5000), (128, 1000, 40), (129, 40, 190), (300, 257, 20),
                                          (700, 129, 33)])
def test_prefix_tiles_beside_own_rows_of_16(B, prefix, own, D, dtype):
    # few and many sequences, either part the longer one, 16 rows of each sequence
    lens = [own - (11 * b) % (own // 2 + 1) for b in range(B)]
    lens[B // 2] = 0
    Case([1] * B, lens, prefix, hq=16, hkv=1, D=D, dtype=dtype, page=16).check()
