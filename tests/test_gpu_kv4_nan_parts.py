"""A row that stands for NaN shows in the heads that see it, however little it would
weigh: units cut into parts join the same as whole ones.

Every key's first element is 0 but for some hot ones at 200, every query's is 20: the
hot keys' scores pass the others' by 20 * 200 / sqrt(D) = 500 (D = 64) or 354 (128), so
that the parts without one weigh exp(-354) at most, nothing in fp32."""
import pytest
import torch

import dispatch_combine_gb300 as moe
from tests.gpu_common import ensure_lib
from tests.test_gpu_kv4_attention import BF16, FP16, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib():
    ensure_lib()


def put(b, seq, r):
    """Row r of a sequence as b.k and b.v have it."""
    slot = (b.table[seq, r // b.page] * b.page + r % b.page).to(torch.int32)[None]
    moe.moe_kv4_append(b.kv, None, b.k[seq][r:r + 1], b.v[seq][r:r + 1], None, slot, None, b.kc, b.vc)


@pytest.mark.parametrize("hq,hkv,D,dtype", [(16, 2, 64, BF16), (16, 2, 128, FP16), (32, 2, 128, BF16), (14, 2, 64, FP16)])
@pytest.mark.parametrize("others", [0, 80])       # few units, joined one way, and many, joined the other
@pytest.mark.parametrize("hot,bad", [(3000, 100), (100, 5000), (5999, 0)])
@pytest.mark.parametrize("what", ["k", "v"])
def test_nan_in_a_part_that_weighs_nothing(hq, hkv, D, dtype, others, hot, bad, what):
    lens, qs = [6000] + [40] * others, [2] + [1] * others
    b = Batch(lens, qs, hq, hkv, D, 16, dtype, seed=3)
    b.q[:, :, 0] = 20.0
    for seq in range(len(lens)):
        b.k[seq][:, :, 0] = 0.0
    b.k[0][hot, :, 0] = 200.0
    everything = torch.cat([(b.table[0].long()[:, None] * 16 + torch.arange(16, device="cuda")).flatten()])
    moe.moe_kv4_append(b.kv, None, b.k[0], b.v[0], None, everything[:6000].to(torch.int32), None, b.kc, b.vc)
    for seq in range(1, len(lens)):
        slots = (b.table[seq, :3].long()[:, None] * 16 + torch.arange(16, device="cuda")).flatten()[:40]
        moe.moe_kv4_append(b.kv, None, b.k[seq], b.v[seq], None, slots.to(torch.int32), None, b.kc, b.vc)
    clean, clean_lse = b.run()
    b.check(clean, clean_lse, rows={0, 1, 2})
    (b.k if what == "k" else b.v)[0][bad, 1, 40] = float("nan")     # head 1, group 1
    put(b, 0, bad)
    o, lse = b.run()
    G = hq // hkv
    if what == "k":
        assert o[:2, G:].isnan().all() and lse[:2, G:].isnan().all()
    else:
        assert o[:2, G:, 32:64].isnan().all()
    # nobody else sees it
    assert torch.equal(o[:2, :G], clean[:2, :G]) and torch.equal(lse[:2, :G], clean_lse[:2, :G])
    assert torch.equal(o[2:], clean[2:]) and torch.equal(lse[2:], clean_lse[2:])
