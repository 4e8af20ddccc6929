"""moe_kv4_attention where the values are small, large, or both, and most of the weight is
elsewhere: a first key without a value that takes it, the others 2^-12 to 2^-24 as likely.

Bounds.  As in test_gpu_kv4_attention.py but for what fp16 does at its lower end.  A
key's probability is held as 2^9 p / peak or more (the largest score of its stretch is put
at 2^9 and may be passed by later ones); half a step of the lowest is 2^-25, so 2^-34 peak.
The value scales of a group are taken times 2^-(x + 1), x the exponent of the group's
largest scale S of the sequence at most, or -16 if that is more: F = max(S, 2^-16), 2^x <= F.
Half a step, 2^-25, is 2^-24 F of a scale, with the weight p; of the product with the
probability it is 2^-33 peak F; and each element is a whole number of at most 7 of
them.  So beside the relative errors there are at most
  sum_j peak (2^-34 |v_j| + 2^-33 7 F) + 2^-24 7 F sum_j p_j,
and the accumulators' cuts, 2^-22 of the sum of magnitudes at each 16 keys of a stretch."""
import math

import pytest
import torch

import dispatch_combine_gb300 as moe
from tests.gpu_common import ensure_lib
from tests.kv4_common import held
from tests.test_gpu_kv4_attention import BF16, FP16, Batch, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib():
    ensure_lib()


class Sink:
    """A sequence's rows that `users` others share, of shrinking lengths, `m` new tokens
    each; so many users and heads that a warp has hundreds of keys in a row.  The first key takes
    the weight (the others 2^-down as likely, give or take) and has no value; values are positive."""

    def __init__(self, n, users, m, hq, hkv, D, page, dtype, down, v_std):
        b = self.b = Batch([n], [1], hq, hkv, D, page, dtype, seed=down, k_std=0.05, v_std=v_std)
        self.lens = [n - 7 * i for i in range(users)]
        self.m, self.k, self.v = m, b.k[0], b.v[0]
        self.q = rand(users * m, hq, D, dtype=dtype, seed=1)
        self.q[:, :, 0] = 8.0
        self.k[:, :, 0] = 0.0
        self.k[0, :, 0] = down * math.log(2) * D ** 0.5 / 8.0
        self.v.abs_()
        self.v[0] = 0.0
        self.table = b.table.expand(users, -1).contiguous()
        self.kv_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.offsets = torch.arange(0, users * m + 1, m, dtype=torch.int32, device="cuda")
        self.ws = moe.Workspace(moe.moe_kv4_attention_workspace_size(b.kv, users * m, users, m))

    def run(self):
        b, n = self.b, self.lens[0]
        slots = (b.table[0, :-(-n // b.page)].long()[:, None] * b.page + torch.arange(b.page, device="cuda")).flatten()[:n]
        moe.moe_kv4_append(b.kv, None, self.k, self.v, None, slots.to(torch.int32), None, b.kc, b.vc)
        return moe.moe_kv4_attention(b.kv, self.q, b.kc, b.vc, self.table, self.kv_lens, self.ws, q_offsets=self.offsets,
                                     max_q=self.m, want_lse=True)

    def check(self, o, lse):
        b = self.b
        G, D, m = b.hq // b.hkv, b.D, self.m
        scale, t = D ** -0.5, torch.finfo(b.dtype)
        kh, ks = held(self.k)
        vh, vs = held(self.v)
        for seq in range(0, len(self.lens), 5):
            for i in range(m):
                at, sees = seq * m + i, self.lens[seq] - m + i + 1
                q = self.q[at].double().unflatten(0, (b.hkv, G))
                k, s, v, sv = (x[:sees].transpose(0, 1) for x in (kh, ks, vh, vs))     # [hkv, keys, D]
                F = sv.amax(1, keepdim=True).clamp(min=2.0 ** -16)
                z = scale * (q @ k.mT)
                ref_lse = torch.logsumexp(z, -1, keepdim=True)
                p = torch.exp(z - ref_lse)
                ref = p @ v
                d = 2.0 ** -20 * scale * 15 * (q.abs() @ s.mT)
                dm = d.amax(-1, keepdim=True)
                e = 2 * 2.0 ** -11 + 2.0 ** -21 + d + dm + sees / 16 * 2.0 ** -22
                peak = p.amax(-1, keepdim=True)
                bound = (p * e) @ (v.abs() + 8 * sv) + 2.0 ** -34 * peak * v.abs().sum(1, keepdim=True) + dm * ref.abs()
                bound = bound + sees * 2.0 ** -33 * peak * 7 * F + 7 * 2.0 ** -24 * F
                assert (bound < 0.1 * ref.abs()).all()          # what is left to the others is well above it
                bound = bound + t.eps / 2 * (ref.abs() + bound) + t.tiny * t.eps / 2
                got, got_lse = (x[at].double().unflatten(0, (b.hkv, G)) for x in (o, lse))
                off = ((got - ref).abs() / bound).amax().item()
                assert off <= 1, (seq, i, off)
                assert ((got_lse[..., None] - ref_lse).abs() <= dm + 2.0 ** -20 * (1 + ref_lse.abs())).all()
        assert moe.moe_get_device_status(self.ws) == 0


# a group's largest element is about 2.1 times what its elements are drawn with
STD = {e: 2.0 ** e * 7 / 2.1 for e in (-14, -12, -10, -8, 0, 3, 10)}
SHAPES = [(2000, 60, 1, 64, 8, 128), (2000, 60, 2, 64, 8, 128), (2100, 120, 1, 28, 4, 64), (1900, 60, 3, 56, 8, 64)]


@pytest.mark.parametrize("n,users,m,hq,hkv,D", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("down,size", [(24, -14), (20, -12), (24, -10), (24, -8), (20, 0), (24, 3)])
def test_small_probabilities(n, users, m, hq, hkv, D, dtype, down, size):
    b = Sink(n, users, m, hq, hkv, D, 16, dtype, down, STD[size])
    b.check(*b.run())


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_many_keys(dtype):
    b = Sink(20000, 24, 1, 64, 8, 128, 64, dtype, 22, STD[-12])
    b.check(*b.run())


@pytest.mark.parametrize("n,users,m,hq,hkv,D", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("down", [12, 20])
def test_groups_of_different_sizes(n, users, m, hq, hkv, D, dtype, down):
    """Small values beside large ones of another group lose nothing to them."""
    b = Sink(n, users, m, hq, hkv, D, 32, dtype, down, 1.0)
    w = b.v.float()
    w[..., :32] *= STD[10]
    w[..., 32:64] *= STD[-10]
    b.v.copy_(w.to(dtype))
    b.check(*b.run())


@pytest.mark.parametrize("n,users,m,hq,hkv,D", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_sizes_that_change_along_the_keys(n, users, m, hq, hkv, D, dtype):
    """Scales that grow, shrink, and grow again, by 2^8 and in other places for each group."""
    b = Sink(n, users, m, hq, hkv, D, 16, dtype, 10, 0.05)
    at = torch.arange(n, device="cuda")[:, None, None]
    g = torch.arange(D, device="cuda")[None, None] // 32
    b.v.copy_((b.v.float() * torch.exp2(4.0 * torch.sin(at / 300.0 + 2.0 * g))).to(dtype))
    b.check(*b.run())


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_one_size_or_another_is_the_same_but_for_the_size(dtype):
    """Values 2^-8 or 2^6 as large: the same codes, scales as much smaller or larger, so the
    outputs too, to the bit but where they are subnormal."""
    b = Sink(2000, 60, 1, 64, 8, 128, 16, dtype, 8, 1.0)
    want, lse = b.run()
    v = b.v.clone()
    for e in (-8, 6):
        b.v.copy_(v * 2.0 ** e)
        got, got_lse = b.run()
        fine = got.abs() >= torch.finfo(dtype).tiny
        assert fine.any() and torch.equal(got_lse, lse)
        assert torch.equal(got.float()[fine], (want.float() * 2.0 ** e)[fine])
