"""moe_verify_drafts against its definition.  Weights are counted here as whole
numbers of 2^-60 too (int64 sums, the border from exact fractions), so every token
has to be equal."""
from fractions import Fraction

import pytest
import torch

import dispatch_combine_gb300 as moe
from tests.gpu_common import ensure_lib

pytestmark = pytest.mark.gpu
FP32, BF16, FP16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _lib():
    ensure_lib()


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def probs(T, V, seed, dtype=FP32, spread=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.softmax(torch.randn(T, V, generator=g, device="cuda") * spread, -1).to(dtype)


def first_past(w, u):
    """The first index at which the running sum of weights passes u times the whole; None: all zero."""
    n = (w.float().nan_to_num(0.0, posinf=1.0).clamp(0, 1).double() * 2.0 ** 60).to(torch.int64).cpu()
    cum = n.cumsum(0)
    total = int(cum[-1])
    if total == 0:
        return None
    border = min(Fraction(max(u, 0.0)) * total // 1, total - 1)
    return int((cum <= border).sum())


def want(target, tokens, uniforms, offsets, draft):
    T, V = target.shape
    out, accepted = torch.full((T,), -1, dtype=torch.int32), []
    tok, u, off = tokens.tolist(), uniforms.tolist(), offsets.tolist()
    for q0, q1 in zip(off, off[1:]):
        if q1 == q0:
            accepted.append(0)
            continue
        n = q1 - q0 - 1
        a = 0
        while a < n:
            x = tok[q0 + a + 1]
            if not 0 <= x < V:
                break
            p, q = float(target[q0 + a, x]), 1.0 if draft is None else float(draft[q0 + a, x])
            if not Fraction(u[q0 + a]) * Fraction(q) < Fraction(p):
                break
            out[q0 + a] = x
            a += 1
        accepted.append(a)
        row = target[q0 + a].float()
        w = row.clone()
        if a < n:
            if draft is not None:
                w = row - draft[q0 + a].float()
            elif 0 <= tok[q0 + a + 1] < V:
                w[tok[q0 + a + 1]] = 0.0
        v = first_past(w, u[q1 - 1])
        if v is None:
            v = first_past(row, u[q1 - 1])
        out[q0 + a] = 0 if v is None else v
    return torch.tensor(accepted, dtype=torch.int32), out


def check(target, tokens, uniforms, offsets, draft, status=0, **kw):
    ws = moe.Workspace(256)
    out = torch.full((target.shape[0],), -5, dtype=torch.int32, device="cuda")
    acc, out = moe.moe_verify_drafts(target, tokens, uniforms, offsets, draft=draft, ws=ws, out_tokens=out, **kw)
    wa, wo = want(target, tokens, uniforms, offsets, draft)
    assert acc.cpu().tolist() == wa.tolist()
    rows = slice(0, int(offsets[-1]))
    assert out[rows].cpu().tolist() == wo[rows].tolist()
    assert (out[int(offsets[-1]):] == -5).all()        # rows behind the last sequence
    assert moe.moe_get_device_status(ws) == status
    return acc


def batch(counts, V, seed, dtype, greedy=False, near=0.7):
    T = sum(counts)
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn(T, V, generator=g, device="cuda") * 2
    target = torch.softmax(logits, -1).to(dtype)
    drafter = torch.softmax(logits + near * torch.randn(T, V, generator=g, device="cuda"), -1)
    drawn = drafter.argmax(-1) if greedy else torch.multinomial(drafter, 1, generator=g)[:, 0]
    off = torch.tensor([sum(counts[:b]) for b in range(len(counts) + 1)], dtype=torch.int32, device="cuda")
    u = torch.rand(T, generator=g, device="cuda")
    return target, drawn.roll(1).to(torch.int32), u, off, None if greedy else drafter.to(dtype)


@pytest.mark.parametrize("V", [1, 2, 31, 33, 257, 1000, 32000, 50021, 131072])
@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("greedy", [False, True])
def test_ragged_batch(V, dtype, greedy):
    counts = [5, 1, 0, 8, 2, 1, 3, 0]
    for seed in range(3):
        check(*batch(counts, V, seed + V, dtype, greedy))


def test_many_drafts_and_many_sequences():
    acc = check(*batch([70, 40, 33], 500, 1, FP32, near=0.02))
    assert acc.max() > 20            # past one warp's drafts
    check(*batch([1 + b % 4 for b in range(300)], 129, 2, FP32))
    check(*batch([1] * 700, 64, 3, BF16, True))
    for n in (80, 160, 310):         # clusters of 4, 2 and 1 where rows are long enough for more
        check(*batch([1 + b % 2 for b in range(n)], 9001, n, FP32))


def test_rows_with_strides_and_room_behind():
    target, tokens, u, off, draft = batch([4, 3, 2], 1001, 5, FP32)
    wide = torch.full((12, 2 * 1001 + 9), 0.5, device="cuda")
    wide[:9, 3:1004], wide[:9, 1005:2006] = target, draft
    more = torch.cat([tokens, i32(4, 4, 4)])
    check(wide[:, 3:1004], more, torch.cat([u, u[:3]]), off, wide[:, 1005:2006])


def test_borders_are_exact():
    """u q = p falls, one step less stands; sums met exactly go on to the next token."""
    V = 64
    target, draft = torch.zeros(4, V, device="cuda"), torch.zeros(4, V, device="cuda")
    target[0, 5], draft[0, 5] = 0.25, 0.5
    target[0, 9], target[0, 10], draft[0, 9] = 0.5, 0.25, 0.5
    target[1:, 3], target[1:, 40] = 0.5, 0.5
    off = i32(0, 2)
    for u0, stands in ((0.5, 0), (0.5 - 2.0 ** -25, 1), (0.0, 1)):
        acc = check(target[:2], i32(1, 5), torch.tensor([u0, 0.5], device="cuda"), off, draft[:2])
        assert acc.item() == stands
    for u, token in ((0.0, 3), (0.5 - 2.0 ** -25, 3), (0.5, 40), (1 - 2.0 ** -24, 40)):
        _, out = moe.moe_verify_drafts(target[1:2].contiguous(), i32(1), torch.tensor([u], device="cuda"), i32(0, 1))
        assert out.item() == token
        check(target[1:2].contiguous(), i32(1), torch.tensor([u], device="cuda"), i32(0, 1), None)


def test_tiny_and_odd_weights():
    V = 3000
    target = probs(6, V, 3, spread=12.0)          # down to fp32's subnormals
    target[0, 7], target[1, 8], target[2, 9] = float("nan"), -0.5, float("inf")
    draft = probs(6, V, 4, spread=12.0)
    draft[3] = target[3]                          # nothing is left of the difference
    target[4], draft[4] = 0.0, 0.0                # nor of the target
    off = i32(0, 2, 4, 6)
    for u in (0.0, 1e-9, 0.3, 0.999999):
        check(target, i32(1, 5, 2, 6, 2, 6), torch.full((6,), u, device="cuda"), off, draft)
    check(target, i32(1, 5, 2, 6, 2, 6), torch.full((6,), 1.0, device="cuda"), off, draft)


def test_certain_rows():
    V = 40000
    for at in (0, 1, 31, 32, 5000, V - 1):
        target = torch.zeros(1, V, device="cuda")
        target[0, at] = 1.0
        for u in (0.0, 0.5, 1 - 2.0 ** -24):
            check(target, i32(0), torch.tensor([u], device="cuda"), i32(0, 1), None)


def test_bad_tokens_and_offsets_are_reported():
    target, tokens, u, off, draft = batch([3, 3], 100, 5, FP32)
    for bad in (-1, 100, 2 ** 31 - 1):
        t = tokens.clone()
        t[1] = bad
        acc = check(target, t, u, off, draft, status=1)
        assert acc[0] == 0
        check(target, t, u, off, None, status=1)
    ws = moe.Workspace(256)
    for bad in ([0, 4, 3], [-1, 3, 6], [0, 3, 7]):
        buf = torch.full((10,), -5, dtype=torch.int32, device="cuda")
        moe.moe_verify_drafts(target, tokens, u, i32(*bad), draft=draft, ws=ws, out_tokens=buf[2:8])
        assert moe.moe_get_device_status(ws) == 1
        assert (buf[:2] == -5).all() and (buf[8:] == -5).all()
    moe.moe_verify_drafts(target, tokens, u, i32(0, 4, 3), draft=draft)      # nobody to report to


def test_nothing_to_do():
    target, tokens, u, off, draft = batch([3], 100, 5, FP32)
    acc, out = moe.moe_verify_drafts(target, tokens, u, i32(0), draft=draft)
    assert acc.shape == (0,)
    acc, out = moe.moe_verify_drafts(target[:0], tokens[:0], u[:0], i32(0, 0, 0))
    assert acc.tolist() == [0, 0] and out.shape == (0,)


def test_distribution():
    """What is kept is distributed as the target's samples: 40000 sequences of one draft over 8 tokens.
    A share's standard deviation is at most 0.5 / 200 = 0.0025: five of them."""
    n, V = 40000, 8
    p, q = probs(1, V, 1, spread=1.0), probs(1, V, 2, spread=1.0)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.multinomial(q[0], n, replacement=True, generator=g)
    tokens = torch.stack([torch.zeros_like(x), x], 1).reshape(-1).to(torch.int32)
    u = torch.rand(2 * n, generator=g, device="cuda")
    off = torch.arange(0, 2 * n + 1, 2, device="cuda", dtype=torch.int32)
    rows = lambda r: r.expand(2 * n, V).contiguous()  # noqa: E731
    acc, out = moe.moe_verify_drafts(rows(p), tokens, u, off, draft=rows(q))
    share = torch.bincount(out[::2].long(), minlength=V).double() / n
    assert ((share - p[0].double()).abs() < 0.0125).all()
    assert abs(acc.double().mean().item() - torch.minimum(p, q).sum().item()) < 0.0125


def test_capture_and_replay():
    target, tokens, u, off, draft = batch([4, 2, 7], 5000, 5, BF16)
    acc, out = moe.moe_verify_drafts(target, tokens, u, off, draft=draft)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_verify_drafts(target, tokens, u, off, draft=draft, accepted=acc, out_tokens=out)
    for seed in range(3):
        u.copy_(torch.rand(13, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        wa, wo = want(target, tokens, u, off, draft)
        assert acc.tolist() == wa.tolist() and out.tolist() == wo.tolist()
