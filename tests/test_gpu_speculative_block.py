"""The example that decodes drafts over a 4-bit cache (append, read back, attention,
verification and the rest of the block together) against the same run in plain torch.

The plain form keeps the block's rounding points and holds keys and values as the
definition of the 4-bit cache says, and calls the same moe_layer; what differs is a
few half steps of bf16 (2^-9 relative) carried through the projections, and now and
then a key's code at a border (one step of its group, a tenth of a few values of
thousands): relative Frobenius below 3e-2, the block with a 16-bit cache's 2e-2 and a
half.  Which drafts stand and which tokens follow is a matter of the run's own
probabilities, and has to be equal.
"""
import torch

import dispatch_combine_gb300 as moe
import pytest

from examples.speculative_block import Block4, serve
from tests.gpu_common import ensure_lib
from tests.kv4_common import held
from tests.test_gpu_verify_drafts import want

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def plain_logits(b, tokens, positions, seen):
    """Logits of one sequence's `tokens` after the rows in `seen` (what is held of keys and values)."""
    def norm(v, w):
        v = v.float()
        return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6) * w.float()

    n, x = tokens.shape[0], b.embedding[tokens.long()]
    q, k, v = (t.unflatten(1, (-1, b.D)) for t in (norm(x, b.w_attn).to(BF16) @ b.w_qkv.T).split(
        [b.hq * b.D, b.hkv * b.D, b.hkv * b.D], dim=1))
    t = (positions.double()[:, None] * b.inv_freq.double())[:, None]
    cos, sin = t.cos().float(), t.sin().float()

    def turn(z):
        a, c = z.float().chunk(2, -1)
        return torch.cat([a * cos - c * sin, c * cos + a * sin], -1)

    k, v = held(turn(k))[0].float(), held(v)[0].float()
    ks, vs = (torch.cat([old, z]) for old, z in zip(seen, (k, v))) if seen else (k, v)
    G, before = b.hq // b.hkv, ks.shape[0] - n
    s = torch.einsum("qhd,khd->hqk", turn(q).to(BF16).float(), ks.repeat_interleave(G, 1)) * b.D ** -0.5
    mask = torch.arange(ks.shape[0], device="cuda") > before + torch.arange(n, device="cuda")[:, None]
    p = torch.softmax(s.masked_fill(mask, float("-inf")), -1)
    o = torch.einsum("hqk,khd->qhd", p, vs.repeat_interleave(G, 1)).to(BF16)
    x = x.float() + (o.flatten(1) @ b.w_o.T).float()
    u = norm(x, b.w_ffn).to(BF16)
    shape = dict(b.shape, T=n)
    y = moe.moe_layer(shape, u, b.w_r, b.bias, b.w_gate_up, b.w_down, moe.Workspace(moe.moe_workspace_size(shape)))
    return (x.to(BF16).float() + norm(y, b.w_post)).to(BF16) @ b.w_out.T, (ks, vs)


@pytest.mark.parametrize("users,prompt,steps,n_drafts,kw", [
    (3, 64, 4, 3, dict(hq=8, hkv=2, head_dim=64, page=16)), (2, 128, 3, 1, dict(hq=4, hkv=4, head_dim=128, page=32)),
])
def test_drafted_steps_over_a_4_bit_cache(users, prompt, steps, n_drafts, kw):
    ensure_lib()
    b = Block4(dict(T=0, d=512, E=8, G=2, topk_group=1, k=2, inter=128, score=0), vocab=300, pages=64, **kw)
    words, said, record = serve(b, users, prompt, steps, n_drafts)
    assert b.status() == 0
    arange = lambda n: torch.arange(n, device="cuda")  # noqa: E731
    _, first = plain_logits(b, words, arange(prompt), None)
    stood = [(first, prompt)] * users
    new = 1 + n_drafts
    for r in record:
        acc, out = want(r["target"], r["tokens"].flatten().to(torch.int32), r["uniforms"], r["offsets"], r["draft"])
        assert r["accepted"].tolist() == acc.tolist() and r["out"].tolist() == out.tolist()
        for u in range(users):
            seen, n = stood[u]
            assert int(r["rows"][u]) == n
            ref, after = plain_logits(b, r["tokens"][u], n + arange(new), seen)
            got = r["logits"][u * new:(u + 1) * new].float()
            off = (got - ref.float()).norm() / ref.float().norm()
            assert off < 3e-2, (u, off)
            n += int(r["accepted"][u]) + 1
            stood[u] = tuple(z[:n] for z in after), n
    for u in range(users):
        assert len(said[u]) == 1 + steps + sum(int(r["accepted"][u]) for r in record)


def test_it_runs_as_a_command():
    ensure_lib()
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "examples/speculative_block.py", "--users", "5", "--prompt", "128", "--steps", "3"],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "MOE_OK" in r.stdout, r.stdout + r.stderr
