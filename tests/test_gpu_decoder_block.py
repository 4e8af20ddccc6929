"""The example block (norms, cache append, shared-prefix attention and the MoE
layer together) against the same block in plain torch.

The plain form keeps the block's own rounding points (bf16 projections, cache
and layer input), takes norms, rotation and attention in fp32 and calls the same
moe_layer, so what differs is a few half steps of bf16 (2^-9 relative) carried
through the projections: relative Frobenius below 2e-2.
"""
import torch

import dispatch_combine_gb300 as moe
import pytest

from examples.decoder_block import Block, serve
from tests.gpu_common import ensure_lib

pytestmark = pytest.mark.gpu
SHAPE = dict(T=0, d=512, E=8, G=2, topk_group=1, k=2, inter=128, score=0)


def plain_block(b, xs, positions, seen):
    """xs [n,d] of one sequence at `positions`, after the rows already in
    `seen` (a list of rotated k and v, extended here)."""
    def norm(v, w):
        v = v.float()
        return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6) * w.float()

    n = xs.shape[0]
    qkv = norm(xs, b.w_attn).to(torch.bfloat16) @ b.w_qkv.T
    q, k, v = (t.unflatten(1, (-1, b.D)) for t in qkv.split(
        [b.hq * b.D, b.hkv * b.D, b.hkv * b.D], dim=1))
    t = (positions.double()[:, None] * b.inv_freq.double())[:, None]
    cos, sin = t.cos().float(), t.sin().float()

    def turn(z):
        a, c = z.float().chunk(2, -1)
        return torch.cat([a * cos - c * sin, c * cos + a * sin], -1).to(torch.bfloat16)

    ks = torch.cat([seen[0], turn(k)]) if seen else turn(k)
    vs = torch.cat([seen[1], v]) if seen else v
    G, before = b.hq // b.hkv, ks.shape[0] - n
    s = torch.einsum("qhd,khd->hqk", turn(q).float(),
                     ks.float().repeat_interleave(G, 1)) * b.D ** -0.5
    mask = torch.arange(ks.shape[0], device="cuda") > before + torch.arange(n, device="cuda")[:, None]
    p = torch.softmax(s.masked_fill(mask, float("-inf")), -1)
    o = torch.einsum("hqk,khd->qhd", p, vs.float().repeat_interleave(G, 1)).to(torch.bfloat16)
    x = xs.float() + (o.flatten(1) @ b.w_o.T).float()
    u = norm(x, b.w_ffn).to(torch.bfloat16)
    x = x.to(torch.bfloat16)
    shape = dict(b.shape, T=n)
    y = moe.moe_layer(shape, u, b.w_r, b.bias, b.w_gate_up, b.w_down,
                      moe.Workspace(moe.moe_workspace_size(shape)))
    return (x.float() + norm(y, b.w_post)).to(torch.bfloat16), (ks, vs)


@pytest.mark.parametrize("users,prompt,steps,graph", [(5, 75, 3, True), (33, 300, 2, False)])
def test_block_serves_users_behind_a_shared_prompt(users, prompt, steps, graph):
    ensure_lib()
    b = Block(SHAPE, hq=8, hkv=2, head_dim=64, page=16, pages=256)
    out_prompt, out = serve(b, users, prompt, steps, graph=graph)
    torch.cuda.synchronize()
    assert b.status() == 0

    g = torch.Generator(device="cuda").manual_seed(1)     # serve()'s own draws
    x = torch.randn(prompt, SHAPE["d"], generator=g, device="cuda").to(torch.bfloat16)
    inputs = torch.randn(steps, users, SHAPE["d"], generator=g, device="cuda").to(torch.bfloat16)
    want, seen = plain_block(b, x, torch.arange(prompt, device="cuda"), None)

    def far(got, ref):
        return ((got.float() - ref.float()).norm() / ref.float().norm()).item()

    assert far(out_prompt, want) < 2e-2
    for user in (0, users // 2, users - 1):
        mine = seen
        for i in range(steps):
            ref, mine = plain_block(b, inputs[i, user:user + 1],
                                    torch.tensor([prompt + i], device="cuda"), mine)
            assert far(out[i, user:user + 1], ref) < 2e-2
