"""One MoE decoder block served to a batch that shares a prompt.

The shared prompt is run once and its keys and values stay in the paged cache;
then every user of the batch decodes tokens of their own behind it:

    norm_in -> q, k, v projection -> kv_append (rotation, paged cache)
            -> prefix_attention (prompt read once for all users)
            -> output projection -> norm_out (residual, next norm)
            -> moe_layer -> norm_out (residual)

The projections are plain torch matrix products.  A decode step is captured
into a CUDA graph once and replayed; positions, slots and lengths change on the
device between replays.

    python examples/decoder_block.py [--users 64] [--prompt 500] [--steps 8]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import dispatch_combine_gb300 as moe


class Block:
    """Random weights of one decoder block, its cache and its workspaces."""

    def __init__(self, shape, hq=16, hkv=4, head_dim=128, page=64, pages=1024, seed=0,
                 device="cuda"):
        self.shape, d = dict(shape), shape["d"]
        self.hq, self.hkv, self.D, self.page = hq, hkv, head_dim, page
        g = torch.Generator(device=device).manual_seed(seed)

        def w(*s, std):
            return (torch.randn(*s, generator=g, device=device) * std).to(torch.bfloat16)

        E, inter = shape["E"], shape["inter"]
        self.w_qkv = w((hq + 2 * hkv) * head_dim, d, std=d ** -0.5)
        self.w_o = w(d, hq * head_dim, std=(hq * head_dim) ** -0.5)
        self.w_r, self.bias = w(d, E, std=0.02), torch.randn(E, generator=g, device=device)
        self.w_gate_up, self.w_down = w(E, 2 * inter, d, std=d ** -0.5), w(E, d, inter, std=inter ** -0.5)
        self.w_attn, self.w_ffn, self.w_post = (1 + w(d, std=0.1) for _ in range(3))
        self.inv_freq = 10000.0 ** (-torch.arange(0, head_dim, 2, device=device,
                                                  dtype=torch.float32) / head_dim)
        self.kv = moe.kv_struct(hq, hkv, head_dim, page, pages, torch.bfloat16)
        self.k_cache = torch.zeros(pages, hkv, page, head_dim, dtype=torch.bfloat16, device=device)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.spaces = {}

    def workspaces(self, T, B, max_q, prefix):
        key = (T, B, max_q, prefix)
        if key not in self.spaces:
            s = dict(self.shape, T=T)
            self.spaces[key] = (
                moe.Workspace(moe.moe_prefix_attention_workspace_size(self.kv, T, B, max_q, prefix)),
                moe.Workspace(moe.moe_workspace_size(s)))
        return self.spaces[key]

    def __call__(self, x, positions, slots, prefix_pages, prefix, table, lens, offsets=None,
                 max_q=1):
        """x [T,d] -> the block's output [T,d] (the residual stream)."""
        T = x.shape[0]
        ws_attn, ws_moe = self.workspaces(T, lens.shape[0], max_q, prefix)
        u = moe.moe_norm_in(x, self.w_attn)
        qkv = u @ self.w_qkv.T
        q, k, v = (t.unflatten(1, (-1, self.D)) for t in qkv.split(
            [self.hq * self.D, self.hkv * self.D, self.hkv * self.D], dim=1))
        q = moe.moe_kv_append(self.kv, q, k, v, positions, slots, self.inv_freq, self.k_cache,
                              self.v_cache, ws_attn)
        o, _ = moe.moe_prefix_attention(self.kv, q, self.k_cache, self.v_cache, prefix_pages,
                                        prefix, table, lens, ws_attn, q_offsets=offsets,
                                        max_q=max_q)
        x, u = moe.moe_norm_out(o.flatten(1) @ self.w_o.T, x, next_weight=self.w_ffn)
        y = moe.moe_layer(dict(self.shape, T=T), u, self.w_r, self.bias, self.w_gate_up,
                          self.w_down, ws_moe)
        return moe.moe_norm_out(y, x, post_weight=self.w_post)[0]

    def status(self):
        return max(moe.moe_get_device_status(w) for pair in self.spaces.values() for w in pair)


def serve(block, users, prompt, steps, seed=1, graph=True):
    """Runs the shared prompt, then `steps` tokens of every user.  Returns the
    prompt's outputs [prompt, d] and the users' [steps, users, d]."""
    dev, page, d = "cuda", block.page, block.shape["d"]
    g = torch.Generator(device=dev).manual_seed(seed)
    n_prompt, n_own = -(-prompt // page), -(-steps // page)
    ids = torch.arange(n_prompt + users * n_own, dtype=torch.int32, device=dev)
    prompt_pages, table = ids[:n_prompt], ids[n_prompt:].reshape(users, n_own).contiguous()

    def rows(pages, at):  # cache rows of positions `at` in a run of pages
        return pages.gather(-1, at // page) * page + (at % page).to(torch.int32)

    # ---- the prompt: one sequence, whose own rows become the others' prefix
    x = torch.randn(prompt, d, generator=g, device=dev).to(torch.bfloat16)
    at = torch.arange(prompt, device=dev)
    out_prompt = block(x, at.to(torch.int32), rows(prompt_pages, at), None, 0,
                       prompt_pages[None].contiguous(),
                       torch.tensor([prompt], dtype=torch.int32, device=dev),
                       torch.tensor([0, prompt], dtype=torch.int32, device=dev), max_q=prompt)
    # ---- decode: buffers that a captured step reads
    x = torch.empty(users, d, dtype=torch.bfloat16, device=dev)
    positions = torch.empty(users, dtype=torch.int32, device=dev)
    slots, lens = torch.empty_like(positions), torch.empty_like(positions)
    inputs = torch.randn(steps, users, d, generator=g, device=dev).to(torch.bfloat16)
    outputs = torch.empty_like(inputs)
    captured, y = None, None
    for i in range(steps):
        x.copy_(inputs[i])
        positions.fill_(prompt + i)
        slots.copy_(rows(table, torch.full((users, 1), i, device=dev))[:, 0])
        lens.fill_(i + 1)
        if captured is not None:
            captured.replay()
        else:
            y = block(x, positions, slots, prompt_pages, prompt, table, lens)
            if graph:  # the same step again, as a graph: it rewrites the same rows
                torch.cuda.synchronize()
                captured = torch.cuda.CUDAGraph()
                with torch.cuda.graph(captured):
                    y = block(x, positions, slots, prompt_pages, prompt, table, lens)
                captured.replay()
        outputs[i] = y
    return out_prompt, outputs


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--users", type=int, default=64)
    ap.add_argument("--prompt", type=int, default=500)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    block = Block(dict(T=0, d=1024, E=16, G=4, topk_group=2, k=2, inter=512, score=0))
    _, out = serve(block, a.users, a.prompt, a.steps)
    torch.cuda.synchronize()
    status = block.status()
    print(f"{a.steps} tokens of {a.users} users behind a prompt of {a.prompt}: "
          f"device status {moe.moe_status_string(status)}, output rms "
          f"{out.float().square().mean().sqrt().item():.3f}")
    return 0 if status == 0 and bool(torch.isfinite(out).all()) else 1


if __name__ == "__main__":
    sys.exit(main())
