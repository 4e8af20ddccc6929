"""One MoE decoder block that decodes drafted tokens over a 4-bit cache.

The users of a batch share a prompt.  It is run once and held in 4 bits; a long
chunk like it is read back to 16 bits for its own attention.  Then every step
takes each user's last token and a few drafts of a small drafter:

    norm_in -> q, k, v projection -> kv4_append (rotation, 4-bit paged cache)
            -> kv4_attention (all new tokens of a user at once)
            -> output projection -> norm_out (residual, next norm)
            -> moe_layer -> norm_out -> logits -> verify_drafts

The rows of drafts that fall are written again by the next step's tokens.
Embedding, projections and the drafter (a table of next-token probabilities) are
plain torch.

    python examples/speculative_block.py [--users 16] [--prompt 512] [--steps 8]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import dispatch_combine_gb300 as moe
from examples.decoder_block import Block


class Block4(Block):
    """The block of the other example with its cache in 4 bits, and a vocabulary."""

    def __init__(self, shape, vocab=1000, seed=0, device="cuda", **kw):
        super().__init__(shape, seed=seed, device=device, **kw)
        n = (self.kv.num_pages, self.hkv, moe.moe_kv4_page_bytes(self.kv))
        self.k_cache, self.v_cache = (torch.zeros(n, dtype=torch.uint8, device=device) for _ in range(2))
        g = torch.Generator(device=device).manual_seed(seed + 1)
        d = shape["d"]
        self.embedding = torch.randn(vocab, d, generator=g, device=device).to(torch.bfloat16)
        self.w_out = (torch.randn(vocab, d, generator=g, device=device) * 3 * d ** -0.5).to(torch.bfloat16)
        # the drafter: what the residual stream would say of a token without the block
        self.drafter = torch.softmax((self.embedding @ self.w_out.T).float(), -1)

    def spaces4(self, T, B, max_q):
        key = ("4 bit", T, B, max_q)
        if key not in self.spaces:
            attn = max(moe.moe_kv4_attention_workspace_size(self.kv, T, B, max_q),
                       moe.moe_prefix_attention_workspace_size(self.kv, T, B, max_q, 0))
            self.spaces[key] = (moe.Workspace(attn), moe.Workspace(moe.moe_workspace_size(dict(self.shape, T=T))))
        return self.spaces[key]

    def __call__(self, tokens, positions, slots, table, lens, offsets, max_q, chunk_slots=None):
        """Logits of the new tokens.  chunk_slots: the rows of a whole sequence, to be read
        back for the attention of a long chunk (one sequence)."""
        T = tokens.shape[0]
        ws, ws_moe = self.spaces4(T, lens.shape[0], max_q)
        x = self.embedding[tokens.long()]
        u = moe.moe_norm_in(x, self.w_attn)
        q, k, v = (t.unflatten(1, (-1, self.D)) for t in (u @ self.w_qkv.T).split(
            [self.hq * self.D, self.hkv * self.D, self.hkv * self.D], dim=1))
        q = moe.moe_kv4_append(self.kv, q, k, v, positions, slots, self.inv_freq, self.k_cache, self.v_cache, ws)
        if chunk_slots is None:
            o, _ = moe.moe_kv4_attention(self.kv, q, self.k_cache, self.v_cache, table, lens, ws, q_offsets=offsets,
                                         max_q=max_q)
        else:
            n, page = chunk_slots.shape[0], self.page
            pages = -(-n // page)
            kv = moe.kv_struct(self.hq, self.hkv, self.D, page, pages, torch.bfloat16)
            caches = [torch.zeros(pages, self.hkv, page, self.D, dtype=torch.bfloat16, device=x.device) for _ in range(2)]
            at = torch.arange(n, dtype=torch.int32, device=x.device)
            moe.moe_kv4_read(self.kv, chunk_slots, self.k_cache, self.v_cache, ws, *caches, dst_slots=at)
            o, _ = moe.moe_prefix_attention(kv, q, *caches, None, 0, torch.arange(pages, dtype=torch.int32,
                                                                                  device=x.device)[None].contiguous(),
                                            lens, ws, q_offsets=offsets, max_q=max_q)
        x, u = moe.moe_norm_out(o.flatten(1) @ self.w_o.T, x, next_weight=self.w_ffn)
        y = moe.moe_layer(dict(self.shape, T=T), u, self.w_r, self.bias, self.w_gate_up, self.w_down, ws_moe)
        return moe.moe_norm_out(y, x, post_weight=self.w_post)[0] @ self.w_out.T


def drafts(block, last, n, g):
    """n tokens after each of `last`, drawn one after the other, and the distributions
    that they were drawn from: ([users, 1 + n], [users, 1 + n, vocab], the last unused)."""
    tokens, rows = [last], []
    for _ in range(n):
        rows.append(block.drafter[tokens[-1].long()])
        tokens.append(torch.multinomial(rows[-1], 1, generator=g)[:, 0])
    rows.append(torch.zeros_like(block.drafter[last.long()]))
    return torch.stack(tokens, 1), torch.stack(rows, 1)


def serve(block, users, prompt, steps, n_drafts=3, seed=1):
    """Runs the shared prompt (its length in whole pages), then `steps` drafted steps.
    Returns the decided tokens of each user and, for each step, what went in and out."""
    dev, page = "cuda", block.page
    if prompt % page:
        raise ValueError("prompt: whole pages, which the users share")
    g = torch.Generator(device=dev).manual_seed(seed)
    vocab, new = block.embedding.shape[0], 1 + n_drafts
    n_prompt, n_own = prompt // page, -(-(steps * new) // page)
    ids = torch.arange(n_prompt + users * n_own, dtype=torch.int32, device=dev)
    table = torch.cat([ids[:n_prompt].expand(users, -1), ids[n_prompt:].reshape(users, n_own)], 1).contiguous()

    def i32(*v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    # ---- the prompt
    words = torch.randint(0, vocab, (prompt,), generator=g, device=dev)
    at = torch.arange(prompt, dtype=torch.int32, device=dev)
    logits = block(words, at, at, None, i32(prompt), i32(0, prompt), prompt, chunk_slots=at)
    first = torch.softmax(logits[-1].float(), -1)
    last = torch.multinomial(first, users, replacement=True, generator=g)
    # ---- drafted steps: `rows` cache rows of each user stand
    rows = torch.full((users,), prompt, dtype=torch.int64, device=dev)
    offsets = torch.arange(0, users * new + 1, new, dtype=torch.int32, device=dev)
    said, record = [[t] for t in last.tolist()], []
    for _ in range(steps):
        tokens, q = drafts(block, last, n_drafts, g)
        at = rows[:, None] + torch.arange(new, device=dev)
        slots = table.long().gather(1, at // page) * page + at % page
        logits = block(tokens.flatten(), at.flatten().to(torch.int32), slots.flatten().to(torch.int32), table,
                       (rows + new).to(torch.int32), offsets, new)
        p = torch.softmax(logits.float(), -1)
        u = torch.rand(users * new, generator=g, device=dev)
        accepted, out = moe.moe_verify_drafts(p, tokens.flatten().to(torch.int32), u, offsets, draft=q.flatten(0, 1),
                                              ws=block.spaces4(users * new, users, new)[0])
        record.append(dict(tokens=tokens, rows=rows.clone(), logits=logits, target=p, draft=q.flatten(0, 1), uniforms=u,
                           offsets=offsets, accepted=accepted, out=out))
        last = out.view(users, new).gather(1, accepted.long()[:, None])[:, 0].long()
        rows = rows + accepted + 1
        for b, (n, row) in enumerate(zip(accepted.tolist(), out.view(users, new).tolist())):
            said[b] += row[:n + 1]
    return words, said, record


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--users", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=512)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    block = Block4(dict(T=0, d=1024, E=16, G=4, topk_group=2, k=2, inter=512, score=0))
    _, said, record = serve(block, a.users, a.prompt, a.steps)
    torch.cuda.synchronize()
    status = block.status()
    stood = torch.stack([r["accepted"] for r in record]).float().mean().item()
    print(f"{a.steps} steps of {a.users} users behind a prompt of {a.prompt}: {sum(map(len, said))} tokens, "
          f"{stood:.2f} of 3 drafts a step stood, device status {moe.moe_status_string(status)}")
    return 0 if status == 0 and all(bool(torch.isfinite(r["logits"]).all()) for r in record) else 1


if __name__ == "__main__":
    sys.exit(main())
