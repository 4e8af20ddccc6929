"""What is measured of the operators around the MoE layer: the norms before and
after a block, the append to the paged key/value cache, and the attention of a
batch that shares a long prefix.

``run`` computes one pass in elementary torch operations, or with the
framework's own operators where ``own`` is true.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one token of one user: the norm in front of a block, pure latency
        dict(name="norm_in_one_token", op="norm_in", T=1, d=7168, kind="rms", bias=False, dtype="bf16"),
        # a prefill step of 16384 tokens
        dict(name="norm_in_prefill", op="norm_in", T=16384, d=7168, kind="rms", bias=False, dtype="bf16"),
        # a decode step: norm after the block, residual, norm before the next block
        dict(name="norm_out_decode", op="norm_out", T=512, d=7168, kind="rms", bias=False, dtype="bf16",
             post=True, gate="none", scale=1.0, next=True),
        # an odd batch of a LayerNorm model whose blocks are gated per token
        dict(name="norm_out_layer_odd", op="norm_out", T=1021, d=4104, kind="layer", bias=True, dtype="fp16",
             post=True, gate="token", scale=0.5, next=True),
        # prefill with a learned scale for each channel of the block's output
        dict(name="norm_out_prefill", op="norm_out", T=16384, d=7168, kind="rms", bias=False, dtype="bf16",
             post=True, gate="channel", scale=1.0, next=True),
        # a decode step's new tokens, one for each of 64 sequences
        dict(name="append_decode", op="append", T=64, hq=64, hkv=8, D=128, page=64, rot=128, style="half",
             pad=0, far=131072, dtype="bf16"),
        # a ragged small batch padded to a captured size, interleaved pairs, half of each head rotated
        dict(name="append_padded_odd", op="append", T=333, hq=28, hkv=4, D=64, page=16, rot=32, style="pairs",
             pad=13, far=1000000, dtype="fp16"),
        # a prefill step of 16384 tokens
        dict(name="append_prefill", op="append", T=16384, hq=64, hkv=8, D=128, page=64, rot=128, style="half",
             pad=0, far=32768, dtype="bf16"),
        # one user, a short system prompt, the first tokens of the answer
        dict(name="attend_one_token", op="attend", B=1, q=1, hq=64, hkv=8, D=128, page=64, prefix=1000, own=9,
             dtype="bf16"),
        # drafted tokens checked for a ragged batch: several queries for each sequence, 7 heads to a key head
        dict(name="attend_drafts_odd", op="attend", B=37, q=6, hq=28, hkv=4, D=64, page=16, prefix=4099, own=777,
             dtype="fp16"),
        # 64 users of one assistant: a prompt of 8192 tokens, up to 1024 tokens of their own
        dict(name="attend_decode", op="attend", B=64, q=1, hq=64, hkv=8, D=128, page=64, prefix=8192, own=1024,
             dtype="bf16"),
        # 256 users asking about one long document
        dict(name="attend_long_prefix", op="attend", B=256, q=1, hq=64, hkv=8, D=128, page=64, prefix=32768, own=512,
             dtype="bf16"),
    ]


def _between(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_in", "norm_out", "append", "attend"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op in ("norm_in", "norm_out"):
        kind = rng.choice(["rms", "layer"])
        d = 8 * _between(rng, 16, 1024)
        case = dict(op=op, T=_between(rng, 1, min(16384, 16384 * 7168 // d)), d=d, kind=kind, bias=kind == "layer",
                    dtype=dtype)
        if op == "norm_out":
            case.update(post=rng.random() < 0.7, gate=rng.choice(["none", "channel", "token", "full"]),
                        scale=rng.choice([1.0, 0.5, 0.25]), next=rng.random() < 0.8)
            case["T"] = max(1, min(case["T"], 12288 * 7168 // d))
        return case
    D, hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    G, page = rng.choice([1, 2, 4, 5, 7, 8, 16]), rng.choice([16, 32, 64, 128])
    G = min(G, 64 // hkv)
    if op == "append":
        T = _between(rng, 1, 8192)
        return dict(op=op, T=T, hq=G * hkv, hkv=hkv, D=D, page=page, rot=rng.choice([D, D // 2]),
                    style=rng.choice(["half", "pairs"]), pad=rng.randrange(0, min(T, 17)),
                    far=_between(rng, 64, 1000000), dtype=dtype)
    q = rng.choice([1, 1, 1, 2, 5, _between(rng, 6, 64)])
    B = _between(rng, 1, 256)
    B = max(1, min(B, 256 // q))
    prefix = rng.choice([0, _between(rng, 1, 32768), _between(rng, 1024, 32768)])
    return dict(op=op, B=B, q=q, hq=G * hkv, hkv=hkv, D=D, page=page, prefix=prefix, own=_between(rng, 1, 1024),
                dtype=dtype)


def _lengths(case):
    """Queries and own (non-shared) length of each sequence: ragged, up to q and own, the same for every seed."""
    rng = random.Random("%d %d %d %d" % (case["B"], case["q"], case["own"], case["prefix"]))
    qs, lens = [], []
    for b in range(case["B"]):
        n = case["q"] if b == 0 else rng.randint(1, case["q"])
        qs.append(n)
        lens.append(max(n, case["own"] if b == 0 else rng.randint(1, case["own"])))
    return qs, lens


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device=dev) * std + mean).to(dt)

    s = dict(case)
    if case["op"] in ("norm_in", "norm_out"):
        T, d = case["T"], case["d"]
        # a residual stream: some channels far larger than the others
        loud = torch.where(torch.rand(d, generator=g, device=dev) < 0.01, 30.0, 1.0)
        s["x"] = (torch.randn(T, d, generator=g, device=dev) * loud).to(dt)
        s["w"], s["b"] = normal(d, std=0.2, mean=1.0), normal(d, std=0.1) if case["bias"] else None
        if case["op"] == "norm_out":
            s["f"] = normal(T, d, std=0.3)
            s["pw"], s["pb"] = (normal(d, std=0.2, mean=1.0), normal(d, std=0.1) if case["bias"] else None) \
                if case["post"] else (None, None)
            shape = {"none": None, "channel": (d,), "token": (T, 1), "full": (T, d)}[case["gate"]]
            s["gate"] = None if shape is None else normal(*shape, std=0.3, mean=0.5)
            s["x_out"] = torch.empty_like(s["x"])
        s["out"] = torch.empty_like(s["x"])
        return s
    hq, hkv, D, page = case["hq"], case["hkv"], case["D"], case["page"]
    if case["op"] == "append":
        T = case["T"]
        pages = -(-T // page) + 3
        # a projection's output: queries, keys and values of a token side by side
        qkv = normal(T, (hq + 2 * hkv) * D)
        s["q"] = qkv[:, :hq * D].unflatten(1, (hq, D))
        s["k"] = qkv[:, hq * D:(hq + hkv) * D].unflatten(1, (hkv, D))
        s["v"] = qkv[:, (hq + hkv) * D:].unflatten(1, (hkv, D))
        s["positions"] = torch.randint(0, case["far"], (T,), generator=g, device=dev, dtype=torch.int32)
        slots = torch.randperm(pages * page, generator=g, device=dev)[:T].to(torch.int32)
        if case["pad"]:
            slots[-case["pad"]:] = -1
        s["slots"] = slots
        s["inv_freq"] = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float32) / case["rot"])
        s["k_cache"], s["v_cache"] = normal(pages, hkv, page, D), normal(pages, hkv, page, D)
        s["q_out"] = torch.empty(T, hq, D, dtype=dt, device=dev)
        nbytes = 256
    else:
        qs, lens = _lengths(case)
        B, T, prefix = case["B"], sum(qs), case["prefix"]
        n_prefix, n_own = -(-prefix // page), -(-max(lens) // page)
        pages = n_prefix + B * n_own
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        s["prefix_pages"], s["page_table"] = order[:n_prefix].contiguous(), order[n_prefix:].reshape(B, n_own).contiguous()
        s["k_cache"], s["v_cache"] = normal(pages, hkv, page, D), normal(pages, hkv, page, D)
        s["query"] = normal(T, hq, D, std=1.5)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["offsets"] = torch.tensor([sum(qs[:b]) for b in range(B + 1)], dtype=torch.int32, device=dev)
        s["out"], s["lse"] = torch.empty(T, hq, D, dtype=dt, device=dev), torch.empty(T, hq, device=dev)
    if own:
        import dispatch_combine_gb300 as moe
        s["heads"] = moe.kv_struct(num_q_heads=hq, num_kv_heads=hkv, head_dim=D, page_size=page, num_pages=pages,
                                   dtype=dt)
        if case["op"] == "attend":
            nbytes = moe.moe_prefix_attention_workspace_size(s["heads"], T, B, case["q"], prefix)
        s["ws"] = moe.Workspace(nbytes)
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

EPS = 1e-6


def _norm(v, w, b, kind):
    if kind == "layer":
        v = v - v.mean(dim=-1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(dim=-1, keepdim=True) + EPS) * w.float()
    return v if b is None else v + b.float()


def _plain_norm_out(s):
    v = s["f"].float()
    if s["pw"] is not None:
        v = _norm(v, s["pw"], s["pb"], s["kind"])
    if s["gate"] is not None:
        v = v * s["gate"].float()
    r = s["x"].float() * s["scale"] + v
    return (r.to(s["x"].dtype), _norm(r, s["w"], s["b"], s["kind"]).to(s["x"].dtype) if s["next"] else None)


def _rotated(v, cos, sin, rot, style):
    a, b = (v[..., :rot // 2], v[..., rot // 2:rot]) if style == "half" else (v[..., 0:rot:2], v[..., 1:rot:2])
    x, y = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat([x, y], -1) if style == "half" else torch.stack([x, y], -1).flatten(-2)
    return torch.cat([turned, v[..., rot:]], -1)


def _plain_append(s):
    dt, page, slots = s["k_cache"].dtype, s["page"], s["slots"].long()
    angle = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _rotated(s["q"].float(), cos, sin, s["rot"], s["style"]).to(dt)
    k = _rotated(s["k"].float(), cos, sin, s["rot"], s["style"]).to(dt)
    # a padding token (slot -1) writes what token 0 writes, where token 0 writes it
    real = slots >= 0
    at = torch.where(real, slots, slots[0])
    real = real[:, None, None]
    s["k_cache"][at // page, :, at % page] = torch.where(real, k, k[:1])
    s["v_cache"][at // page, :, at % page] = torch.where(real, s["v"], s["v"][:1])
    return q, s["k_cache"], s["v_cache"]


def _plain_attend(s):
    hq, hkv, D, B, nq = s["hq"], s["hkv"], s["D"], s["B"], s["q"]
    G, scale = hq // hkv, s["D"] ** -0.5
    query, off, lens = s["query"].float(), s["offsets"].long(), s["lens"].long()
    T = query.shape[0]
    # queries padded to [B, nq], and where each token sits there
    step = torch.arange(nq, device=query.device)
    count = off[1:] - off[:-1]
    padded = query[(off[:-1, None] + step).clamp(max=T - 1)].reshape(B, nq, hkv, G, D)
    token = torch.arange(T, device=query.device)
    seq = (token[:, None] >= off[None, 1:]).sum(-1)
    place = token - off[seq]

    def rows(cache, pages):  # [..., n] page numbers -> [..., hkv, n * page, D]
        return cache[pages.long()].float().movedim(-3, -4).flatten(-3, -2)

    own_k, own_v = rows(s["k_cache"], s["page_table"]), rows(s["v_cache"], s["page_table"])
    pre_k = rows(s["k_cache"], s["prefix_pages"])[:, :s["prefix"]]
    pre_v = rows(s["v_cache"], s["prefix_pages"])[:, :s["prefix"]]
    by_head = padded.permute(2, 0, 1, 3, 4)  # [hkv, B, nq, G, D]
    pre = (by_head.reshape(hkv, -1, D) @ pre_k.transpose(-1, -2)).reshape(hkv, B, nq, G, -1) * scale
    mine = (padded.permute(0, 2, 1, 3, 4).reshape(B, hkv, nq * G, D) @ own_k.transpose(-1, -2)) * scale
    mine = mine.reshape(B, hkv, nq, G, -1)
    limit = lens[:, None] - count[:, None] + step + 1  # [B, nq]
    seen = torch.arange(mine.shape[-1], device=query.device) < limit[..., None]
    mine = mine.masked_fill(~seen[:, None, :, None, :], -math.inf).permute(1, 0, 2, 3, 4)
    top = mine.amax(-1, keepdim=True)
    if s["prefix"]:
        top = torch.maximum(top, pre.amax(-1, keepdim=True))
    top = top.clamp(min=-1e30)  # a row that sees nothing
    pre, mine = torch.exp(pre - top), torch.exp(mine - top)
    total = pre.sum(-1, keepdim=True) + mine.sum(-1, keepdim=True)
    o = (pre.reshape(hkv, B * nq * G, -1) @ pre_v).reshape(hkv, B, nq, G, D)
    own_o = mine.permute(1, 0, 2, 3, 4).reshape(B, hkv, nq * G, -1) @ own_v
    o = o + own_o.reshape(B, hkv, nq, G, D).permute(1, 0, 2, 3, 4)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + torch.log(total))[..., 0]
    o, lse = o.permute(1, 2, 0, 3, 4).reshape(B, nq, hq, D), lse.permute(1, 2, 0, 3).reshape(B, nq, hq)
    return o[seq, place].to(s["query"].dtype), lse[seq, place]


def _own(s):
    import dispatch_combine_gb300 as moe
    if s["op"] in ("norm_in", "norm_out"):
        kind = moe.MOE_NORM_RMS if s["kind"] == "rms" else moe.MOE_NORM_LAYER
        if s["op"] == "norm_in":
            return moe.moe_norm_in(s["x"], s["w"], s["b"], kind=kind, eps=EPS, out=s["out"])
        return moe.moe_norm_out(s["f"], s["x"], post_weight=s["pw"], post_bias=s["pb"], gate=s["gate"],
                                residual_scale=s["scale"], next_weight=s["w"] if s["next"] else None,
                                next_bias=s["b"] if s["next"] else None, kind=kind, eps=EPS, x_out=s["x_out"],
                                next_out=s["out"] if s["next"] else None)
    if s["op"] == "append":
        style = moe.MOE_ROPE_HALF if s["style"] == "half" else moe.MOE_ROPE_PAIRS
        q = moe.moe_kv_append(s["heads"], s["q"], s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"],
                              s["k_cache"], s["v_cache"], s["ws"], style=style, q_out=s["q_out"])
        return q, s["k_cache"], s["v_cache"]
    return moe.moe_prefix_attention(s["heads"], s["query"], s["k_cache"], s["v_cache"], s["prefix_pages"], s["prefix"],
                                    s["page_table"], s["lens"], s["ws"], q_offsets=s["offsets"], max_q=s["q"],
                                    out=s["out"], lse=s["lse"])


def run(state):
    if own:
        return _own(state)
    if state["op"] == "norm_in":
        return _norm(state["x"].float(), state["w"], state["b"], state["kind"]).to(state["x"].dtype)
    return {"norm_out": _plain_norm_out, "append": _plain_append, "attend": _plain_attend}[state["op"]](state)


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _exact_norm(v, w, b, kind):
    mean = v.sum(1, keepdim=True) / v.shape[1] if kind == "layer" else torch.zeros_like(v[:, :1])
    centred = v - mean
    var = centred.pow(2).sum(1, keepdim=True) / v.shape[1]
    out = centred / torch.sqrt(var + EPS) * w.double()
    return out + b.double() if b is not None else out


def _exact_attend(s):
    T, hq, D, page = s["query"].shape[0], s["hq"], s["D"], s["page"]
    G = hq // s["hkv"]
    o = torch.zeros(T, hq, D, dtype=torch.float64, device=s["query"].device)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device=o.device)
    off, lens = s["offsets"].tolist(), s["lens"].tolist()
    for h in range(s["hkv"]):
        k, v = s["k_cache"][:, h].double(), s["v_cache"][:, h].double()
        heads = slice(h * G, (h + 1) * G)
        q = s["query"][:, heads].double() / math.sqrt(D)
        shared = s["prefix_pages"].long()
        pk, pv = (c[shared].reshape(-1, D)[:s["prefix"]] for c in (k, v))
        for b in range(s["B"]):
            mine = s["page_table"][b].long()
            n = lens[b]
            bk, bv = (torch.cat([p, c[mine].reshape(-1, D)[:n]]) for p, c in ((pk, k), (pv, v)))
            for t0 in range(off[b], off[b + 1], 16):
                t1 = min(off[b + 1], t0 + 16)
                z = torch.einsum("tgd,kd->tgk", q[t0:t1], bk)
                last = torch.arange(t0, t1, device=o.device) - off[b + 1] + n + s["prefix"]
                z = torch.where(torch.arange(bk.shape[0], device=o.device) <= last[:, None, None], z, -math.inf)
                lse[t0:t1, heads] = torch.logsumexp(z, -1)
                o[t0:t1, heads] = torch.softmax(z, -1) @ bv
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_in":
        return _exact_norm(s["x"].double(), s["w"], s["b"], s["kind"])
    if case["op"] == "norm_out":
        v = _exact_norm(s["f"].double(), s["pw"], s["pb"], s["kind"]) if case["post"] else s["f"].double()
        r = case["scale"] * s["x"].double() + (v if s["gate"] is None else s["gate"].double() * v)
        return r, _exact_norm(r, s["w"], s["b"], s["kind"]) if case["next"] else None
    if case["op"] == "append":
        half, style = case["rot"] // 2, case["style"]
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           torch.outer(s["positions"].double(), s["inv_freq"].double()))[:, None]

        def turned(v):
            v = v.double().clone()
            pair = v[..., :case["rot"]]
            pair = pair.unflatten(-1, (2, half)).transpose(-1, -2) if style == "half" else pair.unflatten(-1, (half, 2))
            z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
            v[..., :case["rot"]] = (z.transpose(-1, -2) if style == "half" else z).flatten(-2)
            return v

        q, k = turned(s["q"]), turned(s["k"])
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        n = case["T"] - case["pad"]
        at = s["slots"][:n].long()
        page, row = torch.div(at, case["page"], rounding_mode="floor"), at.remainder(case["page"])
        kc[page, :, row], vc[page, :, row] = k[:n], s["v"][:n].double()
        return q, kc, vc
    return _exact_attend(s)


def work(case):
    if case["op"] in ("norm_in", "norm_out"):
        n, row = case["T"] * case["d"], 2 * case["d"]
        streams, flops, small = 2, 5 * n, row * (1 + case["bias"])
        if case["op"] == "norm_out":
            streams = 3 + (case["gate"] == "full") + case["next"]
            small = row * (case["next"] + case["post"]) * (1 + case["bias"])
            small += {"none": 0, "channel": row, "token": 2 * case["T"], "full": 0}[case["gate"]]
            flops = n * (3 + 5 * case["post"] + 5 * case["next"])
        return {"bytes": 2 * n * streams + small, "flops": flops}
    hq, hkv, D = case["hq"], case["hkv"], case["D"]
    if case["op"] == "append":
        T = case["T"]
        real = T - case["pad"]
        return {"bytes": 4 * D * (T * hq + 2 * real * hkv) + 8 * T + 2 * case["rot"],
                "flops": 3 * case["rot"] * (T * hq + real * hkv)}
    qs, lens = _lengths(case)
    T, prefix = sum(qs), case["prefix"]
    seen = sum(n * prefix + sum(m - n + i + 1 for i in range(n)) for n, m in zip(qs, lens))
    return {"bytes": 4 * hkv * D * (prefix + sum(lens)) + 4 * T * hq * D + 4 * T * hq + 4 * sum(-(-m // case["page"]) for m in lens),
            "flops": 4 * D * hq * seen}
