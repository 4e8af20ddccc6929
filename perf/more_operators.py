"""What is measured of serving from a cache held in 4 bits: the append that
rotates and quantises, reading rows back to 16 bits, the attention over it, and
the verification of the tokens that were drafted.

A row of a head is held in groups of 32 elements: one fp16 scale s = max|v| / 7
and a whole number from -7 to 7 for each element, v / s rounded to even.

``run`` computes one pass in elementary torch operations, or with the
framework's own operators where ``own`` is true.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
GROUP = 32


def listed():
    return [
        # a decode step's new tokens, one for each of 64 sequences
        dict(name="append_decode", op="append", T=64, hq=64, hkv=8, D=128, page=64, rot=128, style="half",
             pad=0, far=131072, dtype="bf16"),
        # a ragged small batch padded to a captured size, interleaved pairs, half of each head rotated
        dict(name="append_padded_odd", op="append", T=333, hq=28, hkv=4, D=64, page=16, rot=32, style="pairs",
             pad=13, far=1000000, dtype="fp16"),
        # a prefill step of 16384 tokens
        dict(name="append_prefill", op="append", T=16384, hq=64, hkv=8, D=128, page=64, rot=128, style="half",
             pad=0, far=32768, dtype="bf16"),
        # a conversation's rows for a chunk of new tokens to attend to in 16 bits
        dict(name="read_rows_odd", op="read", n=4099, hkv=4, D=64, page=16, pad=3, paged=False, dtype="fp16"),
        # a long document's rows into a 16-bit cache, where a whole batch shares them
        dict(name="read_prefix", op="read", n=131072, hkv=8, D=128, page=64, pad=0, paged=True, dtype="bf16"),
        # one user, the first tokens of an answer
        dict(name="attend_one_token", op="attend", B=1, q=1, hq=64, hkv=8, D=128, page=64, length=1000,
             dtype="bf16"),
        # drafted tokens checked for a ragged batch: several queries for each sequence, 7 heads to a key head
        dict(name="attend_drafts_odd", op="attend", B=37, q=6, hq=28, hkv=4, D=64, page=16, length=4099,
             dtype="fp16"),
        # 64 users, up to 8192 tokens each
        dict(name="attend_decode", op="attend", B=64, q=1, hq=64, hkv=8, D=128, page=64, length=8192, dtype="bf16"),
        # 16 users with long contexts
        dict(name="attend_long", op="attend", B=16, q=1, hq=64, hkv=8, D=128, page=64, length=131072, dtype="bf16"),
        # one user, four drafts
        dict(name="verify_one", op="verify", B=1, drafts=4, vocab=32000, greedy=False, dtype="fp32"),
        # a ragged batch whose drafter gives tokens without probabilities, an odd vocabulary
        dict(name="verify_greedy_odd", op="verify", B=37, drafts=3, vocab=50021, greedy=True, dtype="bf16"),
        # 64 users, up to 7 drafts each
        dict(name="verify_batch", op="verify", B=64, drafts=7, vocab=131072, greedy=False, dtype="fp32"),
    ]


def _between(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "verify"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "verify":
        drafts, vocab = _between(rng, 1, 15), _between(rng, 1000, 200000)
        most = max(1, 64 * 8 * 131072 // ((drafts + 1) * vocab))
        return dict(op=op, B=_between(rng, 1, min(128, most)), drafts=drafts, vocab=vocab, greedy=rng.random() < 0.3,
                    dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]))
    D, hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    G, page = rng.choice([1, 2, 4, 5, 7, 8, 16]), rng.choice([16, 32, 64, 128])
    G = min(G, 64 // hkv)
    if op == "append":
        T = _between(rng, 1, 8192)
        return dict(op=op, T=T, hq=G * hkv, hkv=hkv, D=D, page=page, rot=rng.choice([D, D // 2]),
                    style=rng.choice(["half", "pairs"]), pad=rng.randrange(0, min(T, 17)),
                    far=_between(rng, 64, 1000000), dtype=dtype)
    if op == "read":
        n = _between(rng, 1, 131072)
        return dict(op=op, n=n, hkv=hkv, D=D, page=page, pad=rng.randrange(0, min(n, 17)), paged=rng.random() < 0.5,
                    dtype=dtype)
    q, B = rng.choice([1, 1, 1, 2, 5, _between(rng, 6, 16)]), _between(rng, 1, 256)
    # rows in all at most the largest listed case's, and so for the products
    most = min(16 * 131072 * 8 * 128 // (B * hkv * D), 16 * 64 * 131072 // (B * G * hkv * q), 131072)
    return dict(op=op, B=B, q=q, hq=G * hkv, hkv=hkv, D=D, page=page, length=_between(rng, 1, max(1, most)),
                dtype=dtype)


def _lengths(case):
    """Queries and length of each sequence: ragged, up to q and length, the same for every seed."""
    rng = random.Random("%d %d %d" % (case["B"], case["q"], case["length"]))
    qs, lens = [], []
    for b in range(case["B"]):
        n = case["q"] if b == 0 else rng.randint(1, case["q"])
        qs.append(n)
        lens.append(max(n, case["length"] if b == 0 else rng.randint(1, case["length"])))
    return qs, lens


def _drafts(case):
    """Drafts of each sequence: ragged, up to drafts, none among them, the same for every seed."""
    rng = random.Random("%d %d %d" % (case["B"], case["drafts"], case["vocab"]))
    return [case["drafts"] if b == 0 else rng.randint(0, case["drafts"]) for b in range(case["B"])]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dt)

    s = dict(case)
    if case["op"] == "verify":
        B, V = case["B"], case["vocab"]
        counts = torch.tensor([n + 1 for n in _drafts(case)], device=dev)
        T = int(counts.sum())
        logits = torch.randn(T, V, generator=g, device=dev) * 3
        s["target"] = torch.softmax(logits, -1).to(dt)
        # a smaller model's opinion: near the target's; each row's token is drawn from it
        logits += torch.randn(T, V, generator=g, device=dev)
        drafter = torch.softmax(logits, -1)
        s["draft"] = None if case["greedy"] else drafter.to(dt)
        noise = torch.rand(T, V, generator=g, device=dev).clamp_(min=1e-9).log_().neg_()
        drawn = (drafter / noise).argmax(-1) if not case["greedy"] else drafter.argmax(-1)
        # tokens[t] is judged by row t - 1 of the same sequence
        s["tokens"] = drawn.roll(1).to(torch.int32)
        s["uniforms"] = torch.rand(T, generator=g, device=dev)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["most"] = case["drafts"] + 1
        s["accepted"] = torch.empty(B, dtype=torch.int32, device=dev)
        s["out"] = torch.empty(T, dtype=torch.int32, device=dev)
        if own:
            import dispatch_combine_gb300 as moe
            s["ws"] = moe.Workspace(256)
        return s
    hkv, D, page = case["hkv"], case["D"], case["page"]
    # channels of keys differ in size
    loud = torch.exp(0.3 * torch.randn(hkv, D, generator=g, device=dev))

    def filled(pages):
        """A cache with a row for every slot."""
        if own:
            import dispatch_combine_gb300 as moe
            heads = moe.kv_struct(num_q_heads=case.get("hq", hkv), num_kv_heads=hkv, head_dim=D, page_size=page,
                                  num_pages=pages, dtype=dt)
            s["heads"] = heads
            s["k_cache"], s["v_cache"] = (torch.zeros(pages, hkv, moe.moe_kv4_page_bytes(heads), dtype=torch.uint8,
                                                      device=dev) for _ in range(2))
        else:
            for x in "kv":
                s[x + "_codes"] = torch.empty(pages, hkv, page, D // 2, dtype=torch.uint8, device=dev)
                s[x + "_scales"] = torch.empty(pages, hkv, page, D // GROUP, dtype=torch.float16, device=dev)
        part = max(1, (1 << 26) // (hkv * page * D))
        for p in range(0, pages, part):
            n = min(part, pages - p)
            k, v = ((torch.randn(n * page, hkv, D, generator=g, device=dev) * size).to(dt) for size in (loud, 1.0))
            if own:
                slots = torch.arange(p * page, (p + n) * page, dtype=torch.int32, device=dev)
                moe.moe_kv4_append(heads, None, k, v, None, slots, None, s["k_cache"], s["v_cache"])
            else:
                for x, rows in (("k", k), ("v", v)):
                    codes, scales = _quantised(rows.float())
                    s[x + "_codes"][p:p + n] = codes.unflatten(0, (n, page)).transpose(1, 2)
                    s[x + "_scales"][p:p + n] = scales.unflatten(0, (n, page)).transpose(1, 2)

    if case["op"] == "append":
        hq, T = case["hq"], case["T"]
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
        s["q_out"] = torch.empty(T, hq, D, dtype=dt, device=dev)
        s["k_out"], s["v_out"] = (torch.zeros(T, hkv, D, dtype=dt, device=dev) for _ in range(2))
        filled(pages)
    elif case["op"] == "read":
        n = case["n"]
        pages = -(-n // page) + 3
        # pages in any order, a page's rows side by side
        order = torch.randperm(pages, generator=g, device=dev)
        slots = (order[:, None] * page + torch.arange(page, device=dev)).reshape(-1)[:n].to(torch.int32)
        if case["pad"]:
            slots[-case["pad"]:] = -1
        s["slots"], s["to"] = slots, None
        shape = (n, hkv, D)
        if case["paged"]:
            s["to"], shape = torch.arange(n, dtype=torch.int32, device=dev), (-(-n // page), hkv, page, D)
        s["k_out"], s["v_out"] = (torch.zeros(shape, dtype=dt, device=dev) for _ in range(2))
        filled(pages)
    else:
        qs, lens = _lengths(case)
        B, T, hq = case["B"], sum(qs), case["hq"]
        each = [-(-n // page) for n in lens]
        pages = sum(each)
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        table = torch.zeros(B, max(each), dtype=torch.int32, device=dev)
        for b, n in enumerate(each):
            table[b, :n] = order[sum(each[:b]):][:n]
        s["page_table"] = table
        s["query"] = normal(T, hq, D, std=1.5)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["offsets"] = torch.tensor([sum(qs[:b]) for b in range(B + 1)], dtype=torch.int32, device=dev)
        s["out"], s["lse"] = torch.empty(T, hq, D, dtype=dt, device=dev), torch.empty(T, hq, device=dev)
        filled(pages)
        if own:
            import dispatch_combine_gb300 as moe
            s["ws"] = moe.Workspace(moe.moe_kv4_attention_workspace_size(s["heads"], T, B, case["q"]))
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _quantised(rows):
    """Codes (two in a byte) and scales of fp32 rows [..., D]."""
    v = rows.unflatten(-1, (-1, GROUP))
    scale = (v.abs().amax(-1) / torch.full((), 7.0, device=v.device)).half()
    s = scale.float()[..., None]
    code = torch.where(s > 0, torch.round(v / s), 0.0).clamp(-7, 7).flatten(-2)
    n = (code + 8).to(torch.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4), scale


def _values(codes, scales):
    """What codes and scales stand for, in fp32."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().sub_(8.0).unflatten(-1, (-1, GROUP))
    return n.mul_(scales.float()[..., None]).flatten(-2)


def _rotated(v, cos, sin, rot, style):
    a, b = (v[..., :rot // 2], v[..., rot // 2:rot]) if style == "half" else (v[..., 0:rot:2], v[..., 1:rot:2])
    x, y = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat([x, y], -1) if style == "half" else torch.stack([x, y], -1).flatten(-2)
    return torch.cat([turned, v[..., rot:]], -1)


def _read_rows(s, x, slots, page):
    return _values(s[x + "_codes"][slots // page, :, slots % page], s[x + "_scales"][slots // page, :, slots % page])


def _plain_append(s):
    page, slots = s["page"], s["slots"].long()
    angle = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _rotated(s["q"].float(), cos, sin, s["rot"], s["style"]).to(s["q"].dtype)
    n = slots.shape[0] - s["pad"]  # padding is not appended, and its rows are left as they were
    at = slots[:n]
    for x, rows in (("k", _rotated(s["k"].float(), cos, sin, s["rot"], s["style"])), ("v", s["v"].float())):
        codes, scales = _quantised(rows[:n])
        s[x + "_codes"][at // page, :, at % page] = codes
        s[x + "_scales"][at // page, :, at % page] = scales
        s[x + "_out"][:n] = _read_rows(s, x, at, page).to(s["k"].dtype)
    return q, s["k_out"], s["v_out"]


def _plain_read(s):
    page, n = s["page"], s["n"] - s["pad"]
    at = s["slots"][:n].long()
    for x in "kv":
        rows, out = _read_rows(s, x, at, page).to(s["k_out"].dtype), s[x + "_out"]
        if s["to"] is None:
            out[:n] = rows
        else:
            to = s["to"][:n].long()
            out[to // page, :, to % page] = rows
    return s["k_out"], s["v_out"]


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
    pages = s["page_table"].long()

    def rows(x):  # [B, hkv, rows, D]
        v = _values(s[x + "_codes"][pages], s[x + "_scales"][pages])
        return v.transpose(1, 2).flatten(2, 3)

    z = padded.permute(0, 2, 1, 3, 4).reshape(B, hkv, nq * G, D) @ rows("k").transpose(-1, -2)
    z = (z * scale).reshape(B, hkv, nq, G, -1)
    limit = lens[:, None] - count[:, None] + step + 1  # [B, nq]
    seen = torch.arange(z.shape[-1], device=query.device) < limit[..., None]
    z = z.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = z.amax(-1, keepdim=True).clamp(min=-1e30)  # a row that sees nothing
    z = torch.exp_(z.sub_(top))
    total = z.sum(-1, keepdim=True)
    o = (z.reshape(B, hkv, nq * G, -1) @ rows("v")).reshape(B, hkv, nq, G, D)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + torch.log(total))[..., 0]
    o, lse = o.permute(0, 2, 1, 3, 4).reshape(B, nq, hq, D), lse.permute(0, 2, 1, 3).reshape(B, nq, hq)
    return o[seq, place].to(s["query"].dtype), lse[seq, place]


def _plain_verify(s):
    B, V = s["B"], s["vocab"]
    off, tokens = s["offsets"].long(), s["tokens"].long()
    T = tokens.shape[0]
    n = off[1:] - off[:-1] - 1  # drafts of each sequence
    step = torch.arange(s["most"], device=off.device)
    row = (off[:-1, None] + step).clamp(max=T - 1)
    word = tokens[(row + 1).clamp(max=T - 1)]
    p = s["target"][row, word].double()
    q = s["draft"][row, word].double() if s["draft"] is not None else torch.ones_like(p)
    # the drafts before the first that is refused
    fine = (s["uniforms"][row].double() * q < p) & (step < n[:, None])
    accepted = fine.to(torch.int64).cumprod(-1).sum(-1)
    at = off[:-1] + accepted
    w = s["target"][at].float()
    refused = (accepted < n)[:, None]
    other = word.gather(1, accepted[:, None])
    if s["draft"] is not None:
        w = torch.where(refused, (w - s["draft"][at].float()).clamp(min=0.0), w)
    else:
        w = torch.where(refused & (torch.arange(V, device=off.device) == other), 0.0, w)
    below = w.double().cumsum(-1)
    last = s["uniforms"][off[1:] - 1].double()
    final = (below <= last[:, None] * below[:, -1:]).sum(-1).clamp(max=V - 1)
    token = torch.arange(T, device=off.device)
    seq = (token[:, None] >= off[None, 1:]).sum(-1)
    place = token - off[seq]
    after = tokens[(token + 1).clamp(max=T - 1)]
    out = torch.where(place < accepted[seq], after, torch.where(place == accepted[seq], final[seq], -1))
    return accepted.to(torch.int32), out.to(torch.int32)


def _own(s):
    import dispatch_combine_gb300 as moe
    if s["op"] == "append":
        style = moe.MOE_ROPE_HALF if s["style"] == "half" else moe.MOE_ROPE_PAIRS
        q = moe.moe_kv4_append(s["heads"], s["q"], s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"],
                               s["k_cache"], s["v_cache"], style=style, q_out=s["q_out"])
        k, v = moe.moe_kv4_read(s["heads"], s["slots"], s["k_cache"], s["v_cache"], k_out=s["k_out"], v_out=s["v_out"])
        return q, k, v
    if s["op"] == "read":
        return moe.moe_kv4_read(s["heads"], s["slots"], s["k_cache"], s["v_cache"], k_out=s["k_out"],
                                v_out=s["v_out"], dst_slots=s["to"])
    if s["op"] == "attend":
        return moe.moe_kv4_attention(s["heads"], s["query"], s["k_cache"], s["v_cache"], s["page_table"], s["lens"],
                                     s["ws"], q_offsets=s["offsets"], max_q=s["q"], out=s["out"], lse=s["lse"])
    return moe.moe_verify_drafts(s["target"], s["tokens"], s["uniforms"], s["offsets"], draft=s["draft"], ws=s["ws"],
                                 accepted=s["accepted"], out_tokens=s["out"])


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "read": _plain_read, "attend": _plain_attend,
            "verify": _plain_verify}[state["op"]](state)


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _exact_cache(s, x):
    """[pages, hkv, page, D] of what the cache holds."""
    c = s[x + "_codes"].to(torch.int64)
    low, high = c.remainder(16) - 8, torch.div(c, 16, rounding_mode="floor") - 8
    whole = torch.empty(*c.shape[:-1], 2 * c.shape[-1], dtype=torch.float64, device=c.device)
    whole[..., ::2], whole[..., 1::2] = low, high
    return whole * s[x + "_scales"].double().repeat_interleave(GROUP, -1)


def _exact_held(v):
    """What rows in 64 bits are held as."""
    g = v.reshape(*v.shape[:-1], v.shape[-1] // GROUP, GROUP)
    scale = (g.abs().max(-1, keepdim=True).values / 7).to(torch.float16).double()
    return torch.where(scale > 0, scale * torch.round(g / scale).clamp(-7, 7), 0.0).reshape(v.shape)


def _exact_attend(s):
    T, hq, D, page = s["query"].shape[0], s["hq"], s["D"], s["page"]
    G = hq // s["hkv"]
    o = torch.zeros(T, hq, D, dtype=torch.float64, device=s["query"].device)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device=o.device)
    off, lens = s["offsets"].tolist(), s["lens"].tolist()
    for b in range(s["B"]):
        n = lens[b]
        mine = s["page_table"][b, :-(-n // page)].long()
        part = {x + y: s[x + y][mine] for x in "kv" for y in ("_codes", "_scales")}
        for h in range(s["hkv"]):
            one = {name: t[:, h:h + 1] for name, t in part.items()}
            k, v = (_exact_cache(one, x).reshape(-1, D)[:n] for x in "kv")
            heads = slice(h * G, (h + 1) * G)
            for t in range(off[b], off[b + 1]):
                sees = n - (off[b + 1] - 1 - t)
                z = (s["query"][t, heads].double() / math.sqrt(D)) @ k[:sees].T
                lse[t, heads] = torch.logsumexp(z, -1)
                o[t, heads] = torch.softmax(z, -1) @ v[:sees]
    return o, lse


def exact(case, seed):
    if case["op"] == "verify":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "append":
        half, style, n = case["rot"] // 2, case["style"], case["T"] - case["pad"]
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           torch.outer(s["positions"].double(), s["inv_freq"].double()))[:, None]

        def turned(v):
            v = v.double().clone()
            pair = v[..., :case["rot"]]
            pair = pair.unflatten(-1, (2, half)).transpose(-1, -2) if style == "half" else pair.unflatten(-1, (half, 2))
            z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
            v[..., :case["rot"]] = (z.transpose(-1, -2) if style == "half" else z).flatten(-2)
            return v

        k, v = _exact_held(turned(s["k"])), _exact_held(s["v"].double())
        k[n:], v[n:] = 0.0, 0.0
        return turned(s["q"]), k, v
    if case["op"] == "read":
        n, page = case["n"] - case["pad"], case["page"]
        outs = []
        for x in "kv":
            rows = _exact_cache(s, x).transpose(1, 2).flatten(0, 1)[s["slots"][:n].long()]
            out = torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda")
            if case["paged"]:
                flat = torch.zeros(out.shape[0] * page, *rows.shape[1:], dtype=torch.float64, device="cuda")
                flat[s["to"][:n].long()] = rows
                out = flat.unflatten(0, (-1, page)).transpose(1, 2).contiguous()
            else:
                out[:n] = rows
            outs.append(out)
        return tuple(outs)
    return _exact_attend(s)


def work(case):
    if case["op"] == "verify":
        rows = 1 if case["greedy"] else 2
        size = 4 if case["dtype"] == "fp32" else 2
        T = sum(_drafts(case)) + case["B"]
        return {"bytes": case["B"] * case["vocab"] * rows * size + T * (12 + 2 * size) + 8 * case["B"],
                "flops": 3 * case["B"] * case["vocab"]}
    hkv, D = case["hkv"], case["D"]
    held = D // 2 + 2 * D // GROUP  # bytes of a head's row
    if case["op"] == "read":
        n = case["n"] - case["pad"]
        return {"bytes": 2 * n * hkv * (held + 2 * D) + 4 * case["n"] * (1 + case["paged"]), "flops": 2 * n * hkv * D}
    hq = case["hq"]
    if case["op"] == "append":
        T = case["T"]
        real = T - case["pad"]
        # queries in and out, keys and values in, held, and out as they are held
        return {"bytes": 4 * D * T * hq + 2 * real * hkv * (4 * D + held) + 8 * T + 2 * case["rot"],
                "flops": 3 * case["rot"] * (T * hq + real * hkv) + 6 * real * hkv * D}
    qs, lens = _lengths(case)
    T = sum(qs)
    seen = sum(m - n + i + 1 for n, m in zip(qs, lens) for i in range(n))
    return {"bytes": 2 * hkv * held * sum(lens) + 4 * T * hq * D + 4 * T * hq + 4 * sum(-(-m // case["page"]) for m in lens),
            "flops": 4 * D * hq * seen}
