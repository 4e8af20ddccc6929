"""The 4-bit cache in plain torch and 64 bits, written from its definition: a
group of 32 elements v is s = fp16(max|v| / 7) and the whole numbers nearest to
v / s from -7 to 7, and stands for their products with s."""
import math

import torch

GROUP = 32


def held(v):
    """(what rows v [..., D] are held as, the scale of each element), 64 bits."""
    g = v.double().unflatten(-1, (-1, GROUP))
    scale = (g.abs().amax(-1, keepdim=True) / 7).to(torch.float16).double()
    n = torch.where(scale > 0, torch.round(g / scale).clamp(-7, 7), 0.0)
    return (n * scale).flatten(-2), scale.expand_as(g).flatten(-2)


def attended(q, k, v, scale, sees):
    """q [T, G, D] over rows k, v [n, D], token i seeing the first sees[i]; (o, lse)."""
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    for i, m in enumerate(sees):
        if m > 0:
            z = scale * (q[i].double() @ k[:m].T)
            lse[i] = torch.logsumexp(z, -1)
            o[i] = torch.softmax(z, -1) @ v[:m]
    return o, lse
