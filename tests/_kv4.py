"""Plain forms of the 4-bit KV cache for its tests: the row format, and attention over it in
64 bits."""
import math

import torch


def turns_of(table):
    return torch.tensor(list(table.turns[: table.head_dim // 2]), dtype=torch.float64)


def rotate(x, pos, table):
    """x [..., d], pos broadcastable to x's leading axes: the rotated vectors in 64 bits."""
    t = turns_of(table).to(x.device)
    a = pos.double().unsqueeze(-1) * t
    a = (a - torch.round(a)) * (2.0 * math.pi)
    c, s = torch.cos(a), torch.sin(a)
    x, d = x.double(), x.shape[-1]
    if table.pairs == 1:
        u, w = x[..., : d // 2], x[..., d // 2:]
        return torch.cat([u * c - w * s, u * s + w * c], -1)
    u, w = x[..., 0::2], x[..., 1::2]
    return torch.stack([u * c - w * s, u * s + w * c], -1).flatten(-2)


def quantise(x):
    """x [..., d] fp32 -> codes [..., G, 32] (int64), s, z fp16 [..., G, 1]."""
    x = x.float().unflatten(-1, (-1, 32))
    z = x.amin(-1, keepdim=True).half()
    s = ((x.amax(-1, keepdim=True) - z.float()) / torch.full_like(z, 15).float()).clamp_min(0).half()
    q = (x - z.float()) / torch.where(s > 0, s.float(), torch.full_like(z, math.inf).float())
    return torch.round(q).clamp(0, 15).long(), s, z


def decode_rows(rows):
    """rows [..., 5d/4] uint8 -> per half (key, value): codes [..., G, 32], s, z [..., G, 1]."""
    d = rows.shape[-1] * 4 // 5
    G = d // 32
    out = []
    for half in range(2):
        b = rows[..., half * d // 2: (half + 1) * d // 2].long()
        nib = torch.stack([b & 15, b >> 4], -1).flatten(-2)  # codes in the order of storage
        codes = torch.empty(*rows.shape[:-1], G, 32, dtype=torch.long, device=rows.device)
        w = 8 if half == 0 else 4
        for u in range(32 // w):       # r (keys) or c (values)
            for g in range(G):
                at = (u * G + g) * w
                codes[..., g, u * w: (u + 1) * w] = nib[..., at: at + w]
        par = rows[..., d + half * d // 8: d + (half + 1) * d // 8].contiguous()
        par = par.view(torch.float16).unflatten(-1, (G, 2))
        out.append((codes, par[..., 0:1], par[..., 1:2]))
    return out


def values(codes, s, z):
    """What the codes stand for, in 64 bits."""
    return (codes.double() * s.double() + z.double()).flatten(-2)


def attend(q, rows, qpos, table, window=0, n_sink=0):
    """q [Hq, Tq, d] rotated, in 64 bits, at positions qpos [Tq], over rows [Hkv, Tk, 5d/4]
    (key n at position n) -> o [Hq, Tq, d], lse [Hq, Tq], and two magnitudes for the error
    bounds: amp = sum p (s n + |z|) and logit = max over the visible keys of
    scale sum |q| (s n + |z|)."""
    Hq, Tq, d = q.shape
    Hkv, Tk = rows.shape[0], rows.shape[1]
    (kc, ks, kz), (vc, vs, vz) = decode_rows(rows)
    k, v = values(kc, ks, kz), values(vc, vs, vz)
    ka, va = values(kc, ks, kz.abs()), values(vc, vs, vz.abs())
    n = torch.arange(Tk, device=q.device)
    dist = qpos[:, None] - n
    seen = dist >= 0
    if window > 0:
        seen &= (dist < window) | (n < n_sink)
    o, lse, amp, logit = [], [], [], []
    for h in range(Hq):
        j = h // (Hq // Hkv)
        x = q[h] @ k[j].T * table.softmax_scale
        a = q[h].abs() @ ka[j].T * table.softmax_scale
        if table.method == 7:
            x = x - 2.0 ** (-8.0 * (h + 1) / Hq) * dist.double()
        x = x.masked_fill(~seen, -math.inf)
        e = torch.logsumexp(x, -1)
        p = torch.exp(x - e[:, None])
        p = p.masked_fill(~seen, 0.0)
        # Masked rows may hold anything: leave them out of the product altogether.
        live = seen.any(0)
        o.append(p[:, live] @ v[j][live])
        amp.append(p[:, live] @ va[j][live])
        logit.append(a.masked_fill(~seen, 0).amax(-1))
        lse.append(e)
    return torch.stack(o), torch.stack(lse), torch.stack(amp), torch.stack(logit)


def decode_bounds(o, lse, amp, logit, n_keys, d):
    """Error bounds of the decode kernel's o (before and after its rounding to bf16) and lse.
    A logit's product sums d terms in fp32 and takes the query in 22 bits and one rounding
    each for scale, product and log2 e: (d + 16) 2^-24 of its magnitude.  p moves by that,
    twice (numerator and sum); p s is rounded to fp16 (2^-11, and 2^-24 of the largest for
    the smallest ones); exp2 and the sum over the keys give (n_keys + 64) 2^-24 (each
    addition at most half a step); o is rounded to bf16 (2^-8)."""
    e = (d + 16) * 2.0 ** -24 * logit + 2.0 ** -21
    rel = 2 * e + 2.0 ** -11 + (n_keys + 64) * 2.0 ** -24
    bo = rel[..., None] * amp + 2.0 ** -8 * o.abs() + 1e-30
    bl = e + (n_keys + 64) * 2.0 ** -24 + 2.0 ** -22 * lse.abs()
    return bo, bl
