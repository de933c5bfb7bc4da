"""Inputs and error bounds for the 4-bit attention kernels that stay small where tests/_kv4.py's
worst-case ones grow past the outputs: over long caches, and for chunks by the prefill kernel.

Two kinds of checks:
  counting   queries of zeros.  Every visible key weighs the same, all products and sums are exact,
             the LSE is the logarithm of the number of visible keys, and a value's element is
             nonzero in every d-th tile of 32 keys only: a key or a tile that is left out, taken
             twice or masked wrongly shows at any length.
  random     ordinary queries; each rounding counted as a random error of its standard deviation,
             the sum of all held to eight of them.
"""
import math

import torch

from tests import _kv4 as R

U11 = 2.0 ** -11 / 3 ** 0.5  # standard deviation of a rounding to fp16, at most, of a value


def visible(qpos, Tk, window=0, n_sink=0):
    """[Tq, Tk] truth values: key n at position n, causal, window and sinks."""
    n = torch.arange(Tk, device=qpos.device)
    dist = qpos[:, None] - n
    seen = dist >= 0
    if window > 0:
        seen &= (dist < window) | (n < n_sink)
    return seen


# ---------------------------------------------------------------------------- counting
def counting_rows(Tk, d, device):
    """Rows [Tk, 5d/4]: arbitrary finite keys; of the values the element j = (n // 32) % d of key n
    stands for (1 + n % 15) / 8, the others for 0."""
    G = d // 32
    gen = torch.Generator(device=device)
    gen.manual_seed(Tk)
    n = torch.arange(Tk, device=device)
    rows = torch.zeros(Tk, 5 * d // 4, dtype=torch.uint8, device=device)
    rows[:, : d // 2] = torch.randint(0, 256, (Tk, d // 2), device=device, generator=gen, dtype=torch.uint8)
    j, code = n // 32 % d, 1 + n % 15
    c, g = j % 32 // 4, j // 32            # value unit c G + g of 4 codes, from the low bits up
    at = (c * G + g) * 4 + j % 4
    rows[n, d // 2 + at // 2] = (code << (4 * (at % 2))).to(torch.uint8)
    par = torch.zeros(Tk, 2, G, 2, dtype=torch.float16, device=device)
    par[:, 0, :, 0], par[:, 0, :, 1], par[:, 1, :, 0] = 0.25, -1.5, 0.125
    rows[:, d:] = par.flatten(1).view(torch.uint8)
    return rows


def counting_result(qpos, Tk, d, window=0, n_sink=0, cached=None):
    """o [Tq, d] and lse [Tq] in 64 bits; keys from `cached` on (the call's own) have values of 0."""
    n = torch.arange(Tk, device=qpos.device)
    v = torch.zeros(Tk, d, dtype=torch.float64, device=qpos.device)
    v[n, n // 32 % d] = (1 + n % 15).double() / 8
    if cached is not None:
        v[cached:] = 0
    seen = visible(qpos, Tk, window, n_sink).double()
    count = seen.sum(-1)
    return seen @ v / count[:, None], torch.log(count)


def counting_bounds(o, lse):
    """Sums are exact; the division rounds to 2^-24 and o to bf16, half a step of 2^-8.  lse is
    (M + log2 sum) ln 2 with both terms below 32: one unit, 2^-19, of the logarithm and half of one
    of the sum, then ln 2 of it and a last rounding of lse."""
    return 2.0 ** -8 * (1 + 2.0 ** -10) * o.abs(), (2.0 ** -19 + 2.0 ** -20) * math.log(2.0) + 2.0 ** -22 * lse.abs()


# ------------------------------------------------------------------------------ random
def attend(q, rows, qpos, table, head0=0, Hq=1, window=0, n_sink=0):
    """q [g, Tq, d] rotated, in 64 bits: query heads head0 .. of Hq that share rows [Tk, 5d/4].
    -> o, lse and what the bounds need."""
    d, scale = q.shape[-1], table.softmax_scale
    (kc, ks, kz), (vc, vs, vz) = R.decode_rows(rows)
    k, v = R.values(kc, ks, kz), R.values(vc, vs, vz)
    ka, va = R.values(kc, ks, kz.abs()), R.values(vc, vs, vz.abs())
    sn = R.values(vc, vs, torch.zeros_like(vz))
    seen = visible(qpos, rows.shape[0], window, n_sink)
    live = seen.any(0)
    k, v, ka, va, sn, seen = k[live], v[live], ka[live], va[live], sn[live], seen[:, live]
    n = torch.arange(rows.shape[0], device=rows.device)[live]
    out = []

    def spread(w, o):  # sum of w (v - o)^2: w the squares of p times a logit's error
        return (w @ v ** 2 - 2 * o * (w @ v) + o ** 2 * w.sum(-1, keepdim=True)).clamp_min(0)
    for h in range(q.shape[0]):
        x = q[h] @ k.T * scale
        if table.method == 7:
            x = x - 2.0 ** (-8.0 * (head0 + h + 1) / Hq) * (qpos[:, None] - n).double()
        x = x.masked_fill(~seen, -math.inf)
        lse = torch.logsumexp(x, -1)
        p = torch.exp(x - lse[:, None])
        o = p @ v
        logit = (q[h].abs() @ ka.T * scale).masked_fill(~seen, 0).amax(-1)
        var = (q[h] ** 2) @ (k ** 2).T * (2 * (scale * U11) ** 2)  # of a logit of fp16 operands
        p2 = p ** 2
        out.append(dict(o=o, lse=lse, amp=p @ va, logit=logit, pn2=p2 @ sn ** 2, pv2=p2 @ v ** 2,
                        spread=spread(p2, o), moved=spread(p2 * var, o), var=(p * var).sum(-1)))
    return {key: torch.stack([x[key] for x in out]) for key in out[0]}


def decode_bounds(r, d, keys_of_a_block, blocks):
    """The decode kernel: a logit's product sums d terms in fp32 and rounds the query to 22 bits,
    scale, product and reference once each, at most (d + 16) 2^-24 of its magnitude, whatever the
    key's value; p s rounds to fp16; the tensor cores cut off up to 2^-22 of a sum at each of the 32 steps between two folds;
    the other sums round to nearest, a lane's own over a sixteenth of the block's keys and then
    folds, lanes, warps and blocks; o rounds to bf16."""
    e = (d + 16) * 2.0 ** -24 * r["logit"] + 2.0 ** -21
    sums = 32 * 2.0 ** -22 + (keys_of_a_block / 16 + blocks + 64) * 2.0 ** -24
    bo = 8 * (e[..., None] * r["spread"].sqrt() + U11 * r["pn2"].sqrt()) + sums * r["amp"] + 2.0 ** -8 * r["o"].abs()
    return bo, e + sums + 2.0 ** -21 + 2.0 ** -22 * r["lse"].abs()


def chunk_bounds(r, n_keys):
    """The prefill kernel: query and key round to fp16 (`var`), and so do p and the value; sums as
    above, cut off at each of n_keys / 16 steps; o rounds to bf16."""
    sums = (n_keys / 16 + 64) * 2.0 ** -22
    e = 2.0 ** -21 * r["logit"] + 2.0 ** -21
    bo = 8 * (r["moved"].sqrt() + e[..., None] * r["spread"].sqrt() + 2 ** 0.5 * U11 * r["pv2"].sqrt()) + \
        sums * r["amp"] + 2.0 ** -8 * r["o"].abs()
    return bo, 8 * r["var"].sqrt() + e + sums + 2.0 ** -22 * r["lse"].abs()
