"""Cases and plain forms of the operators around the 4-bit KV cache.

A cache row holds the rotated key and the value of one token and KV head in 5d/4 bytes:
d/2 bytes of key codes, d/2 bytes of value codes, then an fp16 (scale, minimum) pair for
each group of 32 elements, the key's groups before the value's.  A stored element stands
for scale * code + minimum, code in 0..15.

  write   kv4_write of new rows (keys rotated at their positions), then kv4_read of them
  read    kv4_read of a cached prefix
  decode  attn_decode_kv4: one token per sequence, appended and attended over its cache
  chunk   attn_prefill_chunk_kv4: a chunk of tokens after a cached prefix, then kv4_read
          of the rows that it appended
"""
import math

import torch

own = False

GROUP = 32
LOG2E = 1.4426950408889634


def _case(name, op, **kw):
    c = dict(op=op, B=1, Hq=32, Hkv=8, d=128, T=1, T_max=1, len_lo=0, len_hi=0, window=0,
             n_sink=0, pairs="interleaved", method="yarn", base=500000.0, L_train=8192,
             scale=16.0, dtype="bf16")
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # A 16K prompt of the Llama-3-8B head shape goes into the cache.
        _case("write_16k", "write", T=16384, T_max=16392),
        # A padded batch of short turns appended at each sequence's own length.
        _case("write_ragged_d64_half", "write", B=4, Hkv=4, d=64, T=1003, T_max=3001, len_lo=7,
              len_hi=1990, pairs="half", base=10000.0, L_train=4096, scale=4.0),
        # A cached 124K prefix read back for an attention over it in 16 bits.
        _case("read_124k", "read", T=126976, T_max=131072),
        # Short prefixes of a batch, as fp16 operands; an odd row count.
        _case("read_short_d64_fp16", "read", B=6, Hkv=4, d=64, T=777, T_max=1001, len_lo=1,
              len_hi=224, dtype="fp16"),
        # One user's next token after a short prompt: latency counts.
        _case("decode_b1_1k", "decode", T_max=2048, len_lo=1000, len_hi=1000),
        # A served batch over caches of 32K to 128K keys.
        _case("decode_b8_128k", "decode", B=8, T_max=131073, len_lo=32768, len_hi=131072),
        # Llama-2-7B heads (no sharing of KV heads) over a sliding window with sink tokens.
        _case("decode_b16_mha_window", "decode", B=16, Hkv=32, T_max=16384, len_lo=100,
              len_hi=16383, window=4096, n_sink=4, pairs="half", base=10000.0, L_train=4096,
              scale=4.0),
        # One KV head for 16 query heads, small heads, odd lengths.
        _case("decode_b3_mqa_d64", "decode", B=3, Hq=16, Hkv=1, d=64, T_max=5001, len_lo=63,
              len_hi=4999, base=10000.0, L_train=4096, scale=4.0),
        # A user's next turn after a cached 124K prefix.
        _case("chunk_256_after_124k", "chunk", T=256, T_max=131072, len_lo=126976,
              len_hi=126976),
        # A long prompt taken in pieces of 2048.
        _case("chunk_2k_after_30k", "chunk", T=2048, T_max=32768, len_lo=30720, len_hi=30720),
        # A few tokens to check at once for a batch, sliding window and sinks, odd sizes.
        _case("chunk_33_window_d64_b2", "chunk", B=2, Hq=16, Hkv=4, d=64, T=33, T_max=20011,
              len_lo=19001, len_hi=19001, window=4096, n_sink=4, pairs="half", base=10000.0,
              L_train=4096, scale=4.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "chunk"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 8, 16])
    kw = dict(d=d, Hkv=Hkv, Hq=Hkv * g, pairs=rng.choice(["interleaved", "half"]),
              method=rng.choice(["yarn", "yarn", "rope", "alibi"]))
    if rng.random() < 0.5:
        kw.update(base=10000.0, L_train=4096, scale=4.0)
    if op in ("decode", "chunk") and rng.random() < 0.35:
        kw.update(window=_log_int(rng, 1, 6000), n_sink=rng.choice([0, 1, 4, 9]))
    if op in ("write", "read"):
        B = rng.choice([1, 2, 3])
        kw.update(T=_log_int(rng, 1, min(100000, 1000000 // (B * Hkv))), B=B,
                  dtype=rng.choice(["bf16", "fp16"]) if op == "read" else "bf16")
        lo = rng.randrange(0, 500)
        hi = lo + rng.randrange(0, 3000)
        kw.update(len_lo=lo, len_hi=hi, T_max=hi + kw["T"] + rng.randrange(0, 9))
    elif op == "decode":
        B = _log_int(rng, 1, 32)
        hi = _log_int(rng, 1, max(16, 400000 // B))
        lo = rng.randrange(0, hi + 1)
        kw.update(B=B, len_lo=lo, len_hi=hi, T_max=hi + 1 + rng.randrange(0, 9))
    else:
        T = _log_int(rng, 1, 2048)
        P0 = _log_int(rng, 1, 40000)
        T = min(T, max(1, 2000000000 // (Hkv * g * (P0 + T))))
        kw.update(T=T, len_lo=P0, len_hi=P0, T_max=P0 + T + rng.randrange(0, 9),
                  B=rng.choice([1, 1, 2]) if T <= 256 else 1)
    return _case(None, op, **kw)


def _lens(case):
    """The sequences' cached lengths, spread evenly from len_hi down to len_lo."""
    B = case["B"]
    return [case["len_hi"] - (case["len_hi"] - case["len_lo"]) * b // max(1, B - 1)
            for b in range(B)]


def _counts(case):
    """Valid rows of each sequence of a padded batch (all rows where the batch is not ragged)."""
    B, T = case["B"], case["T"]
    if case["len_lo"] == case["len_hi"]:
        return [T] * B
    return [T - (T * b) // (2 * B) for b in range(B)]


def _turns(case):
    """Rotations per position of each pair, in 64 bits, and the logit multiplier."""
    d, scale = case["d"], case["scale"]
    i = torch.arange(d // 2, dtype=torch.float64)
    theta = torch.exp(-2.0 * i / d * math.log(case["base"]))
    if case["method"] == "yarn":
        r = case["L_train"] * theta / (2.0 * math.pi)
        gamma = ((r - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        theta = theta * (gamma + (1.0 - gamma) / scale)
    elif case["method"] == "alibi":
        theta = torch.zeros_like(theta)
    mscale = 0.1 * math.log(scale) + 1.0 if case["method"] == "yarn" else 1.0
    return theta / (2.0 * math.pi), mscale * mscale / math.sqrt(d)


def _key_length(case):
    """Keys that a query of a decode case can have at most."""
    return max(_lens(case)) + 1


# ------------------------------------------------------------------ the cache's format
def _rotate(x, pos, turns, half):
    """x [..., T, d] in 64 bits, pos [B, 1, T] positions: each pair turned by pos * turns."""
    frac = pos.double().unsqueeze(-1) * turns
    ang = (frac - torch.round(frac)) * (2.0 * math.pi)
    c, s = torch.cos(ang), torch.sin(ang)
    d = x.shape[-1]
    if half:
        a, b = x[..., : d // 2], x[..., d // 2:]
        return torch.cat([a * c - b * s, a * s + b * c], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)


def _quantise(x):
    """x [..., d] fp32 -> codes uint8 [..., d/32, 32], scale and minimum fp16 [..., d/32, 1]."""
    x = x.unflatten(-1, (-1, GROUP))
    z = x.amin(-1, keepdim=True).half()
    # Divided by a tensor: a division by a number is a product with its rounded reciprocal.
    steps = torch.full_like(z, 15.0, dtype=torch.float32)
    s = ((x.amax(-1, keepdim=True) - z.float()) / steps).clamp_min(0.0).half()
    by = torch.where(s > 0, s.float(), torch.full_like(steps, math.inf))
    n = torch.round((x - z.float()) / by).clamp(0.0, 15.0)
    return n.to(torch.uint8), s, z


def _dequantise(n, s, z):
    return (n.float() * s.float() + z.float()).flatten(-2)


def _pack(kq, vq):
    """Codes and (scale, minimum) pairs of keys and values -> rows [..., 5d/4] of bytes."""
    (kn, ks, kz), (vn, vs, vz) = kq, vq
    G = kn.shape[-2]
    # A key word of 8 codes holds elements 32g + 8r .. + 7 of group g; words in (r, g) order.
    kb = kn.unflatten(-1, (4, 4, 2)).movedim(-4, -3)
    # A value unit of 4 codes holds elements 32g + 4c .. + 3; units in (c, g) order.
    vb = vn.unflatten(-1, (8, 2, 2)).movedim(-4, -3)
    kb = (kb[..., 0] | (kb[..., 1] << 4)).flatten(-3)
    vb = (vb[..., 0] | (vb[..., 1] << 4)).flatten(-3)
    par = torch.cat([torch.cat([ks, kz], -1), torch.cat([vs, vz], -1)], -2).flatten(-2)
    assert par.shape[-1] == 4 * G
    return torch.cat([kb, vb, par.contiguous().view(torch.uint8)], -1)


def _unpack(rows, d):
    """Rows [..., 5d/4] of bytes -> keys and values [..., d] in fp32."""
    G = d // GROUP
    kb, vb = rows[..., : d // 2], rows[..., d // 2: d]
    par = rows[..., d:].contiguous().view(torch.float16).float().unflatten(-1, (2, G, 2))
    kn = torch.stack([kb & 15, kb >> 4], -1).flatten(-2).unflatten(-1, (4, G, 8))
    vn = torch.stack([vb & 15, vb >> 4], -1).flatten(-2).unflatten(-1, (8, G, 4))
    kn = kn.movedim(-2, -3).flatten(-2)
    vn = vn.movedim(-2, -3).flatten(-2)
    k = kn.float() * par[..., 0, :, 0:1] + par[..., 0, :, 1:2]
    v = vn.float() * par[..., 1, :, 0:1] + par[..., 1, :, 1:2]
    return k.flatten(-2), v.flatten(-2)


# ----------------------------------------------------------------------------- inputs
def prepare(case, seed):
    """Inputs on the GPU; the cache holds quantised normal keys and values, the keys with
    channels of unlike size as trained models have them, and zeros behind each sequence."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    B, Hq, Hkv, d, T, T_max = (case[n] for n in ("B", "Hq", "Hkv", "d", "T", "T_max"))
    turns, scale = _turns(case)
    chan = torch.exp(0.4 * torch.randn(Hkv, 1, d, device="cuda", generator=gen))

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    rows = torch.zeros(B, Hkv, T_max, 5 * d // 4, dtype=torch.uint8, device="cuda")
    lens = _lens(case)
    held = T if case["op"] == "read" else 0
    for b in range(B):  # a sequence at a time, in pieces: the fp32 copies stay small
        end = min(T_max, lens[b] + held)
        for t0 in range(0, end, 16384):
            n = min(16384, end - t0)
            kq = _quantise(normal(Hkv, n, d) * chan)
            rows[b, :, t0: t0 + n] = _pack(kq, _quantise(normal(Hkv, n, d)))
    s = dict(case=dict(case), rows=rows, scale=scale,
             turns=turns.cuda(),
             starts=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             counts=torch.tensor(_counts(case), dtype=torch.int32, device="cuda"))
    if case["op"] != "read":
        # A decode step's new token has its heads side by side; other rows are [B, H, T, d].
        one = case["op"] == "decode"
        shape = (lambda H: (B, H, d)) if one else (lambda H: (B, H, T, d))
        kc = chan.view(Hkv, d) if one else chan
        s["q"] = normal(*shape(Hq)).bfloat16() if case["op"] != "write" else None
        s["k"] = (normal(*shape(Hkv)) * kc).bfloat16()
        s["v"] = normal(*shape(Hkv)).bfloat16()
    return s


# ------------------------------------------------------------------------- plain forms
def _new_rows(s, pos):
    """The stored values of the new keys and values (k, v [B, Hkv, T, d]) at positions pos."""
    half = s["case"]["pairs"] == "half"
    k = s["k"] if s["k"].dim() == 4 else s["k"].unsqueeze(2)
    v = s["v"] if s["v"].dim() == 4 else s["v"].unsqueeze(2)
    k = _rotate(k.double(), pos, s["turns"], half).float()
    return _dequantise(*_quantise(k)), _dequantise(*_quantise(v.float()))


def _slopes(Hq, device):
    return torch.exp2(-8.0 * (torch.arange(Hq, device=device, dtype=torch.float64) + 1) / Hq)


def _attend(s, q, k, v, qpos):
    """q [B, Hq, Tq, d] at positions qpos [B, Tq] over the keys 0 .. of k, v [B, Hkv, Tk, d]."""
    c = s["case"]
    B, Hq, Tq, d = q.shape
    Hkv, Tk = k.shape[1], k.shape[2]
    q = _rotate(q.double(), qpos.unsqueeze(1), s["turns"], c["pairs"] == "half").float()
    x = torch.matmul(q.reshape(B, Hkv, -1, d), k.transpose(-1, -2)) * s["scale"]
    x = x.view(B, Hq, Tq, Tk)
    kpos = torch.arange(Tk, device=q.device)
    dist = qpos.unsqueeze(-1) - kpos
    seen = dist >= 0
    if c["window"] > 0:
        seen &= (dist < c["window"]) | (kpos < c["n_sink"])
    if c["method"] == "alibi":
        x -= _slopes(Hq, q.device).float().view(1, -1, 1, 1) * dist.unsqueeze(1).float()
    x.masked_fill_(~seen.unsqueeze(1), -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, Hkv, -1, Tk), v).view(B, Hq, Tq, d) / l
    return o, (m + torch.log(l)).squeeze(-1)


def _run_plain(s):
    c = s["case"]
    B, T, d = c["B"], c["T"], c["d"]
    dev = s["rows"].device
    step = torch.arange(T, device=dev)
    if c["op"] == "write":
        live = (step < s["counts"].unsqueeze(1)).view(B, 1, T, 1)
        k, v = _new_rows(s, (s["starts"].unsqueeze(1) + step).unsqueeze(1))
        return (k * live).bfloat16(), (v * live).bfloat16()
    if c["op"] == "read":
        to = torch.bfloat16 if c["dtype"] == "bf16" else torch.float16
        live = (step < s["counts"].unsqueeze(1)).view(B, 1, T, 1)
        at = (s["starts"].unsqueeze(1) + step).clamp_max(c["T_max"] - 1)
        at = at.view(B, 1, T, 1).expand(-1, c["Hkv"], -1, s["rows"].shape[-1])
        k, v = _unpack(s["rows"].gather(2, at.long()), d)
        return (k * live).to(to), (v * live).to(to)
    # The cache with the new rows in place, as values.
    Tk = _key_length(c) if c["op"] == "decode" else c["len_hi"] + T
    k, v = _unpack(s["rows"][:, :, :Tk], d)
    pos = s["starts"].unsqueeze(1) + step
    kn, vn = _new_rows(s, pos.unsqueeze(1))
    at = pos.view(B, 1, T, 1).expand(-1, c["Hkv"], -1, d).long()
    k.scatter_(2, at, kn)
    v.scatter_(2, at, vn)
    q = s["q"] if c["op"] == "chunk" else s["q"].unsqueeze(2)
    o, lse = _attend(s, q, k, v, pos)
    if c["op"] == "chunk":
        return o.bfloat16(), kn.bfloat16(), vn.bfloat16()
    o, lse, kn, vn = (x.squeeze(2) for x in (o, lse, kn, vn))
    return o.bfloat16(), lse, kn.bfloat16(), vn.bfloat16()


# ------------------------------------------------------------------------ the operators
def _kept(s):
    """What a user's program keeps between calls: the frequency table and a workspace."""
    from yarn_position_scaling_b200 import api
    if "table" not in s:
        c = s["case"]
        s["table"] = api.rope_freq_table(c["d"], c["base"], c["L_train"], c["scale"],
                                         c["method"], pairs=c["pairs"])
        n = 0
        if c["op"] == "decode":
            n = api.attn_decode_kv4_workspace_bytes(c["B"], c["Hq"], c["Hkv"], c["d"])
        elif c["op"] == "chunk":
            n = api.attn_prefill_chunk_kv4_workspace_bytes(c["B"], c["Hq"], c["Hkv"], c["T"],
                                                           c["d"], c["len_hi"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return api, s["table"], s["workspace"]


def _run_own(s):
    api, table, ws = _kept(s)
    c = s["case"]
    B, Hkv, T, d = c["B"], c["Hkv"], c["T"], c["d"]
    if c["op"] == "write":
        api.kv4_write(s["k"], s["v"], s["rows"], table, starts=s["starts"], counts=s["counts"])
        return api.kv4_read(s["rows"], T, starts=s["starts"], counts=s["counts"])
    if c["op"] == "read":
        to = torch.bfloat16 if c["dtype"] == "bf16" else torch.float16
        return api.kv4_read(s["rows"], T, starts=s["starts"], counts=s["counts"], dtype=to)
    if c["op"] == "decode":
        lse = torch.empty(B, c["Hq"], device="cuda")
        kn, vn = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        o = api.attn_decode_kv4(s["q"], s["k"], s["v"], s["rows"], s["starts"], table,
                                c["window"], c["n_sink"], lse=lse, k_stored=kn, v_stored=vn,
                                workspace=ws)
        return o, lse, kn, vn
    P0 = c["len_hi"]
    o = api.attn_prefill_chunk_kv4(s["q"], s["k"], s["v"], s["rows"], P0, table, c["window"],
                                   c["n_sink"], workspace=ws)
    return (o,) + tuple(api.kv4_read(s["rows"], T, pos0=P0))


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ------------------------------------------------------------------------------- work
def _visible(c, pos):
    """Keys that the query at position pos sees."""
    if c["window"] <= 0:
        return pos + 1
    w0 = max(0, pos + 1 - c["window"])
    return pos + 1 - w0 + min(w0, c["n_sink"])


def work(case):
    c = case
    B, Hq, Hkv, d, T = (c[n] for n in ("B", "Hq", "Hkv", "d", "T"))
    row, val = 5 * d // 4, 4 * d  # a row in the cache, and its key and value in 16 bits
    if c["op"] == "write":
        n = sum(_counts(c)) * Hkv
        return dict(bytes=float(n * (val + row + val)), flops=float(n * 20 * d))
    if c["op"] == "read":
        n = sum(_counts(c)) * Hkv
        return dict(bytes=float(n * (row + val)), flops=float(n * 4 * d))
    if c["op"] == "decode":
        keys = [_visible(c, n) for n in _lens(c)]
        return dict(bytes=float(Hkv * sum(keys) * row + B * (2 * Hkv * val + 4 * Hq * d)),
                    flops=float(sum(keys) * Hq * 4 * d))
    P0 = c["len_hi"]
    if c["window"] > 0:
        pairs = sum(_visible(c, P0 + t) for t in range(T))
        first = max(0, P0 + 1 - c["window"])
        keys = P0 + T - first + min(first, c["n_sink"])
    else:
        pairs, keys = T * P0 + T * (T + 1) // 2, P0 + T
    return dict(bytes=float(B * (Hkv * (keys * row + 2 * T * val) + 4 * T * Hq * d)),
                flops=float(B * Hq * pairs * 4 * d))


# ------------------------------------------------- the definition, in 64 bits, on its own
def _turned(case, x, pos):
    """x [H, T, d] in 64 bits as complex pairs times e^(i pos theta)."""
    turns, _ = _turns(case)
    turns = turns.to(x.device)
    a = pos.double()[:, None] * turns
    z = torch.polar(torch.ones_like(a), torch.remainder(a, 1.0) * (2.0 * math.pi))
    d = x.shape[-1]
    if case["pairs"] == "half":
        y = torch.complex(x[..., : d // 2].contiguous(), x[..., d // 2:].contiguous()) * z
        return torch.cat([y.real, y.imag], -1)
    y = torch.view_as_complex(x.reshape(*x.shape[:-1], d // 2, 2).contiguous()) * z
    return torch.view_as_real(y).reshape(x.shape)


def _stored(x):
    """What four bits keep of x [H, T, d] in 64 bits."""
    H, T, d = x.shape
    g = x.reshape(H, T, d // GROUP, GROUP)
    lo = g.min(-1, keepdim=True).values.half().double()
    st = ((g.max(-1, keepdim=True).values - lo) / 15.0).half().double().clamp(min=0.0)
    q = torch.where(st > 0, (g - lo) / torch.where(st > 0, st, torch.ones_like(st)),
                    torch.zeros_like(g))
    return (q.round().clamp(0, 15) * st + lo).reshape(H, T, d)


def _half_of_rows(rows, d, which):
    """rows [H, T, 5d/4] of bytes -> the keys (which = 0) or values (1) [H, T, d] in 64 bits."""
    b = rows[..., which * (d // 2): (which + 1) * (d // 2)].to(torch.int64)
    at = d + which * (d // 8)
    par = rows[..., at: at + d // 8].contiguous().view(torch.float16).double()
    e = torch.arange(d, device=rows.device)
    grp, r = e // GROUP, e % GROUP
    # Byte and nibble of element e: a key word is 8 codes, a value unit 4.
    w = 8 if which == 0 else 4
    nib = ((r // w) * (d // GROUP) + grp) * w + r % w
    code = (b[..., nib // 2] >> (4 * (nib % 2))) & 15
    return code.double() * par[..., 2 * grp] + par[..., 2 * grp + 1]


def _held(rows, d):
    return _half_of_rows(rows, d, 0), _half_of_rows(rows, d, 1)


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    dev, d, T = s["rows"].device, c["d"], c["T"]
    lens, counts = _lens(c), _counts(c)
    if c["op"] == "read":
        ks, vs = [], []
        for b in range(c["B"]):
            k = torch.zeros(c["Hkv"], T, d, dtype=torch.float64, device=dev)
            v = torch.zeros_like(k)
            n = counts[b]
            k[:, :n], v[:, :n] = _held(s["rows"][b, :, lens[b]: lens[b] + n], d)
            ks.append(k)
            vs.append(v)
        return torch.stack(ks), torch.stack(vs)
    outs = []
    for b in range(c["B"]):
        pos = lens[b] + torch.arange(T, device=dev)
        kb = s["k"][b].double().reshape(c["Hkv"], T, d)
        vb = s["v"][b].double().reshape(c["Hkv"], T, d)
        kn, vn = _stored(_turned(c, kb, pos)), _stored(vb)
        if c["op"] == "write":
            kn[:, counts[b]:] = 0
            vn[:, counts[b]:] = 0
            outs.append((kn, vn))
            continue
        q = _turned(c, s["q"][b].double().reshape(c["Hq"], T, d), pos)
        end = lens[b] + T
        g = c["Hq"] // c["Hkv"]
        kpos = torch.arange(end, device=dev)
        gap = pos[:, None] - kpos[None, :]
        hide = gap < 0
        if c["window"] > 0:
            hide = hide | ((gap >= c["window"]) & (kpos[None, :] >= c["n_sink"]))
        o, lse = [], []
        for h in range(c["Hkv"]):
            kc, vc = _held(s["rows"][b, h: h + 1, : lens[b]], d)
            kc, vc = torch.cat([kc[0], kn[h]]), torch.cat([vc[0], vn[h]])
            for j in range(h * g, (h + 1) * g):
                x = (q[j] @ kc.T) * s["scale"]
                if c["method"] == "alibi":
                    x = x - 2.0 ** (-8.0 * (j + 1) / c["Hq"]) * gap.double()
                x = x.masked_fill(hide, -math.inf)
                e = torch.logsumexp(x, -1)
                o.append(torch.exp(x - e[:, None]) @ vc)
                lse.append(e)
        outs.append((torch.stack(o), torch.stack(lse), kn, vn) if c["op"] == "decode"
                    else (torch.stack(o), kn, vn))
    outs = [torch.stack(x) for x in zip(*outs)]
    if c["op"] == "decode":
        outs = [x.squeeze(2) for x in outs]
    return tuple(outs)
