"""The 4-bit decode kernel in its steady state -- thousands of keys a block, so that rings are
refilled, references raised and accumulators folded -- in every form, output by output, and chunks
by either kernel against bounds that plain mistakes break (tests/_kv4_bounds.py, which
tests/test_kv4_bounds.py checks on the CPU)."""
import math

import pytest
import torch

from tests import _kv4 as R
from tests import _kv4_bounds as K
from tests.test_gpu_kv4 import gen_of, new_kv, randn, random_rows, table
from yarn_position_scaling_b200 import api, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    api.load()


# Query heads a KV head, for every number of columns that has a form of its own, at each head
# size; 6 x 8 segments of these lengths give a block 7 to 14 thousand keys, three folds a warp or
# more.
LENS = [131071, 100003, 70001, 131070, 90000, 4099]
HKV = 8
FORMS = [(2, 128, "interleaved"), (2, 128, "half"), (4, 128, "interleaved"), (3, 128, "half"),
         (8, 128, "interleaved"), (5, 128, "half"), (16, 128, "interleaved"), (12, 128, "half"),
         (4, 64, "interleaved"), (1, 64, "half"), (8, 64, "half"), (6, 64, "interleaved"),
         (16, 64, "interleaved"), (16, 64, "half")]
# Tokens of a chunk, and heads: one run of tokens, or two and a part.
CHUNKS = [(2, 1, 128, "half"), (4, 1, 128, "interleaved"), (2, 2, 128, "half"), (4, 2, 128, "interleaved"),
          (2, 4, 128, "half"), (8, 2, 128, "interleaved"), (4, 9, 128, "half"), (4, 1, 64, "half"),
          (2, 2, 64, "interleaved"), (8, 1, 64, "half"), (4, 4, 64, "interleaved"), (16, 3, 64, "half")]


def block_keys(total, cols):
    """Keys of a block and blocks of a 131072-key segment: one wave of 2 or 4 blocks an SM."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    keys = total / (sms * (2 if cols > 8 else 4)) + 256
    return keys, 131072 / keys + 2


def counting_cache(B, T_max, d):
    return K.counting_rows(T_max, d, "cuda").expand(B, HKV, -1, -1).contiguous()


def within(o, lse, want_o, want_lse, bounds, times=1):
    bo, bl = bounds
    eo, el = (o.double() - want_o).abs(), (lse.double() - want_lse).abs()
    assert (el <= times * bl).all(), float((el / bl).max())
    assert (eo <= times * bo).all(), float((eo / bo.clamp_min(1e-300)).max())


# ---------------------------------------------------------------------------- counting
@pytest.mark.parametrize("window,n_sink", [(0, 0), (70003, 301)])
@pytest.mark.parametrize("g,d,pairs", FORMS)
def test_decode_counts_every_key_once(g, d, pairs, window, n_sink):
    B, T_max = len(LENS), max(LENS) + 1
    cache, tab = counting_cache(B, T_max, d), table(d, pairs)
    q = torch.zeros(B, HKV * g, d, dtype=torch.bfloat16, device="cuda")
    k = randn(gen_of(g), B, HKV, d).bfloat16()
    cl = torch.tensor(LENS, dtype=torch.int32, device="cuda")
    lse = torch.empty(B, HKV * g, device="cuda")
    o = api.attn_decode_kv4(q, k, torch.zeros_like(k), cache, cl, tab, window, n_sink, lse=lse)
    api.device_status()
    for b, L in enumerate(LENS):
        want, want_lse = K.counting_result(torch.tensor([L], device="cuda"), L + 1, d, window, n_sink, cached=L)
        within(o[b], lse[b], want, want_lse, K.counting_bounds(want, want_lse))


@pytest.mark.parametrize("window,n_sink", [(0, 0), (70003, 301)])
@pytest.mark.parametrize("g,Tq,d,pairs", CHUNKS)
def test_short_chunk_counts_every_key_once(g, Tq, d, pairs, window, n_sink):
    B, P0 = 6, 131000
    cache, tab = counting_cache(B, P0 + Tq, d), table(d, pairs)
    q = torch.zeros(B, HKV * g, Tq, d, dtype=torch.bfloat16, device="cuda")
    k = randn(gen_of(g), B, HKV, Tq, d).bfloat16()
    lse = torch.empty(B, HKV * g, Tq, device="cuda")
    o = api.attn_prefill_chunk_kv4(q, k, torch.zeros_like(k), cache, P0, tab, window, n_sink, lse=lse)
    api.device_status()
    pos = P0 + torch.arange(Tq, device="cuda")
    want, want_lse = K.counting_result(pos, P0 + Tq, d, window, n_sink, cached=P0)
    within(o, lse, want, want_lse, K.counting_bounds(want, want_lse))


@pytest.mark.parametrize("window,n_sink", [(0, 0), (1, 0), (2, 1), (33, 0), (300, 70), (900, 500), (2000, 3)])
@pytest.mark.parametrize("P0,Tq", [(0, 9), (777, 7), (1001, 10), (2047, 129), (300, 400), (1024, 256)])
@pytest.mark.parametrize("d", [64, 128])
def test_chunks_count_every_key_once(P0, Tq, d, window, n_sink):
    """By the decode kernel and, with room for no more than the 16-bit rows, or with more tokens,
    by the prefill kernel, whose split over the keys adds a merge's roundings to lse."""
    B, Hq = 2, 2 * HKV
    tab = table(d)
    q = torch.zeros(B, Hq, Tq, d, dtype=torch.bfloat16, device="cuda")
    k = randn(gen_of(P0), B, HKV, Tq, d).bfloat16()
    pos = P0 + torch.arange(Tq, device="cuda")
    want, want_lse = K.counting_result(pos, P0 + Tq, d, window, n_sink, cached=P0)
    planes = (api.attn_prefill_workspace_bytes(B, HKV, P0 + Tq, d) + 255) // 256 * 256
    full = api.attn_prefill_chunk_kv4_workspace_bytes(B, Hq, HKV, Tq, d, P0)
    for n in (planes, full):
        cache = counting_cache(B, P0 + Tq, d)
        lse = torch.empty(B, Hq, Tq, device="cuda")
        o = api.attn_prefill_chunk_kv4(q, k, torch.zeros_like(k), cache, P0, tab, window, n_sink, lse=lse,
                                       workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))
        api.device_status()
        within(o, lse, want, want_lse, K.counting_bounds(want, want_lse), 4)


# ------------------------------------------------------------------- references that rise
@pytest.mark.parametrize("window,n_sink", [(0, 0), (50001, 130)])
@pytest.mark.parametrize("g,d,pairs", FORMS)
def test_decode_raises_its_references_all_along(g, d, pairs, window, n_sink):
    """ALiBi alone: scores rise by 2^(-8 (h + 1) / Hq) a key, through every tile.  Weights that count
    have scores within 32 log2 units of the best; the slope's roundings (exp2 2^-22, its product,
    quotient and the bias's FMA 2^-24 each) move those by 2^-16.  All terms are positive, so what
    moves the weights (twice), rounds p s (2^-11) or cuts the sums off is relative to the output."""
    B, T_max, Hq = len(LENS), max(LENS) + 1, HKV * g
    cache, tab = counting_cache(B, T_max, d), table(d, pairs, "alibi")
    cache[..., d // 2: d] = torch.randint(0, 256, (T_max, d // 2), device="cuda", generator=gen_of(d), dtype=torch.uint8)
    q = torch.zeros(B, Hq, d, dtype=torch.bfloat16, device="cuda")
    k = randn(gen_of(g), B, HKV, d).bfloat16()
    cl = torch.tensor(LENS, dtype=torch.int32, device="cuda")
    lse = torch.empty(B, Hq, device="cuda")
    o = api.attn_decode_kv4(q, k, k, cache, cl, tab, window, n_sink, lse=lse)
    api.device_status()
    keys, blocks = block_keys(sum(LENS) * HKV, g)
    sums = 32 * 2.0 ** -22 + (keys / 16 + blocks + 64) * 2.0 ** -24
    slope = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device="cuda", dtype=torch.float64) / Hq)
    for b, L in enumerate(LENS):
        n = torch.arange(L + 1, device="cuda")
        seen = K.visible(torch.tensor([L], device="cuda"), L + 1, window, n_sink)
        x = (-slope[:, None] * (L - n).double()).masked_fill(~seen, -math.inf)
        e = torch.logsumexp(x, -1)
        p = torch.exp(x - e[:, None])
        for h in (0, HKV - 1):
            at = slice(h * g, (h + 1) * g)
            (c, s, z) = R.decode_rows(cache[b, h, : L + 1])[1]
            v = R.values(c, s, z)
            want = p[at] @ v
            amp = p[at] @ R.values(c, s, z.abs())   # the new row's minimum is not positive
            bo = (2.0 ** -15 + 2.0 ** -11 + sums) * amp + 2.0 ** -8 * want.abs()
            within(o[b, at], lse[b, at], want, e[at], (bo, 2.0 ** -16 + sums + 2.0 ** -22 * e[at].abs()))


# ------------------------------------------------------------------------------ random
def check_heads(q, rows, pos, tab, o, lse, bounds, h, g, Hq, window=0, n_sink=0):
    """Query heads of KV head h: q [Hq, Tq, d], o and lse likewise, rows [Tk, 5d/4]."""
    at = slice(h * g, (h + 1) * g)
    r = K.attend(R.rotate(q[at], pos, tab), rows, pos, tab, h * g, Hq, window, n_sink)
    within(o[at], lse[at], r["o"], r["lse"], bounds(r))


@pytest.mark.parametrize("method,window,n_sink", [("yarn", 0, 0), ("yarn", 70003, 301), ("alibi", 0, 0)])
@pytest.mark.parametrize("g,d,pairs", FORMS)
def test_decode_over_long_caches(g, d, pairs, method, window, n_sink):
    B, T_max, Hq = len(LENS), max(LENS) + 1, HKV * g
    gen, tab = gen_of(100 + g + d), table(d, pairs, method)
    cache = random_rows(gen, B, HKV, T_max, d)
    q = randn(gen, B, Hq, d).bfloat16()
    k, v = (x.squeeze(2) for x in new_kv(gen, B, HKV, 1, d))
    lse = torch.empty(B, Hq, device="cuda")
    cl = torch.tensor(LENS, dtype=torch.int32, device="cuda")
    o = api.attn_decode_kv4(q, k, v, cache, cl, tab, window, n_sink, lse=lse)
    api.device_status()
    keys, blocks = block_keys(sum(LENS) * HKV, g)
    for b, h in ((0, 0), (1, 5), (2, HKV - 1), (5, 3)):
        L = LENS[b]
        # ALiBi's bias is one more term of the score, rounded with it: of weights that count, at most
        # 32 log2 units beside the score itself.
        def bounds(r):
            r = dict(r, logit=r["logit"] + (32 if method == "alibi" else 0))
            return K.decode_bounds(r, d, keys, blocks)
        check_heads(q[b][:, None], cache[b, h, : L + 1], torch.tensor([L], device="cuda"), tab, o[b][:, None],
                    lse[b][:, None], bounds, h, g, Hq, window, n_sink)


@pytest.mark.parametrize("window,n_sink", [(0, 0), (70003, 301)])
@pytest.mark.parametrize("g,Tq,d,pairs", CHUNKS)
def test_short_chunk_over_a_long_cache(g, Tq, d, pairs, window, n_sink):
    B, P0, Hq = 6, 131000, HKV * g
    gen, tab = gen_of(200 + g + d), table(d, pairs)
    cache = random_rows(gen, B, HKV, P0 + Tq, d)
    q = randn(gen, B, Hq, Tq, d).bfloat16()
    k, v = new_kv(gen, B, HKV, Tq, d)
    lse = torch.empty(B, Hq, Tq, device="cuda")
    o = api.attn_prefill_chunk_kv4(q, k, v, cache, P0, tab, window, n_sink, lse=lse)
    api.device_status()
    keys, blocks = block_keys(B * HKV * P0, g * Tq)
    pos = P0 + torch.arange(Tq, device="cuda")
    for b, h in ((0, 0), (5, HKV - 1)):
        check_heads(q[b], cache[b, h], pos, tab, o[b], lse[b], lambda r: K.decode_bounds(r, d, keys, blocks),
                    h, g, Hq, window, n_sink)


@pytest.mark.parametrize("method,window,n_sink", [("yarn", 0, 0), ("yarn", 1, 0), ("yarn", 5, 2), ("yarn", 64, 4),
                                                  ("yarn", 300, 70), ("yarn", 900, 500), ("alibi", 0, 0),
                                                  ("alibi", 100, 3)])
@pytest.mark.parametrize("g,Hkv,Tq,d,pairs", [(4, 2, 9, 128, "half"), (1, 3, 2, 128, "interleaved"),
                                              (2, 2, 10, 64, "interleaved"), (8, 1, 4, 64, "half"),
                                              (3, 4, 7, 128, "interleaved"), (16, 1, 2, 128, "half")])
def test_short_chunk_within_sharp_bounds(g, Hkv, Tq, d, pairs, method, window, n_sink):
    P0, Hq = 1001, g * Hkv
    gen, tab = gen_of(300 + g + d + window), table(d, pairs, method)
    cache = random_rows(gen, 2, Hkv, P0 + Tq, d)
    q = randn(gen, 2, Hq, Tq, d).bfloat16()
    k, v = new_kv(gen, 2, Hkv, Tq, d)
    lse = torch.empty(2, Hq, Tq, device="cuda")
    o = api.attn_prefill_chunk_kv4(q, k, v, cache, P0, tab, window, n_sink, lse=lse)
    api.device_status()
    pos = P0 + torch.arange(Tq, device="cuda")

    def bounds(r):
        r = dict(r, logit=r["logit"] + (32 if method == "alibi" else 0))
        return K.decode_bounds(r, d, P0 + Tq, 40)
    for b in range(2):
        for h in range(Hkv):
            check_heads(q[b], cache[b, h], pos, tab, o[b], lse[b], bounds, h, g, Hq, window, n_sink)


@pytest.mark.parametrize("method,window,n_sink", [("yarn", 0, 0), ("yarn", 1, 0), ("yarn", 64, 4), ("yarn", 300, 70),
                                                  ("yarn", 900, 500), ("alibi", 0, 0)])
@pytest.mark.parametrize("g,Hkv,P0,Tq,d,pairs", [(4, 2, 777, 513, 128, "half"), (1, 3, 0, 300, 64, "interleaved"),
                                                 (2, 2, 2048, 129, 128, "interleaved"),
                                                 (8, 1, 1000, 200, 64, "half"), (20, 2, 333, 200, 64, "interleaved"),
                                                 (2, 1, 20000, 256, 128, "interleaved")])
def test_chunk_within_sharp_bounds(g, Hkv, P0, Tq, d, pairs, method, window, n_sink):
    """The prefill kernel over fp16 copies of the rows.  ALiBi's bias enters its scores in fp32, as
    one more rounding of a term of at most 32 log2 units where the weight counts."""
    Hq = g * Hkv
    gen, tab = gen_of(400 + g + d + window), table(d, pairs, method)
    cache = random_rows(gen, 1, Hkv, P0 + Tq, d)
    q = randn(gen, 1, Hq, Tq, d).bfloat16()
    k, v = new_kv(gen, 1, Hkv, Tq, d)
    lse = torch.empty(1, Hq, Tq, device="cuda")
    o = api.attn_prefill_chunk_kv4(q, k, v, cache, P0, tab, window, n_sink, lse=lse)
    api.device_status()
    pos = P0 + torch.arange(Tq, device="cuda")

    def bounds(r):
        r = dict(r, logit=r["logit"] + (32 if method == "alibi" else 0))
        return K.chunk_bounds(r, P0 + Tq)
    for h in range(Hkv):
        check_heads(q[0], cache[0, h], pos, tab, o[0], lse[0], bounds, h, g, Hq, window, n_sink)
