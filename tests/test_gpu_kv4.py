"""The 4-bit KV cache on the GPU against plain forms in 64 bits (tests/_kv4.py)."""
import math

import pytest
import torch

from tests import _kv4 as R
from yarn_position_scaling_b200 import api, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    api.load()


def table(d, pairs="interleaved", method="yarn"):
    return api.rope_freq_table(d, 500000.0, 8192, 16.0, method, pairs=pairs)


def randn(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


def gen_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def new_kv(gen, B, Hkv, T, d):
    """Keys whose channels differ in size, values, bf16 [B, Hkv, T, d]."""
    k = randn(gen, B, Hkv, T, d) * torch.exp(0.5 * randn(gen, 1, Hkv, 1, d))
    return k.bfloat16(), randn(gen, B, Hkv, T, d).bfloat16()


def random_rows(gen, B, Hkv, T_max, d):
    """A cache of any bytes in its codes and moderate scales and minima."""
    G = d // 32
    rows = torch.randint(0, 256, (B, Hkv, T_max, 5 * d // 4), device="cuda", generator=gen,
                         dtype=torch.uint8)
    par = torch.stack([0.05 + 0.3 * torch.rand(B, Hkv, T_max, 2 * G, device="cuda", generator=gen),
                       -1.5 + 0.5 * randn(gen, B, Hkv, T_max, 2 * G)], -1)
    rows[..., d:] = par.half().flatten(-2).view(torch.uint8)
    return rows


def stored_rows(k, v, pos, tab):
    """Codes, s, z of keys k at positions pos and of values v, from the format's definition."""
    return R.quantise(R.rotate(k, pos, tab).float()), R.quantise(v.float())


def check_rows(rows, k, v, pos, tab):
    for (c0, s0, z0), (c1, s1, z1) in zip(R.decode_rows(rows), stored_rows(k, v, pos, tab)):
        assert torch.equal(s0, s1) and torch.equal(z0, z1) and torch.equal(c0, c1)


# ----------------------------------------------------------------------------- write, read
@pytest.mark.parametrize("d,pairs", [(64, "interleaved"), (64, "half"), (128, "interleaved"),
                                     (128, "half")])
@pytest.mark.parametrize("B,Hkv,T,pos0", [(1, 1, 1, 0), (2, 3, 17, 5), (1, 8, 257, 131000),
                                          (3, 2, 31, 1)])
def test_write_is_the_formats_definition(d, pairs, B, Hkv, T, pos0):
    gen, tab = gen_of(T * d + Hkv), table(d, pairs)
    k, v = new_kv(gen, B, Hkv, T, d)
    cache = random_rows(gen, B, Hkv, pos0 + T + 3, d)
    before = cache.clone()
    api.kv4_write(k, v, cache, tab, pos0=pos0)
    api.device_status()
    pos = pos0 + torch.arange(T, device="cuda")
    check_rows(cache[:, :, pos0: pos0 + T], k, v, pos, tab)
    assert torch.equal(cache[:, :, :pos0], before[:, :, :pos0])
    assert torch.equal(cache[:, :, pos0 + T:], before[:, :, pos0 + T:])


def test_write_keeps_within_half_a_step():
    gen, d, T = gen_of(3), 128, 700
    tab = table(d)
    k, v = new_kv(gen, 1, 2, T, d)
    cache = api.kv4_cache(1, 2, T, d)
    api.kv4_write(k, v, cache, tab)
    want = (R.rotate(k, torch.arange(T, device="cuda"), tab), v.double())
    for (c, s, z), x in zip(R.decode_rows(cache), want):
        err = (R.values(c, s, z) - x).abs().unflatten(-1, (-1, 32))
        # Half a step; s and z are fp16: up to 15 s 2^-11 at the top code and 2^-11 |z| at the
        # bottom; fp32 rounding of the rotated key below 2^-22 |x|.
        bound = s.double() * (0.5 + 15 * 2.0 ** -11) + z.double().abs() * 2.0 ** -11 + \
            2.0 ** -22 * x.abs().unflatten(-1, (-1, 32))
        assert (err <= bound).all()


@pytest.mark.parametrize("d,pairs", [(64, "half"), (128, "interleaved")])
def test_ragged_batch_with_starts_and_counts(d, pairs):
    gen, tab = gen_of(9), table(d, pairs)
    B, Hkv, T, T_max = 6, 2, 40, 100
    k, v = new_kv(gen, B, Hkv, T, d)
    starts, counts = [0, 60, 7, 55, 3, 99], [40, 40, 0, 33, 1, 1]
    cs = torch.tensor(starts, dtype=torch.int32, device="cuda")
    cc = torch.tensor(counts, dtype=torch.int32, device="cuda")
    cache = random_rows(gen, B, Hkv, T_max, d)
    before = cache.clone()
    api.kv4_write(k, v, cache, tab, starts=cs, counts=cc)
    ko = torch.full((B, Hkv, T, d), 7.0, dtype=torch.bfloat16, device="cuda")
    vo = torch.full_like(ko, 8.0)
    api.kv4_read(cache, T, starts=cs, counts=cc, k=ko, v=vo)
    kz, vz = api.kv4_read(cache, T, starts=cs, counts=cc)
    api.device_status()
    for b in range(B):
        s, n = starts[b], counts[b]
        if n:
            check_rows(cache[b, :, s: s + n], k[b, :, :n], v[b, :, :n],
                       s + torch.arange(n, device="cuda"), tab)
        assert torch.equal(cache[b, :, :s], before[b, :, :s])
        assert torch.equal(cache[b, :, s + n:], before[b, :, s + n:])
        (kc, ks, kz_), (vc, vs, vz_) = R.decode_rows(cache[b, :, s: s + n])
        want_k = R.values(kc, ks, kz_).float().bfloat16()
        want_v = R.values(vc, vs, vz_).float().bfloat16()
        assert torch.equal(ko[b, :, :n], want_k) and torch.equal(vo[b, :, :n], want_v)
        assert (ko[b, :, n:] == 7).all() and (vo[b, :, n:] == 8).all()
        assert torch.equal(kz[b, :, :n], want_k) and torch.equal(vz[b, :, :n], want_v)
        assert not kz[b, :, n:].any() and not vz[b, :, n:].any()


@pytest.mark.parametrize("d", [64, 128])
def test_strided_inputs_and_outputs(d):
    gen, tab = gen_of(4), table(d)
    B, Hkv, T = 2, 3, 37
    k, v = new_kv(gen, B, Hkv, T, d)
    kt = k.transpose(1, 2).contiguous().transpose(1, 2)            # [B, T, H, d] in memory
    wide = torch.zeros(B, Hkv, T, 2 * d, dtype=torch.bfloat16, device="cuda")
    wide[..., d:] = v
    a, b = api.kv4_cache(B, Hkv, T, d), api.kv4_cache(B, Hkv, T, d)
    api.kv4_write(k, v, a, tab)
    api.kv4_write(kt, wide[..., d:], b, tab)
    assert torch.equal(a, b)
    ko, vo = api.kv4_read(a, T)
    k2 = torch.zeros(B, T, Hkv, d, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    v2 = torch.zeros(B, Hkv, T, 3 * d, dtype=torch.bfloat16, device="cuda")
    api.kv4_read(a, T, k=k2, v=v2[..., d: 2 * d])
    api.device_status()
    assert torch.equal(k2, ko) and torch.equal(v2[..., d: 2 * d], vo)
    assert not v2[..., :d].any() and not v2[..., 2 * d:].any()
    # One head and one sequence of a larger tensor: strides of length-one axes do not matter.
    api.kv4_write(k[:1, 1:2], v[:1, 1:2], b[:1, :1].contiguous(), tab)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
def test_read_rounds_once(d, dtype):
    gen = gen_of(11)
    rows = random_rows(gen, 2, 2, 333, d)
    k, v = api.kv4_read(rows, 300, pos0=20, dtype=dtype)
    api.device_status()
    for got, (c, s, z) in zip((k, v), R.decode_rows(rows[:, :, 20:320])):
        assert torch.equal(got, R.values(c, s, z).float().to(dtype))


def test_constant_groups_and_the_ends_of_the_range():
    d, T = 128, 6
    tab = table(d, method="alibi")  # no rotation: the keys stay as they are
    x = torch.zeros(1, 1, T, d)
    x[0, 0, 1] = 5.0
    x[0, 0, 2] = -3.140625
    x[0, 0, 3, ::2] = 65280.0
    x[0, 0, 3, 1::2] = -65280.0
    x[0, 0, 4] = torch.linspace(-1e-6, 1e-6, d)
    x[0, 0, 5, 17] = 1e-30
    x = x.bfloat16().cuda()
    cache = api.kv4_cache(1, 1, T, d)
    api.kv4_write(x, x, cache, tab)
    api.device_status()
    check_rows(cache, x, x, torch.arange(T, device="cuda"), tab)
    k, v = api.kv4_read(cache, T)
    assert torch.equal(k[0, 0, :3].float(), x[0, 0, :3].float().half().float())
    assert torch.equal(k, v) and torch.isfinite(k.float()).all()


@pytest.mark.parametrize("bad", [65536.0, -1e30, math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("which", ["k", "v"])
def test_values_outside_the_range_are_reported_and_stored_finite(bad, which):
    d = 64
    tab = table(d, method="alibi")
    kv = {n: torch.ones(1, 2, 3, d, dtype=torch.bfloat16, device="cuda") for n in "kv"}
    kv[which][0, 1, 2, 40] = bad
    cache = api.kv4_cache(1, 2, 3, d)
    api.kv4_write(kv["k"], kv["v"], cache, tab)
    with pytest.raises(api.YarnAttnError) as ei:
        api.device_status()
    assert ei.value.code == api.YR_ERANGE
    k, v = api.kv4_read(cache, 3)
    api.device_status()
    got = (k if which == "k" else v).float()
    assert torch.isfinite(got).all()
    assert abs(float(got[0, 1, 2, 40])) > 65000
    ones = torch.ones_like(got, dtype=torch.bool)
    ones[0, 1, 2, 32:] = False
    assert (got[ones] == 1).all()


def test_row_ranges_outside_the_cache_are_skipped_and_reported():
    d, T, T_max = 64, 8, 20
    gen, tab = gen_of(1), table(64)
    k, v = new_kv(gen, 5, 1, T, d)
    starts = torch.tensor([13, -1, 0, 0, 12], dtype=torch.int32, device="cuda")
    counts = torch.tensor([8, 8, 9, -1, 8], dtype=torch.int32, device="cuda")
    cache = random_rows(gen, 5, 1, T_max, d)
    before = cache.clone()
    api.kv4_write(k, v, cache, tab, starts=starts, counts=counts)
    with pytest.raises(api.YarnAttnError) as ei:
        api.device_status()
    assert ei.value.code == api.YR_EINVAL
    assert torch.equal(cache[:4], before[:4])
    check_rows(cache[4, :, 12:20], k[4], v[4], 12 + torch.arange(8, device="cuda"), tab)
    ko, vo = api.kv4_read(cache, T, starts=starts, counts=counts)
    with pytest.raises(api.YarnAttnError):
        api.device_status()
    assert not ko[:4].any() and not vo[:4].any() and ko[4].any()
    api.device_status()


# --------------------------------------------------------------------------------- decode
def run_decode(gen, Hq, Hkv, d, lens, T_max, pairs="interleaved", method="yarn", window=0,
               n_sink=0, cache=None, poison=False):
    B, tab = len(lens), table(d, pairs, method)
    cache = random_rows(gen, B, Hkv, T_max, d) if cache is None else cache
    if poison:  # what no query sees holds NaN and infinite scales and minima
        for b, L in enumerate(lens):
            hide = torch.ones(T_max, dtype=torch.bool, device="cuda")
            n = torch.arange(T_max, device="cuda")
            hide &= ~((n <= L) & ((n > L - window) | (n < n_sink))) if window else n > L
            cache[b][:, hide] = 255
    before = cache.clone()
    q = randn(gen, B, Hq, d).bfloat16()
    k, v = (x.squeeze(2) for x in new_kv(gen, B, Hkv, 1, d))
    lse = torch.empty(B, Hq, device="cuda")
    ks, vs = torch.empty_like(k), torch.empty_like(v)
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o = api.attn_decode_kv4(q, k, v, cache, cl, tab, window, n_sink, lse=lse, k_stored=ks,
                            v_stored=vs)
    api.device_status()
    for b, L in enumerate(lens):
        pos = torch.tensor([L], device="cuda")
        check_rows(cache[b, :, L: L + 1], k[b][:, None], v[b][:, None], pos, tab)
        (kc, s0, z0), (vc, s1, z1) = R.decode_rows(cache[b, :, L])
        assert torch.equal(ks[b], R.values(kc, s0, z0).float().bfloat16())
        assert torch.equal(vs[b], R.values(vc, s1, z1).float().bfloat16())
        keep = torch.arange(T_max, device="cuda") != L
        assert torch.equal(cache[b][:, keep], before[b][:, keep])
        qr = R.rotate(q[b][:, None], pos, tab)
        n = torch.arange(L + 1, device="cuda")
        see = torch.ones_like(n, dtype=torch.bool)
        if window:
            see = (n > L - window) | (n < n_sink)
        rows = cache[b, :, : L + 1].clone()
        rows[:, ~see] = 0
        ro, rl, amp, logit = (x.squeeze(1) for x in R.attend(qr, rows, pos, tab, window, n_sink))
        bo, bl = R.decode_bounds(ro, rl, amp, logit, int(see.sum()), d)
        eo, el = (o[b].double() - ro).abs(), (lse[b].double() - rl).abs()
        assert (eo <= bo).all(), (b, L, float((eo / bo).max()))
        assert (el <= bl).all(), (b, L, float((el / bl).max()))
    return o


LENS = [0, 1, 15, 16, 63, 64, 127, 128, 129, 1000, 2499]


@pytest.mark.parametrize("pairs", ["interleaved", "half"])
@pytest.mark.parametrize("Hq,Hkv,d", [(32, 8, 128), (4, 4, 64), (16, 1, 128), (16, 1, 64),
                                      (9, 3, 128), (14, 2, 64), (1, 1, 128), (24, 2, 128)])
def test_decode_heads_and_lengths(Hq, Hkv, d, pairs):
    run_decode(gen_of(Hq + d), Hq, Hkv, d, LENS, 2500, pairs)


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (63, 0), (64, 4), (300, 5), (300, 129),
                                           (2000, 600), (5000, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_window_and_sinks_read_only_what_is_seen(window, n_sink, d):
    run_decode(gen_of(window + d), 8, 2, d, LENS, 2501, window=window, n_sink=n_sink, poison=True)


@pytest.mark.parametrize("window,n_sink", [(0, 0), (200, 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_alibi(window, n_sink, d):
    run_decode(gen_of(5), 12, 4, d, [0, 77, 901, 2400], 2401, method="alibi", window=window,
               n_sink=n_sink, poison=True)


def test_decode_nothing_behind_the_length_is_read():
    run_decode(gen_of(6), 8, 2, 128, [0, 3, 500], 600, poison=True)


def test_decode_many_and_single_sequences():
    run_decode(gen_of(7), 8, 4, 64, [(i * 37) % 200 for i in range(70)], 201)
    run_decode(gen_of(8), 4, 1, 128, [30000], 30001)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_sums_over_many_keys_do_not_drift(d):
    """Values of both signs cancel over 128K keys of like weight, while the codes' own sums only
    grow, and the tensor cores cut their sums off: each 16 keys take up to two units in the last
    place, 2^-22, off a sum that grows evenly over the 512 keys between two folds, 32 / 2 times
    2^-22 of it in all.  That part has one sign: seen in the mean over heads and dimensions, where
    the roundings to nearest (p s to 2^-11 of terms that add up like the root of their number, o
    to 2^-8) are left as their six standard deviations."""
    B, H, L = 24, 8, 131071
    gen, tab = gen_of(30 + d), table(d)
    rows = torch.empty(H, L + 1, 5 * d // 4, dtype=torch.uint8, device="cuda")
    rows[..., :d] = torch.randint(0, 256, (H, L + 1, d), generator=gen, dtype=torch.uint8, device="cuda")
    s = (0.5 + 0.5 * torch.rand(H, L + 1, d // 16, generator=gen, device="cuda")).half()
    par = torch.stack([s, -7.5 * s], -1).flatten(-2)
    par[..., : d // 16] *= 0.25  # keys
    rows[..., d:] = par.view(torch.uint8)
    cache = rows.expand(B, -1, -1, -1).contiguous()
    q, k = randn(gen, H, d).bfloat16(), randn(gen, H, d).bfloat16()
    o = api.attn_decode_kv4(*(x.expand(B, -1, -1).contiguous() for x in (q, k, k)), cache,
                            torch.full((B,), L, dtype=torch.int32, device="cuda"), tab)
    api.device_status()
    pos = torch.tensor([L], device="cuda")
    ro, _, amp, _ = (x.squeeze(1) for x in R.attend(R.rotate(q[:, None], pos, tab), cache[0], pos, tab))
    n_out = ro.numel()
    # Codes up to 15; sum p^2 taken as 4 / keys (scores of deviation 1 give e / keys).
    terms = 2.0 ** -11 / 3 ** 0.5 * 15 * (4 / L) ** 0.5 / n_out ** 0.5
    rounding = 2.0 ** -8 / 3 ** 0.5 * float(ro.pow(2).mean().sqrt()) / n_out ** 0.5
    bound = 16 * 2.0 ** -22 * float(amp.mean()) + 6 * (terms + rounding)
    for b in (0, B // 2, B - 1):
        assert abs(float((o[b].double() - ro).mean())) <= bound, b


def test_decode_scales_of_very_different_size():
    """Value groups whose scales differ by tokens and groups up to 2^30, the smallest with
    the weight: each output keeps its precision relative to what its own group holds."""
    gen, d, L = gen_of(12), 128, 400
    cache = random_rows(gen, 1, 2, L + 1, d)
    par = cache[..., d:].view(torch.float16).unflatten(-1, (8, 2))
    n = torch.arange(L + 1, device="cuda")
    f = torch.where(n % 2 == 0, 2.0 ** -14, 2.0 ** 12)[None, None, :, None]
    g = 2.0 ** torch.tensor([0.0, -3.0, 2.0, -1.0], device="cuda")
    par[..., 4:, 0] = (f * g * 0.5).half()[..., :]
    par[..., 4:, 1] = (f * -3.0).half()
    # Keys of the large tokens score low: their minima follow the query's sign below.
    q = torch.ones(1, 4, d, dtype=torch.bfloat16, device="cuda")
    par[..., :4, 0] = 0.01
    par[..., :4, 1] = torch.where(n % 2 == 0, 1.0, -8.0)[None, None, :, None].half()
    cache[..., d:] = par.flatten(-2).contiguous().view(torch.uint8)
    tab = table(d, method="alibi")
    k = torch.ones(1, 2, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(1, 4, device="cuda")
    cl = torch.tensor([L], dtype=torch.int32, device="cuda")
    o = api.attn_decode_kv4(q, k, k * 2.0 ** -14, cache, cl, tab, lse=lse)
    api.device_status()
    pos = cl.long()
    ro, rl, amp, logit = (x.squeeze(1) for x in R.attend(q[0][:, None].double(), cache[0], pos, tab))
    bo, bl = R.decode_bounds(ro, rl, amp, logit, L + 1, d)
    assert ((o[0].double() - ro).abs() <= bo).all()
    assert ((lse[0].double() - rl).abs() <= bl).all()


@pytest.mark.parametrize("scale", [1e-3, 1e4])
def test_decode_queries_of_any_size(scale):
    """The query is scaled by a power of two before it is split: tiny and huge ones keep
    their 22 bits."""
    gen, d, L = gen_of(13), 128, 300
    cache = random_rows(gen, 1, 1, L + 1, d)
    tab = table(d)
    q = (randn(gen, 1, 4, d) * scale).bfloat16()
    k, v = (x.squeeze(2) for x in new_kv(gen, 1, 1, 1, d))
    lse = torch.empty(1, 4, device="cuda")
    cl = torch.tensor([L], dtype=torch.int32, device="cuda")
    o = api.attn_decode_kv4(q, k, v, cache, cl, tab, lse=lse)
    api.device_status()
    ro, rl, amp, logit = (x.squeeze(1) for x in R.attend(
        R.rotate(q[0][:, None], cl.long(), tab), cache[0], cl.long(), tab))
    bo, bl = R.decode_bounds(ro, rl, amp, logit, L + 1, d)
    assert ((o[0].double() - ro).abs() <= bo).all()
    assert ((lse[0].double() - rl).abs() <= bl).all()


@pytest.mark.parametrize("scale", [0.0, 1e-30, 1e-38])
def test_decode_alibi_of_queries_that_score_nothing(scale):
    """ALiBi alone decides: its slope is kept in the units of the scaled query."""
    gen, d, L = gen_of(16), 64, 700
    cache = random_rows(gen, 1, 2, L + 1, d)
    tab = table(d, method="alibi")
    q = (randn(gen, 1, 8, d) * scale).bfloat16()
    k, v = (x.squeeze(2) for x in new_kv(gen, 1, 2, 1, d))
    lse = torch.empty(1, 8, device="cuda")
    cl = torch.tensor([L], dtype=torch.int32, device="cuda")
    o = api.attn_decode_kv4(q, k, v, cache, cl, tab, lse=lse)
    api.device_status()
    ro, rl, amp, logit = (x.squeeze(1) for x in R.attend(q[0][:, None].double(), cache[0], cl.long(), tab))
    bo, bl = R.decode_bounds(ro, rl, amp, logit, L + 1, d)
    # The bias m (L - n) is one more term of the score, rounded with it: up to L at m = 1.
    slope = 2.0 ** (-torch.arange(1.0, 9.0, device="cuda", dtype=torch.float64))
    extra = (2.0 ** -22 * slope * L)
    assert ((o[0].double() - ro).abs() <= bo + (2 * extra)[:, None] * amp).all()
    assert ((lse[0].double() - rl).abs() <= bl + extra).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_decode_keeps_what_is_not_a_number_to_its_head(bad):
    gen, d, L = gen_of(17), 128, 200
    tab = table(d)
    cache = random_rows(gen, 1, 2, L + 1, d)
    q = randn(gen, 1, 8, d).bfloat16()
    k, v = (x.squeeze(2) for x in new_kv(gen, 1, 2, 1, d))
    cl = torch.tensor([L], dtype=torch.int32, device="cuda")
    want = api.attn_decode_kv4(q, k, v, cache, cl, tab)
    q[0, 5, 77] = bad
    got = api.attn_decode_kv4(q, k, v, cache, cl, tab)
    api.device_status()
    assert torch.isnan(got[0, 5].float()).all()
    keep = torch.arange(8, device="cuda") != 5
    assert torch.equal(got[0, keep], want[0, keep])


def test_decode_reports_bad_lengths():
    gen, d = gen_of(14), 64
    cache = random_rows(gen, 4, 2, 50, d)
    before = cache.clone()
    tab = table(d)
    q = randn(gen, 4, 4, d).bfloat16()
    k, v = (x.squeeze(2) for x in new_kv(gen, 4, 2, 1, d))
    cl = torch.tensor([-1, 10, 50, 49], dtype=torch.int32, device="cuda")
    lse = torch.empty(4, 4, device="cuda")
    o = api.attn_decode_kv4(q, k, v, cache, cl, tab, lse=lse)
    with pytest.raises(api.YarnAttnError) as ei:
        api.device_status()
    assert ei.value.code == api.YR_EINVAL
    for b, ok in enumerate([False, True, False, True]):
        assert torch.isfinite(o[b].float()).all() if ok else torch.isnan(o[b].float()).all()
        assert torch.isfinite(lse[b]).all() if ok else torch.isnan(lse[b]).all()
    assert torch.equal(cache[0], before[0]) and torch.equal(cache[2], before[2])
    alone = api.attn_decode_kv4(q[1:2], k[1:2], v[1:2], cache[1:2], cl[1:2], tab)
    api.device_status()
    ratio = (alone.float() - o[1:2].float()).abs().max()
    assert ratio <= 2 ** -7 * o[1].float().abs().max()


def test_decode_cache_offsets_beyond_32_bits():
    """The last sequence's plane starts beyond 4 GB and its rows beyond 2^31 bytes of it."""
    free, _ = torch.cuda.mem_get_info()
    d, Hkv, T_max = 128, 2, 14_000_000  # 2.24 GB a plane, 4.5 GB a sequence
    if free < 24 << 30:
        pytest.skip("needs 24 GB of free device memory")
    gen, tab = gen_of(15), table(d)
    cache = torch.zeros(2, Hkv, T_max, 160, dtype=torch.uint8, device="cuda")
    lens = [5, T_max - 2]
    for b, L in enumerate(lens):
        lo = max(0, L - 700)
        cache[b, :, lo:L] = random_rows(gen, 1, Hkv, L - lo, d)[0]
    cache[1, :, :3] = random_rows(gen, 1, Hkv, 3, d)[0]
    q = randn(gen, 2, 4, d).bfloat16()
    k, v = (x.squeeze(2) for x in new_kv(gen, 2, Hkv, 1, d))
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o = api.attn_decode_kv4(q, k, v, cache, cl, tab, 500, 3)
    ko, _ = api.kv4_read(cache, 1, starts=cl)
    api.device_status()
    L = lens[1]
    check_rows(cache[1, :, L: L + 1], k[1][:, None], v[1][:, None],
               torch.tensor([L], device="cuda"), tab)
    kc, s, z = R.decode_rows(cache[1, :, L])[0]
    assert torch.equal(ko[1, :, 0], R.values(kc, s, z).float().bfloat16())
    # The same keys in a short cache, with their distances kept: positions only enter the
    # rotation, which rows already carry, so the rows are attended as they are.
    rows = torch.cat([cache[1, :, :3], cache[1, :, L - 499: L + 1]], 1)
    qr = R.rotate(q[1][:, None], torch.tensor([L], device="cuda"), tab)
    pos = torch.tensor([502], device="cuda")
    ro, rl, amp, logit = (x.squeeze(1) for x in R.attend(qr, rows, pos, tab))
    bo, _ = R.decode_bounds(ro, rl, amp, logit, 503, d)
    assert ((o[1].double() - ro).abs() <= bo).all()


# ------------------------------------------------------------------------------------ chunk
# The chunk's attention takes rotated queries, keys, values and probabilities in fp16: a
# logit moves by up to 2 2^-11 of its magnitude scale sum |q||k| (typically far less), p by
# as much, values and p by 2^-11 each; o is rounded to bf16.
def chunk_bounds(o, lse, amp, logit):
    e = 2.0 ** -10 * logit + 2.0 ** -12
    return (2 * e + 2.0 ** -10)[..., None] * amp + 2.0 ** -8 * o.abs() + 1e-6, e + 2.0 ** -20 * lse.abs()


def run_chunk(gen, B, Hq, Hkv, d, P0, Tq, T_max, pairs="interleaved", method="yarn", window=0,
              n_sink=0, poison=False):
    tab = table(d, pairs, method)
    cache = random_rows(gen, B, Hkv, T_max, d)
    if poison:
        n = torch.arange(T_max, device="cuda")
        hide = n >= P0
        if window:
            hide |= (n <= P0 - window) & (n >= n_sink)
        cache[:, :, hide] = 255
    before = cache.clone()
    q = randn(gen, B, Hq, Tq, d).bfloat16()
    k, v = new_kv(gen, B, Hkv, Tq, d)
    lse = torch.empty(B, Hq, Tq, device="cuda")
    o = api.attn_prefill_chunk_kv4(q, k, v, cache, P0, tab, window, n_sink, lse=lse)
    api.device_status()
    pos = P0 + torch.arange(Tq, device="cuda")
    check_rows(cache[:, :, P0: P0 + Tq], k, v, pos, tab)
    keep = torch.ones(T_max, dtype=torch.bool, device="cuda")
    keep[P0: P0 + Tq] = False
    assert torch.equal(cache[:, :, keep], before[:, :, keep])
    for b in range(B):
        rows = cache[b, :, : P0 + Tq].clone()
        if window:
            n = torch.arange(P0 + Tq, device="cuda")
            rows[:, (n <= P0 - window) & (n >= n_sink)] = 0
        ro, rl, amp, logit = R.attend(R.rotate(q[b], pos, tab), rows, pos, tab, window, n_sink)
        bo, bl = chunk_bounds(ro, rl, amp, logit)
        eo, el = (o[b].double() - ro).abs(), (lse[b].double() - rl).abs()
        assert (eo <= bo).all(), float((eo / bo).max())
        assert (el <= bl).all(), float((el / bl).max())


@pytest.mark.parametrize("P0,Tq", [(0, 1), (0, 300), (1, 127), (200, 77), (1000, 1), (777, 513),
                                   (2048, 129)])
def test_chunk_offsets_and_ragged_sizes(P0, Tq):
    run_chunk(gen_of(P0 + Tq), 1, 8, 2, 128, P0, Tq, P0 + Tq + 5, poison=True)


@pytest.mark.parametrize("Hq,Hkv,d,pairs", [(4, 4, 64, "half"), (8, 1, 128, "half"),
                                            (12, 4, 64, "interleaved"), (40, 2, 64, "interleaved")])
def test_chunk_heads(Hq, Hkv, d, pairs):
    run_chunk(gen_of(Hq), 2, Hq, Hkv, d, 333, 200, 600, pairs)


@pytest.mark.parametrize("window,n_sink", [(256, 0), (300, 4), (64, 1), (1, 0), (500, 700),
                                           (3000, 2)])
def test_chunk_window_and_sinks_use_only_what_is_seen(window, n_sink):
    run_chunk(gen_of(window), 2, 4, 2, 64, 1300, 150, 1500, window=window, n_sink=n_sink,
              poison=True)


def test_chunk_alibi():
    run_chunk(gen_of(2), 1, 8, 4, 128, 500, 99, 700, method="alibi")


# A few tokens are taken by the decode kernel, tokens times heads as its columns.
@pytest.mark.parametrize("Hq,Hkv,d,pairs", [(4, 4, 128, "half"), (8, 2, 128, "interleaved"),
                                            (16, 2, 64, "half"), (16, 1, 128, "interleaved"),
                                            (6, 2, 64, "interleaved"), (10, 2, 128, "half")])
@pytest.mark.parametrize("Tq", [1, 2, 3, 7, 16, 17])
def test_short_chunk_heads_and_tokens(Hq, Hkv, d, pairs, Tq):
    run_chunk(gen_of(Hq + Tq), 2, Hq, Hkv, d, 777, Tq, 777 + Tq, pairs, poison=True)


@pytest.mark.parametrize("P0", [0, 1, 30, 31, 32, 33, 127, 4000])
def test_short_chunk_after_any_prefix(P0):
    run_chunk(gen_of(P0), 1, 8, 2, 128, P0, 9, P0 + 11, poison=True)


@pytest.mark.parametrize("window,n_sink", [(1, 0), (3, 0), (5, 2), (40, 0), (64, 4), (300, 70),
                                           (900, 500), (5000, 1)])
@pytest.mark.parametrize("d,Tq", [(64, 10), (128, 5)])
def test_short_chunk_window_and_sinks_use_only_what_is_seen(window, n_sink, d, Tq):
    run_chunk(gen_of(window + d), 2, 8, 4, d, 1001, Tq, 1100, window=window, n_sink=n_sink,
              poison=True)


@pytest.mark.parametrize("window,n_sink", [(0, 0), (100, 3)])
def test_short_chunk_alibi(window, n_sink):
    run_chunk(gen_of(3), 1, 12, 4, 128, 600, 6, 700, method="alibi", window=window, n_sink=n_sink)


@pytest.mark.parametrize("window", [0, 200])
def test_short_chunk_within_a_small_workspace(window):
    """A workspace with room for the 16-bit rows alone takes the other kernel; both are right."""
    gen, d, Hq, Hkv, P0, Tq = gen_of(23), 128, 8, 2, 600, 4
    tab = table(d)
    cache = random_rows(gen, 1, Hkv, P0 + Tq, d)
    q = randn(gen, 1, Hq, Tq, d).bfloat16()
    k, v = new_kv(gen, 1, Hkv, Tq, d)
    planes = (api.attn_prefill_workspace_bytes(1, Hkv, P0 + Tq, d) + 255) // 256 * 256
    full = api.attn_prefill_chunk_kv4_workspace_bytes(1, Hq, Hkv, Tq, d, P0)
    assert planes < full
    pos = P0 + torch.arange(Tq, device="cuda")
    for n in (planes, full):
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        o = api.attn_prefill_chunk_kv4(q, k, v, cache, P0, tab, window, workspace=ws)
        api.device_status()
        rows = cache[0].clone()
        if window:
            rows[:, : P0 + 1 - window] = 0
        ro, rl, amp, logit = R.attend(R.rotate(q[0], pos, tab), rows, pos, tab, window)
        bo, _ = chunk_bounds(ro, rl, amp, logit)
        assert ((o[0].double() - ro).abs() <= bo).all()


def test_short_chunk_meets_the_decode_kernels_bounds():
    """Its queries have 22 bits and its rows are taken exactly, as in a decode step."""
    gen, d, Hq, Hkv, P0, Tq = gen_of(29), 128, 16, 4, 1500, 4
    tab = table(d)
    cache = random_rows(gen, 1, Hkv, P0 + Tq, d)
    q = randn(gen, 1, Hq, Tq, d).bfloat16()
    k, v = new_kv(gen, 1, Hkv, Tq, d)
    lse = torch.empty(1, Hq, Tq, device="cuda")
    o = api.attn_prefill_chunk_kv4(q, k, v, cache, P0, tab, lse=lse)
    api.device_status()
    pos = P0 + torch.arange(Tq, device="cuda")
    ro, rl, amp, logit = R.attend(R.rotate(q[0], pos, tab), cache[0], pos, tab)
    bo, bl = R.decode_bounds(ro, rl, amp, logit, P0 + Tq, d)
    assert ((o[0].double() - ro).abs() <= bo).all()
    assert ((lse[0].double() - rl).abs() <= bl).all()


@pytest.mark.parametrize("d", [64, 128])
def test_chunk_does_not_depend_on_where_a_prompt_is_cut(d):
    """One chunk, two chunks, and decode steps leave the same cache and agree."""
    gen, tab = gen_of(21), table(d)
    T, cut, Hq, Hkv = 90, 70, 4, 2
    q = randn(gen, 1, Hq, T, d).bfloat16()
    k, v = new_kv(gen, 1, Hkv, T, d)
    whole, parts = api.kv4_cache(1, Hkv, T, d), api.kv4_cache(1, Hkv, T, d)
    o = api.attn_prefill_chunk_kv4(q, k, v, whole, 0, tab)

    def part(x, a, b):
        return x[:, :, a:b].contiguous()
    outs = [api.attn_prefill_chunk_kv4(part(q, 0, cut), part(k, 0, cut), part(v, 0, cut), parts,
                                       0, tab)]
    for t in range(cut, T):
        cl = torch.tensor([t], dtype=torch.int32, device="cuda")
        step = api.attn_decode_kv4(q[:, :, t].contiguous(), k[:, :, t].contiguous(),
                                   v[:, :, t].contiguous(), parts, cl, tab)
        outs.append(step.unsqueeze(2))
    api.device_status()
    assert torch.equal(whole, parts)
    # Each side is within its bound of the same 64-bit result.
    ro, rl, amp, logit = R.attend(R.rotate(q[0], torch.arange(T, device="cuda"), tab), whole[0],
                                  torch.arange(T, device="cuda"), tab)
    bo, _ = chunk_bounds(ro, rl, amp, logit)
    both = torch.cat(outs, 2)
    assert ((o[0].double() - ro).abs() <= bo).all()
    assert ((both[0].double() - ro).abs() <= bo).all()


# ------------------------------------------------------------- together, streams and graphs
def test_serving_run_of_all_of_them():
    """A padded batch of prompts is written, a second turn taken as a chunk, then tokens one
    by one; every step against the 64-bit attention over what the cache then holds."""
    gen, d, Hq, Hkv, B = gen_of(31), 128, 8, 2, 3
    tab = table(d, "half")
    T_max = 300
    cache = api.kv4_cache(B, Hkv, T_max, d)
    k, v = new_kv(gen, B, Hkv, 120, d)
    counts = torch.tensor([120, 64, 1], dtype=torch.int32, device="cuda")
    api.kv4_write(k, v, cache, tab, counts=counts)
    lens = counts.clone()
    ws = torch.empty(api.attn_decode_kv4_workspace_bytes(B, Hq, Hkv, d), dtype=torch.uint8,
                     device="cuda")
    for step in range(5):
        q = randn(gen, B, Hq, d).bfloat16()
        kn, vn = (x.squeeze(2) for x in new_kv(gen, B, Hkv, 1, d))
        o = api.attn_decode_kv4(q, kn, vn, cache, lens, tab, workspace=ws)
        api.device_status()
        for b in range(B):
            L = int(lens[b])
            pos = torch.tensor([L], device="cuda")
            r = R.attend(R.rotate(q[b][:, None], pos, tab), cache[b, :, : L + 1], pos, tab)
            ro, rl, amp, logit = (x.squeeze(1) for x in r)
            bo, _ = R.decode_bounds(ro, rl, amp, logit, L + 1, d)
            assert ((o[b].double() - ro).abs() <= bo).all()
        lens += 1
    # The longest sequence's next turn on its own, in the same cache.
    P0, Tq = int(lens[0]), 33
    one = cache[:1]
    q = randn(gen, 1, Hq, Tq, d).bfloat16()
    kn, vn = new_kv(gen, 1, Hkv, Tq, d)
    others = cache[1:].clone()
    o = api.attn_prefill_chunk_kv4(q, kn, vn, one, P0, tab)
    api.device_status()
    pos = P0 + torch.arange(Tq, device="cuda")
    ro, rl, amp, logit = R.attend(R.rotate(q[0], pos, tab), one[0, :, : P0 + Tq], pos, tab)
    bo, _ = chunk_bounds(ro, rl, amp, logit)
    assert ((o[0].double() - ro).abs() <= bo).all()
    assert torch.equal(cache[1:], others)


def _decode_case(seed, L=3000):
    gen, d, Hq, Hkv, B = gen_of(seed), 128, 8, 2, 2
    cache = random_rows(gen, B, Hkv, L + 1, d)
    q = randn(gen, B, Hq, d).bfloat16()
    k, v = (x.squeeze(2) for x in new_kv(gen, B, Hkv, 1, d))
    cl = torch.tensor([L, L // 3], dtype=torch.int32, device="cuda")
    return q, k, v, cache, cl


def test_results_repeat_bit_for_bit_and_on_another_stream():
    tab = table(128)
    q, k, v, cache, cl = _decode_case(41)
    want = api.attn_decode_kv4(q, k, v, cache, cl, tab)
    for _ in range(5):
        assert torch.equal(api.attn_decode_kv4(q, k, v, cache, cl, tab), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = api.attn_decode_kv4(q, k, v, cache, cl, tab)
        kr, vr = api.kv4_read(cache, 100)
    s.synchronize()
    assert torch.equal(got, want)
    a, b = api.kv4_read(cache, 100)
    assert torch.equal(a, kr) and torch.equal(b, vr)


def test_stream_argument_with_outputs_allocated_by_the_call():
    """The call's own outputs and workspaces belong to the stream it runs on, whatever the
    current stream frees and takes meanwhile."""
    tab = table(128)
    q, k, v, cache, cl = _decode_case(43)
    want = api.attn_decode_kv4(q, k, v, cache, cl, tab)
    kw, vw = api.kv4_read(cache, 500)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        for _ in range(20):
            got = api.attn_decode_kv4(q, k, v, cache, cl, tab, stream=stream)
            kr, vr = api.kv4_read(cache, 500, stream=stream)
            churn = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
            del churn
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(kr, kw) and torch.equal(vr, vw)


def test_read_of_keys_or_values_alone():
    gen, d = gen_of(44), 64
    cache = random_rows(gen, 1, 2, 40, d)
    kw, vw = api.kv4_read(cache, 30, pos0=3)
    one = torch.zeros_like(kw)
    k, v = api.kv4_read(cache, 30, pos0=3, k=one)
    assert k is one and v is None and torch.equal(one, kw)
    k, v = api.kv4_read(cache, 30, pos0=3, v=one)
    assert k is None and v is one and torch.equal(one, vw)
    api.device_status()


def test_two_calls_at_once_with_a_workspace_each():
    tab = table(128)
    cases = [_decode_case(51), _decode_case(52, 5000)]
    want = [api.attn_decode_kv4(*c, tab) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(10):
        got = []
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                got.append(api.attn_decode_kv4(*c, tab))
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    api.device_status()


def test_captured_decode_follows_its_lengths():
    """A graph of a decode step, replayed as the lengths advance, with two graphs alive."""
    tab = table(128)
    q, k, v, cache, cl = _decode_case(61, 900)
    big = torch.zeros(2, 2, 1000, 160, dtype=torch.uint8, device="cuda")
    big[:, :, :901] = cache
    ref = big.clone()
    out = [torch.empty_like(q) for _ in range(2)]
    ws = [torch.empty(api.attn_decode_kv4_workspace_bytes(2, 8, 2, 128), dtype=torch.uint8,
                      device="cuda") for _ in range(2)]
    api.attn_decode_kv4(q, k, v, big.clone(), cl, tab)  # set-up before the capture
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            api.attn_decode_kv4(q, k, v, big, cl, tab, out=out[i], workspace=ws[i])
        graphs.append(g)
    for step in range(6):
        q.copy_(torch.randn_like(q))
        graphs[step % 2].replay()
        want = api.attn_decode_kv4(q, k, v, ref, cl, tab)
        assert torch.equal(out[step % 2], want)
        assert torch.equal(big, ref)
        cl += 1
    api.device_status()
