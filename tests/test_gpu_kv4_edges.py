"""Edges of the 4-bit KV cache's calls on the GPU: what their documentation allows, far from the
ordinary sizes and values.  Plain forms in tests/_kv4.py."""
import math
import os
import subprocess
import sys
import textwrap

import pytest
import torch

from tests import _kv4 as R
from tests.test_gpu_kv4 import gen_of, new_kv, randn, random_rows, table
from yarn_position_scaling_b200 import api, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    api.load()


def one_value_rows(z, d):
    """Cache rows [1, 1, T, 5d/4] whose key's elements are all z[t] (exact in fp16), and whose
    values are codes of scale 1/8 and minimum -1."""
    T = z.numel()
    rows = torch.randint(0, 256, (1, 1, T, 5 * d // 4), dtype=torch.uint8, device="cuda",
                         generator=gen_of(T))
    par = torch.zeros(1, 1, T, 2, d // 32, 2, dtype=torch.float16, device="cuda")
    par[:, :, :, 0, :, 1] = z.half().view(1, 1, T, 1)
    par[:, :, :, 1, :, 0] = 0.125
    par[:, :, :, 1, :, 1] = -1.0
    rows[..., d:] = par.flatten(-3).view(torch.uint8)
    return rows


# ------------------------------------------------------------------- scores of any size
# Queries of equal elements a over keys of equal elements z: a score is scale a d z.  Keys 2^-9
# apart are then more than 1000 apart in their scores, so one key has all the weight, and the
# output is its value as stored: s n + z in one rounding.  The score's error is that of its
# factors' and sums' roundings, (d + 16) 2^-24 of it at the most.
HUGE = [1e6, 1e8, 1e10, 1e20, 1e32, 1e35]


@pytest.mark.parametrize("a", HUGE + [-x for x in HUGE])
@pytest.mark.parametrize("Hq,d", [(1, 128), (4, 64), (4, 128), (6, 128), (16, 64), (12, 128)])
def test_decode_takes_the_largest_of_huge_scores(a, Hq, d):
    L = 300
    tab = table(d, method="alibi")  # no rotation, and a bias far below the gaps
    z = 1 + torch.randperm(L, generator=torch.Generator().manual_seed(L)) / 512
    rows = torch.cat([one_value_rows(z, d), torch.zeros(1, 1, 1, 5 * d // 4, dtype=torch.uint8, device="cuda")], 2)
    best = int(z.argmax() if a > 0 else z.argmin())
    q = torch.full((1, Hq, d), a, device="cuda").bfloat16()
    k = torch.full((1, 1, d), 0.5 if a > 0 else 3.0, device="cuda").bfloat16()  # never the best
    lse = torch.empty(1, Hq, device="cuda")
    o = api.attn_decode_kv4(q, k, k, rows, torch.tensor([L], dtype=torch.int32, device="cuda"), tab, lse=lse)
    api.device_status()
    want = R.values(*R.decode_rows(rows[0, :, best])[1]).float().bfloat16()
    assert torch.equal(o[0], want.expand(Hq, d))
    score = float(q[0, 0, 0].double()) * d * float(z[best]) * tab.softmax_scale
    bias = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device="cuda", dtype=torch.float64) / Hq) * (L - best)
    assert (lse.double() - (score - bias)).abs().max() <= (d + 17) * 2.0 ** -24 * abs(score)


@pytest.mark.parametrize("a", [-1e32, 1e32, -1e9, 3e7])
@pytest.mark.parametrize("Hq,d", [(1, 128), (4, 64), (4, 128), (8, 128), (16, 128)])
def test_huge_scores_that_are_equal_share_the_weight(a, Hq, d):
    """Equal scores stay equal however coarse: the output is the mean of the values.  n codes of
    scale 1/8 and p = 1 are summed exactly, the division and bf16 round."""
    L = 700
    tab = api.rope_freq_table(d, 500000.0, 8192, 16.0, "factors", factors=[1e30] * (d // 2))  # no rotation
    rows = torch.cat([one_value_rows(torch.ones(L), d), torch.zeros(1, 1, 1, 5 * d // 4, dtype=torch.uint8, device="cuda")], 2)
    q = torch.full((1, Hq, d), a, device="cuda").bfloat16()
    score = abs(float(q[0, 0, 0])) * d * tab.softmax_scale
    k = torch.ones(1, 1, d, device="cuda").bfloat16()
    lse = torch.empty(1, Hq, device="cuda")
    o = api.attn_decode_kv4(q, k, k, rows, torch.tensor([L], dtype=torch.int32, device="cuda"), tab, lse=lse)
    api.device_status()
    v = R.values(*R.decode_rows(rows[0, 0])[1])
    want = v.mean(0)
    assert ((o[0].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20).all()
    assert (lse.abs().double() - score).abs().max() <= (d + 17) * 2.0 ** -24 * score


@pytest.mark.parametrize("a", [-1e32, 1e32, -1e8])
def test_a_lone_key_of_a_huge_score_has_the_weight(a):
    d = 128
    rows = api.kv4_cache(1, 2, 4, d)
    gen, tab = gen_of(1), table(d)
    q = torch.full((1, 8, d), a, device="cuda").bfloat16()
    k, v = torch.ones(1, 2, d, device="cuda").bfloat16(), randn(gen, 1, 2, d).bfloat16()
    vs = torch.empty_like(v)
    o = api.attn_decode_kv4(q, k, v, rows, torch.zeros(1, dtype=torch.int32, device="cuda"), tab, v_stored=vs)
    api.device_status()
    assert torch.equal(o.view(2, 4, d), vs.view(2, 1, d).expand(2, 4, d))


@pytest.mark.parametrize("a", [1e8, -1e8, 1e32, -1e32])
@pytest.mark.parametrize("Hq,Tq,d", [(1, 2, 128), (2, 4, 64), (4, 4, 128)])
def test_short_chunk_takes_the_largest_of_huge_scores(a, Hq, Tq, d):
    P0 = 300
    tab = table(d, method="alibi")
    z = 1 + torch.randperm(P0, generator=torch.Generator().manual_seed(P0)) / 512
    rows = torch.cat([one_value_rows(z, d), torch.zeros(1, 1, Tq, 5 * d // 4, dtype=torch.uint8, device="cuda")], 2)
    best = int(z.argmax() if a > 0 else z.argmin())
    q = torch.full((1, Hq, Tq, d), a, device="cuda").bfloat16()
    k = torch.full((1, 1, Tq, d), 0.5 if a > 0 else 3.0, device="cuda").bfloat16()
    o = api.attn_prefill_chunk_kv4(q, k, k, rows, P0, tab)
    api.device_status()
    want = R.values(*R.decode_rows(rows[0, :, best])[1]).float().bfloat16()
    assert torch.equal(o[0], want.expand(Hq, Tq, d))


@pytest.mark.parametrize("Hq,d", [(1, 128), (4, 64), (16, 128)])
def test_a_temperature_that_leaves_no_score_gives_the_mean(Hq, d):
    """A softmax scale below fp32's range: every score is 0, in the partly filled tile too."""
    L = 70
    tab = api.rope_freq_table(d, 500000.0, 8192, 16.0, "factors", factors=[1.0] * (d // 2), attn_factor=1e-30)
    gen = gen_of(d)
    rows = torch.cat([one_value_rows(torch.ones(L), d), torch.zeros(1, 1, 1, 5 * d // 4, dtype=torch.uint8, device="cuda")], 2)
    q, k = randn(gen, 1, Hq, d).bfloat16(), randn(gen, 1, 1, d).bfloat16()
    lse = torch.empty(1, Hq, device="cuda")
    o = api.attn_decode_kv4(q, k, k * 0, rows, torch.tensor([L], dtype=torch.int32, device="cuda"), tab, lse=lse)
    api.device_status()
    want = R.values(*R.decode_rows(rows[0, 0])[1]).mean(0)
    assert ((o[0].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20).all()
    assert (lse.double() - math.log(L + 1)).abs().max() <= 2.0 ** -20


# ----------------------------------------------------------------------- far positions
def exact_angles(pos, tab):
    """(cos, sin) of pos times the table's turns, the product without a rounding: turns split into
    a 24-bit part, whose product with a position below 2^29 is exact, and the rest."""
    t = R.turns_of(tab).cuda()
    hi = t.float().double()
    n = pos.double().unsqueeze(-1)
    frac = n * hi
    frac = (frac - torch.round(frac) + n * (t - hi)) * (2.0 * math.pi)
    return torch.cos(frac), torch.sin(frac)


def turn(x, c, s, pairs):
    """Pairs of x [..., T, d] in 64 bits turned by the angles of c, s [T, d/2]."""
    if pairs == "half":
        u, w = x.chunk(2, -1)
        return torch.cat([u * c - w * s, u * s + w * c], -1)
    u, w = x[..., 0::2], x[..., 1::2]
    return torch.stack([u * c - w * s, u * s + w * c], -1).flatten(-2)


@pytest.mark.parametrize("pairs", ["interleaved", "half"])
@pytest.mark.parametrize("pos0", [(1 << 20) - 17, (1 << 28) - 17, (1 << 28) + 12345])
def test_far_positions_are_rotated_as_defined(pos0, pairs):
    """Keys whose rotated elements lie within a few hundredths of a large number: a step of a code
    is 2^-11 of that number, so an angle that is off by 2^-25, the rounding of position times turns
    at 2^28, moves one code in some thousands.  The rows are those of the definition, and a decode
    step writes the same ones."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    d, T = 64, 1000
    tab = api.rope_freq_table(d, 10000.0, 8192, 1.0, "rope", pairs=pairs)
    cache = torch.empty(1, 1, pos0 + T, 80, dtype=torch.uint8, device="cuda")
    gen = gen_of(pos0 % 1000)
    pos = pos0 + torch.arange(T, device="cuda")
    c, s = exact_angles(pos, tab)
    for _ in range(40):
        y = 1000.0 + randn(gen, 1, 1, T, d)
        k = turn(y.double(), c, -s, pairs).bfloat16()
        v = randn(gen, 1, 1, T, d).bfloat16()
        api.kv4_write(k, v, cache, tab, pos0=pos0)
        rows = cache[:, :, pos0:]
        want = R.quantise(turn(k.double(), c, s, pairs).float()), R.quantise(v.float())
        for got, w in zip(R.decode_rows(rows), want):
            assert all(torch.equal(a, b) for a, b in zip(got, w))
    api.device_status()
    written = cache[:, :, pos0: pos0 + 64].clone()
    cache[:, :, pos0: pos0 + 64] = 0
    ws = torch.empty(api.attn_decode_kv4_workspace_bytes(1, 1, 1, d), dtype=torch.uint8, device="cuda")
    for t in range(64):
        api.attn_decode_kv4(k[:, :, t].contiguous(), k[:, :, t].contiguous(), v[:, :, t].contiguous(), cache,
                            torch.tensor([pos0 + t], dtype=torch.int32, device="cuda"), tab, window=1,
                            workspace=ws)
    api.device_status()
    assert torch.equal(cache[:, :, pos0: pos0 + 64], written)


# ---------------------------------------------------------- first use inside a capture
CAPTURE_CHILD = textwrap.dedent(f"""
    import sys
    sys.path.insert(0, {os.path.dirname(os.path.dirname(os.path.abspath(__file__)))!r})
    import torch
    from yarn_position_scaling_b200 import api
    from tests.test_gpu_kv4 import gen_of, random_rows, randn, table
    tab, gen, L = table(128), gen_of(1), 100
    q, k = randn(gen, 1, 16, 128).bfloat16(), randn(gen, 1, 2, 128).bfloat16()
    kv, cl = random_rows(gen, 1, 2, L + 1, 128), torch.tensor([L], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(api.attn_decode_kv4_workspace_bytes(1, 16, 2, 128), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.attn_decode_kv4(q, k, k, kv, cl, tab, out=out, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(api.attn_decode_kv4(q, k, k, kv, cl, tab), out)
    api.device_status()
    print("CAPTURED")
""")


def test_first_call_of_a_process_may_be_captured():
    """A kernel form is set up at its first launch, which may be one into a graph."""
    r = subprocess.run([sys.executable, "-c", CAPTURE_CHILD], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "CAPTURED" in r.stdout, r.stdout + r.stderr


# ------------------------------------------------------------------- two threads at once
def test_two_threads_call_at_once():
    """First calls of a form from two threads, each on a stream of its own: the one-time set-up is
    shared, the results are those of calls in turn."""
    import threading
    cases = []
    for i, Hq in enumerate((8, 24)):
        gen, L = gen_of(70 + i), 2000
        q = randn(gen, 1, Hq, 64).bfloat16()
        k, v = (x.squeeze(2) for x in new_kv(gen, 1, 2, 1, 64))
        cases.append((q, k, v, random_rows(gen, 1, 2, L + 1, 64), torch.tensor([L], dtype=torch.int32, device="cuda")))
    kc = torch.randn(1, 2, 100, 64, device="cuda").bfloat16()
    tab, got = table(64, "half"), [None, None]
    torch.cuda.synchronize()
    start = threading.Barrier(2)

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            start.wait()
            for _ in range(20):
                got[i] = api.attn_decode_kv4(*cases[i], tab)
                api.attn_decode(*cases[i][:3], kc.clone(), kc.clone(), torch.tensor([50], dtype=torch.int32, device="cuda"), tab)
            torch.cuda.current_stream().synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    api.device_status()
    for c, g in zip(cases, got):
        assert torch.equal(api.attn_decode_kv4(*c, tab), g)


# ----------------------------------------------------- the largest windows and sinks
BIG = 2 ** 31 - 1


@pytest.mark.parametrize("window,n_sink", [(BIG, 0), (BIG, BIG), (BIG - 100, 3), (1, BIG), (64, BIG - 60)])
@pytest.mark.parametrize("Tq", [1, 5, 200])
def test_largest_windows_and_sinks_over_the_4_bit_cache(window, n_sink, Tq):
    """They hide nothing: windows of the whole length, bit for bit."""
    gen, tab, P0, d = gen_of(Tq), table(128), 700, 128
    rows = random_rows(gen, 1, 2, P0 + Tq, d)
    q = randn(gen, 1, 8, Tq, d).bfloat16()
    k, v = new_kv(gen, 1, 2, Tq, d)
    lse = [torch.empty(1, 8, Tq, device="cuda") for _ in range(2)]
    plain = (window, P0 + Tq) if window < BIG - 100 else (P0 + Tq, 0)
    want = api.attn_prefill_chunk_kv4(q, k, v, rows, P0, tab, *plain, lse=lse[0])
    got = api.attn_prefill_chunk_kv4(q, k, v, rows, P0, tab, window, n_sink, lse=lse[1])
    assert torch.equal(got, want) and torch.equal(*lse)
    if Tq == 1:
        one = [x.squeeze(2).contiguous() for x in (q, k, v)]
        cl = torch.tensor([P0], dtype=torch.int32, device="cuda")
        want = api.attn_decode_kv4(*one, rows, cl, tab, *plain)
        assert torch.equal(api.attn_decode_kv4(*one, rows, cl, tab, window, n_sink), want)
    api.device_status()


@pytest.mark.parametrize("window,n_sink", [(BIG, 0), (BIG, BIG), (BIG - 100, 3), (1, BIG)])
def test_largest_windows_and_sinks_of_a_prefill(window, n_sink):
    gen, tab, T, d = gen_of(5), table(64), 300, 64
    q = randn(gen, 1, 4, T, d).bfloat16()
    k, v = new_kv(gen, 1, 2, T, d)
    plain = (window, T) if window == 1 else (T, 0)
    want = api.attn_prefill(q, k, v, tab, window=plain[0], n_sink=plain[1])
    got = api.attn_prefill(q, k, v, tab, window=window, n_sink=n_sink)
    api.device_status()
    assert torch.equal(got, want)


# ------------------------------------------------------------- workspaces, tiny caches, graphs
def guarded(n, fill):
    """A workspace of n bytes of `fill`, and the bytes behind it, which must stay as they are."""
    whole = torch.full((n + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
    whole[:n] = fill
    return whole[:n], whole[n:]


@pytest.mark.parametrize("lens", [[0], [0, 0, 0], [1, 300, 0, 5000], [127] * 40, [3] * 300, [20000, 1]])
@pytest.mark.parametrize("Hq,Hkv,d", [(2, 2, 128), (8, 2, 128), (16, 2, 64), (32, 2, 128)])
def test_decode_reads_only_what_it_wrote_into_its_workspace(lens, Hq, Hkv, d):
    gen, tab, B, T_max = gen_of(len(lens)), table(d), len(lens), max(lens) + 1
    rows = random_rows(gen, B, Hkv, T_max, d)
    q = randn(gen, B, Hq, d).bfloat16()
    k, v = (x.squeeze(2) for x in new_kv(gen, B, Hkv, 1, d))
    cl, outs = torch.tensor(lens, dtype=torch.int32, device="cuda"), []
    for fill in (0, 255):
        ws, behind = guarded(api.attn_decode_kv4_workspace_bytes(B, Hq, Hkv, d), fill)
        lse = torch.empty(B, Hq, device="cuda")
        outs.append((api.attn_decode_kv4(q, k, v, rows, cl, tab, workspace=ws, lse=lse), lse))
        assert (behind == 0xAB).all()
    api.device_status()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert torch.isfinite(outs[0][0].float()).all() and torch.isfinite(outs[0][1]).all()


@pytest.mark.parametrize("P0,Tq,window,n_sink", [(0, 1, 0, 0), (0, 5, 0, 0), (3000, 7, 0, 0), (3000, 7, 100, 5),
                                                 (700, 130, 0, 0), (3000, 130, 500, 200)])
@pytest.mark.parametrize("B,Hq,Hkv,d", [(1, 2, 2, 128), (3, 8, 2, 64), (1, 16, 1, 128)])
def test_chunk_reads_only_what_it_wrote_into_its_workspace(B, Hq, Hkv, d, P0, Tq, window, n_sink):
    gen, tab = gen_of(P0 + Tq), table(d)
    rows = random_rows(gen, B, Hkv, P0 + Tq, d)
    q = randn(gen, B, Hq, Tq, d).bfloat16()
    k, v = new_kv(gen, B, Hkv, Tq, d)
    outs = []
    for fill in (0, 255):
        ws, behind = guarded(api.attn_prefill_chunk_kv4_workspace_bytes(B, Hq, Hkv, Tq, d, P0), fill)
        lse = torch.empty(B, Hq, Tq, device="cuda")
        outs.append((api.attn_prefill_chunk_kv4(q, k, v, rows, P0, tab, window, n_sink, workspace=ws, lse=lse), lse))
        assert (behind == 0xAB).all()
    api.device_status()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert torch.isfinite(outs[0][0].float()).all() and torch.isfinite(outs[0][1]).all()


def test_decode_of_very_many_sequences():
    """More sequences than a grid axis holds: zero queries, so the LSE counts each one's keys."""
    B, d = 70000, 64
    rows = torch.zeros(B, 1, 9, 80, dtype=torch.uint8, device="cuda")
    lens = torch.arange(B, device="cuda", dtype=torch.int32) % 9
    q, tab = torch.zeros(B, 1, d, dtype=torch.bfloat16, device="cuda"), table(d)
    v = (torch.arange(B, device="cuda") % 128 + 1.0).bfloat16().view(B, 1, 1).expand(B, 1, d).contiguous()
    lse = torch.empty(B, 1, device="cuda")
    o = api.attn_decode_kv4(q, v, v, rows, lens, tab, lse=lse)
    api.device_status()
    n = (lens + 1).double().view(B, 1)
    # Scales of 0 put the reference at -32 and log2 of the sum between 32 and 64, where its unit is
    # 2^-18; their sum is exact, and ln 2 of it rounds once.
    assert (lse.double() - n.log()).abs().max() <= 2.0 ** -18 * math.log(2.0) + 2.0 ** -22
    want = v.double() / n.unsqueeze(-1)  # the new row alone is not 0, and is its minimum, exactly
    assert ((o.double() - want).abs() <= 2.0 ** -8 * want).all()


@pytest.mark.parametrize("Tq", [3, 150])
def test_captured_write_chunk_and_read(Tq):
    """One graph of a ragged write, a chunk by either kernel and a read, replayed with new inputs."""
    gen, tab, d, Hq, Hkv, P0, T = gen_of(Tq), table(128), 128, 8, 2, 400, 60
    q = randn(gen, 1, Hq, Tq, d).bfloat16()
    k, v = new_kv(gen, 1, Hkv, Tq, d)
    kp, vp = new_kv(gen, 1, Hkv, T, d)
    starts = torch.tensor([7], dtype=torch.int32, device="cuda")
    counts = torch.tensor([50], dtype=torch.int32, device="cuda")
    first = random_rows(gen, 1, Hkv, P0 + Tq, d)
    ws = torch.empty(api.attn_prefill_chunk_kv4_workspace_bytes(1, Hq, Hkv, Tq, d, P0), dtype=torch.uint8, device="cuda")

    def run(rows, o, kr, vr):
        api.kv4_write(kp, vp, rows, tab, starts=starts, counts=counts)
        api.attn_prefill_chunk_kv4(q, k, v, rows, P0, tab, out=o, workspace=ws)
        api.kv4_read(rows, T, starts=starts, counts=counts, k=kr, v=vr)

    def outs():
        return torch.zeros_like(q), torch.zeros_like(kp), torch.zeros_like(vp)
    rows, captured = first.clone(), outs()
    run(rows, *captured)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(rows, *captured)
    for step in range(3):
        for x in (q, k, v, kp, vp):
            x.copy_(torch.randn_like(x))
        starts.fill_(11 * step)
        counts.fill_(60 - 30 * step)
        rows.copy_(first)
        for x in captured:
            x.zero_()
        graph.replay()
        other, plain = first.clone(), outs()
        run(other, *plain)
        assert torch.equal(rows, other) and all(torch.equal(a, b) for a, b in zip(captured, plain))
    api.device_status()


# --------------------------------------------------- values outside the range, appended
@pytest.mark.parametrize("bad", [65536.0, -1e30, math.inf, math.nan])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("Tq", [0, 3, 150])
def test_appended_values_outside_the_range_are_reported_and_stored_finite(bad, which, Tq):
    """By a decode step (Tq = 0) and by chunks of either kernel; other heads' rows are as without."""
    gen, tab, d, P0, n = gen_of(Tq), table(64), 64, 90, max(Tq, 1)
    rows = random_rows(gen, 1, 2, P0 + n, d)
    q = randn(gen, 1, 4, n, d).bfloat16()
    kv = dict(zip("kv", new_kv(gen, 1, 2, n, d)))

    def call(rows):
        if Tq == 0:
            one = [x.squeeze(2).contiguous() for x in (q, kv["k"], kv["v"])]
            return api.attn_decode_kv4(*one, rows, torch.tensor([P0], dtype=torch.int32, device="cuda"), tab)
        return api.attn_prefill_chunk_kv4(q, kv["k"], kv["v"], rows, P0, tab)
    plain = rows.clone()
    want = call(plain)
    api.device_status()
    kv[which][0, 1, n - 1, 40] = bad
    got = call(rows)
    with pytest.raises(api.YarnAttnError) as ei:
        api.device_status()
    assert ei.value.code == api.YR_ERANGE
    assert torch.equal(rows[:, 0], plain[:, 0]) and torch.equal(rows[:, 1, : P0 + n - 1], plain[:, 1, : P0 + n - 1])
    for x in api.kv4_read(rows, P0 + n):
        assert torch.isfinite(x.float()).all()
    api.device_status()
    assert torch.equal(got.view(2, -1)[0], want.view(2, -1)[0])
