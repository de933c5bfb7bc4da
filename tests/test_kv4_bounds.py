"""The error bounds of tests/_kv4_bounds.py on the CPU: they hold for operands rounded as the
kernels round them, and plain mistakes (a mask one key off, a tile left out, a tenth too much)
break them."""
import math

import pytest
import torch

from tests import _kv4 as R
from tests import _kv4_bounds as K
from yarn_position_scaling_b200 import api, build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    api.load()


def inputs(d, g, Tq, Tk, seed=0, method="yarn"):
    gen = torch.Generator().manual_seed(seed)
    tab = api.rope_freq_table(d, 500000.0, 8192, 16.0, method)
    rows = torch.randint(0, 256, (Tk, 5 * d // 4), generator=gen, dtype=torch.uint8)
    par = torch.stack([0.05 + 0.3 * torch.rand(Tk, d // 16, generator=gen),
                       -1.5 + 0.5 * torch.randn(Tk, d // 16, generator=gen)], -1)
    rows[:, d:] = par.half().flatten(1).view(torch.uint8)
    qpos = Tk - Tq + torch.arange(Tq)
    q = R.rotate(torch.randn(g, Tq, d, generator=gen).bfloat16(), qpos, tab)
    return q, rows, qpos, tab


def emulated(q, rows, qpos, tab, window, n_sink, prefill, drop=None, shift=0, factor=1.0):
    """The attention with the kernels' roundings (or the prefill kernel's fp16 operands), and
    with mistakes: keys drop[0] .. drop[1] left out, a mask or a window shifted by keys."""
    (kc, ks, kz), (vc, vs, vz) = R.decode_rows(rows)
    k, v = R.values(kc, ks, kz), R.values(vc, vs, vz)
    seen = K.visible(qpos + shift, rows.shape[0], window, n_sink)
    if drop is not None:
        seen[:, drop[0]: drop[1]] = False
    if prefill:
        q, k, v = q.half().double(), k.half().double(), v.half().double()
    x = (q @ k.T * tab.softmax_scale).masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    lse = (m + p.sum(-1, keepdim=True).log()).squeeze(-1)
    if prefill:
        o = p.half().double() @ v
    else:
        s, G = vs.double(), rows.shape[1] * 4 // 5 // 32
        n, z = vc.double(), vz.double()
        o = torch.cat([(256 * p * s[:, g, 0]).half().double() / 256 @ n[:, g] + p @ z[:, g].expand(-1, 32)
                       for g in range(G)], -1)
    return (o / p.sum(-1, keepdim=True) * factor).bfloat16().double(), lse


CASES = [(128, 4, 7, 784, 0, 0), (128, 2, 40, 1040, 0, 0), (64, 4, 10, 1011, 300, 70), (64, 2, 129, 2177, 0, 0),
         (128, 1, 1, 30001, 0, 0), (128, 2, 10, 1011, 900, 500)]


@pytest.mark.parametrize("d,g,Tq,Tk,window,n_sink", CASES)
@pytest.mark.parametrize("prefill", [False, True])
def test_bounds_hold_for_the_kernels_roundings_and_break_for_mistakes(d, g, Tq, Tk, window, n_sink, prefill):
    q, rows, qpos, tab = inputs(d, g, Tq, Tk, seed=Tk + window)
    r = K.attend(q, rows, qpos, tab, 0, g, window, n_sink)
    bo, bl = K.chunk_bounds(r, Tk) if prefill else K.decode_bounds(r, d, Tk, 40)

    def fails(**mistake):
        o, lse = emulated(q, rows, qpos, tab, window, n_sink, prefill, **mistake)
        return bool(((o - r["o"]).abs() > bo).any()), bool(((lse - r["lse"]).abs() > bl).any())
    assert fails() == (False, False)
    assert fails(factor=1.1)[0] and fails(factor=0.0)[0]
    if Tk <= 2500:
        assert any(fails(shift=-1))
        if window == 0 or Tk - window > 100:
            assert any(fails(drop=(Tk - 64, Tk - 32)))
    # Not a bound that outputs cannot pass: a tenth of the outputs' size at the most.
    assert float(bo.mean()) <= 0.1 * float(r["o"].pow(2).mean().sqrt())


@pytest.mark.parametrize("Tk,window,n_sink", [(131072, 0, 0), (131072, 70001, 300), (1011, 300, 70), (33, 0, 0)])
def test_counting_shows_one_key(Tk, window, n_sink):
    d = 64
    rows = K.counting_rows(Tk, d, "cpu")
    (_, _, _), (vc, vs, vz) = R.decode_rows(rows)
    qpos = torch.tensor([Tk - 1])
    o, lse = K.counting_result(qpos, Tk, d, window, n_sink)
    seen = K.visible(qpos, Tk, window, n_sink).double()
    assert torch.allclose(seen @ R.values(vc, vs, vz) / seen.sum(), o, rtol=1e-14, atol=0)
    bo, bl = K.counting_bounds(o, lse)
    count = float(seen.sum())
    for other in (count - 1, count + 1):
        assert abs(math.log(other) - float(lse)) > 1.5 * float(bl)
    n = torch.arange(Tk)
    mid = int(seen[0].nonzero()[len(seen[0].nonzero()) // 2]) // 32 * 32
    less = seen.clone()
    less[:, mid: mid + 32] = 0       # a tile left out, and the count of keys as if it were there
    bad = less @ R.values(vc, vs, vz) / count
    assert ((bad - o).abs() > bo).any()
