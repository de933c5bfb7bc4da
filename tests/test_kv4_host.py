"""The 4-bit KV cache's entry points refuse bad arguments on the host, before any CUDA call."""
import ctypes

import pytest
import torch

from yarn_position_scaling_b200 import api, build

FAKE = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 8)
NUL = ctypes.c_void_p(0)
NOST = ctypes.POINTER(ctypes.c_int64)()


@pytest.fixture(scope="module")
def lib():
    build.build()
    return api.load()


@pytest.fixture(scope="module")
def tab(lib):
    return api.rope_freq_table(64, 10000.0, 64, 4.0, "yarn")


def _err(lib, rc, code, name):
    assert rc == code, lib.yr_last_error()
    assert lib.yr_last_error().decode().startswith(name)


WRITE = dict(k=FAKE, v=FAKE, kv4=FAKE, B=2, Hkv=2, T=8, d=64, T_max=64, ks=NOST, vs=NOST, pos0=0,
             starts=NUL, counts=NUL, tab=True)
ROWS_BAD = [
    (dict(kv4=NUL), api.YR_EINVAL), (dict(kv4=ODD), api.YR_EINVAL), (dict(B=0), api.YR_EINVAL),
    (dict(Hkv=0), api.YR_EINVAL), (dict(T=0), api.YR_EINVAL), (dict(T_max=0), api.YR_EINVAL),
    (dict(B=65536), api.YR_EINVAL), (dict(Hkv=65536), api.YR_EINVAL),
    (dict(d=96), api.YR_EUNSUPPORTED), (dict(d=256), api.YR_EUNSUPPORTED),
    (dict(pos0=-1), api.YR_EINVAL), (dict(pos0=57), api.YR_EINVAL), (dict(T=65), api.YR_EINVAL),
    (dict(T_max=(1 << 30) + 1), api.YR_EINVAL), (dict(pos0=(1 << 30) + 1, starts=FAKE), api.YR_EINVAL),
    (dict(starts=ctypes.c_void_p((1 << 20) + 2)), api.YR_EINVAL),
    (dict(counts=ctypes.c_void_p((1 << 20) + 1)), api.YR_EINVAL),
    (dict(k=ODD), api.YR_EINVAL), (dict(v=ODD), api.YR_EINVAL),
    (dict(ks=(ctypes.c_int64 * 3)(1024, 512, 60)), api.YR_EINVAL),
    (dict(vs=(ctypes.c_int64 * 3)(1024, 0, 64)), api.YR_EINVAL),
    (dict(vs=(ctypes.c_int64 * 3)(-1024, 512, 64)), api.YR_EINVAL),
]


@pytest.mark.parametrize("kw,code", ROWS_BAD + [(dict(k=NUL), api.YR_EINVAL),
                                                (dict(v=NUL), api.YR_EINVAL),
                                                (dict(tab=False), api.YR_EINVAL),
                                                (dict(d=128), api.YR_EINVAL)])
def test_write_refuses(lib, tab, kw, code):
    a = dict(WRITE, **kw)
    rc = lib.yr_kv4_write(a["k"], a["v"], a["kv4"], a["B"], a["Hkv"], a["T"], a["d"], a["T_max"],
                          a["ks"], a["vs"], a["pos0"], a["starts"], a["counts"],
                          ctypes.byref(tab) if a["tab"] else None, NUL)
    _err(lib, rc, code, "yr_kv4_write")


@pytest.mark.parametrize("kw,code", ROWS_BAD + [(dict(k=NUL, v=NUL), api.YR_EINVAL),
                                                (dict(type=2), api.YR_EINVAL),
                                                (dict(type=-1), api.YR_EINVAL)])
def test_read_refuses(lib, kw, code):
    a = dict(WRITE, type=0, **kw) if "type" not in kw else dict(WRITE, **kw)
    rc = lib.yr_kv4_read(a["kv4"], a["k"], a["v"], a["type"], a["B"], a["Hkv"], a["T"], a["d"],
                         a["T_max"], a["ks"], a["vs"], a["pos0"], a["starts"], a["counts"], 0, NUL)
    _err(lib, rc, code, "yr_kv4_read")


@pytest.mark.parametrize("kw,code", [
    (dict(q=NUL), api.YR_EINVAL), (dict(k=NUL), api.YR_EINVAL), (dict(v=NUL), api.YR_EINVAL),
    (dict(kv4=NUL), api.YR_EINVAL), (dict(cl=NUL), api.YR_EINVAL), (dict(o=NUL), api.YR_EINVAL),
    (dict(ws=NUL), api.YR_EINVAL), (dict(tab=False), api.YR_EINVAL), (dict(q=ODD), api.YR_EINVAL),
    (dict(kv4=ODD), api.YR_EINVAL), (dict(ks=ODD), api.YR_EINVAL),
    (dict(cl=ctypes.c_void_p((1 << 20) + 2)), api.YR_EINVAL),
    (dict(lse=ctypes.c_void_p((1 << 20) + 2)), api.YR_EINVAL), (dict(Hq=7), api.YR_EINVAL),
    (dict(B=0), api.YR_EINVAL), (dict(T_max=0), api.YR_EINVAL),
    (dict(T_max=(1 << 30) + 1), api.YR_EINVAL), (dict(d=80), api.YR_EUNSUPPORTED),
    (dict(d=128), api.YR_EINVAL), (dict(Hq=34), api.YR_EUNSUPPORTED),
    (dict(window=-1), api.YR_EINVAL), (dict(n_sink=2), api.YR_EINVAL),
    (dict(n_sink=-1, window=4), api.YR_EINVAL), (dict(ws_bytes=8), api.YR_EINVAL),
    (dict(ws=ODD), api.YR_EINVAL), (dict(B=1 << 28, Hq=8), api.YR_EINVAL),
])
def test_decode_refuses(lib, tab, kw, code):
    a = dict(q=FAKE, k=FAKE, v=FAKE, kv4=FAKE, cl=FAKE, o=FAKE, lse=NUL, ks=NUL, B=2, Hq=8, Hkv=2,
             d=64, T_max=64, tab=True, window=0, n_sink=0, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    rc = lib.yr_attn_decode_kv4(a["q"], a["k"], a["v"], a["kv4"], a["cl"], a["o"], a["lse"],
                                a["ks"], NUL, a["B"], a["Hq"], a["Hkv"], a["d"], a["T_max"],
                                ctypes.byref(tab) if a["tab"] else None, a["window"], a["n_sink"],
                                a["ws"], a["ws_bytes"], NUL)
    _err(lib, rc, code, "yr_attn_decode_kv4")


@pytest.mark.parametrize("kw,code", [
    (dict(q=NUL), api.YR_EINVAL), (dict(k=NUL), api.YR_EINVAL), (dict(v=NUL), api.YR_EINVAL),
    (dict(kv4=NUL), api.YR_EINVAL), (dict(o=NUL), api.YR_EINVAL), (dict(ws=NUL), api.YR_EINVAL),
    (dict(tab=False), api.YR_EINVAL), (dict(k=ODD), api.YR_EINVAL), (dict(q=ODD), api.YR_EINVAL),
    (dict(kv4=ODD), api.YR_EINVAL), (dict(Hq=7), api.YR_EINVAL), (dict(Hq=0), api.YR_EINVAL),
    (dict(Tq=0), api.YR_EINVAL), (dict(P0=-1), api.YR_EINVAL), (dict(P0=57), api.YR_EINVAL),
    (dict(d=96), api.YR_EUNSUPPORTED), (dict(d=128), api.YR_EINVAL),
    (dict(window=-1), api.YR_EINVAL), (dict(n_sink=1), api.YR_EINVAL),
    (dict(ws_bytes=8), api.YR_EINVAL), (dict(ws=ODD), api.YR_EINVAL),
])
def test_chunk_refuses(lib, tab, kw, code):
    a = dict(q=FAKE, k=FAKE, v=FAKE, kv4=FAKE, o=FAKE, B=2, Hq=8, Hkv=2, Tq=8, d=64, P0=8,
             T_max=64, tab=True, window=0, n_sink=0, ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    rc = lib.yr_attn_prefill_chunk_kv4(a["q"], a["k"], a["v"], a["kv4"], a["o"], NUL, a["B"],
                                       a["Hq"], a["Hkv"], a["Tq"], a["d"], a["P0"], a["T_max"],
                                       ctypes.byref(tab) if a["tab"] else None, a["window"],
                                       a["n_sink"], a["ws"], a["ws_bytes"], NUL)
    _err(lib, rc, code, "yr_attn_prefill_chunk_kv4")


def test_sizes(lib):
    assert [api.kv4_row_bytes(d) for d in (64, 128, 96, 0, -64)] == [80, 160, 0, 0, 0]
    assert api.attn_decode_kv4_workspace_bytes(2, 8, 3, 64) == 0
    assert api.attn_decode_kv4_workspace_bytes(2, 8, 2, 96) == 0
    assert api.attn_decode_kv4_workspace_bytes(2, 8, 2, 64) >= 4 * 4 * 66 * 4
    planes = api.attn_prefill_workspace_bytes(1, 8, 1256, 128)
    split = api.attn_prefill_chunk_split_bytes(1, 32, 256, 128)
    assert api.attn_prefill_chunk_kv4_workspace_bytes(1, 32, 8, 256, 128, 1000) == planes + split
    assert api.attn_prefill_chunk_kv4_workspace_bytes(1, 32, 8, 256, 128, -1) == 0
    # a few tokens: room for a partial result of each block and segment, 16 rows of d + 2 each
    few = api.attn_prefill_chunk_kv4_workspace_bytes(1, 32, 8, 4, 128, 0)
    assert few >= (592 + 8) * 16 * 130 * 4
    huge = (1 << 29) + 5  # sizes whose products pass 32 bits
    planes = api.attn_prefill_workspace_bytes(1, 1, huge, 64)
    split = api.attn_prefill_chunk_split_bytes(1, 16, huge, 64)
    assert api.attn_prefill_chunk_kv4_workspace_bytes(1, 16, 1, huge, 64, 0) == \
        (planes + 255) // 256 * 256 + split
    assert api.attn_prefill_chunk_kv4_workspace_bytes(1, 32, 8, 256, 128, 1 << 30) == 0


def test_python_checks_need_no_gpu(lib, tab):
    kv = torch.zeros(1, 2, 8, 80, dtype=torch.uint8)
    k = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        api.kv4_write(k, k, kv, tab)
    with pytest.raises(ValueError, match="CUDA"):
        api.kv4_read(kv, 4)
    with pytest.raises(ValueError, match="dtype"):
        api.kv4_read(kv, 4, dtype=torch.float32)
    with pytest.raises(ValueError, match="64 or 128"):
        api.kv4_cache(1, 2, 8, 96, device="cpu")
    assert api.kv4_cache(1, 2, 8, 64, device="cpu").shape == (1, 2, 8, 80)
