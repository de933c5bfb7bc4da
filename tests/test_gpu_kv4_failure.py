"""The 4-bit decode kernel's wait limit, without a GPU fault.

A test hook, compiled only into the test build of the library
(libyarnattn_faulthooks.so), makes warp 0 of one block leave out one bulk copy, so that a
wait which nothing will complete runs out of its (here 300 ms) limit.  The kernel must
record the timeout, return, and leave no output that an earlier call's partial results
could pass for: the heads whose keys the block has not read are NaN, all others and the
cache are those of a clean call, and the next call on the same context is clean.  It runs
in child processes so that the short limit and the hook stay out of this one.
"""
import os
import subprocess
import sys
import textwrap

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = textwrap.dedent(f"""
    import os, sys
    sys.path.insert(0, {ROOT!r})
    import torch
    from tests.test_gpu_kv4 import gen_of, new_kv, random_rows, randn, table
    from yarn_position_scaling_b200 import api, build
    api.load(build.build(fault_hooks=True), make_default=True)
    kind, drop = sys.argv[1:3]
    B, Hq, Hkv, d, L, Tq, first = map(int, sys.argv[3:])
    gen, tab, T_max, g = gen_of(Hq + d), table(d), L + Tq, Hq // Hkv
    start = random_rows(gen, B, Hkv, T_max, d)
    cache = start.clone()
    q, earlier = (randn(gen, B, Hq, Tq, d).bfloat16() for _ in range(2))
    k, v = new_kv(gen, B, Hkv, Tq, d)
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    n = (api.attn_decode_kv4_workspace_bytes(B, Hq, Hkv, d) if kind == "decode" else
         api.attn_prefill_chunk_kv4_workspace_bytes(B, Hq, Hkv, Tq, d, L))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")

    def call(q):
        if kind == "decode":
            lse = torch.empty(B, Hq, device="cuda")
            o = api.attn_decode_kv4(q[:, :, 0].contiguous(), k[:, :, 0].contiguous(),
                                    v[:, :, 0].contiguous(), cache, lens, tab, lse=lse,
                                    workspace=ws)
        else:
            lse = torch.empty(B, Hq, Tq, device="cuda")
            o = api.attn_prefill_chunk_kv4(q, k, v, cache, L, tab, lse=lse, workspace=ws)
        return o, lse

    want, want_lse = call(q)
    api.device_status()
    clean = cache.clone()
    call(earlier)                 # leaves finite partial results of another query
    api.device_status()
    cache.copy_(start)
    os.environ["YR_FAULT_DROP_KV4_COPY"] = drop
    got, lse = call(q)
    try:
        api.device_status()
        print("NO TIMEOUT REPORTED")
        sys.exit(3)
    except api.YarnAttnError as e:
        assert e.code == api.YR_ETIMEOUT and "decode-load-timeout" in str(e), str(e)
    del os.environ["YR_FAULT_DROP_KV4_COPY"]
    assert torch.equal(cache, clean), "rows"
    # Outputs by (sequence, KV head) segment, in the order in which the blocks take them.
    def by_segment(x):
        return x.float().reshape(B * Hkv, g, -1)
    bad = torch.isnan(by_segment(got)) & torch.isnan(by_segment(lse)).any(-1, keepdim=True)
    n_bad = int(bad.any(-1).any(-1).sum())
    assert n_bad >= 1, "stale results"
    assert bad.any(-1).any(-1)[first: first + n_bad].all(), "not one run of segments"
    if kind == "decode":
        assert bad[first: first + n_bad].all()
    if L < 32:                    # short segments: the block's share holds several
        assert 2 <= n_bad < B * Hkv // 4, n_bad
    else:                         # a long one: the other heads' keys are elsewhere
        assert n_bad == 1, n_bad
    same = ~bad
    assert torch.equal(by_segment(got)[same], by_segment(want)[same]), "unaffected outputs"
    ok = ~torch.isnan(lse)
    assert torch.equal(lse[ok], want_lse[ok]), "unaffected lse"
    again, again_lse = call(q)
    api.device_status()
    assert torch.equal(again, want) and torch.equal(again_lse, want_lse)
    print("CLEAN AFTER TIMEOUT")
""")


@pytest.mark.parametrize("kind,drop,B,Hq,Hkv,d,L,Tq,first", [
    # the second piece of a block that holds about a dozen short segments
    ("decode", "0:1", 1000, 16, 8, 128, 5, 1, 1),
    ("decode", "0:1", 1000, 32, 4, 64, 20, 1, 1),
    # long segments: the first keys (blocks of 128 units, of which a segment's first 256 are not
    # keys), and a copy in the ring's steady state
    ("decode", "2:0", 1, 32, 2, 128, 5000, 1, 0),
    ("decode", "0:11", 2, 4, 2, 64, 1200000, 1, 0),
    # several tokens
    ("chunk", "2:0", 1, 8, 2, 128, 5000, 3, 0),
])
def test_a_copy_that_does_not_land_leaves_nan(kind, drop, B, Hq, Hkv, d, L, Tq, first):
    env = dict(os.environ, YR_WAIT_TIMEOUT_MS="300")
    env.pop("YR_FAULT_DROP_KV4_COPY", None)
    args = [kind, drop] + [str(x) for x in (B, Hq, Hkv, d, L, Tq, first)]
    r = subprocess.run([sys.executable, "-c", CHILD] + args, env=env, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0 and "CLEAN AFTER TIMEOUT" in r.stdout, r.stdout + r.stderr
