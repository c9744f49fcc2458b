"""Failure detection in the attention kernels without a GPU fault: a bounded wait
that runs out must end the kernel with the workspace error set, and the context
and the workspace must stay usable.

A failure-path build (-DSPEC_TEST_HOOKS, waits limited to 50 ms) leaves out the
first copy of one CTA (register kernel), or the commit of its first scores
(tcgen05 kernel).  Every wait that depends on it gives up, the CTA's roles run
out, and the kernel returns; the same call with the hook off gives the normal
result.  In a child process with its own copy of the library."""
import json
import os
import subprocess
import sys
import textwrap

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = textwrap.dedent("""
    import ctypes, json, sys, time
    sys.path.insert(0, sys.argv[2])
    import torch
    import speculative_decoding_draft_sampling_gb300 as sv
    from speculative_decoding_draft_sampling_gb300 import _build
    sv.build()
    sv.LIB_PATH = _build.build(force=True, extra_flags=["-DSPEC_TEST_HOOKS", "-DSPEC_WAIT_LIMIT_NS=50000000ull"],
                               out=sys.argv[1])
    sv._lib = None
    L = sv.lib()
    dev = torch.device("cuda", 0)
    D, P, H, T = 128, 64, 2, 900
    table = torch.randperm(40, device=dev).to(torch.int32)[:32].view(2, 16)
    pool = torch.zeros((40, H, sv.cache_block_bytes(D, P)), dtype=torch.uint8, device=dev)
    k = torch.randn((2, T + 64, H, D), device=dev).to(torch.bfloat16)
    sv.cache_append(k, k, pool, table, torch.zeros(2, dtype=torch.int32, device=dev))
    ctx = torch.full((2,), T, dtype=torch.int32, device=dev)
    res = {}
    for name, n, hook in (("registers", 3, L.spec_test_drop_copy), ("tcgen05", 64, L.spec_test_drop_commit)):
        hook.argtypes, hook.restype = [ctypes.c_int], ctypes.c_int
        q = torch.randn((2, n, 4 * H, D), device=dev).to(torch.bfloat16)
        call = lambda: sv.cache_attend(q, pool, table, ctx, want_lse=True)
        ref = call()
        want = (ref.out.clone(), ref.lse.clone())
        e0 = sv.workspace_error(ref.ws)
        assert hook(1) == 0
        t0 = time.perf_counter()
        bad = call()
        torch.cuda.synchronize()
        dt = time.perf_counter() - t0
        e1 = sv.workspace_error(bad.ws)
        assert hook(0) == 0
        control_left = int(bad.ws[256:16384].count_nonzero())
        bad.ws[:256].zero_()
        again = call()
        e2 = sv.workspace_error(again.ws)
        res[name] = dict(e0=e0, e1=e1, e2=e2, seconds=dt, control_left=control_left,
                         same=bool(torch.equal(again.out, want[0]) and torch.equal(again.lse, want[1])))
    print(json.dumps(res))
""")


def test_bounded_waits_run_out_and_report(tmp_path):
    script = tmp_path / "child.py"
    script.write_text(CHILD)
    r = subprocess.run([sys.executable, str(script), str(tmp_path / "libspecverify_hooks.so"), ROOT],
                       capture_output=True, text=True, timeout=900, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    for name, res in json.loads([ln for ln in r.stdout.splitlines() if ln.startswith("{")][-1]).items():
        assert res["e0"] == 0, (name, res)
        assert res["e1"] & 1, (name, res)             # SPEC_WS_ERR_WAIT: a wait gave up
        assert res["seconds"] < 30.0, (name, res)     # the kernel returned after its waits ran out
        assert res["control_left"] == 0, (name, res)
        assert res["e2"] == 0 and res["same"], (name, res)
