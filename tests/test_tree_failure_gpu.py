"""A bounded wait of the tree attention that runs out, without a GPU fault: with the test
hook PA_OPT_DROP_FIRST_FILL the first stage of every CTA never becomes full.  The call must
return, report PA_DEVERR_TIMEOUT and leave the output rows as they were, those of items that
several CTAs share too, and the next call must be right.  In a child process: the limit is
read once per process."""
import os
import subprocess
import sys
import textwrap

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = textwrap.dedent("""
    import sys, time
    sys.path.insert(0, {root!r}), sys.path.insert(0, {root!r} + "/tests")
    import torch
    from paged_kv_cache_132_gb300 import api, native
    from test_tree_attention_gpu import Case
    native.load()
    cases = [([17], [5], 8, 2, 64), ([2000, 0, 131], [9, 3, 70], 8, 2, 128), ([300] * 40, [16] * 40, 16, 8, 64),
             ([30000], [8], 8, 8, 128)]
    for before, nodes, h, hkv, d in cases:
        c = Case(before, nodes, h, hkv, d, 16, torch.bfloat16)
        want = c.call()
        assert api.get_device_error() == (0, 0)
        out = torch.full_like(want, 7.0)
        api.set_option("drop_first_fill", True)
        start = time.time()
        c.call(out=out)
        status, code = api.get_device_error()
        elapsed = time.time() - start
        api.set_option("drop_first_fill", False)
        assert (status, code) == (-6, native.DEVERR_TIMEOUT), (status, code)
        assert 0.1 < elapsed < 20.0, elapsed
        assert bool((out == 7).all()), "rows were written"
        assert torch.equal(c.call(out=out), want)
        assert api.get_device_error() == (0, 0)
        print("timeout-detected", round(elapsed, 3), flush=True)
""")


def test_a_wait_that_runs_out_writes_nothing():
    env = dict(os.environ, PA_WAIT_TIMEOUT_MS="200")
    env.pop("PA_DEBUG_DROP_FIRST_FILL", None)
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(root=ROOT)], env=env, cwd=ROOT, timeout=300,
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.count("timeout-detected") == 4, r.stdout
