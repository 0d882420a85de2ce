"""A bounded wait of the prompt attention that runs out, without a GPU fault.

With the test hook PA_OPT_DROP_FIRST_FILL the first stage of every CTA never becomes
full, so that the wait for it runs out after PA_WAIT_TIMEOUT_MS.  The call must
return, report PA_DEVERR_TIMEOUT and leave the output rows as they were, and the next
call must be right.  In a child process: the limit is read once per process.
"""
import os
import subprocess
import sys
import textwrap

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = textwrap.dedent("""
    import sys, time
    sys.path.insert(0, {root!r})
    import torch
    from paged_kv_cache_132_gb300 import api, native
    native.load()
    cases = [([17], 8, 2, 64), ([200, 0, 131], 6, 2, 128),   # an item a CTA at most, no list
             ([90, 700, 1, 300] * 20, 16, 8, 64), ([129] * 60, 40, 40, 128), ([5000], 8, 8, 128)]
    for lens, h, hkv, d in cases:
        t = sum(lens)
        g = torch.Generator(device="cuda").manual_seed(t)
        q, k, v = (torch.randn(t, n, d, generator=g, device="cuda").bfloat16() for n in (h, hkv, hkv))
        loc = torch.tensor([0] + lens).cumsum(0).int().cuda()
        want = api.prompt_attention(q, k, v, loc, 0.1)
        assert api.get_device_error() == (0, 0)
        out = torch.full_like(q, 7.0)
        api.set_option("drop_first_fill", True)
        start = time.time()
        api.prompt_attention(q, k, v, loc, 0.1, out=out)
        status, code = api.get_device_error()
        elapsed = time.time() - start
        api.set_option("drop_first_fill", False)
        assert (status, code) == (-6, native.DEVERR_TIMEOUT), (status, code)
        assert 0.1 < elapsed < 20.0, elapsed
        assert bool((out == 7).all()), "rows were written"
        assert torch.equal(api.prompt_attention(q, k, v, loc, 0.1, out=out), want)
        assert api.get_device_error() == (0, 0)
        print("timeout-detected", t, round(elapsed, 3), flush=True)
""")


def test_a_wait_that_runs_out_writes_nothing():
    env = dict(os.environ, PA_WAIT_TIMEOUT_MS="200")
    env.pop("PA_DEBUG_DROP_FIRST_FILL", None)
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(root=ROOT)], env=env, cwd=ROOT, timeout=300,
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.count("timeout-detected") == 5, r.stdout
    print(r.stdout)
