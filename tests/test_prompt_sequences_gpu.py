"""Attention over packed prompts of thousands of sequences: more than one pass of the
planning kernel, with sequences of few and of many units in each."""
import pytest
import torch

from paged_kv_cache_132_gb300 import api, native
from test_prompt_gpu import check, rows, run, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    native.load()


@pytest.mark.parametrize("n", [1023, 1024, 1025, 2500])
@pytest.mark.parametrize("h,hkv,d,dtype", [(4, 4, 64, torch.bfloat16), (16, 2, 128, torch.float16)])
def test_thousands_of_sequences(n, h, hkv, d, dtype):
    g = torch.Generator().manual_seed(n)
    lens = (torch.randint(0, 12, (n,), generator=g) * torch.randint(0, 2, (n,), generator=g)).tolist()
    for at in (0, 5, 1000, n - 1):  # long ones (many units) among them, in every pass
        lens[at] = 700 + at % 600
    run(lens, h, hkv, d, dtype, seed=n, fused=True, extra=30, first=4)


def test_bad_start_rows_in_every_pass():
    """Some start rows out of range: their sequences are skipped, the others computed."""
    lens = [3] * 2200
    q, k, v = rows(6600, 8, 4, 64, torch.float16, 51)
    loc = starts(lens)
    loc[[700, 1500, 2200]] = torch.tensor([-5, 10000, 7000], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    api.prompt_attention(q, k, v, loc, 0.125, out=out)
    assert api.get_device_error() == (-5, native.DEVERR_CONTEXT_LEN)
    skipped = torch.zeros(2200, dtype=torch.bool)
    skipped[[699, 700, 1499, 1500, 2199]] = True
    bad = skipped.repeat_interleave(3).cuda()
    assert bool((out[bad] == 7).all())
    want = torch.full_like(q, 7.0)
    api.prompt_attention(q, k, v, starts(lens), 0.125, out=want)
    assert torch.equal(out[~bad], want[~bad])
    check(q, k, v, lens[:300], 0.125, want[:900])
