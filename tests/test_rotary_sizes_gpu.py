"""Rotary embedding with cache write from few tokens to many: the number of threads of a
token's CTA changes with tokens and rows, and each of its forms is held against the
definition in 64 bits, on both sides of the change.  Tolerance as in test_rotary_gpu.py.
"""
import pytest
import torch

from paged_kv_cache_132_gb300 import native
from test_rotary_gpu import case, run_and_check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    native.load()


# A head row has ceil(d * bytes / 32) lanes: 12 rows of 4 or 8, 18 of 5 or 9, 4 of 16 or 32.
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("h,hkv,d,rot", [(8, 2, 64, 64), (12, 3, 72, 32), (2, 1, 256, 128)])
@pytest.mark.parametrize("side", [-1, 0, 1])
def test_both_sides_of_the_change(h, hkv, d, rot, interleaved, dtype, side):
    lanes = -(-(d * torch.empty((), dtype=dtype).element_size()) // 32)
    tokens = 2 * (h + 2 * hkv) * lanes + side
    run_and_check(case(tokens, h, hkv, d, rot, dtype, fused=True, padding=5, seed=d), rot, interleaved, True, tokens)
    run_and_check(case(tokens, h, hkv, d, rot, dtype, bs=8, seed=d + 1), rot, interleaved, False, tokens)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens", [1024, 1025, 3001])
@pytest.mark.parametrize("h,hkv,d,rot", [(8, 2, 128, 128), (5, 5, 24, 16), (40, 40, 128, 64)])
def test_many_tokens(h, hkv, d, rot, tokens, interleaved, dtype):
    run_and_check(case(tokens, h, hkv, d, rot, dtype, fused=True, padding=7, far=131072), rot, interleaved, True, tokens)
