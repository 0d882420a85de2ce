"""Tensor maps of the pools are encoded once, however many activations pass by: the host
part of the library with a counting encoder in place of CUDA's (map_lookups.cu)."""
import os
import subprocess

import pytest

from paged_kv_cache_132_gb300.build import ARCH, INCLUDE, cuda_home

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("maps") / "map_lookups")
    subprocess.run([os.path.join(cuda_home(), "bin", "nvcc"), *ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-cudart", "shared", "-I", INCLUDE,
                    "-o", exe, os.path.join(HERE, "map_lookups.cu")], check=True, capture_output=True, text=True)
    return exe


def counts(program, *args):
    out = subprocess.run([program, *map(str, args)], check=True, capture_output=True, text=True).stdout
    return [int(x) for x in out.split()]


@pytest.mark.parametrize("layers", [1, 4, 8])
def test_prompts_leave_the_pools_maps(program, layers):
    assert counts(program, layers, 5) == [2 * layers, 3 * 5 * layers]


def test_decode_and_prefill_beside_prompts(program):
    """Each has its own view of a pool: four layers' fill the pools' 16 maps."""
    assert counts(program, 4, 5, "prefill") == [4 * 2 * 2, 4 * 5 * 4]
