"""pa_commit_tree refuses pools that share memory, on the host: a path's rows would move twice."""
import ctypes

import pytest

from paged_kv_cache_132_gb300 import build, native

FAKE = 0x10000000  # aligned, never dereferenced: without sequences nothing is launched
BYTES = 8 * 2 * 16 * 64 * 2


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return native.load()


def _commit(lib, k, v):
    n = len(k)
    kp, vp = (ctypes.c_void_p * n)(*k), (ctypes.c_void_p * n)(*v)
    desc = native.CacheDesc(8, 2, 16, 64, native.PA_BF16)
    return lib.pa_commit_tree(kp, vp, n, ctypes.byref(desc), FAKE, 0, 0, None, None, None, None, None, 4, None, 0, None,
                              None, None)


def _apart(n, step=BYTES):
    return [FAKE + 2 * i * step for i in range(n)], [FAKE + (2 * i + 1) * step for i in range(n)]


@pytest.mark.parametrize("layers", [1, 2, 32, 256])
def test_pools_that_share_memory(lib, layers):
    k, v = _apart(layers)
    assert _commit(lib, k, v) in (0, -4)             # -4: no device here
    assert _commit(lib, v[::-1], k) in (0, -4)
    assert _commit(lib, k, k) == -1
    for at in {0, layers // 2, layers - 1}:
        for other in (k[at] + 16, k[at] + BYTES - 16):
            assert _commit(lib, k, v[:at] + [other] + v[at + 1:]) == -1
    if layers > 1:
        assert _commit(lib, [k[0]] * layers, v) == -1
        assert _commit(lib, k, [v[-1]] + v[1:]) == -1
    k, v = _apart(layers, BYTES - 16)
    assert _commit(lib, k, v) == -1
