"""Reading an int8 cache back wants two outputs, on the host (no GPU is touched)."""
import ctypes as C

import pytest

from semi_ar_draft_gb300 import binding as b


@pytest.fixture(scope="module")
def L():
    from semi_ar_draft_gb300 import build

    build.build()
    return b.lib()


def test_keys_and_values_over_one_another_are_refused(L):
    """Each element of the overlap would be the key's or the value's, by chance."""
    T, Hk, D = 4, 2, 64
    p = b.AppendParams(T, Hk, D, 16, 10, b.BF16, b.I8, Hk * D, D, Hk * D, D, 16 * Hk * D, Hk * D, D)
    x = b.BlockExponents(0x900000, 0xa00000, 8, 4, 1, 2)
    pools = [C.c_void_p(0x10000), C.c_void_p(0x20000), C.c_void_p(0x30000)]
    n = T * Hk * D * 2
    for k, v in ((0x40000, 0x40000), (0x40000, 0x40000 + n - 16), (0x40000 + 16, 0x40000)):
        assert L.dspark_cache_read_i8(C.byref(p), C.byref(x), *pools, C.c_void_p(k), C.c_void_p(v), None) == 1
    q = b.AppendParams(0, Hk, D, 16, 10, b.BF16, b.I8, Hk * D, D, Hk * D, D, 16 * Hk * D, Hk * D, D)
    assert L.dspark_cache_read_i8(C.byref(q), C.byref(x), *pools, C.c_void_p(0x40000), C.c_void_p(0x40000), None) == 0  # no tokens
