"""Addresses that are no element's are refused before anything is launched (on the host: no GPU is touched)."""
import ctypes as C

import pytest

from semi_ar_draft_gb300 import binding as b


@pytest.fixture(scope="module")
def L():
    from semi_ar_draft_gb300 import build

    build.build()
    return b.lib()


def at(x):
    return C.c_void_p(x)


def test_slots(L):
    p = b.AppendParams(4, 2, 64, 16, 10, b.BF16, b.I8, 128, 64, 128, 64, 2048, 128, 64)
    x = b.BlockExponents(0x900000, 0xa00000, 8, 4, 1, 2)
    for off in (1, 2, 4):
        assert L.dspark_cache_append_i8(C.byref(p), C.byref(x), at(0x1000), at(0x2000), at(0x10000), at(0x20000), at(0x30000 + off), None, None) == 1
        assert L.dspark_cache_read_i8(C.byref(p), C.byref(x), at(0x10000), at(0x20000), at(0x30000 + off), at(0x1000), at(0x2000), None) == 1


@pytest.mark.parametrize("i8", [True, False])
def test_lengths_tables_offsets_and_lse(L, i8):
    p = b.AttentionParams(4, 4, 8, 2, 128, 16, 9, 3, 1, b.BF16, b.I8 if i8 else b.BF16, 1, 0, 0.1, 0.0, 1024, 128, 4096, 256, 128, None)
    size = b.dspark_paged_attention_workspace_size(p)
    x = b.BlockExponents(0x900000, 0xa00000, 8, 4, 1, 2)
    for i in range(4):
        for off in (1, 2):
            a = [0x40000, 0x50000, 0x60000, 0x70000]  # table, seq_len, offsets, lse
            a[i] += off
            table, seq, offsets, lse = map(at, a)
            first, last = (at(0x10000), at(0x20000), at(0x30000), table, seq, offsets), (at(0x80000), lse, at(0x100000), size, None)
            if i8:
                assert L.dspark_paged_attention_i8(C.byref(p), C.byref(x), *first, *last) == 1, i
            else:
                assert L.dspark_paged_attention(C.byref(p), *first, None, None, *last) == 1, i
