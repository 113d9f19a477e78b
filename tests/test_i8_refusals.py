"""Refusals of the int8 paged cache, on the host (no GPU is touched)."""
import ctypes as C

import pytest
import torch

from semi_ar_draft_gb300 import api, paged


@pytest.fixture(scope="module")
def L():
    from semi_ar_draft_gb300 import build

    build.build()
    from semi_ar_draft_gb300 import binding

    return binding.lib()


A = [C.c_void_p(0x10000 * (i + 1)) for i in range(16)]  # addresses that nothing reads


def append_params(**kw):
    from semi_ar_draft_gb300 import binding as b

    p = b.AppendParams(4, 2, 128, 16, 10, b.BF16, b.I8, 256, 128, 256, 128, 16 * 256, 256, 128)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def exps(**kw):
    from semi_ar_draft_gb300 import binding as b

    x = b.BlockExponents(0x900000, 0xa00000, 8, 4, 1, 2)
    for k, v in kw.items():
        setattr(x, k, v)
    return x


BAD = [({"T": -1}, {}, 1), ({"Hk": 0}, {}, 1), ({"D": 0}, {}, 1), ({"D": 24}, {}, 2), ({"D": 272}, {}, 2), ({"page_size": 24}, {}, 1),
       ({"page_size": 8192}, {}, 1), ({"num_pages": 0}, {}, 1), ({"dtype": 0}, {}, 1), ({"dtype": 4}, {}, 1), ({"kv_dtype": 1}, {}, 1),
       ({"kv_dtype": 3}, {}, 1), ({"kv_page_stride": 8}, {}, 1), ({"kv_token_stride": 24}, {}, 1), ({"kv_head_stride": 4}, {}, 1),
       ({}, {"k": None}, 1), ({}, {"v": None}, 1), ({}, {"block": 0}, 1), ({}, {"block": 3}, 1), ({}, {"block": 32}, 1),
       ({"page_size": 256}, {"block": 256}, 1), ({}, {"page_stride": -1}, 1), ({}, {"block_stride": -1}, 1), ({}, {"head_stride": -1}, 1)]


@pytest.mark.parametrize("p,x,status", BAD)
def test_parameters(L, p, x, status):
    q, y = append_params(**p), exps(**x)
    assert L.dspark_cache_append_i8(C.byref(q), C.byref(y), A[0], A[1], A[2], A[3], A[4], None, None) == status
    assert L.dspark_cache_read_i8(C.byref(q), C.byref(y), A[2], A[3], A[4], A[0], A[1], None) == status


def test_addresses(L):
    p, x = append_params(), exps()
    good = [A[0], A[1], A[2], A[3], A[4], None, None]
    for i in range(5):
        args = list(good)
        args[i] = None
        assert L.dspark_cache_append_i8(C.byref(p), C.byref(x), *args) == 1, i
    for i, off in ((0, 1), (1, 1), (2, 8), (3, 4), (5, 2)):
        args = list(good)
        args[i] = C.c_void_p(0x50000 + off)
        assert L.dspark_cache_append_i8(C.byref(p), C.byref(x), *args) == 1, i
    assert L.dspark_cache_append_i8(None, C.byref(x), *good) == 1 and L.dspark_cache_append_i8(C.byref(p), None, *good) == 1
    args = list(good)
    args[3] = args[2]  # keys and values into one pool
    assert L.dspark_cache_append_i8(C.byref(p), C.byref(x), *args) == 1
    for kw in ({"v": 0x900000}, {"page_stride": 0}, {"block_stride": 0}, {"head_stride": 0}):  # exponents that two blocks share
        y = exps(**kw)
        assert L.dspark_cache_append_i8(C.byref(p), C.byref(y), *good) == 1
    for i in range(5):
        args = [A[2], A[3], A[4], A[0], A[1], None]
        args[i] = None
        assert L.dspark_cache_read_i8(C.byref(p), C.byref(x), *args) == 1, i
    for i, off in ((3, 8), (4, 2)):
        args = [A[2], A[3], A[4], A[0], A[1], None]
        args[i] = C.c_void_p(0x50000 + off)
        assert L.dspark_cache_read_i8(C.byref(p), C.byref(x), *args) == 1, i
    for kw in ({"k_token_stride": 512}, {"v_token_stride": 512}, {"k_head_stride": 256}, {"v_head_stride": 256}):
        q = append_params(**kw)  # the outputs are dense
        assert L.dspark_cache_read_i8(C.byref(q), C.byref(x), A[2], A[3], A[4], A[0], A[1], None) == 1


def test_attention_takes_int8_pools_with_exponents_only(L):
    from semi_ar_draft_gb300 import binding as b

    p = b.AttentionParams(4, 4, 8, 2, 128, 16, 9, 3, 1, b.BF16, b.I8, 1, 0, 0.1, 0.0, 1024, 128, 4096, 256, 128, None)
    size = b.dspark_paged_attention_workspace_size(p)
    assert size > 256
    x = exps()
    args = lambda: [A[0], A[1], A[2], A[3], A[4], A[5]]  # noqa: E731  q, k, v, table, seq_len, offsets
    assert L.dspark_paged_attention(C.byref(p), *args(), None, None, A[6], None, A[7], size, None) == 1
    assert L.dspark_paged_attention_i8(C.byref(p), None, *args(), A[6], None, A[7], size, None) == 1
    for kw in ({"block": 32}, {"block": 5}, {"k": None}, {"head_stride": -2}):
        y = exps(**kw)
        assert L.dspark_paged_attention_i8(C.byref(p), C.byref(y), *args(), A[6], None, A[7], size, None) == 1
    assert L.dspark_paged_attention_i8(C.byref(p), C.byref(x), *args(), A[6], None, A[7], size - 1, None) == 6
    for scale in (2.0 ** -33, -2.0 ** 33, 1e30):
        p.scale = scale
        assert L.dspark_paged_attention_i8(C.byref(p), C.byref(x), *args(), A[6], None, A[7], size, None) == 2
    p.scale = 0.1
    # offsets that do not fit 32 bits of the strides' common power of two (16 bytes here), or of a byte of the exponents
    p.kv_token_stride, p.kv_page_stride = 272, 16 * (2 ** 32 // 8)
    assert L.dspark_paged_attention_i8(C.byref(p), C.byref(x), *args(), A[6], None, A[7], size, None) == 2
    p.kv_token_stride, p.kv_page_stride = 256, 4096
    y = exps(page_stride=2 ** 29)
    assert L.dspark_paged_attention_i8(C.byref(p), C.byref(y), *args(), A[6], None, A[7], size, None) == 2
    for kv in (b.BF16, b.E4M3):
        p.kv_dtype = kv
        assert L.dspark_paged_attention_i8(C.byref(p), C.byref(x), *args(), A[6], None, A[7], 1 << 30, None) == 1


def z(*s, dtype=torch.bfloat16, device="cpu"):
    return torch.zeros(s, dtype=dtype, device=device)


def test_tensors():
    """Types and shapes are looked at before any address."""
    i8, u8, i64, i32 = torch.int8, torch.uint8, torch.int64, torch.int32
    pools = lambda: [z(5, 16, 2, 64, dtype=i8), z(5, 16, 2, 64, dtype=i8), z(5, 2, 4, dtype=u8), z(5, 2, 4, dtype=u8)]  # noqa: E731
    k, slots = z(4, 2, 64), z(4, dtype=i64)
    table, seq = z(4, 3, dtype=i32), z(4, dtype=i32)

    def calls(p):
        return (lambda: api.cache_append_i8(k, k, *p, slots), lambda: api.cache_read_i8(*p, slots),
                lambda: api.paged_attention_i8(z(4, 4, 64), *p, table, seq, ws=z(256, dtype=u8)))

    for i, t, error in ((0, z(5, 16, 2, 64), TypeError), (1, z(5, 16, 2, 64), TypeError), (2, z(5, 2, 4, dtype=i8), ValueError),
                        (3, z(5, 2, 4), ValueError), (2, z(4, 2, 4, dtype=u8), ValueError), (3, z(5, 1, 4, dtype=u8), ValueError),
                        (3, z(5, 2, 8, dtype=u8), ValueError), (1, z(5, 16, 2, 32, dtype=i8), ValueError),
                        (2, z(5, 4, 2, dtype=u8).transpose(1, 2), ValueError), (2, z(5, 8, dtype=u8), ValueError)):
        p = pools()
        p[i] = t
        for f in calls(p):
            with pytest.raises(error):
                f()
    p = pools()
    p[2] = p[3] = z(5, 2, 3, dtype=u8)  # no whole blocks
    for f in calls(p):
        with pytest.raises(ValueError, match="exp"):
            f()
    for f in calls(pools()):
        with pytest.raises(ValueError, match="device tensors"):
            f()
    p = pools()
    p[3] = z(5, 2, 4, dtype=u8, device="meta")
    for f in calls(p):
        with pytest.raises(ValueError, match="one device"):
            f()
    p = pools()
    for bad in (z(4, 2, 32), z(4, 3, 64), z(2, 64)):
        with pytest.raises(ValueError):
            api.cache_append_i8(bad, bad, *p, slots)
    with pytest.raises(ValueError):
        api.cache_append_i8(k, k.half(), *p, slots)
    with pytest.raises(ValueError):
        api.cache_read_i8(*p, slots, out=(z(3, 2, 64), z(3, 2, 64)))
    # the calls of the other caches do not take int8 pages
    with pytest.raises(TypeError):
        api.cache_append(k, k, p[0], p[1], slots)
    with pytest.raises(TypeError):
        api.paged_attention(z(4, 4, 64), p[0], p[1], table, seq, ws=z(256, dtype=u8))


def test_paged_cache():
    make = lambda **kw: paged.PagedCache(2, 4, 16, 2, 1, 1, 64, 8, device="cpu", **kw)  # noqa: E731
    for block in (0, 3, 32, -1):
        with pytest.raises(ValueError, match="scale_block"):
            make(kv_dtype=torch.int8, scale_block=block)
    with pytest.raises(ValueError, match="scale_block"):
        make(scale_block=8)
    with pytest.raises(ValueError, match="scales"):
        make(kv_dtype=torch.int8, k_scale=torch.ones(1, 1))
    assert make(kv_dtype=torch.int8).k_exp.shape == (1, 4, 1, 1)
    assert make(kv_dtype=torch.int8, scale_block=1).v_exp.shape == (1, 4, 1, 16)
    with pytest.raises(ValueError, match="read"):
        make().read(0)
