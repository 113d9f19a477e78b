"""Layouts and types that the paged-cache calls take and refuse, on the host (no GPU is touched)."""
import pytest
import torch

from semi_ar_draft_gb300 import api


@pytest.fixture(scope="module", autouse=True)
def built():
    from semi_ar_draft_gb300 import build

    build.build()


def z(*s, dtype=torch.bfloat16):
    return torch.zeros(s, dtype=dtype)


def alike(make):
    """Two tensors of one layout whose strides differ where there is one index only."""
    x = make()
    i = list(x.shape).index(1)
    stride = list(x.stride())
    stride[i] = 16 * x.numel()
    y = x.as_strided(x.shape, stride)
    assert x.stride() != y.stride()
    return x, y


def test_a_stride_that_one_index_never_uses_is_no_layout():
    """Pools and exponents of one kv head, one page or one block a page, whichever way round they were made."""
    k, slots = z(4, 1, 64), z(4, dtype=torch.int64)
    table, seq, u8 = z(4, 3, dtype=torch.int32), z(4, dtype=torch.int32), torch.uint8
    for pages, n in ((5, 4), (5, 1), (1, 4), (1, 1)):
        kp, vp = alike(lambda: z(pages, 16, 1, 64, dtype=torch.int8))
        ke, ve = alike(lambda: z(pages, 1, n, dtype=u8))
        for f in (lambda: api.cache_append_i8(k, k, kp, vp, ke, ve, slots), lambda: api.cache_read_i8(kp, vp, ke, ve, slots),
                  lambda: api.paged_attention_i8(z(4, 4, 64), kp, vp, ke, ve, table, seq, ws=z(256, dtype=u8))):
            with pytest.raises(ValueError, match="device tensors"):  # (nothing else is wrong with them)
                f()
        kp, vp = alike(lambda: z(pages, 16, 1, 64))
        for f in (lambda: api.cache_append(k, k, kp, vp, slots), lambda: api.paged_attention(z(4, 4, 64), kp, vp, table, seq, ws=z(256, dtype=u8))):
            with pytest.raises(ValueError, match="device tensors"):
                f()


def test_layouts_that_differ_are_refused():
    k, slots = z(4, 2, 64), z(4, dtype=torch.int64)
    i8, u8 = torch.int8, torch.uint8
    kp, ke = z(5, 16, 2, 64, dtype=i8), z(5, 2, 4, dtype=u8)
    other_pool, other_exp = z(5, 2, 16, 64, dtype=i8).transpose(1, 2), z(5, 4, 2, dtype=u8).transpose(1, 2)
    for args in ((kp, other_pool, ke, ke), (kp, kp, ke, other_exp), (kp, kp, other_exp, ke)):
        with pytest.raises(ValueError, match="layout"):
            api.cache_append_i8(k, k, *args, slots)
        with pytest.raises(ValueError, match="layout"):
            api.cache_read_i8(*args, slots)
