"""An int8 cache takes the 16-bit type that it was made for, and no other (on the host: no GPU is touched)."""
import pytest
import torch

from semi_ar_draft_gb300 import paged


@pytest.mark.parametrize("dtype,other", [(torch.bfloat16, torch.float16), (torch.float16, torch.bfloat16), (torch.bfloat16, torch.float32)])
def test_keys_values_and_queries_are_of_the_cache_s_type(dtype, other):
    """Its exponents stand for another range in the other type: they would be clamped without a word."""
    cache = paged.PagedCache(2, 4, 16, 2, 1, 1, 64, 8, dtype=dtype, kv_dtype=torch.int8, device="cpu")
    good, bad = torch.zeros((8, 1, 64), dtype=dtype), torch.zeros((8, 1, 64), dtype=other)
    for k, v in ((bad, good), (good, bad), (bad, bad)):
        with pytest.raises(TypeError, match="int8 cache"):
            cache.append(0, k, v)
    with pytest.raises(TypeError, match="int8 cache"):
        cache.attend(0, bad)
    with pytest.raises(ValueError, match="device tensors"):  # (of the right type: refused for where they are)
        cache.append(0, good, good)
    with pytest.raises(ValueError, match="device tensors"):
        cache.attend(0, good, out=good)


@pytest.mark.parametrize("dtype", [torch.float32, torch.int8, torch.float8_e4m3fn])
def test_no_int8_cache_of_other_types(dtype):
    with pytest.raises(ValueError, match="bf16 or fp16"):
        paged.PagedCache(2, 4, 16, 2, 1, 1, 64, 8, dtype=dtype, kv_dtype=torch.int8, device="cpu")
