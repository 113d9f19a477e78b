"""How far a stored value may be off: half a step of its block's scale, and less than a step past 127 of the largest ones."""
import pytest
import torch

import i8_reference as R
from semi_ar_draft_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("block", [1, 16])
def test_values_up_to_the_largest_of_the_type(dtype, block):
    """Rows of every magnitude, those of the type's largest number among them: bf16's is 127.5 steps of its last scale and half a
    step off; fp16's last scale is 2^9, and 65504, 127.94 steps of it, is stored as 65024."""
    T, Hk, D, page = 96, 2, 64, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    top = torch.finfo(dtype).max
    x = (torch.rand((T, Hk, D), generator=g, device="cuda", dtype=torch.float64) * 2 - 1) * top
    x *= 2.0 ** -torch.randint(0, 12, (T, Hk, 1), generator=g, device="cuda").double()
    x[::16] = x[::16].sign() * top
    x = x.to(dtype).clamp(-top, top)
    codes = [torch.zeros((T // page, page, Hk, D), dtype=torch.int8, device="cuda") for _ in range(2)]
    exps = [torch.zeros((T // page, Hk, page // block), dtype=torch.uint8, device="cuda") for _ in range(2)]
    slots = torch.arange(T, device="cuda")
    api.cache_append_i8(x, -x, *codes, *exps, slots)
    e = R.exponents(exps[0], dtype).repeat_interleave(block, 2).transpose(1, 2).reshape(T, Hk, 1)
    step = R.two_to(e)
    for back, want in zip(api.cache_read_i8(*codes, *exps, slots, dtype), (x.double(), -x.double())):
        off = (back.double() - want).abs() / step
        held = want.abs() <= 127 * step  # (where it is not, the scale is the last one)
        assert bool((off[held] <= 0.5).all()) and bool((off < 1).all())
        assert bool((e.expand_as(held)[~held] == R.RANGE[dtype][1]).all())
        worst = 0.5 if dtype == torch.bfloat16 else 480 / 512
        assert float(off[::16].max()) == worst
