"""Masks, caps and scales in the int8 kernel for up to eight rows, and keys of small codes in every kernel."""
import pytest
import torch

import i8_bounds as bounds
from semi_ar_draft_gb300 import api, binding
from test_gpu_i8_attention import make_case

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16]


def check(c, lens, offsets, kernel, max_new, scale=None, causal=True, window=0, softcap=0.0):
    assert bounds.kernel_of(c, max_new) == kernel
    out, lse, ws = api.paged_attention_i8(c["q"], *c["codes"], *c["exps"], c["table"], c["seq"], c["offsets"], lse=True, max_new=max_new,
                                          scale=scale, causal=causal, window=window, softcap=softcap)
    assert binding.dspark_get_device_status(ws) == 0
    bounds.compare(out, lse, bounds.attention(c, lens, offsets, kernel, scale, causal, window, softcap))
    return out, lse


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("causal,window,softcap,scale", [(True, 0, 0.0, None), (False, 0, 0.0, None), (True, 1, 0.0, None), (True, 20, 0.0, 0.3),
                                                         (False, 100, 0.0, None), (True, 0, 30.0, None), (True, 50, 2.0, None),
                                                         (True, 0, 0.0, -0.05), (True, 0, 1e4, None), (True, 3, 0.5, -1.0)])
@pytest.mark.parametrize("G,Hk,D,max_new", [(4, 4, 64, 1), (8, 2, 128, 1), (2, 2, 128, 4), (1, 1, 256, 8), (1, 2, 96, 8), (2, 4, 64, 4),
                                            (4, 3, 80, 2), (2, 3, 192, 3), (5, 8, 48, 1)])
def test_masks(dtype, causal, window, softcap, scale, G, Hk, D, max_new):
    """Groups of four, two and one heads, every width of a row, one to eight new tokens in a tile; requests without new
    tokens, padding."""
    lens, news = [300, 8, 64, 129, 17, 700, 40], [9, 8, 1, 16, 17, 0, 12]
    news = [min(n, max_new) for n in news]
    c, lens, offsets = make_case(lens, news, Hk * G, Hk, D, 32, 8, dtype, 7, pad=3)
    out, lse = check(c, lens, offsets, "few", max_new, scale, causal, window, softcap)
    assert not out[offsets[-1]:].any() and not torch.isfinite(lse[offsets[-1]:]).any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("kernel,G,max_new", [("few", 4, 1), ("few", 2, 4), ("rows", 5, 3), ("wide", 32, 2)])
def test_keys_of_small_codes(dtype, D, kernel, G, max_new):
    """Blocks whose scale one token has set: the others' codes are -1, 0 and 1."""
    n = max_new
    c, lens, offsets = make_case([500, 77, 9], [n] * 3, G, 1, D, 16, 16, dtype, D)
    g = torch.Generator(device="cuda").manual_seed(G)
    k = c["codes"][0]
    k.copy_(torch.randint(-1, 2, k.shape, generator=g, device="cuda"))
    k[:, 3] = torch.randint(0, 2, k[:, 3].shape, generator=g, device="cuda").to(torch.int8) * 254 - 127
    c["exps"][0].fill_(127 - 3)
    check(c, lens, offsets, kernel, max_new)
