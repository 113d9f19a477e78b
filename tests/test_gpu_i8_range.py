"""Int8 attention over the range of queries, keys and scores, in each of its kernels."""
import math

import pytest
import torch

import i8_bounds as bounds
from semi_ar_draft_gb300 import api, binding
from test_gpu_i8_attention import make_case

pytestmark = pytest.mark.gpu

KERNELS = [("few", 4, 1), ("rows", 5, 3), ("wide", 32, 2)]  # name, query heads of a kv head, the most new tokens


def attend(c, kernel, **kw):
    assert bounds.kernel_of(c, kw.get("max_new", 0)) == kernel
    out, lse, ws = api.paged_attention_i8(c["q"], *c["codes"], *c["exps"], c["table"], c["seq"], c["offsets"], lse=True, **kw)
    assert binding.dspark_get_device_status(ws) == 0
    return out, lse


def queries(shape, E, seed=1):
    """bf16 of about 2^E, the largest of a row between 2^E and 2^(E + 1)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.rand(shape, generator=g, device="cuda", dtype=torch.float64) * 2 - 1
    x = x / x.abs().amax(-1, keepdim=True) * 1.5
    return (x * 2.0 ** E).to(torch.bfloat16)


@pytest.mark.parametrize("kernel,G,max_new", KERNELS)
@pytest.mark.parametrize("E,scale,softcap", [(60, None, 0.0), (100, None, 0.0), (116, None, 0.0), (118, 1.0, 0.0), (121, None, 0.0), (124, None, 0.0),
                                             (126, None, 0.0), (127, None, 0.0), (87, 2.0 ** 32, 0.0), (95, 2.0 ** 32, 0.0), (121, None, 5.0),
                                             (110, None, 1e-4), (40, None, 2.0 ** -90), (127, None, 1e4), (-100, None, 0.0), (-100, None, 2.0 ** 60),
                                             (-110, 2.0 ** -6, 2.0 ** 99), (-117, None, 30.0)])
def test_queries_of_any_size(kernel, G, max_new, E, scale, softcap):
    """bf16 queries as large and as small as the type has them, over keys whose scales bring the scores back to a few (or as
    near to it as scales go): the factors on the way leave fp32, the scores do not."""
    D = 64
    c, lens, offsets = make_case([90, 41, 3], [max_new, 1, 1], G, 1, D, 16, 8, torch.bfloat16, 8)
    c["q"] = queries(c["q"].shape, E)
    s = D ** -0.5 if scale is None else scale
    e = max(-126, min(121, round(-E - math.log2(s) - 6 - 3)))  # sums of 64 products of 2^E and 2^6 2^e: about 2^3 more
    g = torch.Generator(device="cuda").manual_seed(4)
    c["exps"][0].copy_(torch.randint(max(e - 1, -126), e + 2, c["exps"][0].shape, generator=g, device="cuda") + 127)
    c["codes"][0][c["table"][1, 0], 2:5] = 0  # keys of zeros
    out, lse = attend(c, kernel, scale=scale, softcap=softcap, max_new=max_new)
    bounds.compare(out, lse, bounds.attention(c, lens, offsets, kernel, scale, softcap=softcap))


@pytest.mark.parametrize("kernel,G,max_new", KERNELS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("e", [-10, 0, 9])
@pytest.mark.parametrize("scale", [None, -0.25])
def test_a_row_of_one_key_is_its_value(kernel, G, max_new, dtype, e, scale):
    """However large the score (60, 6e4, 3e7 and up to twice that): keys so far below one that nothing else has a weight, and
    requests of few keys.  The weight and the output are rounded once each, the rest is fp32's."""
    u = torch.finfo(dtype).eps / 2
    u_p = u if kernel == "wide" else 2.0 ** -11
    D, n = 128, max_new
    c, lens, offsets = make_case([n, 300, 40, n], [n] * 4, G, 1, D, 16, 1, dtype, 5)
    g = torch.Generator(device="cuda").manual_seed(2)
    sign = torch.randint(0, 2, (D,), generator=g, device="cuda") * 2 - 1
    c["q"] = ((0.5 + 0.5 * torch.rand(c["q"].shape, generator=g, device="cuda")) * 64 * sign).to(dtype)
    c["exps"][0].fill_(e + 127)
    V, want = bounds.R.values(c["codes"][1], c["exps"][1], dtype), []
    for j, length in enumerate(lens):
        for l in range(length):
            at = (int(c["table"][j, l // 16]), l % 16, 0)
            c["codes"][0][at] = (sign * (120 if (l == length // 2) == (scale is None) else -120)).to(torch.int8)
            if l == length // 2:
                want += [V[at]] * n
    out, _ = attend(c, kernel, scale=scale, max_new=n, causal=False)
    want = torch.stack(want)[:, None]
    err = (out.double() - want).abs()
    assert bool((err <= want.abs() * (u + u_p + u * u_p + 2.0 ** -18) + 2.0 ** -40).all()), float(err.max())


@pytest.mark.parametrize("kernel,G,max_new", KERNELS)
@pytest.mark.parametrize("E", [-127, -130, -133])
def test_queries_below_the_normal_numbers(kernel, G, max_new, E):
    """Rows of subnormal bf16 queries, over keys that bring the scores to 2^-3 .. 2^4."""
    c, lens, offsets = make_case([90, 41, 3], [max_new, 1, 1], G, 1, 64, 16, 8, torch.bfloat16, 8)
    c["q"] = queries(c["q"].shape, E)
    assert bool((c["q"].float().abs().amax(-1) > 0).all()) and float(c["q"].float().abs().max()) < 2.0 ** -126
    c["exps"][0].fill_(121 + 127)
    out, lse = attend(c, kernel, scale=2.0 ** 4, max_new=max_new)
    bounds.compare(out, lse, bounds.attention(c, lens, offsets, kernel, 2.0 ** 4))


@pytest.mark.parametrize("kernel,G,Hk,D,max_new", [("few", 2, 4, 64, 3), ("few", 4, 2, 96, 2), ("few", 8, 1, 256, 1), ("rows", 5, 2, 128, 3), ("wide", 16, 2, 64, 4)])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_rows_of_every_size_in_one_call(kernel, G, Hk, D, max_new, softcap):
    """Each row of a magnitude of its own, from subnormal to the largest, over keys of the smallest scales: nearly equal weights
    beside dominating ones, in one tile.  A row's bits are the same when the others are ordinary."""
    c, lens, offsets = make_case([300, 41, 77], [max_new, 1, max_new], G * Hk, Hk, D, 16, 8, torch.bfloat16, 9)
    g = torch.Generator(device="cuda").manual_seed(D)
    T, Hq = c["q"].shape[:2]
    plain = queries((T, Hq, D), 0)
    E = torch.randint(-132, 128, (T, Hq, 1), generator=g, device="cuda").double()
    c["q"] = torch.where(E < 0, plain.double() * torch.exp2(E.clamp(-132, 0)), plain.double() * torch.exp2(E.clamp(0, 127))).to(torch.bfloat16)
    c["exps"][0].copy_(torch.randint(1, 5, c["exps"][0].shape, generator=g, device="cuda"))
    out, lse = attend(c, kernel, max_new=max_new, softcap=softcap)
    bounds.compare(out, lse, bounds.attention(c, lens, offsets, kernel, softcap=softcap))
    some = torch.rand((T, Hq), generator=g, device="cuda") < 0.5
    c["q"] = torch.where(some[..., None], c["q"], plain)
    again, again_lse = attend(c, kernel, max_new=max_new, softcap=softcap)
    assert torch.equal(again[some], out[some]) and torch.equal(again_lse[some], lse[some])
