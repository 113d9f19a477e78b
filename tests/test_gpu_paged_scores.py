"""Attention's scores at the ends of their range: softcaps far above them, probabilities far below the largest."""
import math

import pytest
import torch

from semi_ar_draft_gb300 import api, binding

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
TYPES = [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16), (torch.bfloat16, E4M3), (torch.float16, E4M3)]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def one_head(q, k, v, G, n, dtype, cache, **kw):
    """Attention of n tokens of G equal-kv heads (q [n G, D]) over k, v [L, D] in pages of 16; (out, lse) [n G, ...]."""
    L, D = k.shape
    pages = -(-L // 16)
    pool = torch.zeros((2, pages * 16, D), device="cuda")
    pool[0, :L], pool[1, :L] = k, v
    kp, vp = (x.to(cache).view(pages, 16, 1, D) for x in pool)
    out, lse, ws = api.paged_attention(q.to(dtype).view(n, G, D), kp, vp, i32([list(range(pages))]), i32([L]), i32([0, n]),
                                       lse=True, causal=False, **kw)
    assert binding.dspark_get_device_status(ws) == 0
    return out.view(n * G, D).double(), lse.view(n * G).double()


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("max_new", [1, 17])
@pytest.mark.parametrize("c", [0.5, 5.0, 50.0, 300.0, 1e4, 1e6, 1e9, 1e20, 2.0 ** 100, 3e38])
def test_softcap_is_c_tanh_of_s_over_c(dtype, cache, max_new, c):
    """One key a request: lse is the score itself.  Queries and keys of one value each, so that q . k is exact in fp32
    and the score's own error shows.  2^-18 of it covers the tanh (2e-6), the scale's product,
    the constants' roundings and two roundings into and out of the log2 domain; 2^-21 the one probability's exponent, an
    fp32 number below 8 (halves are taken against a reference up to 7 lower), and its logarithm."""
    G, D, n = 16, 64, 17
    x = torch.cat([torch.logspace(-4, 1.5, 136, device="cuda"), -torch.logspace(-4, 1.5, 136, device="cuda")]).to(dtype)
    q = torch.zeros((n * G, D), device="cuda")
    q[:, 0] = x.float()
    k = torch.zeros((1, D), device="cuda")
    k[0, 0] = 8.0
    v = torch.ones((1, D), device="cuda")
    out, lse = one_head(q, k, v, G, n, dtype, cache, scale=0.75, softcap=c, max_new=max_new)
    s = x.double() * 8.0 * 0.75
    want = c * torch.tanh(s / c)
    assert bool((out == 1).all())
    assert bool(((lse - want).abs() <= 2.0 ** -18 * want.abs() + 2.0 ** -21).all()), float(((lse - want) / want).abs().max())


@pytest.mark.parametrize("max_new", [1, 17])
def test_a_large_softcap_changes_nothing(max_new):
    """c tanh(s / c) is s within 2^-21 of it where |s| < 2^-10 c."""
    g = torch.Generator(device="cuda").manual_seed(4)
    G, D, n, L = 16, 128, 17, 200
    q, k, v = (torch.randn((m, D), generator=g, device="cuda") for m in (n * G, L, L))
    ref, ref_lse = one_head(q, k, v, G, n, torch.bfloat16, torch.bfloat16, max_new=max_new)
    for c in (1e5, 1e7, 1e12):
        out, lse = one_head(q, k, v, G, n, torch.bfloat16, torch.bfloat16, max_new=max_new, softcap=c)
        # scores below 8 move by 8 2^-18 at most; an output by twice that of the largest value, and by the roundings of
        # its probabilities and its own on either side
        assert bool(((lse - ref_lse).abs() <= 2.0 ** -15).all())
        big = float(v.abs().max())
        assert bool(((out - ref).abs() <= 2 * big * 2.0 ** -15 + 2 * 2.0 ** -8 * (ref.abs() + big)).all())


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("lead", [10.0, 14.0, 16.0, 18.0])
@pytest.mark.parametrize("L,max_new", [(700, 1), (700, 17), (9000, 1), (9000, 17)])
def test_a_key_that_dominates_with_a_small_value(dtype, cache, lead, L, max_new):
    """An attention sink: the first key leads by `lead` nats and its value is 0, so the output is what the other keys'
    small probabilities make of their values.

    Bound: probabilities are taken against a reference r with at least one at 1 or more, times 2^7 as halves: half a
    step of the subnormal halves is 2^-25, so each is off by 2^-32 / sum at most, or by its rounding (u_p); the output
    by one rounding more (2 u |o|, 2^-25 where it is a subnormal half); scores in fp32 by 2^-18 (20 nats, D = 64
    products and a few roundings)."""
    G, D, n = 16, 64, 17
    g = torch.Generator(device="cuda").manual_seed(int(lead) + L)
    q = torch.zeros((n * G, D), device="cuda")
    q[:, 0] = 1.0
    q[:, 1] = torch.rand(n * G, generator=g, device="cuda").to(torch.float16).float() * 0.25
    k = torch.zeros((L, D), device="cuda")
    k[0, 0] = lead
    k[1:, 1] = torch.randint(-4, 5, (L - 1,), generator=g, device="cuda") * 0.25
    v = 100.0 + 10.0 * torch.randint(0, 20, (L, D), generator=g, device="cuda")
    v[0] = 0.0
    v = v.to(cache).float()
    k = k.to(cache).float()
    out, lse = one_head(q, k, v, G, n, dtype, cache, scale=1.0, max_new=max_new)
    s = q.to(dtype).double() @ k.double().T
    p = torch.softmax(s, -1)
    want = p @ v.double()
    assert bool((s[:, 0] - s[:, 1:].amax(-1) > lead - 1).all())
    u = torch.finfo(dtype).eps / 2
    u_p = u if cache != E4M3 else 2.0 ** -11
    absolute = 0.0 if (dtype, cache) == (torch.bfloat16, torch.bfloat16) else 2.0 ** -32
    away = p[:, 1:] @ v[1:].double()
    tol = away * (u_p + 2.0 ** -17) + absolute * v.double().sum(0) + 2 * u * want + 2.0 ** -25
    err = (out - want).abs()
    assert bool((err <= tol).all()), (float((err / want).max()), float((err - tol).max()))
