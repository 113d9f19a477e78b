"""Attention over prompts and over many items a block, against plain attention in 64 bits by whole matrices."""
import math

import pytest
import torch

from semi_ar_draft_gb300 import api, binding

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
TYPES = [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16), (torch.bfloat16, E4M3), (torch.float16, E4M3)]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(lens, news, Hq, Hk, D, page, dtype, cache, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    blocks = [-(-x // page) for x in lens]
    P, width = sum(blocks) + 2, max(max(blocks), 1)
    perm = torch.randperm(P, generator=g, device="cuda").tolist()
    table, used = [], 0
    for n in blocks:
        table.append(perm[used:used + n] + [-1] * (width - n))
        used += n
    std = 30.0 if cache == E4M3 else 1.0
    kp, vp = ((torch.randn((P, page, Hk, D), generator=g, device="cuda") * std).to(cache) for _ in range(2))
    ks, vs = (None, None) if cache != E4M3 else ((0.5 + torch.rand(Hk, generator=g, device="cuda")) / std for _ in range(2))
    offsets = [0]
    for n in news:
        offsets.append(offsets[-1] + n)
    q = (torch.randn((offsets[-1], Hq, D), generator=g, device="cuda") * 1.5).to(dtype)
    return dict(q=q, k_pages=kp, v_pages=vp, block_table=i32(table), seq_len=i32(lens), offsets=i32(offsets), k_scale=ks, v_scale=vs)


def check(c, lens, news, causal=True, window=0, max_new=0):
    """The bound of tests/paged_reference.py, by matrices: u = finfo.eps / 2; a score is a sum of D products in fp32 (each
    step within 2^-23 of the magnitudes' sum) with a few roundings more; the probabilities are rounded by u_p, the
    exponential is within 2^-21, fp32 sums over N keys by 16 lanes within (N / 16 + 400) 2^-24, the output once by u."""
    out, lse, ws = api.paged_attention(**c, causal=causal, window=window, max_new=max_new, lse=True)
    assert binding.dspark_get_device_status(ws) == 0
    T, Hq, D = c["q"].shape
    page, Hk = c["k_pages"].shape[1:3]
    G, scale = Hq // Hk, D ** -0.5
    u = torch.finfo(c["q"].dtype).eps / 2
    u_p = 2.0 ** -11 if c["k_pages"].dtype == E4M3 else u
    a = 0
    for j, (L, n) in enumerate(zip(lens, news)):
        if n == 0:
            continue
        l = torch.arange(L, device="cuda")
        pos = L - n + torch.arange(n, device="cuda")[:, None]
        see = (l <= pos) if causal else torch.ones((n, L), dtype=torch.bool, device="cuda")
        if window:
            see = see & (l > pos - window)
        pages = c["block_table"][j].long()[l // page]
        k, v = (x[pages, l % page].double() * (1.0 if s is None else s.double()[:, None])
                for x, s in ((c["k_pages"], c["k_scale"]), (c["v_pages"], c["v_scale"])))  # [L, Hk, D]
        x = c["q"][a:a + n].double().view(n, Hk, G, D)
        s = torch.einsum("nhgd,lhd->nhgl", x, k) * scale
        mag = torch.einsum("nhgd,lhd->nhgl", x.abs(), k.abs()) * scale
        see = see[:, None, None, :]
        s = s.masked_fill(~see, -math.inf)
        ls = torch.logsumexp(s, -1)
        p = torch.exp(s - ls[..., None])
        o, away = (torch.einsum("nhgl,lhd->nhgd", p, y) for y in (v, v.abs()))
        d = torch.where(see, D * mag * 2.0 ** -23 + 8 * s.abs() * 2.0 ** -24, 0.0).amax(-1) + 2.0 ** -21
        steps = (see.sum(-1) / 16 + 400) * 2.0 ** -24
        tol = u * (o.abs() + 2 * u_p * away) + away * (u_p + 2 * d + 2 * steps)[..., None]
        if c["q"].dtype == torch.float16:
            tol = tol + 2.0 ** -25
        got, gl = out[a:a + n].view(n, Hk, G, D).double(), lse[a:a + n].view(n, Hk, G).double()
        assert bool(((got - o).abs() <= tol).all()), (j, float((got - o).abs().max()))
        assert bool(((gl - ls).abs() <= d + steps + ls.abs() * 2.0 ** -22).all()), (j, float((gl - ls).abs().max()))
        a += n


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("Hq,Hk,D", [(4, 1, 128), (3, 3, 64), (2, 1, 256)])
@pytest.mark.parametrize("window", [0, 1, 100, 333])
def test_prompts(dtype, cache, Hq, Hk, D, window):
    """Whole prompts, a chunk behind a cached prefix, and single tokens beside them."""
    lens, news = [700, 1100, 1, 900, 257], [700, 400, 1, 1, 257]
    check(make(lens, news, Hq, Hk, D, 16, dtype, cache, D + window), lens, news, window=window)


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_a_long_block_that_all_see(dtype, cache):
    lens, news = [600, 300], [515, 300]
    check(make(lens, news, 4, 2, 64, 32, dtype, cache, 3), lens, news, causal=False)
    check(make(lens, news, 4, 2, 64, 32, dtype, cache, 4), lens, news, causal=False, window=77)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("D,Hk,most", [(64, 16, 60), (128, 8, 200), (256, 8, 100), (128, 16, 500)])
def test_many_items_a_block(dtype, cache, D, Hk, most):
    """Row tiles of 128 with dozens of items a block, most of one or two key tiles, some empty."""
    g = torch.Generator().manual_seed(D + most)
    B = 400 if most < 500 else 120
    news = torch.randint(0, 21, (B,), generator=g).tolist()
    lens = [n + int(x) for n, x in zip(news, torch.randint(0, most, (B,), generator=g))]
    c = make(lens, news, 8 * Hk, Hk, D, 16, dtype, cache, D)
    check(c, lens, news, max_new=20)
