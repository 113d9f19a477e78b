"""The paged-cache operators on the GPU against plain implementations (whole numbers exactly; attention
in 64 bits, within the bound tests/paged_reference.py derives)."""
import math

import pytest
import torch

import paged_reference as R
from semi_ar_draft_gb300 import api, binding

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def status(ws):
    return binding.dspark_get_device_status(ws)


# ------------------------------------------------------------------ plan and commit
def run_plan(cache_len, new_len, table, n_blocks, free, n_free, page, max_tokens, extra):
    t = i32(table)
    *out, ws = api.cache_plan(i32(cache_len), i32(new_len), t, i32(n_blocks), i32(free), i32([n_free]), page, max_tokens,
                              extra=extra)
    seq, off, slots, pos, held, left = [x.tolist() for x in out]
    return (seq, off, slots, pos, held, left[0], t.tolist(), status(ws) == 8), status(ws)


@pytest.mark.parametrize("B,page,most,new,extra", [
    (1, 16, 1, 1, 0), (1, 1, 9, 3, 1), (3, 16, 100, 9, 1), (32, 16, 500, 9, 1), (33, 64, 1000, 1, 0), (7, 128, 300, 700, 0),
    (700, 32, 90, 17, 1), (2100, 2, 20, 5, 0), (48, 4096, 9000, 5000, 0)])
def test_plan_and_commit(B, page, most, new, extra):
    g = torch.Generator().manual_seed(B * 7 + page)
    rnd = lambda lo, hi: torch.randint(lo, hi + 1, (B,), generator=g).tolist()  # noqa: E731
    cache_len, new_len = rnd(0, most), rnd(0, new)
    n_blocks = [-(-x // page) for x in cache_len]
    width = max(-(-(c + n + extra) // page) for c, n in zip(cache_len, new_len)) + 1
    P = sum(n_blocks) + sum(-(-(c + n + extra) // page) for c, n in zip(cache_len, new_len)) + 3
    perm = torch.randperm(P, generator=g).tolist()
    table, used = [], 0
    for n in n_blocks:
        table.append(perm[used:used + n] + [-7] * (width - n))
        used += n
    free, n_free = perm[used:] + [-1] * used, P - used
    total = sum(new_len) + extra * B
    got, st = run_plan(cache_len, new_len, table, n_blocks, free, n_free, page, total + 5, extra)
    ref = R.plan(cache_len, new_len, table, n_blocks, free, n_free, page, total + 5, extra, P)
    assert st == 0 and got == ref

    # some are rejected, some requests end
    add = [min(int(x), n) for x, n in zip(rnd(0, new), new_len)]
    done = [int(x) for x in torch.rand(B, generator=g) < 0.3]
    f = i32(free)
    length, held, left, ws = api.cache_commit(i32(cache_len), i32(add), i32(got[6]), i32(got[4]), f, i32([got[5]]), page,
                                              extra=extra, done=torch.tensor(done, dtype=torch.uint8, device="cuda"))
    ref = R.commit(cache_len, add, got[6], got[4], free, got[5], page, extra, done, P)
    assert status(ws) == 0
    assert (length.tolist(), held.tolist(), left.item(), f.tolist(), False) == ref


def test_many_steps_lose_no_page():
    """Rounds of plan and commit: at every point each page is in one request's table or on the stack, once."""
    B, page, P, width = 24, 8, 400, 60
    g = torch.Generator().manual_seed(5)
    cache_len, n_blocks, n_free = i32([0] * B), i32([0] * B), i32([P])
    free, table = torch.randperm(P, generator=g).int().cuda(), torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    for _ in range(40):
        new = torch.randint(0, 17, (B,), generator=g).int()
        seq, off, slots, _, n_blocks, n_free, ws = api.cache_plan(cache_len, new.cuda(), table, n_blocks, free, n_free, page,
                                                                  17 * B + B, extra=1)
        assert status(ws) == 0
        live = slots[: int(off[-1])]
        assert int(live.min()) >= 0 and live.unique().numel() == live.numel()
        acc = (torch.rand(B, generator=g) * (new + 1)).int().cuda()
        done = (torch.rand(B, generator=g) < 0.15).cuda()
        cache_len, n_blocks, n_free, ws = api.cache_commit(cache_len, acc, table, n_blocks, free, n_free, page, extra=1,
                                                           done=done)
        assert status(ws) == 0
        held = [p for j in range(B) for p in table[j, : int(n_blocks[j])].tolist()]
        assert sorted(held + free[: int(n_free)].tolist()) == list(range(P))
        assert n_blocks.tolist() == [-(-x // page) for x in cache_len.tolist()]


def test_plan_without_new_lengths_and_positions():
    out = api.cache_plan(i32([5, 0]), None, i32([[3, -1], [-1, -1]]), i32([1, 0]), i32([7, 2, 1, 0, 0, 0, 0, 0]), i32([3]), 8, 3,
                         extra=1, positions=False)
    assert out[3] is None and out[0].tolist() == [6, 1] and out[2].tolist() == [3 * 8 + 5, 8, -1] and out[5].item() == 2


@pytest.mark.parametrize("what", ["pool", "table", "tokens", "length", "count", "blocks", "stack", "page"])
def test_plan_reports_what_does_not_fit(what):
    cache_len, new_len, page, T = [20, 3, 40], [30, 1, 60], 16, 120
    n_blocks, width, P = [2, 1, 3], 8, 20
    table = [[0, 1] + [-1] * 6, [2] + [-1] * 7, [3, 4, 5] + [-1] * 5]
    free, n_free = list(range(6, 20)) + [0] * 6, 14
    if what == "pool":
        n_free = 3  # four are wanted
    if what == "table":
        table, width = [r[:5] for r in table], 5
    if what == "tokens":
        T = 50
    if what == "length":
        cache_len[1] = -4
    if what == "count":
        new_len[0] = -3
    if what == "blocks":
        n_blocks[2] = 9
    if what == "stack":
        n_free = 21
    if what == "page":
        table[0][1] = 77
    got, st = run_plan(cache_len, new_len, table, n_blocks, free, n_free, page, T, 0)
    ref = R.plan(cache_len, new_len, table, n_blocks, free, n_free, page, T, 0, P)
    assert got[:7] == ref[:7]
    assert st == (0 if what == "page" else 8)  # a page outside the pool shows in its tokens' slots


def test_commit_reports_what_does_not_fit():
    table, free, P = [[0, 1, 2], [3, 4, 5]], [6, 7, 0, 0, 0, 0, 0, 0], 8
    for cache_len, add, n_blocks, n_free in (([50, 10], [0, 0], [3, 3], 2), ([10, -5], [0, 2], [3, 3], 2),
                                             ([10, 10], [1, 1], [4, 3], 2), ([0, 0], [0, 0], [3, 3], 5)):
        f = i32(free)
        length, held, left, ws = api.cache_commit(i32(cache_len), i32(add), i32(table), i32(n_blocks), f, i32([n_free]), 16)
        ref = R.commit(cache_len, add, table, n_blocks, free, n_free, 16, 0, [0, 0], P)
        assert ref[4] and status(ws) == 8
        assert (length.tolist(), held.tolist(), left.item(), f.tolist()) == ref[:4]


# ------------------------------------------------------------------ append
def make_pool(P, page, Hk, D, dtype, g, heads_first=False, std=1.0):
    shape = (P, Hk, page, D) if heads_first else (P, page, Hk, D)
    x = torch.randn(shape, generator=g, device="cuda") * std
    x = x.to(dtype)
    return x.transpose(1, 2) if heads_first else x


@pytest.mark.parametrize("dtype,cache", [(torch.bfloat16,) * 2, (torch.float16,) * 2, (torch.bfloat16, E4M3), (torch.float16, E4M3)])
@pytest.mark.parametrize("T,Hk,D,page,heads_first,shift", [
    (1, 1, 64, 16, False, 0), (7, 8, 128, 16, False, 0), (300, 2, 96, 1, True, 0), (129, 3, 80, 64, False, 1), (2000, 16, 256, 32, True, 8)])
def test_append(dtype, cache, T, Hk, D, page, heads_first, shift):
    g = torch.Generator(device="cuda").manual_seed(T + D)
    P = -(-T // page) + 3
    kp, vp = (make_pool(P, page, Hk, D, cache, g, heads_first) for _ in range(2))
    buf = torch.randn(T * 3 * Hk * D + 16, generator=g, device="cuda").mul(3).to(dtype)
    qkv = buf[shift: shift + T * 3 * Hk * D].view(T, 3 * Hk, D)  # shift: rows that start between 16-byte boundaries
    k, v = qkv[:, Hk: 2 * Hk], qkv[:, 2 * Hk:]
    ks = vs = None
    if cache == E4M3:
        ks, vs = (0.003 + 0.01 * torch.rand(Hk, generator=g, device="cuda") for _ in range(2))
    slots = torch.randperm(P * page, generator=g, device="cuda")[:T]
    slots[T // 2] = -1 if T > 1 else slots[0]
    if T > 3:
        slots[1] = P * page  # past the pool: skipped
    want = []
    for x, pool, s in ((k, kp, ks), (v, vp, vs)):
        y = x.float() if s is None else (x.float() / s[:, None]).clamp(-448, 448)
        new = pool.clone()
        for i, at in enumerate(slots.tolist()):
            if 0 <= at < P * page:
                new[at // page, at % page] = y[i].to(cache)
        want.append(new)
    api.cache_append(k, v, kp, vp, slots, ks, vs)
    for got, ref in zip((kp, vp), want):
        assert torch.equal(got.contiguous().view(torch.uint8), ref.contiguous().view(torch.uint8))


def test_append_rounds_every_half_and_keeps_nan():
    """All 2^16 halves through an e4m3 cache: the nearest e4m3 value, ties to even, clamped; NaN stays NaN."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.float16).cuda().view(256, 1, 256)
    kp, vp = (torch.zeros((16, 16, 1, 256), dtype=E4M3, device="cuda") for _ in range(2))
    one = torch.ones(1, device="cuda")
    api.cache_append(x, x, kp, vp, torch.arange(256, device="cuda"), one, None)
    got = kp.view(256, 256).double().cpu()
    ref = x.view(256, 256).double().cpu()  # on the host, where powers of two are exact
    assert torch.equal(got.isnan(), ref.isnan()) and torch.equal(vp.view(torch.uint8), kp.view(torch.uint8))
    ref = ref.clamp(-448, 448)
    exponent = torch.frexp(ref.abs()).exponent.clamp(min=-5) - 4  # of the grid's step: 3 bits below the value's
    ref = torch.ldexp(torch.round(torch.ldexp(ref, -exponent)), exponent)  # half to even, exact in 64 bits
    ok = ~ref.isnan()
    assert torch.equal(got[ok], ref[ok])


# ------------------------------------------------------------------ attention
def make_case(lens, news, Hq, Hk, D, page, dtype, cache, seed, pad=0, spare=3, heads_first=False, q_shift=0):
    """A scattered cache of requests with `lens` tokens (new ones included), `news` of them new."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B = len(lens)
    blocks = [-(-x // page) for x in lens]
    P, width = sum(blocks) + spare, max(max(blocks), 1)
    perm = torch.randperm(P, generator=g, device="cuda").int().tolist()
    table, used = [], 0
    for n in blocks:
        table.append(perm[used:used + n] + [-1] * (width - n))
        used += n
    std = 30.0 if cache == E4M3 else 1.0
    kp, vp = (make_pool(P, page, Hk, D, cache, g, heads_first, std) for _ in range(2))
    ks = vs = None
    if cache == E4M3:
        ks, vs = ((0.5 + torch.rand(Hk, generator=g, device="cuda")) / std for _ in range(2))
    offsets = [0]
    for n in news:
        offsets.append(offsets[-1] + n)
    T = offsets[-1] + pad
    W = Hq + 2 * Hk
    buf = (torch.randn(T * W * D + 16, generator=g, device="cuda") * 1.5).to(dtype)
    q = buf[q_shift: q_shift + T * W * D].view(T, W, D)[:, :Hq]
    return {"q": q, "k_pages": kp, "v_pages": vp, "block_table": i32(table), "seq_len": i32(lens), "offsets": i32(offsets),
            "k_scale": ks, "v_scale": vs}, lens, offsets


def attend(c, **kw):
    out, lse, ws = api.paged_attention(c["q"], c["k_pages"], c["v_pages"], c["block_table"], c["seq_len"], c["offsets"],
                                       k_scale=c["k_scale"], v_scale=c["v_scale"], lse=True, **kw)
    return out, lse, ws


def check(c, lens, offsets, causal=True, window=0, softcap=0.0, scale=None, **kw):
    out, lse, ws = attend(c, causal=causal, window=window, softcap=softcap, scale=scale, **kw)
    assert status(ws) == 0
    scale = c["q"].shape[2] ** -0.5 if scale is None else scale
    ro, rl, to, tl = R.attention(c["q"], c["k_pages"], c["v_pages"], c["block_table"], lens, offsets, scale, causal, window,
                                 softcap, c["k_scale"], c["v_scale"])
    dead = rl == -math.inf
    assert torch.equal(lse == -math.inf, dead) and not out[dead].any()
    err = (out.double() - ro).abs()
    assert bool((err <= to).all()), f"out: {float((err - to).max())} past the bound, worst {float(err.max())}"
    el = (lse.double() - rl).abs()[~dead]
    assert bool((el <= tl[~dead]).all()), f"lse: worst {float(el.max())}"
    return out, lse


TYPES = [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16), (torch.bfloat16, E4M3), (torch.float16, E4M3)]


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("Hq,Hk,D,page", [(4, 4, 64, 16), (8, 1, 128, 16), (8, 2, 256, 32), (5, 1, 80, 1), (14, 2, 96, 64),
                                          (32, 2, 192, 8), (3, 3, 16, 128), (64, 1, 64, 16), (104, 2, 128, 64)])
def test_one_token(dtype, cache, Hq, Hk, D, page):
    lens = [1, 15, 16, 17, 0, 63, 64, 65, 300]
    c, lens, offsets = make_case(lens, [1] * len(lens), Hq, Hk, D, page, dtype, cache, D + page)
    out, lse = check(c, lens, offsets)
    again, lse2, _ = attend({**c, "offsets": None})
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("Hq,Hk,D,page", [(4, 4, 64, 16), (8, 2, 128, 16), (16, 2, 128, 64), (8, 1, 256, 32), (7, 1, 96, 4), (14, 2, 80, 16)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("max_new", [1, 33])  # what chooses between row tiles of 16 and of 128
def test_several_tokens(dtype, cache, Hq, Hk, D, page, causal, max_new):
    news = [1, 17, 0, 5, 9, 2, 33]
    lens = [1, 17, 0, 70, 129, 300, 40]
    c, lens, offsets = make_case(lens, news, Hq, Hk, D, page, dtype, cache, 3 * D + page, pad=3)
    out, lse = check(c, lens, offsets, causal=causal, max_new=max_new)
    assert not out[offsets[-1]:].any() and bool((lse[offsets[-1]:] == -math.inf).all())


@pytest.mark.parametrize("window", [1, 7, 64, 100])
@pytest.mark.parametrize("softcap", [0.0, 5.0])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("cache", [torch.bfloat16, E4M3])
@pytest.mark.parametrize("Hq,max_new", [(8, 1), (8, 17), (32, 17)])
def test_window_and_softcap(window, softcap, causal, cache, Hq, max_new):
    news, lens = [1, 9, 4, 17], [500, 9, 130, 201]
    c, lens, offsets = make_case(lens, news, Hq, 2, 128, 16, torch.bfloat16, cache, window)
    check(c, lens, offsets, causal=causal, window=window, softcap=softcap, max_new=max_new)


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
@pytest.mark.parametrize("max_new", [1, 17])
def test_other_scales(scale, max_new):
    c, lens, offsets = make_case([200, 9], [3, 2], 16, 1, 64, 16, torch.float16, torch.float16, 1)
    check(c, lens, offsets, scale=scale, max_new=max_new)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("lens,news,Hq,Hk,D", [([20000], [1], 8, 1, 128), ([9000, 1, 5000], [1, 1, 4], 4, 1, 256),
                                               ([33, 12000, 700], [2, 17, 3], 8, 2, 64), ([15000, 2000], [9, 1], 16, 1, 128),
                                               ([9000, 500], [16, 1], 64, 8, 64), ([11000], [13], 9, 1, 256)])
@pytest.mark.parametrize("max_new", [1, 17])
def test_long_caches_are_split_and_joined(dtype, cache, lens, news, Hq, Hk, D, max_new):
    c, lens, offsets = make_case(lens, news, Hq, Hk, D, 64, dtype, cache, sum(lens))
    out, lse = check(c, lens, offsets, max_new=max_new)
    again, lse2, _ = attend(c, max_new=max_new)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("max_new", [1, 40])
def test_many_requests(max_new):
    g = torch.Generator().manual_seed(3)
    news = torch.randint(0, 4, (900,), generator=g).tolist()
    lens = [n + int(x) for n, x in zip(news, torch.randint(0, 60, (900,), generator=g))]
    c, lens, offsets = make_case(lens, news, 16, 1, 64, 16, torch.bfloat16, torch.bfloat16, 8)
    check(c, lens, offsets, max_new=max_new)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("Hq,Hk", [(4, 1), (8, 2), (16, 1), (32, 1)])
@pytest.mark.parametrize("max_new", [1, 17])
def test_what_is_not_seen_does_not_matter(dtype, cache, Hq, Hk, max_new):
    """NaN and inf in later tokens, before the window, past a request's length and in pages of nobody."""
    D, page, news, lens = 128, 16, [9, 1, 5], [100, 37, 200]
    c, lens, offsets = make_case(lens, news, Hq, Hk, D, page, dtype, cache, 77)
    for kw in ({"causal": True}, {"causal": True, "window": 20}, {"causal": False, "window": 30}):
        kw["max_new"] = max_new
        ref, ref_lse, _ = attend(c, **kw)
        bad = {**c, "k_pages": c["k_pages"].clone(), "v_pages": c["v_pages"].clone()}
        owned = torch.zeros(bad["k_pages"].shape[:2], dtype=torch.bool, device="cuda")
        last = {}
        for j, n in enumerate(lens):
            for pos in range(n):
                owned[c["block_table"][j, pos // page], pos % page] = True
            # the request's last token: unseen by its other rows when causal
            last[j] = (int(c["block_table"][j, (n - 1) // page]), (n - 1) % page)
        nan, inf = (float("nan"), float("inf")) if cache != E4M3 else (0x7F, 0x7F)  # e4m3 has no inf
        for pool in (bad["k_pages"], bad["v_pages"]):
            pool = pool.view(torch.uint8) if cache == E4M3 else pool
            pool[~owned] = nan
            if kw["causal"]:
                for j, (p, s) in last.items():
                    if news[j] > 1:
                        pool[p, s] = nan if j else inf
            if kw.get("window"):
                for j, n in enumerate(lens):
                    first = n - news[j] - kw["window"]  # the last position that no row sees
                    for pos in range(max(first - 3, 0), first + 1):
                        pool[c["block_table"][j, pos // page].long(), pos % page] = nan
        out, lse, ws = attend(bad, **kw)
        assert status(ws) == 0
        for j in range(len(lens)):
            rows = slice(offsets[j], offsets[j + 1] - (1 if kw["causal"] and news[j] > 1 else 0))
            assert bool(out[rows].isfinite().all()), (kw, j)
            # an edge slice is then summed key by key: the same terms, unrounded probabilities
            u = torch.finfo(dtype).eps / 2
            away = 8.0 * float(c["v_scale"].max() * 30 if cache == E4M3 else 1.0)
            assert bool(((out[rows] - ref[rows]).abs().double() <= 4 * u * away).all()), (kw, j)
            assert bool(((lse[rows] - ref_lse[rows]).abs() <= 1e-5).all()), (kw, j)
            if kw["causal"] and news[j] > 1:
                assert not bool(out[offsets[j + 1] - 1].isfinite().all())


@pytest.mark.parametrize("max_new", [1, 17])
def test_values_that_are_seen_go_through(max_new):
    """A NaN or an infinite value that a row sees reaches it, and only it."""
    c, lens, offsets = make_case([50, 60], [3, 2], 16, 1, 64, 16, torch.bfloat16, torch.bfloat16, 4)
    ref, _, _ = attend(c, max_new=max_new)
    c["v_pages"][c["block_table"][0, 2].long(), 15, 0, 5] = float("nan")  # request 0, position 47: its first new token
    c["v_pages"][c["block_table"][1, 3].long(), 11, 0, 6] = float("inf")  # request 1, position 59: its last
    out, _, _ = attend(c, max_new=max_new)
    assert bool(out[0:3, :, 5].isnan().all()) and bool((out[4, :, 6] == math.inf).all())
    out[0:3, :, 5] = ref[0:3, :, 5]
    out[4, :, 6] = ref[4, :, 6]
    assert bool(((out - ref).abs() <= 8 * 2.0 ** -8 * 4).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("max_new", [1, 8])
def test_every_8_bit_value(dtype, max_new):
    """Eight equal keys and values: an output is the value itself, and a one-hot query's lse is its key plus ln 8."""
    codes = torch.arange(256, dtype=torch.uint8).view(2, 1, 1, 128).expand(2, 8, 1, 128).clone()  # a page a request
    keys = codes.clone()
    keys[(codes & 0x7F) == 0x7F] = 0  # (a NaN key is a NaN score for every query)
    pool = lambda x: torch.cat([x, torch.zeros_like(x)]).view(E4M3).cuda()
    q = torch.eye(128).view(1, 8, 16, 128).expand(2, 8, 16, 128).reshape(16, 16, 128).to("cuda", dtype)
    c = {"q": q, "k_pages": pool(keys), "v_pages": pool(codes), "block_table": i32([[0], [1]]), "seq_len": i32([8, 8]),
         "offsets": i32([0, 8, 16]), "k_scale": None, "v_scale": None}
    out, lse, ws = attend(c, causal=False, scale=1.0, max_new=max_new)
    assert status(ws) == 0
    v = codes[:, 0, 0].view(E4M3).float().cuda()
    assert torch.equal(out.float().nan_to_num(nan=1e9), v.view(2, 1, 1, 128).expand(2, 8, 16, 128).reshape(16, 16, 128).nan_to_num(nan=1e9))
    k = keys[:, 0, 0].view(E4M3).double().cuda().view(16, 16)
    # products with the two logarithms' constants, the sum and the logarithm of 8: a few roundings of fp32
    assert bool(((lse.double() - k - math.log(8)).abs() <= 2.0 ** -21 * (k.abs() + 3)).all())


@pytest.mark.parametrize("max_new", [1, 17])
def test_rows_that_see_nothing(max_new):
    """More new tokens than the cache holds: the first rows stand before position 0."""
    c, lens, offsets = make_case([4, 1, 0], [4, 3, 2], 16, 2, 64, 16, torch.float16, torch.float16, 2)
    for window in (0, 3):
        out, lse, ws = attend(c, window=window, max_new=max_new)
        assert not out[4:6].any() and bool((lse[4:6] == -math.inf).all()) and not out[7:].any()
        assert bool((lse[6].isfinite()).all()) and status(ws) == 0
        check(c, lens, offsets, window=window, max_new=max_new)


@pytest.mark.parametrize("q_shift", [0, 1, 2, 8])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("cache", [torch.bfloat16, E4M3])
@pytest.mark.parametrize("max_new", [1, 17])
def test_strides_and_alignment(q_shift, heads_first, cache, max_new):
    c, lens, offsets = make_case([33, 100, 7], [2, 9, 1], 32, 2, 128, 16, torch.bfloat16, cache, 6, heads_first=heads_first,
                                 q_shift=q_shift)
    check(c, lens, offsets, max_new=max_new)


@pytest.mark.parametrize("cache", [torch.bfloat16, E4M3])
@pytest.mark.parametrize("max_new", [1, 10])
def test_pools_past_4_gib(cache, max_new):
    """Pages whose byte offsets pass 32 bits."""
    page, Hk, D, P = 64, 8, 128, 70000 if cache == torch.bfloat16 else 140000
    kp, vp = (torch.empty((P, page, Hk, D), dtype=cache, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(1)
    use = [P - 1, 3, P - 5, P // 2 + 9]
    T = 10
    slots = torch.tensor([use[i // page] * page + i % page for i in range(200)], device="cuda")
    k, v = (torch.randn((200, Hk, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    api.cache_append(k, v, kp, vp, slots)
    q = torch.randn((T, 64, D), generator=g, device="cuda").to(torch.bfloat16)
    c = {"q": q, "k_pages": kp, "v_pages": vp, "block_table": i32([use]), "seq_len": i32([200]), "offsets": i32([0, T]),
         "k_scale": None, "v_scale": None}
    check(c, [200], [0, T], max_new=max_new)


@pytest.mark.parametrize("max_new", [1, 17])
def test_large_scores_and_queries(max_new):
    """Scores far apart, and bf16 queries beyond the halves' range over an 8-bit cache."""
    for cache in (torch.bfloat16, E4M3):
        c, lens, offsets = make_case([300, 40], [2, 3], 32, 1, 128, 16, torch.bfloat16, cache, 11)
        c["q"].mul_(20.0)
        check(c, lens, offsets, max_new=max_new)
        c["q"].mul_(2.0 ** 60)
        check(c, lens, offsets, scale=2.0 ** -63, max_new=max_new)
        c["q"].mul_(2.0 ** -160)
        check(c, lens, offsets, scale=2.0 ** 97, max_new=max_new)


@pytest.mark.parametrize("max_new", [1, 17])
def test_pages_before_the_window_may_be_gone(max_new):
    """A sliding window's caller gives old pages back: their table entries are not looked at."""
    for cache in (torch.bfloat16, E4M3):
        c, lens, offsets = make_case([400, 130], [3, 2], 64, 2, 128, 16, torch.bfloat16, cache, 5)
        ref, _, ws = attend(c, window=70, max_new=max_new)
        c["block_table"][0, : (400 - 3 - 70 + 1) // 16] = -1
        c["block_table"][1, : (130 - 2 - 70 + 1) // 16] = 1 << 30
        out, _, ws = attend(c, window=70, max_new=max_new)
        assert status(ws) == 0 and torch.equal(out, ref)


@pytest.mark.parametrize("max_new", [1, 17])
def test_no_tokens_at_all(max_new):
    c, lens, offsets = make_case([40, 50], [0, 0], 4, 1, 64, 16, torch.bfloat16, torch.bfloat16, 9, pad=2)
    out, lse, ws = attend(c, max_new=max_new)
    assert not out.any() and bool((lse == -math.inf).all()) and status(ws) == 0
    c["q"] = c["q"][:0]
    out, lse, ws = attend(c, max_new=max_new)
    assert out.numel() == 0 and status(ws) == 0
    seq, off, slots, pos, *_ = api.cache_plan(i32([3]), None, i32([[0]]), i32([1]), i32([1]), i32([0]), 16, 0)
    assert slots.numel() == 0 and off.tolist() == [0, 0] and seq.tolist() == [3]


@pytest.mark.parametrize("max_new", [1, 17])
def test_bad_tables_are_reported(max_new):
    c, lens, offsets = make_case([40, 50], [1, 1], 32 if max_new > 1 else 4, 1, 64, 16, torch.bfloat16, torch.bfloat16, 9)
    ref, _, _ = attend(c, max_new=max_new)
    for what in ("page", "negative", "long", "offsets"):
        d = {**c, "block_table": c["block_table"].clone(), "seq_len": c["seq_len"].clone(), "offsets": c["offsets"].clone()}
        if what == "page":
            d["block_table"][0, 1] = 1 << 20
        if what == "negative":
            d["block_table"][0, 1] = -1
        if what == "long":
            d["seq_len"][0] = 1 << 30
        if what == "offsets":
            d["offsets"][0] = -5
        out, _, ws = attend(d, max_new=max_new)
        assert status(ws) == 8, what
        assert torch.equal(out[1], ref[1])
        _, _, ws = attend(c, max_new=max_new)
        assert status(ws) == 0


@pytest.mark.parametrize("max_new", [1, 5])
def test_other_stream_and_graph(max_new):
    """On a side stream, and replayed from a graph after the lengths changed."""
    Hq = 32
    c, lens, offsets = make_case([700, 200, 64], [1, 5, 2], Hq, 2, 128, 16, torch.bfloat16, torch.bfloat16, 12)
    ref, ref_lse, _ = attend(c, max_new=max_new)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        out, lse, _ = attend(c, max_new=max_new)
    side.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    out, lse, _ = attend(c, max_new=max_new, stream=side)
    side.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    out = torch.zeros_like(ref)
    ws = torch.empty(api.b.dspark_paged_attention_workspace_size(api.b.AttentionParams(
        8, 3, Hq, 2, 128, 16, 100, 50, max_new, api.b.BF16, api.b.BF16, 1, 0, 1.0, 0.0, 1, 1, 8, 8, 8)), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attend(c, out=out, ws=ws, max_new=max_new)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    c["seq_len"].copy_(i32([333, 150, 2]))
    graph.replay()
    torch.cuda.synchronize()
    want, _, _ = attend(c, max_new=max_new)
    assert torch.equal(out, want) and not torch.equal(out, ref)


def test_launches_are_counted():
    c, _, _ = make_case([40], [1], 4, 1, 64, 16, torch.bfloat16, torch.bfloat16, 9)
    n = binding.dspark_kernel_launches()
    attend(c)
    assert binding.dspark_kernel_launches() == n + 2
