"""Attention over the int8 paged cache against the definition in 64 bits, within the bound tests/i8_reference.py derives."""
import math

import pytest
import torch

import i8_reference as R
from semi_ar_draft_gb300 import api, binding

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def status(ws):
    return binding.dspark_get_device_status(ws)


def make_case(lens, news, Hq, Hk, D, page, block, dtype, seed, pad=0, spare=3, heads_first=False, q_shift=0, lo=119, hi=124):
    """A scattered cache of requests with `lens` tokens (new ones included), `news` of them new; blocks whose scales
    differ by up to 2^(hi - lo - 1)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    blocks = [-(-x // page) for x in lens]
    P, width = sum(blocks) + spare, max(max(blocks), 1)
    perm = torch.randperm(P, generator=g, device="cuda").int().tolist()
    table, used = [], 0
    for n in blocks:
        table.append(perm[used:used + n] + [-1] * (width - n))
        used += n
    shape = (P, Hk, page, D) if heads_first else (P, page, Hk, D)
    codes = [(torch.randn(shape, generator=g, device="cuda") * 36).round().clamp(-127, 127).to(torch.int8) for _ in range(2)]
    shape = (P, page // block, Hk) if heads_first else (P, Hk, page // block)
    exps = [torch.randint(lo, hi, shape, generator=g, device="cuda").to(torch.uint8) for _ in range(2)]
    if heads_first:
        codes, exps = ([x.transpose(1, 2) for x in y] for y in (codes, exps))
    offsets = [0]
    for n in news:
        offsets.append(offsets[-1] + n)
    T, W = offsets[-1] + pad, Hq + 2 * Hk
    buf = (torch.randn(T * W * D + 16, generator=g, device="cuda") * 1.5).to(dtype)
    q = buf[q_shift: q_shift + T * W * D].view(T, W, D)[:, :Hq]
    return {"q": q, "codes": codes, "exps": exps, "table": i32(table), "seq": i32(lens), "offsets": i32(offsets)}, lens, offsets


def attend(c, **kw):
    return api.paged_attention_i8(c["q"], *c["codes"], *c["exps"], c["table"], c["seq"], c["offsets"], lse=True, **kw)


def takes_wide(c, max_new):
    """Whether the call goes to the kernel of many rows."""
    G, T, B = c["q"].shape[1] // c["codes"][0].shape[2], c["q"].shape[0], len(c["seq"])
    limit = 31 if c["q"].shape[2] <= 128 else 32
    return G * T > limit * B and (max_new <= 0 or G * max_new > limit)


def check(c, lens, offsets, causal=True, window=0, softcap=0.0, scale=None, max_new=0):
    out, lse, ws = attend(c, causal=causal, window=window, softcap=softcap, scale=scale, max_new=max_new)
    assert status(ws) == 0
    ro, rl, to, tl = R.attention(c["q"], c["codes"], c["exps"], c["table"], lens, offsets,
                                 c["q"].shape[2] ** -0.5 if scale is None else scale, causal, window, softcap, takes_wide(c, max_new))
    dead = rl == -math.inf
    assert torch.equal(lse == -math.inf, dead) and not out[dead].any()
    err = (out.double() - ro).abs()
    assert bool((err <= to).all()), f"out: {float((err - to).max())} past the bound, worst {float(err.max())}"
    el = (lse.double() - rl).abs()[~dead]
    assert bool((el <= tl[~dead]).all()), f"lse: worst {float(el.max())}"
    return out, lse


DTYPES = [torch.bfloat16, torch.float16]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("Hq,Hk,D,page,block", [(4, 4, 64, 16, 16), (8, 1, 128, 16, 4), (8, 2, 256, 32, 32), (5, 1, 80, 1, 1), (14, 2, 96, 64, 1),
                                                (16, 1, 16, 16, 8), (20, 1, 192, 128, 128), (7, 1, 240, 4, 2), (32, 8, 128, 16, 16),
                                                (48, 4, 64, 16, 4), (24, 8, 48, 32, 16), (60, 4, 96, 16, 1), (36, 6, 32, 16, 16)])
def test_decoding_heads_and_pages(dtype, Hq, Hk, D, page, block):
    """One token a request; contexts of one token, of a page, of its edges, of many slices; orders of both layouts."""
    lens = [1, page, page + 1, max(page - 1, 1), 2 * page + 3, 33, 257, 1000, 31, 64]
    for heads_first in (False, True):
        c, lens, offsets = make_case(lens, [1] * len(lens), Hq, Hk, D, page, block, dtype, Hq + D, heads_first=heads_first)
        check(c, lens, offsets)
    c["offsets"] = None
    out, lse, _ = attend(c)
    c["offsets"] = i32(offsets)
    assert torch.equal(out, attend(c)[0])


@pytest.mark.parametrize("D", [16, 48, 80, 96, 112, 144, 176, 192, 208])
@pytest.mark.parametrize("G", [5, 12, 40])
def test_heads_that_do_not_fill_their_rows(D, G):
    """Every kernel, with one kv head and with groups of them; parts of a request in several blocks."""
    for Hk, lens in ((3, [1, 17, 130, 700, 40]), (2, [5000]), (4, [63, 64, 65])):
        c, lens, offsets = make_case(lens, [1] * len(lens), G * Hk, Hk, D, 32, 8, torch.bfloat16, D + G)
        check(c, lens, offsets)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("causal,window,softcap,scale", [(True, 0, 0.0, None), (False, 0, 0.0, None), (True, 1, 0.0, None), (True, 20, 0.0, 0.3),
                                                         (False, 100, 0.0, None), (True, 0, 30.0, None), (True, 50, 2.0, None),
                                                         (True, 0, 0.0, -0.05), (True, 0, 1e4, None)])
@pytest.mark.parametrize("G,D,max_new", [(4, 128, 4), (4, 64, 0), (16, 128, 0), (8, 256, 0), (3, 128, 0), (12, 256, 3), (1, 64, 0)])
def test_masks(dtype, causal, window, softcap, scale, G, D, max_new):
    """Several new tokens a request, at both kernels' row counts; requests without new tokens, padding."""
    lens, news = [300, 5, 64, 129, 17, 700, 40], [9, 5, 1, 16, 17, 0, 12]
    if max_new:
        news = [min(n, max_new) for n in news]
    c, lens, offsets = make_case(lens, news, 2 * G, 2, D, 32, 8, dtype, 7, pad=3)
    out, lse = check(c, lens, offsets, causal, window, softcap, scale, max_new)
    assert not out[offsets[-1]:].any() and bool((lse[offsets[-1]:] == -math.inf).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("G,Hk,max_new", [(4, 1, 1), (5, 4, 2), (32, 1, 8)])
def test_long_contexts_split_over_blocks(dtype, G, Hk, max_new):
    for D in (64, 128, 256):
        n = max_new
        c, lens, offsets = make_case([20000, 7000, 1], [n, n, 1], G * Hk, Hk, D, 64, 16, dtype, D)
        check(c, lens, offsets, max_new=max_new)
        check(c, lens, offsets, max_new=max_new, window=5000)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("max_new", [1, 17])
def test_scales_over_the_whole_range(dtype, max_new):
    """Blocks whose values differ by up to 2^30 (fp16: 2^20) and blocks of zeros with the smallest scale there is, a scale
    for every token; keys of one scale, so that every value has a weight that counts."""
    lo, hi = (100, 131) if dtype == torch.bfloat16 else (104, 125)
    G = 4 if max_new == 1 else 8
    n = min(max_new, 9)
    c, lens, offsets = make_case([500, 333, 40], [n, n, n], G, 1, 128, 16, 1, dtype, 3, lo=lo, hi=hi)
    c["exps"][0].fill_(121)
    g = torch.Generator(device="cuda").manual_seed(max_new)
    dead = torch.rand(c["exps"][1].shape, generator=g, device="cuda") < 0.3
    c["exps"][1][dead] = 0
    page = c["codes"][1].view(-1, 1, 16, 128)
    page[dead.view(-1, 16)[:, None].expand(-1, 1, -1)] = 0
    check(c, lens, offsets, max_new=max_new)
    check(c, lens, offsets, max_new=max_new, scale=2.0)  # a few keys take all


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [3, 16, 40])
def test_every_code_at_every_scale_is_read_exactly(dtype, D, G):
    """Queries of zeros over one key a request: the weight is 1, and the output the value, bit for bit."""
    every = torch.arange(-127, 128, device="cuda")
    lo, hi = (-126, 121) if dtype == torch.bfloat16 else (-24, 9)
    scales = sorted({lo, lo + 1, -1, 0, 1, hi - 1, hi, 5, -13})
    per = -(-255 // D)
    rows = torch.cat([every, every[:per * D - 255]]).view(per, D).to(torch.int8)
    codes = rows.repeat(len(scales), 1)[:, None, None].contiguous()  # [pages of one token, 1, 1, D]
    exps = torch.tensor([e + 127 for e in scales for _ in range(per)], dtype=torch.uint8, device="cuda")[:, None, None].contiguous()
    B = per * len(scales)
    c = {"q": torch.zeros((B, G, D), dtype=dtype, device="cuda"), "codes": [codes, codes], "exps": [exps, exps],
         "table": i32([[b] for b in range(B)]), "seq": i32([1] * B), "offsets": i32(list(range(B + 1)))}
    out, lse, ws = attend(c)
    assert status(ws) == 0 and not lse.any()
    want = R.values(codes, exps, dtype)[:, 0]  # [B, 1, D]
    assert torch.equal(out.double(), want.expand(B, G, D))


@pytest.mark.parametrize("G,max_new", [(4, 1), (1, 3), (8, 3)])
def test_values_up_to_the_type_s_largest(G, max_new):
    """Sums of such values are past fp32's range, averages are not: short contexts, and long ones split over blocks."""
    for lens in ([3000, 40], [60000], [7] * 50):
        c, lens, offsets = make_case(lens, [min(max_new, n) for n in lens], G, 1, 128, 16, 4, torch.bfloat16, 11 + G)
        c["exps"][0].fill_(121)
        g = torch.Generator(device="cuda").manual_seed(G)
        c["exps"][1].copy_(torch.randint(240, 249, c["exps"][1].shape, generator=g, device="cuda").to(torch.uint8))
        c["codes"][1][..., :8] = 127  # an average as large as the values
        c["codes"][1][..., 8:16] = -127
        out, _ = check(c, lens, offsets, max_new=max_new)
        assert bool(out.isfinite().all())


def test_one_key_far_above_with_a_small_value():
    """A dominating key whose values are 2^40 below the others' (as an attention sink's): its row keeps its bits."""
    c, lens, offsets = make_case([100], [1], 2, 1, 64, 16, 1, torch.bfloat16, 5)
    c["exps"][0].fill_(121)
    c["exps"][1].fill_(125)
    page = int(c["table"][0, 2])
    c["codes"][0][page, 3] = torch.where(c["q"][0, 0] >= 0, 127, -127).to(torch.int8)
    c["exps"][1][page, 0, 3] = 85
    for scale in (0.05, 0.5, 5.0):
        check(c, lens, offsets, scale=scale)


@pytest.mark.parametrize("max_new", [1, 17])
@pytest.mark.parametrize("dtype", DTYPES)
def test_magnitudes_of_keys_and_queries(dtype, max_new):
    """Keys of large and small scales under queries and a scale that bring the scores back; a scale past 2^+-32, beside which
    the products leave fp32, is refused."""
    G = 4 if max_new == 1 else 32
    lo, hi = R.RANGE[dtype]
    for e, s in ((hi - 1, 2.0 ** -(hi + 4)), (lo + 1, 2.0 ** min(-lo - 9, 110)), (0, 2.0 ** -8), (min(hi - 1, 25), 2.0 ** -32),
                 (max(lo + 1, -41), 2.0 ** 32)):
        c, lens, offsets = make_case([90, 41], [3, 1], G, 1, 64, 16, 8, dtype, 8)
        g = torch.Generator(device="cuda").manual_seed(4)
        c["exps"][0].copy_(torch.randint(e - 1, e + 2, c["exps"][0].shape, generator=g, device="cuda") + 127)
        if 2.0 ** -32 <= s <= 2.0 ** 32:
            check(c, lens, offsets, scale=s, max_new=max_new)
        else:
            with pytest.raises(binding.DsparkError, match="unsupported"):
                attend(c, scale=s, max_new=max_new)
    for std in (2.0 ** -12, 2.0 ** 12):
        c["q"] = (c["q"].float() * std).to(dtype)
        c["exps"][0].fill_(121)
        check(c, lens, offsets, scale=0.1 / std, max_new=max_new)


@pytest.mark.parametrize("G,max_new", [(4, 1), (5, 3), (32, 4)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_what_is_hidden_does_not_touch_a_row(dtype, G, max_new):
    """Keys and values behind a row's last one, before its window, behind the request's end and in other pages, set to the
    largest there are with every exponent's byte: not a bit changes."""
    n = max_new
    c, lens, offsets = make_case([70, 45], [n, 1], G, 1, 128, 16, 4, dtype, 6)
    ref, ref_lse, _ = attend(c, max_new=max_new)
    win, win_lse, _ = attend(c, max_new=max_new, window=10)
    page = 16
    seen = {(int(c["table"][j, l // page]), l % page) for j, x in enumerate(lens) for l in range(x)}
    for byte in (255, 0, 254, 1):
        d = {**c, "codes": [x.clone() for x in c["codes"]], "exps": [x.clone() for x in c["exps"]]}
        for p in range(d["codes"][0].shape[0]):
            for i in range(page):
                if (p, i) not in seen:
                    for x in d["codes"]:
                        x[p, i] = 127 if byte > 1 else -128
            for b in range(page // 4):
                if not any((p, i) in seen for i in range(4 * b, 4 * b + 4)):
                    for x in d["exps"]:
                        x[p, :, b] = byte
        out, lse, ws = attend(d, max_new=max_new)
        assert status(ws) == 0 and torch.equal(out, ref) and torch.equal(lse, ref_lse)
        # every key before the windows: the first token's starts at 70 - n - 9
        for l in range((70 - n - 9) // 4 * 4):
            for x in d["codes"]:
                x[int(c["table"][0, l // page]), l % page] = 127
            for x in d["exps"]:
                x[int(c["table"][0, l // page]), :, l % page // 4] = byte
        out, lse, ws = attend(d, max_new=max_new, window=10)
        assert status(ws) == 0 and torch.equal(out, win) and torch.equal(lse, win_lse)
    if n > 1:  # the last token's key and value, which the others of its request do not see (its block is its own)
        c, lens, offsets = make_case([69, 45], [n, 1], G, 1, 128, 16, 4, dtype, 6)
        ref, ref_lse, _ = attend(c, max_new=max_new)
        p = int(c["table"][0, 68 // page])
        for x, y in zip(c["codes"], c["exps"]):
            x[p, 68 % page], y[p, :, 68 % page // 4] = 127, 254
        out, lse, _ = attend(c, max_new=max_new)
        others = [t for t in range(n + 1) if t != n - 1]
        assert torch.equal(out[others], ref[others]) and torch.equal(lse[others], ref_lse[others])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,block", [(64, 8), (128, 16), (256, 1)])
def test_the_same_as_attention_over_what_is_read_back(dtype, D, block):
    """The framework's own attention over the 16-bit copy of the cache: both within their bounds of the same numbers."""
    c, lens, offsets = make_case([400, 77, 1000], [4, 1, 3], 8, 2, D, 16, block, dtype, D)
    P = c["codes"][0].shape[0]
    k, v = api.cache_read_i8(*c["codes"], *c["exps"], torch.arange(P * 16, device="cuda"), dtype)
    out, lse = check(c, lens, offsets, max_new=4)
    ref, ref_lse, _ = api.paged_attention(c["q"], k.view(P, 16, 2, D), v.view(P, 16, 2, D), c["table"], c["seq"], c["offsets"],
                                          lse=True, max_new=4)
    _, _, tol, tol_lse = R.attention(c["q"], c["codes"], c["exps"], c["table"], lens, offsets, D ** -0.5, True, 0, 0.0, True)
    assert bool(((out.double() - ref.double()).abs() <= 2 * tol).all())
    assert bool(((lse.double() - ref_lse.double()).abs() <= 2 * tol_lse).all())


@pytest.mark.parametrize("max_new", [1, 17])
def test_pages_before_the_window_may_be_gone_and_bad_tables_are_reported(max_new):
    Hq = 4 if max_new == 1 else 64
    c, lens, offsets = make_case([400, 130], [3, 2], Hq, 1, 128, 16, 16, torch.bfloat16, 5)
    ref, _, ws = attend(c, window=70, max_new=max_new)
    c["table"][0, : (400 - 3 - 70 + 1) // 16] = -1
    c["table"][1, : (130 - 2 - 70 + 1) // 16] = 1 << 30
    out, _, ws = attend(c, window=70, max_new=max_new)
    assert status(ws) == 0 and torch.equal(out, ref)
    c, lens, offsets = make_case([40, 50], [1, 1], Hq, 1, 64, 16, 2, torch.bfloat16, 9)
    ref, _, _ = attend(c, max_new=max_new)
    for what in ("page", "negative", "long", "offsets"):
        d = {**c, "table": c["table"].clone(), "seq": c["seq"].clone(), "offsets": c["offsets"].clone()}
        if what == "page":
            d["table"][0, 1] = 1 << 20
        if what == "negative":
            d["table"][0, 1] = -1
        if what == "long":
            d["seq"][0] = 1 << 30
        if what == "offsets":
            d["offsets"][0] = -5
        error = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, _, ws = attend(d, max_new=max_new, error=error)
        assert status(ws) == 8 and int(error) == 8, what
        assert torch.equal(out[1], ref[1])


@pytest.mark.parametrize("dtype", DTYPES)
def test_queries_at_any_element(dtype):
    c, lens, offsets = make_case([100, 40], [7, 2], 32, 1, 64, 16, 16, dtype, 3, q_shift=5)
    check(c, lens, offsets)
    check(c, lens, offsets, max_new=7)
    c, lens, offsets = make_case([100, 40], [1, 2], 6, 2, 80, 16, 16, dtype, 3, q_shift=3)
    check(c, lens, offsets)


@pytest.mark.parametrize("G,max_new", [(8, 1), (6, 3), (40, 2)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_a_query_that_is_not_finite_stays_in_its_row(dtype, G, max_new):
    n = max_new
    c, lens, offsets = make_case([300, 45], [n, 1], G, 1, 128, 16, 4, dtype, 6)
    ref, ref_lse, _ = attend(c, max_new=max_new)
    for bad in (math.nan, math.inf, -math.inf):
        c["q"][0, 2, 5] = bad
        out, lse, ws = attend(c, max_new=max_new)
        others = torch.ones(ref_lse.shape, dtype=torch.bool, device="cuda")
        others[0, 2] = False
        assert status(ws) == 0 and not torch.isfinite(out[0, 2].float()).all()
        assert torch.equal(out[others], ref[others]) and torch.equal(lse[others], ref_lse[others])


@pytest.mark.parametrize("G,max_new", [(8, 1), (12, 1), (40, 1)])
def test_pools_past_32_bits(G, max_new):
    """Pages whose offsets in bytes do not fit 32 bits (pools of 4.4 GB): the same bits as from a small pool."""
    page, D = 128, 256
    P = (1 << 32) // (page * D) + 3000
    c, lens, offsets = make_case([700, 90], [1, 1], G, 1, D, page, 64, torch.bfloat16, 4)
    ref, ref_lse, _ = attend(c, max_new=max_new)
    small = c["codes"][0].shape[0]
    big = [torch.empty((P, page, 1, D), dtype=torch.int8, device="cuda") for _ in range(2)]
    exps = [torch.zeros((P, 1, 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
    for x, y in zip((*big, *exps), (*c["codes"], *c["exps"])):
        x[P - small:] = y
    table = torch.where(c["table"] >= 0, c["table"] + (P - small), c["table"])
    out, lse, ws = attend({**c, "codes": big, "exps": exps, "table": table}, max_new=max_new)
    assert status(ws) == 0 and torch.equal(out, ref) and torch.equal(lse, ref_lse)


@pytest.mark.parametrize("G,max_new", [(4, 1), (5, 4), (32, 5)])
def test_other_stream_and_graph(G, max_new):
    """On a side stream, and replayed from a graph after the lengths, the codes and the scales changed."""
    c, lens, offsets = make_case([700, 200, 64], [1, 5 if max_new > 1 else 1, 1], G, 1, 128, 16, 8, torch.bfloat16, 12)
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
    out, graph = torch.zeros_like(ref), torch.cuda.CUDAGraph()
    ws = torch.empty(api.b.dspark_paged_attention_workspace_size(api._attention_sizes(c["q"], c["codes"][0], c["seq"], max_new)),
                     dtype=torch.uint8, device="cuda")
    with torch.cuda.graph(graph):
        attend(c, out=out, ws=ws, max_new=max_new)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    c["seq"].copy_(i32([333, 150, 2]))
    c["codes"][0].neg_(), c["exps"][1].add_(1)
    graph.replay()
    torch.cuda.synchronize()
    want, _, _ = attend(c, max_new=max_new)
    assert torch.equal(out, want) and not torch.equal(out, ref)


@pytest.mark.parametrize("max_new", [1, 17])
def test_no_tokens_at_all(max_new):
    c, lens, offsets = make_case([40, 50], [0, 0], 64, 1, 64, 16, 16, torch.bfloat16, 9, pad=2)
    out, lse, ws = attend(c, max_new=max_new)
    assert not out.any() and bool((lse == -math.inf).all()) and status(ws) == 0
    c["q"] = c["q"][:0]
    out, lse, ws = attend(c, max_new=max_new)
    assert out.numel() == 0 and status(ws) == 0
