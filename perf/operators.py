"""Cases of the paged-cache operators: the step between the verify schedule and the verification.

  plan    block tables, slots and positions of a step's new tokens, from the requests' lengths
  commit  lengths after the verification, pages past them given back
  append  the new keys and values written into their pages
  attend  attention of the new tokens over the paged cache

`run` computes the plain form with elementary torch operations, or, where `own` is true, calls the
framework's operators.  Block lengths, batches and the verify budget are those of this repository's
workloads (gamma 4, 8 and 16; 1, 32, 128 and 512 requests; 2048 verified tokens)."""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases
def _attend(name, B, new, length, hq, hk, d, page, dtype="bf16", cache=None, causal=True, window=0, softcap=0.0,
            lse=False):
    return {"name": name, "op": "attend", "B": B, "new": new, "len": length, "hq": hq, "hk": hk, "d": d, "page": page,
            "dtype": dtype, "cache": cache or dtype, "causal": causal, "window": window, "softcap": softcap, "lse": lse}


def _append(name, T, pad, hk, d, page, dtype="bf16", cache=None):
    return {"name": name, "op": "append", "T": T, "pad": pad, "hk": hk, "d": d, "page": page, "dtype": dtype,
            "cache": cache or dtype}


def listed():
    return [
        # a verify step of 32 requests, gamma 8: each feeds its anchor and 1..8 drafted tokens
        {"name": "plan_b32_verify", "op": "plan", "B": 32, "new": 8, "len": 4096, "page": 16, "pad": 17},
        # prompts admitted together: up to 8192 new tokens each, some behind a cached prefix
        {"name": "plan_b48_prompts", "op": "plan", "B": 48, "new": 8192, "len": 1000, "page": 32, "pad": 0},
        # after the verification of 32 requests: few pages come back
        {"name": "commit_b32", "op": "commit", "B": 32, "new": 8, "len": 4096, "page": 16, "done": 0.0},
        # after the verification of 512 requests of which some are finished and give all their pages back
        {"name": "commit_b512_done", "op": "commit", "B": 512, "new": 16, "len": 8000, "page": 16, "done": 0.1},
        # the keys and values of one decoding step of 32 requests, with padding to a fixed token count
        _append("append_b32", 32 * 9 - 41, 41, 8, 128, 16),
        # a prompt chunk into an 8-bit cache
        _append("append_prompt_e4m3", 16384 + 77, 0, 8, 128, 64, cache="e4m3"),
        # one user, one token, a short context: latency
        _attend("attend_b1_short", 1, 1, 1024, 32, 8, 128, 16),
        # decoding, one token a request, ragged contexts
        _attend("attend_b32_decode", 32, 1, 8192, 32, 8, 128, 16, lse=True),
        # decoding over an 8-bit cache
        _attend("attend_b128_e4m3", 128, 1, 8000, 64, 8, 128, 64, cache="e4m3"),
        # the scheduled verify of 512 requests: 1 + L tokens a request, 2048 drafted tokens in all
        _attend("attend_b512_verify", 512, 16, 4096, 32, 4, 128, 32),
        # a draft block of 16 positions that see the context and each other
        _attend("attend_b32_block", 32, 15, 4100, 32, 8, 64, 32, dtype="fp16", causal=False),
        # few requests with long contexts, wide heads, softcapped logits
        _attend("attend_b3_long_softcap", 3, 4, 200000, 16, 2, 256, 128, softcap=30.0, lse=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


def draw(rng):
    kind = rng.random()
    page = rng.choice([16, 16, 32, 64, 128])
    if kind < 0.14:
        if rng.random() < 0.6:
            return {"op": "plan", "B": _log_int(rng, 1, 2000), "new": rng.choice([1, 4, 8, 16]), "len": _log_int(rng, 16, 8192),
                    "page": page, "pad": rng.randrange(64)}
        B = _log_int(rng, 1, 200)
        return {"op": "plan", "B": B, "new": _log_int(rng, 64, 8192 * 48 // max(B, 48)), "len": _log_int(rng, 16, 4096),
                "page": page, "pad": rng.randrange(64)}
    if kind < 0.24:
        return {"op": "commit", "B": _log_int(rng, 1, 512), "new": rng.choice([4, 8, 16]), "len": _log_int(rng, 64, 8000),
                "page": page, "done": rng.choice([0.0, 0.05, 0.1, 0.5])}
    hk = rng.choice([1, 2, 4, 8, 16])
    d = rng.choice([64, 128, 128, 128, 256, 80, 96, 192])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    cache = rng.choice([dtype, dtype, "e4m3"])
    if kind < 0.38:
        return {"op": "append", "T": _log_int(rng, 1, max(1, 16000 * 1024 // (hk * d))), "pad": rng.randrange(50), "hk": hk,
                "d": d, "page": page, "dtype": dtype, "cache": cache}
    if rng.random() < 0.85:  # many requests, or few, below the largest case's cache
        B = _log_int(rng, 1, 512)
        length = _log_int(rng, 32, min(65536, max(64, 3 * 2 ** 29 // (B * hk * d * 2))))
    else:  # few requests, long contexts
        B = rng.randrange(1, 5)
        length = _log_int(rng, 20000, min(260000, 3 * 2 ** 29 // (B * hk * d * 2)))
    group = rng.choice([1, 2, 4, 4, 5, 7, 8, 8, 16])
    new = rng.choice([1, 1, 1, 4, 8, 16])
    c = {"op": "attend", "B": B, "new": new, "len": length, "hq": hk * group, "hk": hk, "d": d, "page": page,
         "dtype": dtype, "cache": cache, "causal": rng.random() < 0.75,
         "window": rng.choice([0, 0, 0, 0, 128, 1000, 4096]), "softcap": rng.choice([0.0, 0.0, 0.0, 30.0, 50.0]),
         "lse": rng.random() < 0.5}
    for less in ({"new": 1}, {"hq": hk}):  # keeps the arithmetic below the largest listed case's
        if 4.0 * B * (new + 1) * c["hq"] * length * d > 7.5e10:
            c |= less
    return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)


def _lengths(c):
    """[(cache_len, new_len)] of the requests, which the case alone decides: contexts spread evenly from an
    eighth of the longest up, one request that has just begun; verified tokens 1..gamma, few of them many
    (a mean of 4 where gamma is 16: a budget of 2048 over 512 requests), or one each, or whole prompts."""
    B, new, length = c["B"], c["new"], c["len"]
    rng = random.Random("%d %d %d" % (B, new, length))
    pairs = []
    for j in range(B):
        n = new
        if 1 < new <= 16 and j:
            n = max(1, min(new, 1 + int(-2.6 * math.log1p(-rng.random() * (1 - math.exp(-new / 3.0))))))
        elif new > 16:
            n = rng.randint(1, new)
        pairs.append((0 if B > 2 and j == B // 2 else rng.randint(max(1, length // 8), length), n))
    return pairs


def _shuffled(c, g):
    """cache_len [B] and new_len [B]: the requests in an order of the seed's."""
    pairs = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")
    pairs = pairs[torch.randperm(c["B"], generator=g, device="cuda")]
    return pairs[:, 0].contiguous(), pairs[:, 1].contiguous()


def _new_tokens(c, n):
    """Tokens a request feeds when n of its drafted tokens are verified: the anchor too; all of a draft block."""
    if c["new"] == 1 or c["new"] > 16:
        return n
    return n + 1 if c.get("causal", True) else c["new"] + 1


def _blocks(length, page):
    return (length + page - 1) // page


def _tables(g, blocks, spare):
    """A block table whose pages are scattered over the pool, -1 past each request's pages, and the pool's
    other pages as the free stack."""
    B = blocks.numel()
    used = int(blocks.sum())
    P = used + spare
    perm = torch.randperm(P, generator=g, device="cuda").int()
    first = torch.cumsum(blocks, 0) - blocks
    width = int(blocks.max()) if B else 0
    return P, perm, first, width


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    op = c["op"]
    if op in ("plan", "commit"):
        page = c["page"]
        cache_len, new_len = _shuffled(c, g)
        extra = 1 if 1 < c["new"] <= 16 else 0
        have = _blocks(cache_len, page) if op == "plan" else _blocks(cache_len + new_len + extra, page)
        after = _blocks(cache_len + new_len + extra, page)
        P, perm, first, _ = _tables(g, have, int((after - have).sum()) + 100)
        width = int(after.max()) + 1
        cols = torch.arange(width, device="cuda")
        table = torch.where(cols < have[:, None], perm[(first[:, None] + cols).clamp(max=P - 1)], -1).int().contiguous()
        n_free = torch.tensor([P - int(have.sum())], dtype=torch.int32, device="cuda")
        free = torch.full((P,), -1, dtype=torch.int32, device="cuda")
        free[: int(n_free)] = perm[int(have.sum()):]
        i32 = dict(dtype=torch.int32, device="cuda")
        s = {"case": c, "cache_len": cache_len, "table": table, "n_blocks": have.int().contiguous(), "free": free,
             "n_free": n_free, "P": P, "extra": extra, "ws": torch.zeros(256, dtype=torch.uint8, device="cuda")}
        if op == "plan":
            T = int((new_len + extra).sum()) + c["pad"]
            s |= {"new_len": new_len, "T": T,
                  "out": (torch.empty(c["B"], **i32), torch.empty(c["B"] + 1, **i32),
                          torch.empty(T, dtype=torch.int64, device="cuda"), torch.empty(T, **i32),
                          torch.empty(c["B"], **i32), torch.empty(1, **i32))}
        else:
            u = torch.rand((c["B"],), generator=g, device="cuda")
            s |= {"accepted": (new_len * u).round().int(),
                  "done": (torch.rand((c["B"],), generator=g, device="cuda") < c["done"]).to(torch.uint8),
                  "out": (torch.empty(c["B"], **i32), torch.empty(c["B"], **i32), torch.empty(1, **i32))}
        return s

    dtype, cache, hk, d, page = DTYPES[c["dtype"]], DTYPES[c["cache"]], c["hk"], c["d"], c["page"]
    scales = [None, None]
    if c["cache"] == "e4m3":  # a scale a head, as a calibration gives them
        scales = [0.01 + 0.02 * torch.rand((hk,), generator=g, device="cuda") for _ in range(2)]

    def pool(P):
        x = torch.randn((P, page, hk, d), generator=g, device="cuda", dtype=torch.float16 if c["cache"] == "e4m3" else dtype)
        return (x * 60).to(cache) if c["cache"] == "e4m3" else x

    if op == "append":
        T, pad = c["T"], c["pad"]
        P = _blocks(T, page) + 5
        # the tokens of a step, consecutive in their pages, the pages scattered
        perm = torch.randperm(P, generator=g, device="cuda")
        t = torch.arange(T, device="cuda") + 3
        slots = torch.cat([perm[t // page] * page + t % page, torch.full((pad,), -1, device="cuda", dtype=torch.int64)])
        qkv = torch.randn((T + pad, 3 * hk, d), generator=g, device="cuda", dtype=dtype)
        return {"case": c, "k": qkv[:, hk:2 * hk], "v": qkv[:, 2 * hk:], "k_pages": pool(P), "v_pages": pool(P),
                "slots": slots.contiguous(), "k_scale": scales[0], "v_scale": scales[1]}

    cache_len, new_len = _shuffled(c, g)
    n = _new_tokens(c, new_len) + torch.zeros_like(new_len)
    seq_len = (cache_len + n).int().contiguous()
    offsets = torch.zeros(c["B"] + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(n, 0)
    blocks = _blocks(seq_len, page)
    P, perm, first, width = _tables(g, blocks, 7)
    cols = torch.arange(width, device="cuda")
    table = torch.where(cols < blocks[:, None], perm[(first[:, None] + cols).clamp(max=P - 1)], -1).int().contiguous()
    T = int(offsets[-1])
    qkv = torch.randn((T, c["hq"] + 2 * hk, d), generator=g, device="cuda", dtype=dtype) * 1.5
    return {"case": c, "q": qkv[:, : c["hq"]], "k_pages": pool(P), "v_pages": pool(P), "table": table, "seq_len": seq_len,
            "offsets": None if c["new"] == 1 else offsets, "k_scale": scales[0], "v_scale": scales[1],
            "max_new": int(n.max()), "max_len": int(seq_len.max()), "scale": 1.0 / math.sqrt(d),
            "out": torch.empty((T, c["hq"], d), dtype=dtype, device="cuda"),
            "lse": torch.empty((T, c["hq"]), device="cuda") if c["lse"] else None}


# ------------------------------------------------------------------ the plain forms
def _plain_plan(s):
    c = s["case"]
    B, page, T = c["B"], c["page"], s["T"]
    n = s["new_len"] + s["extra"]
    seq = s["cache_len"] + n
    offsets = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), torch.cumsum(n, 0).int()])
    need = (_blocks(seq, page) - s["n_blocks"]).clamp(min=0)
    before = torch.cumsum(need, 0) - need
    n_blocks = s["n_blocks"] + need
    cols = torch.arange(s["table"].shape[1], device="cuda")
    fresh = (cols >= s["n_blocks"][:, None]) & (cols < n_blocks[:, None])
    k = before[:, None] + cols - s["n_blocks"][:, None]
    page_of = s["free"][(s["n_free"].long() - 1 - k).clamp(0, s["P"] - 1)]
    table = torch.where(fresh, page_of, s["table"])
    t = torch.arange(T, device="cuda")
    j = torch.searchsorted(offsets[1:].contiguous(), t, right=True).clamp(max=B - 1)
    pos = s["cache_len"][j] + t - offsets[j]
    live = t < offsets[B]
    block = table[j, (pos // page).clamp(0, table.shape[1] - 1)].long()
    slots = torch.where(live, block * page + pos % page, -1)
    return {"seq_len": seq, "offsets": offsets, "slots": slots, "positions": torch.where(live, pos, -1).int(),
            "n_blocks": n_blocks.int(), "n_free": (s["n_free"] - need.sum()).int(), "table": table}


def _plain_commit(s):
    c = s["case"]
    length = torch.where(s["done"] != 0, 0, s["cache_len"] + s["accepted"] + s["extra"])
    keep = torch.minimum(_blocks(length, c["page"]), s["n_blocks"])
    back = s["n_blocks"] - keep
    before = torch.cumsum(back, 0) - back
    cols = torch.arange(s["table"].shape[1], device="cuda")
    out = (cols >= keep[:, None]) & (cols < s["n_blocks"][:, None])
    at = s["n_free"].long() + before[:, None] + cols - keep[:, None]
    at = torch.where(out, at, s["P"])  # what stays goes to a place past the stack's end
    free = torch.cat([s["free"], s["free"][:1]]).scatter(0, at.reshape(-1), s["table"].reshape(-1))[: s["P"]]
    return {"cache_len": length.int(), "n_blocks": keep.int(), "n_free": (s["n_free"] + back.sum()).int(), "free": free}


def _plain_append(s):
    live = (s["slots"] >= 0)[:, None, None]
    at = torch.where(s["slots"] >= 0, s["slots"], s["slots"][0])  # padding writes the first token once more

    def into(x, pages, scale):
        y = x.float()
        if scale is not None:
            y = (y / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        y = y.to(pages.dtype)
        bits = torch.uint8 if pages.dtype == torch.float8_e4m3fn else torch.int16
        y = y.view(bits)
        pages.view(bits).view(-1, *x.shape[1:]).index_copy_(0, at, torch.where(live, y, y[:1]))
        return pages

    return {"k_pages": into(s["k"], s["k_pages"], s["k_scale"]), "v_pages": into(s["v"], s["v_pages"], s["v_scale"])}


def _plain_attend(s):
    c = s["case"]
    B, hk, d, page = c["B"], c["hk"], c["d"], c["page"]
    group = c["hq"] // hk
    q, seq = s["q"].float(), s["seq_len"].long()
    offsets = s["offsets"] if s["offsets"] is not None else torch.arange(B + 1, device="cuda")
    N, L = s["max_new"], s["max_len"]
    n = (offsets[1:] - offsets[:-1]).long()
    i, l = torch.arange(N, device="cuda"), torch.arange(L, device="cuda")
    token = (offsets[:-1, None] + i).clamp(max=q.shape[0] - 1)  # [B, N]
    qb = q[token].view(B, N, hk, group, d).permute(0, 2, 1, 3, 4).reshape(B, hk, N * group, d)
    blocks = s["table"][:, l // page].clamp(min=0).long()  # [B, L]

    def rows(pages, scale):
        x = pages[blocks, l % page].float()  # [B, L, hk, d]
        return (x if scale is None else x * scale[:, None]).permute(0, 2, 1, 3)

    z = torch.matmul(qb, rows(s["k_pages"], s["k_scale"]).transpose(2, 3)) * s["scale"]
    if c["softcap"]:
        z = c["softcap"] * torch.tanh(z / c["softcap"])
    p_i = (seq - n)[:, None, None] + i[:, None]  # [B, N, 1]
    see = (l < seq[:, None, None]).expand(B, N, L)
    if c["causal"]:
        see = see & (l <= p_i)
    if c["window"]:
        see = see & (l > p_i - c["window"])
    see = see[:, None, :, None, :].expand(B, hk, N, group, L).reshape(B, hk, N * group, L)
    z = torch.where(see, z, -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = torch.exp(z - m)
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, rows(s["v_pages"], s["v_scale"])) / torch.where(total == 0, 1.0, total)
    lse = (m + torch.log(total))[..., 0]
    t = torch.arange(q.shape[0], device="cuda")
    j = torch.searchsorted(offsets[1:].contiguous(), t, right=True)
    k = t - offsets[j]
    o = o.view(B, hk, N, group, d)[j, :, k].reshape(q.shape[0], c["hq"], d)
    out = {"out": o.to(s["q"].dtype)}
    if c["lse"]:
        out["lse"] = lse.view(B, hk, N, group)[j, :, k].reshape(q.shape[0], c["hq"])
    return out


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    if not own:
        return {"plan": _plain_plan, "commit": _plain_commit, "append": _plain_append, "attend": _plain_attend}[c["op"]](s)
    from semi_ar_draft_gb300 import api

    if c["op"] == "plan":
        seq, offsets, slots, positions, n_blocks, n_free, _ = api.cache_plan(
            s["cache_len"], s["new_len"], s["table"], s["n_blocks"], s["free"], s["n_free"], c["page"], s["T"],
            extra=s["extra"], out=s["out"], ws=s["ws"])
        return {"seq_len": seq, "offsets": offsets, "slots": slots, "positions": positions, "n_blocks": n_blocks,
                "n_free": n_free, "table": s["table"]}
    if c["op"] == "commit":
        length, n_blocks, n_free, _ = api.cache_commit(s["cache_len"], s["accepted"], s["table"], s["n_blocks"], s["free"],
                                                       s["n_free"], c["page"], extra=s["extra"], done=s["done"],
                                                       out=s["out"], ws=s["ws"])
        return {"cache_len": length, "n_blocks": n_blocks, "n_free": n_free, "free": s["free"]}
    if c["op"] == "append":
        api.cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["slots"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    out, lse, _ = api.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["seq_len"], s["offsets"],
                                      scale=s["scale"], causal=c["causal"], window=c["window"], softcap=c["softcap"],
                                      k_scale=s["k_scale"], v_scale=s["v_scale"], max_new=s["max_new"],
                                      out=s["out"], lse=s["lse"])
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] in ("plan", "commit"):
        B, page = c["B"], c["page"]
        pairs = [(old, old + _new_tokens(c, n), n) for old, n in _lengths(c)]
        if c["op"] == "plan":
            tokens = sum(seq - old for old, seq, _ in pairs)
            pages = sum(-(-seq // page) - -(-old // page) for old, seq, _ in pairs)
            return {"bytes": 4 * (3 * B + 1) + 8 * pages + 4 * B + 12 * (tokens + c["pad"]) + 4 * (3 * B + 2), "flops": 0}
        pages = sum(c["done"] * -(-seq // page) + (1 - c["done"]) * n / 2 / page for _, seq, n in pairs)
        return {"bytes": 4 * 3 * B + B + 8 * pages + 4 * (2 * B + 2), "flops": 0}
    size = 1 if c["cache"] == "e4m3" else 2
    if c["op"] == "append":
        return {"bytes": 2.0 * c["T"] * c["hk"] * c["d"] * (2 + size) + 8 * (c["T"] + c["pad"]), "flops": 0}
    rows = tokens = seen = 0  # cache rows that somebody sees, new tokens, (token, cache row) pairs
    for old, n in _lengths(c):
        n = _new_tokens(c, n)
        w = c["window"] or old + n
        rows += min(old + n, w + n - 1)
        tokens += n
        seen += sum(min((old + i + 1), w) if c["causal"] else min(old + n, w + n - 1 - i) for i in range(n))
    return {"bytes": rows * (2.0 * c["hk"] * c["d"] * size + 4.0 / c["page"])
            + tokens * c["hq"] * (4.0 * c["d"] + (4 if c["lse"] else 0)),
            "flops": 4.0 * c["hq"] * c["d"] * seen}


# ------------------------------------------------------------------ the definition in 64 bits
def _round_e4m3(x):
    """Round to nearest even on the e4m3 grid: 3 mantissa bits, smallest exponent -6, largest value 448."""
    x = x.clamp(-E4M3_MAX, E4M3_MAX)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6)
    step = torch.pow(2.0, e - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    c = case
    if c["op"] in ("plan", "commit"):
        return None  # whole numbers
    s = prepare(case, seed)
    if c["op"] == "append":
        out = {}
        for name in ("k", "v"):
            x = s[name][: c["T"]].double()
            if s[name + "_scale"] is not None:
                x = _round_e4m3(x / s[name + "_scale"].double()[:, None])
            pages = s[name + "_pages"].double()
            pages.view(-1, c["hk"], c["d"])[s["slots"][: c["T"]]] = x
            out[name + "_pages"] = pages
        return out
    hk, group, page = c["hk"], c["hq"] // c["hk"], c["page"]
    seqs = s["seq_len"].tolist()
    offs = s["offsets"].tolist() if s["offsets"] is not None else list(range(c["B"] + 1))
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for j, seq in enumerate(seqs):
        a, b = offs[j], offs[j + 1]
        n = b - a
        first = seq - n  # position of the request's first new token
        lo = max(0, first - c["window"] + 1) if c["window"] else 0
        l = torch.arange(lo, seq, device="cuda")
        pages = s["table"][j].long()[l // page]
        k, v = (s[x + "_pages"][pages, l % page].double() * (1.0 if s[x + "_scale"] is None else s[x + "_scale"].double()[:, None])
                for x in ("k", "v"))
        q = s["q"][a:b].double().view(n, hk, group, -1)
        z = torch.einsum("nhgd,lhd->nhgl", q, k) * s["scale"]
        if c["softcap"]:
            z = c["softcap"] * torch.tanh(z / c["softcap"])
        pos = torch.arange(first, seq, device="cuda")[:, None]
        hide = torch.zeros((n, l.numel()), dtype=torch.bool, device="cuda")
        if c["causal"]:
            hide |= l > pos
        if c["window"]:
            hide |= l <= pos - c["window"]
        z.masked_fill_(hide[:, None, None, :], -math.inf)
        ls = torch.logsumexp(z, -1)
        out[a:b] = torch.einsum("nhgl,lhd->nhgd", torch.exp(z - ls[..., None]), v).reshape(n, c["hq"], -1)
        lse[a:b] = ls.reshape(n, c["hq"])
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}
