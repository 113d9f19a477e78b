"""Cases of the int8 paged cache: keys and values held as 8-bit integers with a scale for each block of tokens
and kv head.

  store   a step's keys and values quantised into their pages, and the blocks that the step touched read back
          as 16-bit values (a prompt's own attention over what later steps will see; a copy for a second tier)
  read    cached tokens read back to 16 bits by their slots (a shared prefix handed to another engine)
  attend  attention of the new tokens over the int8 pages

A value is code * 2^(exponent - 127): `codes` int8 in [-127, 127], `exponent` uint8 of its block and head.  A block is
`block` adjacent tokens of a page.  Its scale is the smallest power of two that holds its largest magnitude in 127
steps; a block that already holds tokens keeps a scale that is larger, and its codes are rounded again (to nearest, ties
to even) where the scale has to grow.  A block is begun anew when its first token is written.

`run` computes the plain form with elementary torch operations, or, where `own` is true, calls the framework's
operators.  Block lengths, batches and the verify budget are those of this repository's workloads (gamma 4, 8 and
16; 1, 32, 128 and 512 requests; 2048 verified tokens)."""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
RANGE = {"bf16": (-126, 121), "fp16": (-24, 9)}  # exponents whose 127 steps are numbers of the 16-bit type


# ------------------------------------------------------------------ cases
def _store(name, B, new, length, pad, hk, d, page, block, dtype="bf16"):
    return {"name": name, "op": "store", "B": B, "new": new, "len": length, "pad": pad, "hk": hk, "d": d, "page": page,
            "block": block, "dtype": dtype}


def _read(name, T, skip, hk, d, page, block, dtype="bf16"):
    return {"name": name, "op": "read", "T": T, "skip": skip, "hk": hk, "d": d, "page": page, "block": block, "dtype": dtype}


def _attend(name, B, new, length, hq, hk, d, page, block, dtype="bf16", causal=True, window=0, softcap=0.0, lse=False):
    return {"name": name, "op": "attend", "B": B, "new": new, "len": length, "hq": hq, "hk": hk, "d": d, "page": page,
            "block": block, "dtype": dtype, "causal": causal, "window": window, "softcap": softcap, "lse": lse}


def listed():
    return [
        # the keys and values of one verify step of 32 requests, gamma 8, whose blocks are partly filled, padded to a
        # fixed token count
        _store("store_b32_step", 32, 8, 1000, 41, 8, 128, 16, 16),
        # four prompts admitted together, some behind a cached prefix
        _store("store_prompts", 4, 8192, 300, 0, 8, 128, 64, 32),
        # a prompt into a cache with a scale for every token, heads of 80
        _store("store_prompt_token", 1, 5000, 0, 0, 4, 80, 16, 1, "fp16"),
        # the last tokens of one request, a few of them skipped: latency
        _read("read_tail", 129, 3, 8, 128, 16, 16),
        # a long shared prefix, its pages scattered over the pool
        _read("read_prefix", 60000, 0, 8, 128, 16, 16),
        # one user, one token, a short context: latency
        _attend("attend_b1_short", 1, 1, 1024, 32, 8, 128, 16, 16),
        # decoding, one token a request, ragged contexts
        _attend("attend_b32_decode", 32, 1, 8192, 32, 8, 128, 16, 16, lse=True),
        # decoding of many requests, large pages and blocks
        _attend("attend_b128_decode", 128, 1, 8000, 64, 8, 128, 64, 64),
        # the scheduled verify of 512 requests: 1 + L tokens a request, 2048 drafted tokens in all
        _attend("attend_b512_verify", 512, 16, 4096, 32, 4, 128, 32, 16),
        # a draft block of 16 positions that see the context and each other, heads of 64
        _attend("attend_b32_block", 32, 15, 4100, 32, 8, 64, 32, 32, dtype="fp16", causal=False),
        # few requests with long contexts, wide heads, softcapped logits
        _attend("attend_b3_long_softcap", 3, 4, 200000, 16, 2, 256, 128, 128, softcap=30.0, lse=True),
        # a scale for every token, a sliding window, five query heads a kv head
        _attend("attend_b48_window_token", 48, 4, 6000, 20, 4, 96, 16, 1, dtype="fp16", window=1000),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


def draw(rng):
    kind = rng.random()
    page = rng.choice([16, 16, 32, 64, 128])
    block = rng.choice([x for x in (1, 2, 4, 8, 16, 16, 32, 64, 128) if x <= page])
    hk = rng.choice([1, 2, 4, 8, 16])
    d = rng.choice([64, 128, 128, 128, 256, 80, 96, 192])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    more = {"hk": hk, "d": d, "page": page, "block": block, "dtype": dtype}
    if kind < 0.25:
        most = 16000 * 1024 // (hk * d)  # tokens of a call
        if rng.random() < 0.5:
            B, new = _log_int(rng, 1, min(512, max(1, most // 17))), rng.choice([1, 4, 8, 16])
            return {"op": "store", "B": B, "new": new, "len": _log_int(rng, 16, 1000), "pad": rng.randrange(64)} | more
        B = _log_int(rng, 1, 16)
        return {"op": "store", "B": B, "new": _log_int(rng, 32, max(64, most // B)), "len": rng.choice([0, 100, 1000]),
                "pad": rng.randrange(64)} | more
    if kind < 0.4:
        return {"op": "read", "T": _log_int(rng, 1, 60000 * 1024 // (hk * d)), "skip": rng.randrange(20)} | more
    if rng.random() < 0.85:  # many requests, or few, below the largest case's cache
        B = _log_int(rng, 1, 512)
        length = _log_int(rng, 32, min(65536, max(64, 3 * 2 ** 29 // (B * hk * d * 2))))
    else:  # few requests, long contexts
        B = rng.randrange(1, 5)
        length = _log_int(rng, 20000, min(260000, 3 * 2 ** 29 // (B * hk * d * 2)))
    group = rng.choice([1, 2, 4, 4, 5, 7, 8, 8, 16])
    c = {"op": "attend", "B": B, "new": rng.choice([1, 1, 1, 4, 8, 16]), "len": length, "hq": hk * group,
         "causal": rng.random() < 0.75, "window": rng.choice([0, 0, 0, 0, 128, 1000, 4096]),
         "softcap": rng.choice([0.0, 0.0, 0.0, 30.0, 50.0]), "lse": rng.random() < 0.5} | more
    for less in ({"new": 1}, {"hq": hk}):  # keeps the arithmetic below the largest listed case's
        if 4.0 * B * (c["new"] + 1) * c["hq"] * length * d > 7.5e10:
            c |= less
    return c


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)


def _lengths(c):
    """[(cached tokens, new tokens)] of the requests, which the case alone decides: contexts spread evenly from an
    eighth of the longest up, one request that has just begun; the tokens a request feeds are its anchor and 1..gamma
    drafted ones, few of them many, or one, or a whole draft block, or a prompt."""
    B, new, length = c["B"], c["new"], c["len"]
    rng = random.Random("%d %d %d" % (B, new, length))
    pairs = []
    for j in range(B):
        n = new
        if 1 < new <= 16:
            if j:
                n = max(1, min(new, 1 + int(-2.6 * math.log1p(-rng.random() * (1 - math.exp(-new / 3.0))))))
            n = n + 1 if c.get("causal", True) else new + 1
        elif new > 16 and j:
            n = rng.randint(1, new)
        pairs.append((0 if length == 0 or (B > 2 and j == B // 2) else rng.randint(max(1, length // 8), length), n))
    return pairs


def _shuffled(c, g):
    """cached and new tokens [B]: the requests in an order of the seed's."""
    pairs = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")
    pairs = pairs[torch.randperm(c["B"], generator=g, device="cuda")]
    return pairs[:, 0].contiguous(), pairs[:, 1].contiguous()


def _blocks(length, page):
    return (length + page - 1) // page


def _pools(c, g, P):
    """Codes as a quantised normal distribution leaves them, and the scales of blocks of different magnitude (values
    of about one)."""
    hk, d, page, nb = c["hk"], c["d"], c["page"], c["page"] // c["block"]
    out = []
    for _ in range(2):
        x = torch.randn((P, page, hk, d), generator=g, device="cuda", dtype=torch.float16)
        out.append((x * 33).round_().clamp_(-127, 127).to(torch.int8))
        del x
    for _ in range(2):
        out.append(torch.randint(120, 124, (P, hk, nb), generator=g, device="cuda", dtype=torch.uint8))
    return dict(zip(("k_pages", "v_pages", "k_exp", "v_exp"), out))


def _layout(c, g):
    """Lengths, CSR offsets and a block table whose pages are scattered over the pool, -1 past each request's."""
    old, n = _shuffled(c, g)
    seq = (old + n).int().contiguous()
    offsets = torch.zeros(c["B"] + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(n, 0)
    have = _blocks(seq, c["page"])
    P = int(have.sum()) + 7
    perm = torch.randperm(P, generator=g, device="cuda").int()
    first = torch.cumsum(have, 0) - have
    cols = torch.arange(int(have.max()), device="cuda")
    table = torch.where(cols < have[:, None], perm[(first[:, None] + cols).clamp(max=P - 1)], -1).int().contiguous()
    return old, seq, offsets, table, P


def _slots_of(c, table, first, last):
    """Slots of the requests' tokens first .. last - 1, one request after the other."""
    n = (last - first).long()
    start = torch.cumsum(n, 0) - n
    j = torch.repeat_interleave(torch.arange(c["B"], device="cuda"), n)
    pos = first.long()[j] + torch.arange(j.numel(), device="cuda") - start[j]
    return table[j, pos // c["page"]].long() * c["page"] + pos % c["page"]


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    op, dtype, hk, d, page = c["op"], DTYPES[c["dtype"]], c["hk"], c["d"], c["page"]
    if op == "read":
        T = c["T"]
        P = _blocks(T, page) + 5
        perm = torch.randperm(P, generator=g, device="cuda")
        t = torch.arange(T, device="cuda") + 3
        slots = perm[t // page] * page + t % page
        slots[torch.randint(0, T, (c["skip"],), generator=g, device="cuda")] = -1
        return {"case": c, "slots": slots.contiguous(), **_pools(c, g, P),
                "out": tuple(torch.empty((T, hk, d), dtype=dtype, device="cuda") for _ in range(2))}
    old, seq, offsets, table, P = _layout(c, g)
    T = int(offsets[-1])
    if op == "store":
        pad = torch.full((c["pad"],), -1, dtype=torch.int64, device="cuda")
        slots = torch.cat([_slots_of(c, table, old, seq), pad])
        back = _slots_of(c, table, old // c["block"] * c["block"], seq)  # every token of the blocks that are written to
        qkv = torch.randn((T + c["pad"], 3 * hk, d), generator=g, device="cuda", dtype=dtype)
        qkv *= 0.5 + 4 * torch.rand((T + c["pad"], 3 * hk, 1), generator=g, device="cuda", dtype=dtype) ** 4
        return {"case": c, "k": qkv[:, hk:2 * hk], "v": qkv[:, 2 * hk:], "slots": slots, "back": back, **_pools(c, g, P),
                "out": tuple(torch.empty((back.numel(), hk, d), dtype=dtype, device="cuda") for _ in range(2))}
    qkv = torch.randn((T, c["hq"] + 2 * hk, d), generator=g, device="cuda", dtype=dtype) * 1.5
    n = offsets[1:] - offsets[:-1]
    return {"case": c, "q": qkv[:, : c["hq"]], **_pools(c, g, P), "table": table, "seq_len": seq,
            "offsets": None if c["new"] == 1 else offsets, "max_new": int(n.max()), "max_len": int(seq.max()),
            "scale": 1.0 / math.sqrt(d), "out": torch.empty((T, c["hq"], d), dtype=dtype, device="cuda"),
            "lse": torch.empty((T, c["hq"]), device="cuda") if c["lse"] else None}


# ------------------------------------------------------------------ the plain forms
def _power(e):
    """2^e in fp32, e whole numbers in [-126, 127]."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _exponents(exp, lohi):
    return (exp.int() - 127).clamp(*lohi)


def _plain_append(s, name):
    """Quantises the step's keys (or values) into their pages, in place."""
    c, x, slots, codes, exp = s["case"], s[name].float(), s["slots"], s[name + "_pages"], s[name + "_exp"]
    P, hk, nb = exp.shape
    block, lohi = c["block"], RANGE[c["dtype"]]
    live = slots >= 0
    at = torch.where(live, slots, slots[0])  # padding counts as the first token
    x = torch.where(live[:, None, None], x, x[:1])
    of = at // block  # block of each token, over the pool
    largest = torch.zeros((P * nb, hk), device="cuda").scatter_reduce(0, of[:, None].expand(-1, hk), x.abs().amax(-1), "amax")
    written = torch.zeros(P * nb, device="cuda").index_fill(0, of, 1.0) > 0
    begun = torch.zeros(P * nb, device="cuda").scatter_reduce(0, of, (at % block == 0).float(), "amax") > 0
    m, e = torch.frexp(largest)  # largest = m 2^e with m in [1/2, 1): 127 steps of 2^(e - 7) hold it up to m = 127 / 128
    e = torch.where(largest == 0, lohi[0], torch.where(m <= 127.0 / 128.0, e - 7, e - 6)).clamp(*lohi)
    before = _exponents(exp, lohi).transpose(1, 2).reshape(P * nb, hk)
    after = torch.where(begun[:, None], e, torch.maximum(e, before))
    grown = torch.where(written[:, None] & ~begun[:, None], after - before, 0)  # [blocks, hk]
    y = codes.view(P * nb, block, hk, -1).float() * _power(-grown.clamp(max=126))[:, None, :, None]
    y = torch.round(y).to(torch.int8).view(P * c["page"], hk, -1)
    new = torch.round(x * _power(-after)[of][..., None]).clamp(-127, 127).to(torch.int8)
    codes.copy_(y.index_copy(0, at, new).view_as(codes))
    byte = torch.where(written[:, None], (after + 127).to(torch.uint8), exp.transpose(1, 2).reshape(P * nb, hk))
    exp.copy_(byte.view(P, nb, hk).transpose(1, 2))


def _plain_read(s, name, slots):
    c, codes, exp = s["case"], s[name + "_pages"], s[name + "_exp"]
    at = slots.clamp(min=0)
    page, i = at // c["page"], at % c["page"]
    x = codes[page, i].float() * _power(_exponents(exp, RANGE[c["dtype"]]))[page, :, i // c["block"]][..., None]
    return torch.where((slots >= 0)[:, None, None], x, 0.0).to(DTYPES[c["dtype"]])


def _plain_store(s):
    _plain_append(s, "k")
    _plain_append(s, "v")
    return {"k": _plain_read(s, "k", s["back"]), "v": _plain_read(s, "v", s["back"]), "k_exp": s["k_exp"], "v_exp": s["v_exp"]}


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

    def rows(name):  # [B, hk, L, d]
        exp = _power(_exponents(s[name + "_exp"], RANGE[c["dtype"]]))[blocks, :, l % page // c["block"]]  # [B, L, hk]
        return (s[name + "_pages"][blocks, l % page].float() * exp[..., None]).permute(0, 2, 1, 3)

    z = torch.matmul(qb, rows("k").transpose(2, 3)) * s["scale"]
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
    o = torch.matmul(e, rows("v")) / torch.where(total == 0, 1.0, total)
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
        if c["op"] == "read":
            return {"k": _plain_read(s, "k", s["slots"]), "v": _plain_read(s, "v", s["slots"])}
        return _plain_store(s) if c["op"] == "store" else _plain_attend(s)
    from semi_ar_draft_gb300 import api

    pools = (s["k_pages"], s["v_pages"], s["k_exp"], s["v_exp"])
    if c["op"] == "store":
        api.cache_append_i8(s["k"], s["v"], *pools, s["slots"])
        k, v = api.cache_read_i8(*pools, s["back"], out=s["out"])
        return {"k": k, "v": v, "k_exp": s["k_exp"], "v_exp": s["v_exp"]}
    if c["op"] == "read":
        k, v = api.cache_read_i8(*pools, s["slots"], out=s["out"])
        return {"k": k, "v": v}
    out, lse, _ = api.paged_attention_i8(s["q"], *pools, s["table"], s["seq_len"], s["offsets"], scale=s["scale"],
                                         causal=c["causal"], window=c["window"], softcap=c["softcap"], max_new=s["max_new"],
                                         out=s["out"], lse=s["lse"])
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    row = 2.0 * c["hk"] * c["d"]  # values of a token, keys and values
    if c["op"] == "read":
        real = max(c["T"] - c["skip"], 1)
        return {"bytes": row * (real + 2 * c["T"]) + 8 * c["T"] + 2 * c["hk"] * _blocks(real, c["block"]), "flops": 0}
    if c["op"] == "store":
        new = back = blocks = 0
        for old, n in _lengths(c):
            new += n
            back += n + old % c["block"]
            blocks += _blocks(old % c["block"] + n, c["block"])
        # the step's values read and their codes written; of the blocks' older tokens the codes read; the values written
        return {"bytes": row * (2 * new + new + (back - new) + 2 * back) + 8 * (new + c["pad"] + back) + 2 * c["hk"] * blocks,
                "flops": 0}
    rows = blocks = tokens = seen = 0  # cache rows and blocks that somebody sees, new tokens, (token, cache row) pairs
    for old, n in _lengths(c):
        w = c["window"] or old + n
        rows += min(old + n, w + n - 1)
        blocks += _blocks(min(old + n, w + n - 1), c["block"])
        tokens += n
        seen += sum(min((old + i + 1), w) if c["causal"] else min(old + n, w + n - 1 - i) for i in range(n))
    return {"bytes": rows * (row + 4.0 / c["page"]) + 2.0 * c["hk"] * blocks
            + tokens * c["hq"] * (4.0 * c["d"] + (4 if c["lse"] else 0)),
            "flops": 4.0 * c["hq"] * c["d"] * seen}


# ------------------------------------------------------------------ the definition in 64 bits
def _two_to(e):
    """2^e in fp64, bit by bit (a power that is off in its last place moves what lies half way between two codes)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _steps(largest, lohi):
    """The scale: the smallest power of two of the range of which 127 reach the largest magnitude (its last otherwise)."""
    tried = _two_to(torch.arange(lohi[0], lohi[1] + 1, device="cuda"))
    k = torch.searchsorted(127.0 * tried, largest.double().contiguous())  # the first that is not below it
    return tried[k.clamp(max=len(tried) - 1)]


def _true_exponent(byte, lohi):
    return _two_to((byte.long() - 127).clamp(lohi[0], lohi[1]))


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    lohi, hk, page, block = RANGE[c["dtype"]], c["hk"], c["page"], c["block"]
    if c["op"] == "read":
        out = {}
        for name in ("k", "v"):
            x = torch.zeros((c["T"], hk, c["d"]), dtype=torch.float64, device="cuda")
            t = torch.nonzero(s["slots"] >= 0)[:, 0]
            p, i = s["slots"][t] // page, s["slots"][t] % page
            x[t] = s[name + "_pages"][p, i].double() * _true_exponent(s[name + "_exp"][p, :, i // block], lohi)[..., None]
            out[name] = x
        return out
    if c["op"] == "store":
        slots, back = s["slots"].tolist(), s["back"].tolist()
        tokens = {}  # block over the pool: [(token of the step, place in the block)]
        for t, slot in enumerate(slots):
            if slot >= 0:
                tokens.setdefault(slot // block, []).append((t, slot % block))
        order = {b: i for i, b in enumerate(tokens)}
        rows = torch.tensor([order[slot // block] * block + slot % block for slot in back], device="cuda")
        out = {"k": None, "v": None, "k_exp": None, "v_exp": None}
        for name in ("k", "v"):
            held = torch.zeros((len(tokens), block, hk, c["d"]), dtype=torch.float64, device="cuda")
            for i, (b, new) in enumerate(tokens.items()):
                page_at, first = b * block // page, b * block % page
                x = s[name][[t for t, _ in new]].double()
                scale = _steps(x.abs().amax((0, 2)), lohi)  # [hk]
                if min(at for _, at in new) > 0:
                    was = _true_exponent(s[name + "_exp"][page_at, :, first // block], lohi)
                    scale = torch.maximum(scale, was)
                    codes = s[name + "_pages"][page_at, first:first + block].double()
                    held[i] = torch.round(codes * (was / scale)[:, None]) * scale[:, None]
                held[i, [at for _, at in new]] = torch.round(x / scale[:, None]).clamp(-127, 127) * scale[:, None]
            out[name] = held.view(-1, hk, c["d"])[rows]
        return out
    group = c["hq"] // hk
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
        k, v = (s[x + "_pages"][pages, l % page].double()
                * _true_exponent(s[x + "_exp"][pages, :, l % page // block], lohi)[..., None] for x in ("k", "v"))
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
