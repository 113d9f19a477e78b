"""Plan, append, read back, attention and commit on an int8 PagedCache, round after round, against the definition; the C names
against the checked calls; decoding rounds on such a cache."""
import math

import pytest
import torch

import i8_reference as R
from semi_ar_draft_gb300 import api, binding as b
from semi_ar_draft_gb300 import decode_round as D
from semi_ar_draft_gb300 import paged

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype,block,Hq,Hk,d", [(torch.bfloat16, None, 8, 2, 64), (torch.float16, 1, 4, 4, 128), (torch.bfloat16, 8, 24, 1, 96)])
def test_rounds_against_the_definition(dtype, block, Hq, Hk, d):
    """Prompts, then rounds in which some tokens are rejected and written over; what every layer holds, reads back and
    attends to."""
    B, page, P, width, layers, most = 3, 16, 40, 12, 2, 96
    g = torch.Generator(device="cuda").manual_seed(d)
    r = torch.Generator().manual_seed(d)
    cache = paged.PagedCache(B, P, page, width, layers, Hk, d, most, dtype=dtype, kv_dtype=torch.int8, scale_block=block)
    pools = [[x[i].cpu().clone() for x in (cache.k_pages, cache.v_pages, cache.k_exp, cache.v_exp)] for i in range(layers)]
    for n_round in range(7):
        new = [30, 1, 17] if n_round == 0 else torch.randint(0, 9, (B,), generator=r).tolist()
        T = sum(new) + B + n_round % 3  # padding
        cache.plan(i32(new), extra=1, max_new=max(new) + 1, tokens=T)
        lens, offs, slots = cache.seq_len.tolist(), cache.offsets.tolist(), cache.slots.tolist()
        for layer in range(layers):
            q, k, v = (torch.randn((T, h, d), generator=g, device="cuda").to(dtype) for h in (Hq, Hk, Hk))
            k = k * torch.exp2(torch.randint(-4, 5, (T, Hk, 1), generator=g, device="cuda").float()).to(dtype)
            cache.append(layer, k, v)
            kc, vc, ke, ve = pools[layer]
            assert R.append(k.cpu(), kc, ke, slots) and R.append(v.cpu(), vc, ve, slots)
            for got, want in zip((cache.k_pages, cache.v_pages, cache.k_exp, cache.v_exp), pools[layer]):
                assert torch.equal(got[layer].cpu(), want)
            live = torch.tensor(slots) >= 0
            for got, c, e in zip(cache.read(layer), (kc, vc), (ke, ve)):
                want = R.values(c, e, dtype).reshape(P * page, Hk, d)[torch.tensor(slots).clamp(min=0)]
                assert got.dtype == dtype and torch.equal(got.cpu().double()[live], want[live]) and not got.cpu()[~live].any()
            out, lse = cache.attend(layer, q, lse=True)
            mean = Hq // Hk * T / B
            ro, rl, to, tl = R.attention(q, [cache.k_pages[layer], cache.v_pages[layer]], [cache.k_exp[layer], cache.v_exp[layer]],
                                         cache.block_table, lens, offs, d ** -0.5, True, 0, 0.0, mean > (31 if d <= 128 else 32))
            assert bool(((out.double() - ro).abs() <= to).all())
            dead = rl == -math.inf
            assert torch.equal(lse == -math.inf, dead) and bool(((lse.double() - rl).abs()[~dead] <= tl[~dead]).all())
        keep = [int(torch.randint(0, n + 1, (1,), generator=r)) for n in new]
        cache.commit(i32(keep), extra=1)
        assert cache.status() == 0


def test_status_covers_the_append():
    cache = paged.PagedCache(1, 4, 16, 4, 1, 1, 64, 8, kv_dtype=torch.int8)
    cache.plan(i32([4]))
    k, v = (torch.ones((8, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[5:] = math.nan  # rows without a slot
    cache.append(0, k, v)
    assert cache.status() == 0
    v[2, 0, 3] = math.inf
    cache.append(0, k, v)
    assert cache.status() == 9 and cache.status() == 0


def test_a_round_replayed_from_a_graph():
    """Plan, append, attention and commit of one round captured once and replayed: the same pools and outputs as eagerly."""
    def make():
        c = paged.PagedCache(2, 20, 16, 8, 1, 2, 128, 24, kv_dtype=torch.int8, scale_block=4)
        c.plan(i32([19, 5]))
        g = torch.Generator(device="cuda").manual_seed(1)
        c.append(0, *(torch.randn((24, 2, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)))
        c.commit(i32([19, 5]))
        return c

    eager, replayed = make(), make()
    new, keep = i32([3, 2]), i32([2, 1])
    q, k, v = (torch.zeros((8, h, 128), dtype=torch.bfloat16, device="cuda") for h in (8, 2, 2))

    def one(c):
        c.plan(new, extra=1, max_new=4, tokens=8)
        c.append(0, k, v)
        out, _ = c.attend(0, q)
        c.commit(keep, extra=1)
        return out

    spare = make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one(spare)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = one(replayed)
    g = torch.Generator(device="cuda").manual_seed(2)
    for n in range(5):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda") * 2.0 ** n)
        graph.replay()
        want = one(eager)
        assert torch.equal(out, want)
        for name in ("k_pages", "v_pages", "k_exp", "v_exp", "block_table", "cache_len"):
            assert torch.equal(getattr(eager, name), getattr(replayed, name)), name
    assert eager.status() == 0 and replayed.status() == 0


def test_a_step_through_the_c_names():
    B, page, P, width, T, Hq, Hk, d, block = 3, 16, 30, 6, 21, 8, 2, 64, 4
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((T, h, d), generator=g, device="cuda").to(torch.bfloat16) for h in (Hq, Hk, Hk))
    table, seq, off = i32([[0, 1, -1, -1, -1, -1], [2] + [-1] * 5, [3] + [-1] * 5]), i32([17, 3, 1]), i32([0, 17, 20, 21])
    slots = torch.tensor([*range(16), 16, 32, 33, 34, 48], dtype=torch.int64, device="cuda")
    sets = [[torch.zeros((P, page, Hk, d), dtype=torch.int8, device="cuda") for _ in range(2)]
            + [torch.zeros((P, Hk, page // block), dtype=torch.uint8, device="cuda") for _ in range(2)] for _ in range(2)]
    api.cache_append_i8(k, v, *sets[0], slots)
    x = b.block_exponents(sets[1][2], sets[1][3], page)
    strides = sets[1][0].stride()[:3]
    error = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = b.AppendParams(T, Hk, d, page, P, b.BF16, b.I8, *k.stride()[:2], *v.stride()[:2], *strides)
    b.dspark_cache_append_i8(p, x, k, v, *sets[1][:2], slots, error)
    assert all(torch.equal(y, z) for y, z in zip(*sets)) and int(error) == 0
    want = api.cache_read_i8(*sets[0], slots)
    got = tuple(torch.empty((T, Hk, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    b.dspark_cache_read_i8(p, x, *sets[1][:2], slots, *got)
    assert all(torch.equal(y, z) for y, z in zip(got, want))
    want, want_lse, _ = api.paged_attention_i8(q, *sets[0], table, seq, off, lse=True)
    a = b.AttentionParams(T, B, Hq, Hk, d, page, P, width, 0, b.BF16, b.I8, 1, 0, d ** -0.5, 0.0, *q.stride()[:2], *strides)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    work = b.workspace(b.dspark_paged_attention_workspace_size(a))
    b.dspark_paged_attention_i8(a, x, q, *sets[1][:2], table, seq, off, out, lse, work)
    assert torch.equal(out, want) and torch.equal(lse, want_lse) and b.dspark_get_device_status(work) == 0


def test_decoding_rounds_keep_their_pages():
    target = D.ToyTarget(512, 64, 1, 4, 1, 64, 256, seed=5)
    draft = D.ToyDraft(4, target)
    prompts = torch.randint(0, 512, (5, 9), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda", dtype=torch.int32)
    out, _, cache = D.generate(target, draft, prompts, 6, page_size=4, kv_dtype=torch.int8, max_len=128)
    assert cache.status() == 0 and cache.k_exp is not None
    held = cache._blocks[0].tolist()
    assert held == [-(-n // 4) for n in cache.cache_len.tolist()]
    assert sum(held) + int(cache.n_free) == cache.free_pages.numel()
    assert [len(x) for x in out] == [n - 9 + 1 for n in cache.cache_len.tolist()]


def test_example_runs(capsys):
    D.main(["--requests", "4", "--rounds", "3", "--int8"])
    assert "status 0" in capsys.readouterr().out
