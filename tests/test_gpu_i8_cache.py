"""The int8 paged cache on the GPU: what is written against the definition bit for bit, what is read back exactly."""
import math

import pytest
import torch

import i8_reference as R
from semi_ar_draft_gb300 import api, binding

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make_pools(P, page, Hk, D, block, g, heads_first=False, lo=100, hi=140):
    """Codes and exponents that another request has left, in either layout of the pages."""
    shape = (P, Hk, page, D) if heads_first else (P, page, Hk, D)
    codes = [torch.randint(-127, 128, shape, generator=g, device="cuda").to(torch.int8) for _ in range(2)]
    if heads_first:
        codes = [c.transpose(1, 2) for c in codes]
    shape = (P, page // block, Hk) if heads_first else (P, Hk, page // block)
    exps = [torch.randint(lo, hi, shape, generator=g, device="cuda").to(torch.uint8) for _ in range(2)]
    if heads_first:
        exps = [e.transpose(1, 2) for e in exps]
    return codes, exps


def step(k, v, codes, exps, slots, error=None):
    """Runs the append on the pools and on copies of them by the definition, and compares every byte."""
    want_c, want_e = [c.cpu().clone() for c in codes], [e.cpu().clone() for e in exps]
    fine = [R.append(x.cpu(), c, e, slots) for x, c, e in zip((k, v), want_c, want_e)]
    api.cache_append_i8(k, v, *codes, *exps, torch.tensor(slots, dtype=torch.int64, device="cuda"), error=error)
    for name, got, want in zip(("k_exp", "v_exp", "k_pages", "v_pages"), (*exps, *codes), (*want_e, *want_c)):
        assert torch.equal(got.cpu(), want), (name, int((got.cpu() != want).sum()))
    return all(fine)


def rows(T, Hk, D, dtype, g, shift=0, wild=True):
    """k, v as slices of a projection's output, tokens of very different magnitude."""
    buf = torch.randn(T * 3 * Hk * D + 16, generator=g, device="cuda")
    x = buf[shift: shift + T * 3 * Hk * D].view(T, 3 * Hk, D)
    if wild:
        x = x * torch.exp2(torch.randint(-9, 5, (T, 3 * Hk, 1), generator=g, device="cuda").float())
    y = torch.empty(T * 3 * Hk * D + 16, dtype=dtype, device="cuda")
    y[shift: shift + T * 3 * Hk * D] = x.reshape(-1).to(dtype)
    y = y[shift: shift + T * 3 * Hk * D].view(T, 3 * Hk, D)
    return y[:, Hk:2 * Hk], y[:, 2 * Hk:]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("Hk,D,page,block,heads_first,shift", [
    (1, 16, 1, 1, False, 0), (2, 64, 16, 16, False, 0), (8, 128, 16, 4, True, 0), (3, 80, 32, 8, False, 3), (2, 256, 128, 128, False, 0),
    (4, 96, 64, 1, True, 1), (5, 192, 64, 32, False, 0), (1, 128, 4096, 64, False, 0), (2, 48, 16, 2, True, 8)])
def test_steps_of_several_requests(dtype, Hk, D, page, block, heads_first, shift):
    """Prompts, then steps of one to nine tokens into blocks that are partly filled, some of them taken back."""
    g = torch.Generator(device="cuda").manual_seed(D + page + block)
    r = torch.Generator().manual_seed(D * page + block)
    B, per = 5, 2 if page > 1000 else -(-260 // page)
    P = B * per + 3
    table = torch.randperm(P, generator=r)[: B * per].view(B, per).tolist()
    codes, exps = make_pools(P, page, Hk, D, block, g, heads_first)
    lens = [0] * B
    for n_step in range(9):
        slots = []
        for j in range(B):
            n = [150, 3, 0, 17, 64][j] if n_step == 0 else int(torch.randint(0, 10, (1,), generator=r))
            n = min(n, per * page - lens[j])
            slots += [table[j][i // page] * page + i % page for i in range(lens[j], lens[j] + n)]
            lens[j] += n if n_step == 0 else int(torch.randint(0, n + 1, (1,), generator=r))  # the rest is rejected
        slots += [-1] * (n_step % 3)
        k, v = rows(len(slots), Hk, D, dtype, g, shift)
        assert step(k, v, codes, exps, slots)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,Hk,D,page,block", [(1, 8, 128, 16, 16), (3000, 8, 64, 64, 32), (5000, 1, 128, 128, 128), (2500, 2, 256, 32, 32),
                                               (4100, 4, 48, 16, 1), (999, 2, 240, 64, 64)])
def test_prompts(dtype, T, Hk, D, page, block):
    """Runs of whole blocks, more than the registers of a warp hold among them, at windows of every size."""
    g = torch.Generator(device="cuda").manual_seed(T)
    P = -(-(T + 5) // page) + 2
    codes, exps = make_pools(P, page, Hk, D, block, g)
    perm = torch.randperm(P, generator=torch.Generator().manual_seed(T)).tolist()
    k, v = rows(T, Hk, D, dtype, g)
    assert step(k, v, codes, exps, [perm[t // page] * page + t % page for t in range(5, T + 5)])


def test_skipped_entries_and_orders():
    """Any order within a block, up to 31 skipped entries between its tokens, slots outside the pool, a slot twice."""
    g = torch.Generator(device="cuda").manual_seed(1)
    P, page, Hk, D, block = 6, 64, 2, 64, 32
    out = [-1, P * page, 1 << 40, -(1 << 62)]
    for slots in ([5, 3, 4, 9, 8], [40] + [-1] * 31 + [41] + [-1] * 31 + [33], [70, 71] + out * 7 + [69], list(range(95, 63, -1)),
                  [130, 130, 131, 130], [200] * 70 + [201], [7] + [-1] * 31 + [6, 100] + [-1] * 12 + [101] + [-1] * 40 + [330, 331],
                  out * 20, out * 20 + [12], [12] + out * 20, [-1] * 33 + [13, 14] + [-1] * 29 + [15]):
        codes, exps = make_pools(P, page, Hk, D, block, g)
        k, v = rows(len(slots), Hk, D, torch.bfloat16, g)
        assert step(k, v, codes, exps, slots)


def test_no_tokens():
    codes, exps = make_pools(2, 16, 1, 64, 16, torch.Generator(device="cuda").manual_seed(1))
    n = binding.dspark_kernel_launches()
    step(torch.empty((0, 1, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((0, 1, 64), dtype=torch.bfloat16, device="cuda"), codes, exps, [])
    k, v = api.cache_read_i8(*codes, *exps, torch.empty(0, dtype=torch.int64, device="cuda"))
    assert k.shape == v.shape == (0, 1, 64) and binding.dspark_kernel_launches() == n


@pytest.mark.parametrize("dtype", DTYPES)
def test_magnitudes_from_the_smallest_to_the_largest(dtype):
    """Every power of two of the type and its neighbours as a block's largest value: the smallest scale that holds it."""
    g = torch.Generator(device="cuda").manual_seed(2)
    info = torch.finfo(dtype)
    m = torch.tensor([1.0, 1.5, 127 / 64, 1.9921875, 1.25], dtype=torch.float64)
    lowest = math.frexp(info.smallest_normal * info.eps)[1] - 1
    e = torch.arange(lowest, math.frexp(info.max)[1], dtype=torch.float64)
    top = torch.cat([(m * torch.exp2(e)[:, None]).reshape(-1), torch.tensor([0.0, info.max])]).to(dtype)
    T, D, page = len(top), 32, 16
    x = (torch.rand((T, 1, D), generator=g, device="cuda") * 2 - 1).double() * top.double().cuda()[:, None, None]
    x = x.to(dtype)
    x[:, 0, 7] = top.cuda()
    P = -(-T // page)
    codes, exps = make_pools(P, page, 1, D, 1, g)
    assert step(x, -x, codes, exps, list(range(T)))
    written = exps[0].reshape(-1)[:T].long() - 127  # (one head, a token a block: slots in order)
    assert (int(written.min()), int(written.max())) == R.RANGE[dtype]
    codes, exps = make_pools(P, page, 1, D, 1, g)
    exps[0].zero_(), exps[1].fill_(255)  # bytes that no append has written
    assert step(x, -x, codes, exps, list(range(T)))


@pytest.mark.parametrize("dtype", DTYPES)
def test_scales_grow_by_any_number_of_steps(dtype):
    """All codes re-rounded by 0 to 20 binades, to nearest even, and left alone where a block is begun anew."""
    P, page, D, block = 21, 256, 16, 128
    codes = [torch.arange(-128, 128, device="cuda").to(torch.int8)[None, :, None, None].expand(P, page, 1, D).contiguous() for _ in range(2)]
    exps = [torch.full((P, 1, 2), 110, dtype=torch.uint8, device="cuda") for _ in range(2)]
    x = (127 * torch.exp2(torch.arange(P, device="cuda") - 17.0)).to(dtype)[:, None, None].expand(P, 1, D).contiguous()
    for at in (5, 128 + 127, 128):
        assert step(x, x * 2, codes, exps, [p * page + at for p in range(P)])


def test_values_that_are_not_finite_are_stored_and_reported():
    for dtype in DTYPES:
        g = torch.Generator(device="cuda").manual_seed(3)
        codes, exps = make_pools(8, 16, 2, 64, 16, g)
        k, v = rows(100, 2, 64, dtype, g)
        error = torch.zeros(1, dtype=torch.int32, device="cuda")
        assert step(k, v, codes, exps, list(range(100)), error) and int(error) == 0
        for at, bad in ((3, math.nan), (40, math.inf), (41, -math.inf)):
            v[at, 1, 5] = bad
        v[70:75] = math.nan  # a token without a finite value
        v[99] = math.inf
        assert not step(k, v, codes, exps, list(range(100)), error)
        assert int(error) == 9
        error.fill_(8)
        assert not step(k, v, codes, exps, list(range(100)), error)
        assert int(error) == 8  # the first one stays
        v[:] = math.nan
        error.zero_()
        before = [x.clone() for x in (*codes, *exps)]
        assert step(k, v, codes, exps, [-1] * 100, error)  # nobody looks at skipped rows
        assert int(error) == 0 and all(torch.equal(x, y) for x, y in zip(before, (*codes, *exps)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads_first", [False, True])
def test_every_code_and_exponent_reads_back(dtype, heads_first):
    P, page, Hk, D, block = 64, 16, 4, 256, 16  # a byte of exponent for each (page, head) of all 256
    g = torch.Generator(device="cuda").manual_seed(4)
    codes, exps = make_pools(P, page, Hk, D, block, g, heads_first)
    codes[0][:] = torch.arange(-128, 128, device="cuda").to(torch.int8)
    for e in exps:
        e.copy_(torch.arange(256, device="cuda").to(torch.uint8).view(P, Hk, 1))
    slots = torch.randperm(P * page, generator=g, device="cuda")
    slots[5], slots[77], slots[78] = -1, P * page, 1 << 50
    k, v = api.cache_read_i8(*codes, *exps, slots, dtype=dtype)
    live = (slots >= 0) & (slots < P * page)
    for got, c, e in zip((k, v), codes, exps):
        want = R.values(c.cpu(), e.cpu(), dtype).reshape(P * page, Hk, D)[slots.clamp(0, P * page - 1).cpu()][live.cpu()]
        codes_ok = (c.reshape(P * page, Hk, D)[slots.clamp(0, P * page - 1)][live] != -128).cpu()  # (-128 is no code)
        assert torch.equal(got[live].cpu().double()[codes_ok], want[codes_ok]) and not got[~live].any()


@pytest.mark.parametrize("T,Hk,D,page,block", [(1, 1, 16, 1, 1), (777, 3, 80, 32, 4), (20000, 8, 128, 64, 64)])
def test_what_is_written_reads_back(T, Hk, D, page, block):
    """Within half a step of the scale, which is at most 1/63.5 of the block's largest value; given outputs are used."""
    g = torch.Generator(device="cuda").manual_seed(T)
    P = -(-T // page) + 1
    codes, exps = make_pools(P, page, Hk, D, block, g)
    slots = torch.randperm(P, generator=g, device="cuda").repeat_interleave(page)[:T] * page + torch.arange(T, device="cuda") % page
    k, v = rows(T, Hk, D, torch.bfloat16, g)
    api.cache_append_i8(k, v, *codes, *exps, slots)
    out = tuple(torch.full((T, Hk, D), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    got = api.cache_read_i8(*codes, *exps, slots, out=out)
    assert got[0] is out[0] and got[1] is out[1]
    b = torch.arange(T, device="cuda") // block
    for x, y in zip((k, v), got):
        top = torch.zeros((int(b[-1]) + 1, Hk), dtype=torch.float64, device="cuda").scatter_reduce(
            0, b[:, None].expand(-1, Hk), x.double().abs().amax(-1), "amax")[b]
        assert bool(((x.double() - y.double()).abs() <= (top / 127)[..., None]).all())


def test_other_stream_and_graph():
    """A step on a side stream, and replayed from a graph with other values and slots."""
    g = torch.Generator(device="cuda").manual_seed(6)
    P, page, Hk, D, block, T = 20, 16, 4, 128, 16, 50
    codes, exps = make_pools(P, page, Hk, D, block, g)
    k, v = (x.contiguous() for x in rows(T, Hk, D, torch.float16, g))
    slots = torch.arange(T, device="cuda") + 37
    want = [x.clone() for x in (*codes, *exps)]
    api.cache_append_i8(k, v, *want, slots)
    ref = api.cache_read_i8(*want, slots, torch.float16)
    side = torch.cuda.Stream()
    first = [x.clone() for x in (*codes, *exps)]
    torch.cuda.synchronize()
    api.cache_append_i8(k, v, *first, slots, stream=side)
    got = api.cache_read_i8(*first, slots, torch.float16, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((*first, *got), (*want, *ref)))
    graph, out = torch.cuda.CUDAGraph(), tuple(torch.empty_like(k) for _ in range(2))
    with torch.cuda.graph(graph):
        api.cache_append_i8(k, v, *codes, *exps, slots)
        api.cache_read_i8(*codes, *exps, slots, out=out)
    for n in range(3):
        k2, v2 = rows(T, Hk, D, torch.float16, g)
        k.copy_(k2), v.copy_(v2), slots.copy_(torch.arange(T, device="cuda") + 37 + 50 * n)
        api.cache_append_i8(k, v, *want, slots)
        ref = api.cache_read_i8(*want, slots, torch.float16)
        if n == 0:
            for x, y in zip((*codes, *exps), first):
                x.copy_(y)  # both have seen the first step
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((*codes, *exps, *out), (*want, *ref)))


def test_pools_past_32_bits():
    """Slots and strides whose offsets do not fit 32 bits (a pool of 4.4 GB)."""
    page, Hk, D, block = 128, 1, 256, 64
    P = (1 << 32) // (page * Hk * D) + 3000
    codes = [torch.empty((P, page, Hk, D), dtype=torch.int8, device="cuda") for _ in range(2)]
    exps = [torch.zeros((P, Hk, page // block), dtype=torch.uint8, device="cuda") for _ in range(2)]
    g = torch.Generator(device="cuda").manual_seed(7)
    k, v = rows(300, Hk, D, torch.bfloat16, g)
    first = (P - 4) * page + 64
    slots = torch.arange(300, device="cuda") + first
    api.cache_append_i8(k, v, *codes, *exps, slots)
    got = api.cache_read_i8(*codes, *exps, slots)
    small_c = [torch.zeros((4, page, Hk, D), dtype=torch.int8, device="cuda") for _ in range(2)]
    small_e = [torch.zeros((4, Hk, page // block), dtype=torch.uint8, device="cuda") for _ in range(2)]
    assert step(k, v, small_c, small_e, list(range(64, 364)))
    ref = api.cache_read_i8(*small_c, *small_e, slots - (P - 4) * page)
    assert all(torch.equal(x, y) for x, y in zip(got, ref))
