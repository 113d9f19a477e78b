"""The C-named functions of `binding` for the paged cache against the checked calls of `api`."""
import pytest
import torch

from semi_ar_draft_gb300 import api, binding as b

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("cache", [torch.bfloat16, torch.float8_e4m3fn])
def test_a_step_through_the_c_names(cache):
    B, page, P, width, T, Hq, Hk, D = 3, 16, 30, 6, 40, 8, 2, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    cache_len, new, n_blocks, n_free = i32([20, 0, 5]), i32([17, 3, 1]), i32([2, 0, 1]), i32([27])
    free = torch.cat([torch.arange(26, -1, -1), torch.zeros(3)]).int().cuda()
    tables = [i32([[27, 28, -1, -1, -1, -1], [-1] * 6, [29, -1, -1, -1, -1, -1]]) for _ in range(2)]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    ref = api.cache_plan(cache_len, new, tables[0], n_blocks, free, n_free, page, T, extra=1)
    out = [torch.empty_like(x) for x in ref[:6]]
    b.dspark_cache_plan(b.CacheParams(B, page, P, width, T, 1), cache_len, new, tables[1], n_blocks, free, n_free, *out, ws)
    assert all(torch.equal(x, y) for x, y in zip(out, ref)) and torch.equal(*tables) and b.dspark_get_device_status(ws) == 0

    seq, off, slots, held, left = out[0], out[1], out[2], out[4], out[5]
    q, k, v = (torch.randn((T, h, D), generator=g, device="cuda").to(torch.bfloat16) for h in (Hq, Hk, Hk))
    scales = [None, None] if cache is torch.bfloat16 else [torch.full((Hk,), 0.02, device="cuda") for _ in range(2)]
    pools = [[torch.zeros((P, page, Hk, D), device="cuda").to(cache) for _ in range(2)] for _ in range(2)]
    api.cache_append(k, v, *pools[0], slots, *scales)
    code = b.cache_dtype_code(cache)
    strides = pools[1][0].stride()[:3]
    b.dspark_cache_append(b.AppendParams(T, Hk, D, page, P, b.BF16, code, *k.stride()[:2], *v.stride()[:2], *strides), k, v,
                          *pools[1], slots, *scales)
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(*pools))

    want, want_lse, _ = api.paged_attention(q, *pools[0], tables[0], seq, off, k_scale=scales[0], v_scale=scales[1], lse=True)
    p = b.AttentionParams(T, B, Hq, Hk, D, page, P, width, 0, b.BF16, code, 1, 0, D ** -0.5, 0.0, *q.stride()[:2], *strides)
    got, lse = torch.empty_like(want), torch.empty_like(want_lse)
    work = b.workspace(b.dspark_paged_attention_workspace_size(p))
    b.dspark_paged_attention(p, q, *pools[0], tables[0], seq, off, *scales, got, lse, work)
    assert torch.equal(got, want) and torch.equal(lse, want_lse) and b.dspark_get_device_status(work) == 0

    add, done = i32([3, 3, 0]), torch.tensor([0, 0, 1], dtype=torch.uint8, device="cuda")
    stacks = [free.clone() for _ in range(2)]
    ref = api.cache_commit(cache_len, add, tables[0], held, stacks[0], left, page, extra=1, done=done)
    out = [torch.empty_like(x) for x in ref[:3]]
    b.dspark_cache_commit(b.CacheParams(B, page, P, width, 0, 1), cache_len, add, done, tables[0], held, stacks[1], left, *out, ws)
    assert all(torch.equal(x, y) for x, y in zip(out, ref)) and torch.equal(*stacks) and b.dspark_get_device_status(ws) == 0
