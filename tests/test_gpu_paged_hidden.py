"""Keys that a row does not see change none of its bits where the references of its exponents have moved: the 16-bit and
e4m3 caches."""
import pytest
import torch

from semi_ar_draft_gb300 import api, binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G,Hk,D,n", [(1, 4, 64, 4), (2, 2, 128, 4), (4, 1, 256, 4), (3, 2, 80, 5), (16, 1, 128, 4)])
def test_the_last_token_s_key_changes_no_other_row(dtype, e4m3, G, Hk, D, n):
    page, lens = 64, [6000 + 131 * j for j in range(24 // Hk)]
    g = torch.Generator(device="cuda").manual_seed(D + n)
    blocks = [-(-x // page) for x in lens]
    P, B = sum(blocks), len(lens)
    table, used = torch.full((B, max(blocks)), -1, dtype=torch.int32, device="cuda"), 0
    perm = torch.randperm(P, generator=g, device="cuda").int()
    for j, m in enumerate(blocks):
        table[j, :m] = perm[used:used + m]
        used += m
    k, v = (torch.randn((P, page, Hk, D), generator=g, device="cuda").to(dtype) for _ in range(2))
    q = (torch.randn((B * n, Hk * G, D), generator=g, device="cuda") * 1.5).to(dtype)
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    offsets = torch.arange(B + 1, dtype=torch.int32, device="cuda") * n
    outs = []
    for size in (0.0, 8.0):
        for j, length in enumerate(lens):
            at = (int(table[j, (length - 1) // page]), (length - 1) % page)
            k[at] = (torch.sign(q[(j + 1) * n - 1].view(Hk, G, D)[:, 0].float()) * size).to(dtype)
            v[at] = size
        pools = [x.to(torch.float8_e4m3fn) if e4m3 else x for x in (k, v)]
        out, lse, ws = api.paged_attention(q, *pools, table, seq, offsets, lse=True, max_new=n)
        assert binding.dspark_get_device_status(ws) == 0
        outs.append((out.view(B, n, -1), lse.view(B, n, -1)))
    for x, y in zip(*outs):
        assert torch.equal(x[:, :-1], y[:, :-1]) and not torch.equal(x[:, -1], y[:, -1])
