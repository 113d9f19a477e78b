"""With a scale for every token, nothing that a verify step appends changes what it says of the positions before."""
import pytest
import torch

from semi_ar_draft_gb300 import decode_round as D
from semi_ar_draft_gb300 import paged

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Hq,Hk,n", [(4, 2, 4), (8, 2, 4), (32, 2, 5)])  # kernels of 8, 16 and 128 rows
def test_later_drafts_do_not_reach_earlier_positions(dtype, Hq, Hk, n):
    """The last two drafts of every request, ordinary and 2^6 times as large: the outputs before them and what the cache holds
    of the tokens before them, bit for bit."""
    B, d, got = 3, 64, []
    for size in (1.0, 64.0):
        g = torch.Generator(device="cuda").manual_seed(n)
        cache = paged.PagedCache(B, 60, 16, 16, 1, Hk, d, 400, dtype=dtype, kv_dtype=torch.int8, scale_block=1)
        rnd = lambda T, h: torch.randn((T, h, d), generator=g, device="cuda")  # noqa: E731
        cache.plan(i32([100, 37, 203]), tokens=340)
        cache.append(0, rnd(340, Hk).to(dtype), rnd(340, Hk).to(dtype))
        cache.commit(i32([100, 37, 203]))
        cache.plan(i32([n] * B), max_new=n, tokens=B * n)
        q, k, v = rnd(B * n, Hq), rnd(B * n, Hk), rnd(B * n, Hk)
        for x in (q, k, v):
            x.view(B, n, -1)[:, -2:] *= size
        cache.append(0, k.to(dtype), v.to(dtype))
        out, lse = cache.attend(0, q.to(dtype), lse=True)
        slots = torch.cat([cache.block_table[j].repeat_interleave(16) * 16 + torch.arange(256, device="cuda") % 16 for j in range(B)]).long()
        keep = torch.cat([torch.arange(256, device="cuda") < m + n - 2 for m in (100, 37, 203)])
        held = [x[keep] for x in cache.read(0, slots)]
        assert cache.status() == 0
        got.append([out.view(B, n, Hq, d)[:, :-2], lse.view(B, n, Hq)[:, :-2], *held])
    assert all(torch.equal(x, y) for x, y in zip(*got))


def quantised(x):
    """bf16 as a cache with a scale for every token and head holds it."""
    m, e = torch.frexp(x.double().abs().amax(-1, keepdim=True) / 127)  # m 2^e with m in [1/2, 1): the power of two at or above
    two = torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e).int())
    return torch.round(x.double() / two) * two


def test_greedy_rounds_give_the_tokens_of_decoding_one_by_one():
    V, gamma, prompt, B = 512, 4, 13, 7
    target = D.ToyTarget(V, 64, 2, 4, 2, 64, 256, seed=4)
    draft = D.ToyDraft(gamma, target)
    prompts = torch.randint(0, V, (B, prompt), generator=torch.Generator(device="cuda").manual_seed(8), device="cuda", dtype=torch.int32)
    out, mean, cache = D.generate(target, draft, prompts, 12, budget=B * 3, page_size=8, max_len=200, kv_dtype=torch.int8)
    assert cache.status() == 0 and mean > 1.0 and cache.k_exp.shape[-1] == 8  # a scale for every token
    checked = 0
    for j in range(B):
        tokens = prompts[j].tolist() + out[j][:-1]
        n = len(tokens)
        x = target.embed[torch.tensor(tokens, device="cuda")] + target.place[:n]
        hide = torch.ones((n, n), device="cuda").triu(1).bool()
        for w, p in zip(target.qkv, target.proj):
            q, k, v = (torch.nn.functional.rms_norm(x, (64,)) @ w).view(n, -1, target.D).split([target.Hq, target.Hk, target.Hk], dim=1)
            k, v = (quantised(y).repeat_interleave(target.Hq // target.Hk, 1) for y in (k, v))
            s = torch.einsum("nhd,lhd->hnl", q.double(), k) * target.D ** -0.5
            o = torch.einsum("hnl,lhd->nhd", torch.softmax(s.masked_fill(hide, float("-inf")), -1), v).to(torch.bfloat16)
            x = x + o.reshape(n, -1) @ p
        logits = (torch.nn.functional.rms_norm(x, (64,)) @ target.head).float()[prompt - 1:]
        for i, tok in enumerate(out[j]):
            best = logits[i].max()  # (a token may be another one within what bf16 activations and logits can move it)
            assert float(best - logits[i, tok]) <= 2.0 ** -4 * max(1.0, float(best.abs())), (j, i)
            checked += int(logits[i].argmax()) == tok
    total = sum(map(len, out))
    assert checked >= 0.9 * total, (checked, total)
