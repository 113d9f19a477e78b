"""Decoding rounds on a paged cache (draft, schedule, plan, append, attention, verify, commit) emit, at
temperature 0, what the target says when it decodes one token at a time with plain attention."""
import pytest
import torch

from semi_ar_draft_gb300 import decode_round as D
from semi_ar_draft_gb300 import paged

pytestmark = pytest.mark.gpu

V, DIM, GAMMA, PROMPT = 512, 64, 4, 13


def plain_logits(target, tokens):
    """Logits after each of `tokens` (a list): full attention in 64 bits over the bf16 keys and values."""
    t = torch.tensor(tokens, device="cuda")
    x = target.embed[t] + target.place[: len(tokens)]
    n = len(tokens)
    hide = torch.ones((n, n), device="cuda").triu(1).bool()
    for w, p in zip(target.qkv, target.proj):
        h = torch.nn.functional.rms_norm(x, (x.shape[-1],))
        q, k, v = (h @ w).view(n, -1, target.D).split([target.Hq, target.Hk, target.Hk], dim=1)
        k, v = (y.double().repeat_interleave(target.Hq // target.Hk, 1) for y in (k, v))
        s = torch.einsum("nhd,lhd->hnl", q.double(), k) * target.D ** -0.5
        o = torch.einsum("hnl,lhd->nhd", torch.softmax(s.masked_fill(hide, float("-inf")), -1), v).to(torch.bfloat16)
        x = x + o.reshape(n, -1) @ p
    h = torch.nn.functional.rms_norm(x, (x.shape[-1],))
    return (h @ target.head).float()


def test_greedy_rounds_give_the_targets_tokens():
    target = D.ToyTarget(V, DIM, 2, 4, 2, 64, 256, seed=4)
    draft = D.ToyDraft(GAMMA, target)
    g = torch.Generator(device="cuda").manual_seed(8)
    B = 7
    prompts = torch.randint(0, V, (B, PROMPT), generator=g, device="cuda", dtype=torch.int32)
    out, mean, cache = D.generate(target, draft, prompts, 12, budget=B * 3, page_size=8, max_len=200)
    assert cache.status() == 0 and mean > 1.0
    lens = cache.cache_len.tolist()
    checked = 0
    for j in range(B):
        assert lens[j] == PROMPT + len(out[j]) - 1  # the last correction is not fed yet
        logits = plain_logits(target, prompts[j].tolist() + out[j][:-1])[PROMPT - 1:]
        for i, tok in enumerate(out[j]):
            best = logits[i].max()
            # the kernels round differently than the plain attention: a token may be another one whose logit is
            # within what bf16 activations (2^-8 each, over two layers and a head of std 3) and the bf16 logits
            # of the verification can move it
            assert float(best - logits[i, tok]) <= 2.0 ** -4 * max(1.0, float(best.abs())), (j, i)
            checked += int(logits[i].argmax()) == tok
    total = sum(map(len, out))
    assert checked >= 0.9 * total, (checked, total)  # and nearly all are the plain argmax itself


def test_rounds_do_not_lose_pages():
    target = D.ToyTarget(V, DIM, 1, 4, 1, 64, 256, seed=5)
    draft = D.ToyDraft(GAMMA, target)
    prompts = torch.randint(0, V, (5, 9), device="cuda", dtype=torch.int32)
    for kv in (None, torch.float8_e4m3fn):
        out, _, cache = D.generate(target, draft, prompts, 6, T=1.0, page_size=4, kv_dtype=kv, max_len=128)
        assert cache.status() == 0
        held = cache._blocks[0].tolist()
        assert held == [-(-n // 4) for n in cache.cache_len.tolist()]
        assert sum(held) + int(cache.n_free) == cache.free_pages.numel()
        cache.commit(None, done=torch.ones(5, dtype=torch.bool, device="cuda"))
        assert cache.status() == 0 and int(cache.n_free) == cache.free_pages.numel()
        assert sorted(cache.free_pages.tolist()) == list(range(cache.free_pages.numel()))


def test_cache_reports_a_full_pool():
    cache = paged.PagedCache(2, 3, 4, 8, 1, 1, 64, 40)
    cache.plan(torch.tensor([9, 9], dtype=torch.int32, device="cuda"))
    assert cache.status() == 8 and int(cache.n_free) == 0


def test_example_runs(capsys):
    D.main(["--requests", "4", "--rounds", "3"])
    assert "status 0" in capsys.readouterr().out
