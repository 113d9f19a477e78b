"""Semi-autoregressive decoding rounds on one GPU, end to end: a draft block, the verify lengths, the target's
pass over the flattened verify tokens on a paged cache, the verification, and the cache's commit.

    python -m semi_ar_draft_gb300.decode_round [--requests 32] [--rounds 16] [--e4m3]

The target here is a toy: two attention layers with random weights (the operators of the library do the
drafting, scheduling, cache, attention and verification; torch does the projections).  Its purpose is the flow: every
length stays on the device, and with temperature 0 the tokens are those of decoding one by one."""
from __future__ import annotations

import argparse

import torch

from . import api
from .paged import PagedCache


class ToyTarget:
    """layers x (causal attention + projection) over token and position embeddings; fp32 logits over V ids."""

    def __init__(self, V, d, layers, Hq, Hk, D, max_len, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s, std: (torch.randn(s, generator=g, device=device) * std).to(torch.bfloat16)  # noqa: E731
        self.Hq, self.Hk, self.D = Hq, Hk, D
        self.embed, self.place = rnd(V, d, std=1.0), rnd(max_len, d, std=0.2)
        self.qkv = [rnd(d, (Hq + 2 * Hk) * D, std=d ** -0.5) for _ in range(layers)]
        self.proj = [rnd(Hq * D, d, std=0.5 * (Hq * D) ** -0.5) for _ in range(layers)]
        self.head = rnd(d, V, std=3.0 * d ** -0.5)

    def places(self, positions):
        """The positions' embeddings; -1 (padding) and what lies past the table read its first and last row."""
        return self.place[positions.long().clamp(0, len(self.place) - 1)]

    def forward(self, tokens, positions, cache):
        """Logits [T, V] fp32 of the planned tokens, whose keys and values go into the cache."""
        x = self.embed[tokens] + self.places(positions)
        for layer, (w, p) in enumerate(zip(self.qkv, self.proj)):
            h = torch.nn.functional.rms_norm(x, (x.shape[-1],))
            qkv = (h @ w).view(len(tokens), self.Hq + 2 * self.Hk, self.D)
            q, k, v = qkv.split([self.Hq, self.Hk, self.Hk], dim=1)
            cache.append(layer, k, v)
            o, _ = cache.attend(layer, q)
            x = x + o.reshape(len(tokens), -1) @ p
        return (torch.nn.functional.rms_norm(x, (x.shape[-1],)) @ self.head).float()


class ToyDraft:
    """The target without its attention: a Markov head with W1 = the normalised embeddings and W2 = the target's
    head, over flat base logits, and falling confidences."""

    def __init__(self, gamma, target):
        self.gamma = gamma
        self.W1 = torch.nn.functional.rms_norm(target.embed, (target.embed.shape[1],)).contiguous()
        self.W2 = target.head.T.contiguous()

    def block(self, B):
        base = torch.zeros((B, self.gamma, len(self.W1)), dtype=self.W1.dtype, device=self.W1.device)
        return base, 0.95 ** torch.arange(1.0, self.gamma + 1, device=base.device).expand(B, -1).contiguous()


def generate(target, draft, prompts, rounds, T=0.0, budget=None, page_size=16, kv_dtype=None, seed=0, max_len=512):
    """prompts [B, n] int32 on the device.  Returns (per request the tokens emitted in `rounds` rounds, the mean
    number of tokens a round, the cache).  A round adds up to gamma + 1 tokens to a request: ValueError if a request
    could outgrow max_len or the target's positions."""
    B, n = prompts.shape
    dev, gamma = prompts.device, draft.gamma
    longest = n + rounds * (gamma + 1)
    if longest > min(max_len, len(target.place)):
        raise ValueError(f"a request may grow to {longest} tokens; the cache holds {max_len}, the target places {len(target.place)}")
    budget = budget or B * gamma
    most = max(budget + B, B * n)
    blocks = -(-max_len // page_size)
    cache = PagedCache(B, B * blocks, page_size, blocks, len(target.qkv), target.Hk, target.D, most, kv_dtype=kv_dtype, device=dev)
    rows = torch.arange(most, device=dev)

    def flat(table):  # table [B, width]: the planned tokens' values, request by request
        t = rows[: len(cache.slots)]
        j = torch.searchsorted(cache.offsets[1:], t, right=True).clamp(max=B - 1)
        i = (t - cache.offsets[j]).clamp(0, table.shape[1] - 1)
        return table[j, i].long()

    # the prompts, whose last position gives the first token
    cache.plan(None, extra=n, max_new=n, tokens=B * n)
    logits = target.forward(flat(prompts), cache.positions, cache)
    anchor = logits[(cache.offsets[1:] - 1).long()].argmax(-1).int()
    cache.commit(None, extra=n)
    emitted = [anchor.tolist()]
    counts = []
    for r in range(rounds):
        base, conf = draft.block(B)
        tok, lse, zat, _ = api.markov_sample_block(base, draft.W1, draft.W2, anchor, T, seed + r)
        L, _, _, _ = api.schedule_verify_len(conf, budget)
        cache.plan(L, extra=1, max_new=gamma + 1, tokens=budget + B)
        logits = target.forward(flat(torch.cat([anchor[:, None], tok], 1)), cache.positions, cache)
        # draft logits are bf16, so the target's are rounded to it for the verification
        n_acc, corr, _ = api.verify(base, draft.W1, draft.W2, anchor, tok, lse, zat, logits.to(base.dtype), T, seed + r,
                                    verify_len=L, target_row_offsets=cache.offsets)
        cache.commit(n_acc, extra=1)
        emitted.append((tok.tolist(), n_acc.tolist(), corr.tolist()))
        counts.append(n_acc.float().mean() + 1)
        anchor = corr
    out = [[t] for t in emitted[0]]
    for tok, n_acc, corr in emitted[1:]:
        for j in range(B):
            out[j] += tok[j][: n_acc[j]] + [corr[j]]
    return out, float(torch.stack(counts).mean()) if counts else 0.0, cache


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--requests", type=int, default=32)
    ap.add_argument("--rounds", type=int, default=16)
    ap.add_argument("--e4m3", action="store_true", help="an 8-bit cache")
    a = ap.parse_args(argv)
    V, d, gamma, n = 4096, 64, 8, 24
    max_len = max(512, n + a.rounds * (gamma + 1))
    target = ToyTarget(V, d, 2, 8, 2, 64, max_len)
    draft = ToyDraft(gamma, target)
    g = torch.Generator(device="cuda").manual_seed(3)
    prompts = torch.randint(0, V, (a.requests, n), generator=g, device="cuda", dtype=torch.int32)
    out, mean, cache = generate(target, draft, prompts, a.rounds, budget=a.requests * gamma // 2, max_len=max_len,
                                kv_dtype=torch.float8_e4m3fn if a.e4m3 else None)
    print(f"{a.requests} requests, {a.rounds} rounds: {mean:.2f} tokens a request and round "
          f"({sum(map(len, out))} in all), cache status {cache.status()}, {int(cache.n_free)} pages free")
    print("request 0:", " ".join(map(str, out[0][:16])))


if __name__ == "__main__":
    main()
