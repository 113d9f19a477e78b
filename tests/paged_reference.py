"""Plain implementations of the paged-cache operators for the tests: whole numbers in Python, attention
in 64 bits from the definition, and the bound its result is held to."""
import math

import torch


def plan(cache_len, new_len, table, n_blocks, free, n_free, page, max_tokens, extra, num_pages):
    """Lists in, (seq_len, offsets, slots, positions, n_blocks, n_free, table, bad) out, every input clamped
    as the header says."""
    B, width = len(cache_len), len(table[0])
    table = [list(r) for r in table]
    left = min(max(n_free, 0), num_pages)
    bad = left != n_free
    seq, offsets, slots, positions, held = [], [0], [], [], []
    for j in range(B):
        old = max(cache_len[j], 0)
        n = max(new_len[j] + extra, 0)
        have = min(max(n_blocks[j], 0), width)
        want = -(-(old + n) // page)
        bad |= cache_len[j] < 0 or new_len[j] + extra < 0 or have != n_blocks[j] or want > width
        for blk in range(have, min(want, width)):
            if left == 0:
                bad = True
                break
            left -= 1
            table[j][blk] = free[left]
            have += 1
        for pos in range(old, old + n):
            blk = pos // page
            p = table[j][blk] if blk < have else -1
            slots.append(p * page + pos % page if 0 <= p < num_pages else -1)
            positions.append(pos)
        seq.append(old + n)
        offsets.append(offsets[-1] + n)
        held.append(have)
    bad |= len(slots) > max_tokens
    pad = max_tokens - len(slots)
    return (seq, offsets, (slots + [-1] * pad)[:max_tokens], (positions + [-1] * pad)[:max_tokens], held, left, table, bad)


def commit(cache_len, add_len, table, n_blocks, free, n_free, page, extra, done, num_pages):
    """(cache_len, n_blocks, n_free, free, bad)."""
    free = list(free)
    top = min(max(n_free, 0), num_pages)
    bad = top != n_free
    length, held = [], []
    for j in range(len(cache_len)):
        have = min(max(n_blocks[j], 0), len(table[0]))
        bad |= have != n_blocks[j]
        n = 0 if done[j] else cache_len[j] + add_len[j] + extra
        bad |= n < 0 or n > have * page
        n = min(max(n, 0), have * page)
        keep = -(-n // page)
        for blk in range(keep, have):
            if top == num_pages:
                bad = True
                break
            free[top] = table[j][blk]
            top += 1
        length.append(n)
        held.append(keep)
    return length, held, top, free, bad


def attention(q, k_pages, v_pages, table, seq_len, offsets, scale, causal, window, softcap, k_scale=None, v_scale=None):
    """out [T, Hq, D], lse [T, Hq] in float64 and the bounds (out, lse) of what the kernels may differ by.

    With u = finfo.eps / 2 of the 16-bit types: the output is rounded once (u |o|) and the probabilities
    once (u_p sum p |v|; halves with an 8-bit cache).  A score is a sum of D products in fp32, each step
    off by at most 2^-23 of the sum of magnitudes, then scaled and capped (8 roundings of its value, and
    1e-6 c for the tanh); an error d of the scores changes out by at most 2 d sum p |v| and lse by d.  The
    hardware exponential and logarithm are within 2^-21 and the fp32 sums over N keys, taken by 16 lanes
    and joined, within (N / 16 + 400) 2^-24."""
    T, Hq, D = q.shape
    page, Hk = k_pages.shape[1], k_pages.shape[2]
    G = Hq // Hk
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=q.device)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    u = torch.finfo(q.dtype).eps / 2
    u_p = 2.0 ** -11 if k_pages.dtype == torch.float8_e4m3fn else u
    ks = k_scale.double() if k_scale is not None else torch.ones(Hk, dtype=torch.float64, device=q.device)
    vs = v_scale.double() if v_scale is not None else torch.ones(Hk, dtype=torch.float64, device=q.device)
    for j, seq in enumerate(seq_len):
        a, b = offsets[j], offsets[j + 1]
        for i in range(b - a):
            pos = seq - (b - a) + i
            lo = max(pos - window + 1, 0) if window else 0
            hi = min(pos + 1, seq) if causal else seq
            if hi <= lo:
                continue
            l = torch.arange(lo, hi, device=q.device)
            pages = table[j].long()[l // page]
            for h in range(Hq):
                k = k_pages[pages, l % page, h // G].double() * ks[h // G]
                v = v_pages[pages, l % page, h // G].double() * vs[h // G]
                x = q[a + i, h].double()
                s = (k @ x) * scale
                mag = (k.abs() @ x.abs()) * abs(scale)
                if softcap:
                    s = softcap * torch.tanh(s / softcap)
                ls = torch.logsumexp(s, 0)
                p = torch.exp(s - ls)
                o = p @ v
                out[a + i, h], lse[a + i, h] = o, ls
                d = float((D * mag * 2.0 ** -23 + 8 * s.abs() * 2.0 ** -24).max()) + 1e-6 * softcap + 2.0 ** -21
                n = (hi - lo) / 16 + 400
                away = p @ v.abs()
                tol[a + i, h] = u * (o.abs() + 2 * u_p * away) + away * (u_p + 2 * d + 2 * n * 2.0 ** -24)
                tol_lse[a + i, h] = d + n * 2.0 ** -24 + abs(float(ls)) * 2.0 ** -22
    if q.dtype == torch.float16:
        tol += 2.0 ** -25  # half a step of the subnormal halves
    return out, lse, tol, tol_lse
