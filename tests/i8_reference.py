"""Plain implementations of the int8 paged cache for the tests: the format and the append from their definition, block by
block in 64 bits, and attention in 64 bits with the bound that the kernels are held to."""
import math

import torch

RANGE = {torch.bfloat16: (-126, 121), torch.float16: (-24, 9)}


def two_to(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def exponents(byte, dtype):
    return (byte.long() - 127).clamp(*RANGE[dtype])


def values(codes, exps, dtype):
    """The pool's values [P, page, Hk, D] in 64 bits."""
    P, page, Hk, D = codes.shape
    e = exponents(exps, dtype).repeat_interleave(page // exps.shape[2], 2)  # [P, Hk, page]
    return codes.double() * two_to(e).transpose(1, 2)[..., None]


def smallest_exponent(m, dtype):
    """The smallest e of the range with m <= 127 2^e, the last one if there is none."""
    lo, hi = RANGE[dtype]
    for e in range(lo, hi):
        if m <= 127 * 2.0 ** e:
            return e
    return hi


def append(x, codes, exps, slots):
    """One of k and v [T, Hk, D] into codes [P, page, Hk, D] and exps [P, Hk, page / block], in place (all on the host).
    Returns whether every value was finite."""
    P, page, Hk, D = codes.shape
    block, dtype = page // exps.shape[2], x.dtype
    of = {}
    for t, slot in enumerate(slots):
        if 0 <= slot < P * page:
            of.setdefault(slot // block, []).append((t, slot % block))
    fine = True
    for b, tokens in of.items():
        p, i0 = b * block // page, b * block % page
        mine = {at: t for t, at in tokens}  # (of two tokens of one slot the later one)
        for h in range(Hk):
            y = x[[t for t, _ in tokens], h].double()
            ok = torch.isfinite(y)
            fine &= bool(ok.all())
            e = smallest_exponent(float(y[ok].abs().max()) if bool(ok.any()) else 0.0, dtype)
            old = int(exponents(exps[p, h, i0 // block], dtype))
            if 0 not in mine:
                e = max(e, old)
                others = [i0 + at for at in range(block) if at not in mine]
                if e > old and others:
                    codes[p, others, h] = torch.round(codes[p, others, h].double() * 2.0 ** (old - e)).to(torch.int8)
            exps[p, h, i0 // block] = e + 127
            for at, t in mine.items():
                q = (x[t, h].double() * 2.0 ** -e).clamp(-127, 127)
                codes[p, i0 + at, h] = torch.round(torch.where(q.isnan(), 0.0, q)).to(torch.int8)
    return fine


def attention(q, codes, exps, table, seq_len, offsets, scale, causal, window, softcap, wide):
    """out [T, Hq, D], lse [T, Hq] in 64 bits, and the bounds (out, lse) of what a kernel may differ by; codes and exps of
    (k, v), wide: the call may go to the kernel of many rows, whose probabilities are of q's type, or to the other one, where
    they are halves (else only to that one).

    With u = finfo.eps / 2: the output is rounded once (u |o|), the probabilities once (u_p sum p |v|).  A score is a sum
    of D products in fp32, each step off by at most 2^-23 of the sum of magnitudes, then scaled and capped (8 roundings of
    its value, and 2e-6 of it for the tanh).  The weight of a value is 2^(s + e), whose exponent is rounded four times at a
    magnitude of at most |s| + |e| + 8, with s in the log2 domain.  An error d of the exponents changes out by at most 2 d
    sum p |v| and lse by d.  The hardware exponential and logarithm are within 2^-21 and the fp32 sums over N keys, taken
    by 16 lanes and joined, within (N / 16 + 400) 2^-24.  A weight below 2^-21 of the largest is a subnormal half, off by
    at most 2^-32 of the largest weight, times 127; in the kernel of many rows, where the values carry their scales, so is a
    probability (fp16), times its value."""
    T, Hq, D = q.shape
    P, page, Hk, _ = codes[0].shape
    G, dtype, dev = Hq // Hk, q.dtype, q.device
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=dev)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=dev)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    u = torch.finfo(dtype).eps / 2
    u_p = u if wide else 2.0 ** -11
    K, V = values(codes[0], exps[0], dtype), values(codes[1], exps[1], dtype)
    ve = exponents(exps[1], dtype).repeat_interleave(page // exps[1].shape[2], 2).transpose(1, 2)  # [P, page, Hk]
    for j, seq in enumerate(seq_len):
        a, b = offsets[j], offsets[j + 1]
        n = b - a
        if n == 0 or seq == 0:
            continue
        l = torch.arange(seq, device=dev)
        pages = table[j].long()[l // page].clamp(0, P - 1)  # (pages before a window may be gone)
        pos = torch.arange(seq - n, seq, device=dev)[:, None]
        see = torch.ones((n, seq), dtype=torch.bool, device=dev)
        if causal:
            see &= l <= pos
        if window:
            see &= l > pos - window
        for h in range(Hk):
            k, v, e = K[pages, l % page, h], V[pages, l % page, h], ve[pages, l % page, h].double()
            x = q[a:b, h * G:(h + 1) * G].double()  # [n, G, D]
            s = torch.einsum("ngd,ld->ngl", x, k) * scale
            mag = torch.einsum("ngd,ld->ngl", x.abs(), k.abs()) * abs(scale)
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            z = s.masked_fill(~see[:, None], -math.inf)
            ls = torch.logsumexp(z, -1)
            dead = ls == -math.inf
            p = torch.where(dead[..., None], 0.0, torch.exp(z - torch.where(dead, 0.0, ls)[..., None]))
            o, away = torch.einsum("ngl,ld->ngd", p, v), torch.einsum("ngl,ld->ngd", p, v.abs())
            err = D * mag * 2.0 ** -23 + 8 * s.abs() * 2.0 ** -24 + (2e-6 * s.abs() if softcap else 0) + 2.0 ** -21
            err = err + 4 * (1.5 * s.abs() + e.abs() + 8) * 2.0 ** -24
            d = torch.where(see[:, None], err, 0.0).amax(-1)  # [n, G]
            N = see.sum(-1)[:, None] / 16 + 400
            w = p * two_to(e.long())
            top = w.amax(-1, keepdim=True)
            tiny = 127 * 2.0 ** -32 * top[..., 0] * ((w < 2.0 ** -21 * top) & see[:, None]).sum(-1)
            if wide and dtype == torch.float16:  # 2^7 p / p_ref with p_ref within 2^-8 .. 1 of the largest, off by 2^-25
                most = p.amax(-1, keepdim=True)
                small = ((p < 2.0 ** -21 * most) & see[:, None]).double()
                away_tiny = 2.0 ** -32 * most * torch.einsum("ngl,ld->ngd", small, v.abs())
            else:
                away_tiny = 0.0
            rows = slice(h * G, (h + 1) * G)
            out[a:b, rows], lse[a:b, rows] = o, ls
            tol[a:b, rows] = (u * (o.abs() + 2 * u_p * away) + away * (u_p + 2 * d + 2 * N * 2.0 ** -24)[..., None]
                              + tiny[..., None] + away_tiny)
            tol_lse[a:b, rows] = d + N * 2.0 ** -24 + torch.where(dead, 0.0, ls).abs() * 2.0 ** -22
    if dtype == torch.float16:
        tol += 2.0 ** -25  # half a step of the subnormal halves
    return out, lse, tol, tol_lse
