"""What int8 attention may be off by, kernel by kernel, and which kernel a call takes."""
import math

import torch

import i8_reference as R


def kernel_of(c, max_new):
    """The kernel of a call: "few" (row tiles of 8), "rows" (of 16) or "wide" (of 128), as the library decides by the rows of
    a request and kv head."""
    q, Hk = c["q"], c["codes"][0].shape[2]
    T, Hq, D = q.shape
    G, B, limit = Hq // Hk, len(c["seq"]), 31 if D <= 128 else 32
    aligned = q.data_ptr() % 16 == 0 and q.stride(0) % 8 == 0 and q.stride(1) % 8 == 0
    if G * T > limit * B and (max_new <= 0 or G * max_new > limit):
        return "wide" if aligned else "rows"
    return "few" if G * T <= 8 * B or 0 < G * max_new <= 8 else "rows"


def attention(c, lens, offsets, kernel, scale=None, causal=True, window=0, softcap=0.0):
    """out [T, Hq, D], lse [T, Hq] in 64 bits and the bounds (out, lse) of what `kernel` may differ by.

    With u = finfo.eps / 2: the output is rounded once (u |o|), a weight once (u_p sum p |v|; halves, "wide": q's type).
    "wide" sums D products of a score in fp32, each step off by at most 2^-23 of sum |q||c| 2^e.  The other two add
    (c + 128) q to a sum that begins at -128 sum q, and so pass sums of up to sum |q|(|c| + 128): D steps, and one for the
    beginning, each off by at most 2^-23 of that.  Then a score is scaled and capped (8 roundings of its value, and 2e-6
    of it for the tanh).  An exponent is the score less its row's reference, at most 2^-24 of a difference whose weight is
    2^-difference, plus the value's exponent less the difference of both references: four roundings at magnitudes of at
    most |e| + 32, whatever the score.  An error d of the exponents changes out by at most 2 d sum p |v| and lse by d.  The
    hardware exponential and logarithm are within 2^-21 and the fp32 sums over N keys, taken by 16 lanes and joined, within
    (N / 16 + 400) 2^-24.  A weight below 2^-21 of the largest is a subnormal half, off by at most 2^-32 of the largest
    weight, times 127; in "wide" with fp16 so is a probability, times its value."""
    q, codes, exps = c["q"], c["codes"], c["exps"]
    T, Hq, D = q.shape
    P, page, Hk, _ = codes[0].shape
    G, dtype, dev, wide = Hq // Hk, q.dtype, q.device, kernel == "wide"
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=dev)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=dev)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    u = torch.finfo(dtype).eps / 2
    u_p = u if wide else 2.0 ** -11
    K, V = R.values(codes[0], exps[0], dtype), R.values(codes[1], exps[1], dtype)
    block = page // exps[0].shape[2]
    ke, ve = (R.exponents(x, dtype).repeat_interleave(block, 2).transpose(1, 2) for x in exps)  # [P, page, Hk]
    for j, seq in enumerate(lens):
        a, b = offsets[j], offsets[j + 1]
        n = b - a
        if n == 0 or seq == 0:
            continue
        l = torch.arange(seq, device=dev)
        pages = c["table"][j].long()[l // page].clamp(0, P - 1)
        pos = torch.arange(seq - n, seq, device=dev)[:, None]
        see = torch.ones((n, seq), dtype=torch.bool, device=dev)
        if causal:
            see &= l <= pos
        if window:
            see &= l > pos - window
        for h in range(Hk):
            k, v, e = K[pages, l % page, h], V[pages, l % page, h], ve[pages, l % page, h]
            x = q[a:b, h * G:(h + 1) * G].double()  # [n, G, D]
            s = torch.einsum("ngd,ld->ngl", x, k) * scale
            mag = torch.einsum("ngd,ld->ngl", x.abs(), k.abs()) * abs(scale)
            if not wide:
                mag = mag + 128 * x.abs().sum(-1, keepdim=True) * R.two_to(ke[pages, l % page, h]) * abs(scale)
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            z = s.masked_fill(~see[:, None], -math.inf)
            ls = torch.logsumexp(z, -1)
            dead = ls == -math.inf
            p = torch.where(dead[..., None], 0.0, torch.exp(z - torch.where(dead, 0.0, ls)[..., None]))
            o, away = torch.einsum("ngl,ld->ngd", p, v), torch.einsum("ngl,ld->ngd", p, v.abs())
            err = (D + 1) * mag * 2.0 ** -23 + (8 * 2.0 ** -24 + (2e-6 if softcap else 0)) * s.abs() + 2.0 ** -21
            d_lse = torch.where(see[:, None], err, 0.0).amax(-1)  # [n, G]
            d = d_lse + torch.where(see, 4 * (e.abs() + 32) * 2.0 ** -24, 0.0).amax(-1)[:, None]
            N = see.sum(-1)[:, None] / 16 + 400
            w = p * R.two_to(e.long())
            top = w.amax(-1, keepdim=True)
            tiny = 127 * 2.0 ** -32 * top[..., 0] * ((w < 2.0 ** -21 * top) & see[:, None]).sum(-1)
            if wide and dtype == torch.float16:
                most = p.amax(-1, keepdim=True)
                small = ((p < 2.0 ** -21 * most) & see[:, None]).double()
                away_tiny = 2.0 ** -32 * most * torch.einsum("ngl,ld->ngd", small, v.abs())
            else:
                away_tiny = 0.0
            rows = slice(h * G, (h + 1) * G)
            out[a:b, rows], lse[a:b, rows] = o, ls
            tol[a:b, rows] = (u * (o.abs() + 2 * u_p * away) + away * (u_p + 2 * d + 2 * N * 2.0 ** -24)[..., None]
                              + tiny[..., None] + away_tiny)
            tol_lse[a:b, rows] = d_lse + N * 2.0 ** -24 + torch.where(dead, 0.0, ls).abs() * 2.0 ** -22
    if dtype == torch.float16:
        tol += 2.0 ** -25  # half a step of the subnormal halves
    return out, lse, tol, tol_lse


def compare(out, lse, want):
    """Outputs against attention()'s."""
    ro, rl, to, tl = want
    dead = rl == -math.inf
    assert torch.equal(lse == -math.inf, dead) and not out[dead].any()
    err = (out.double() - ro).abs()
    assert bool((err <= to).all()), f"out: {float((err - to).max())} past the bound, worst {float(err.max())}"
    el = (lse.double() - rl).abs()[~dead]
    assert bool((el <= tl[~dead]).all()), f"lse: worst {float(el.max())}"
