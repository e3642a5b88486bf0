"""The attention layers' operators in 64 bits, and their test inputs.  Plain
torch on any device; nothing of the library is used."""

import math

import torch

KINDS = {"bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


def freqs(rot, base=10000.0, scaling="plain", factor=1.0, context=0.0, low=1.0, high=32.0):
    """Frequencies one by one, from the definition."""
    out = []
    for i in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if scaling == "ntk" else base
        f = math.exp(-2.0 * i / rot * math.log(b))
        if scaling == "linear":
            f /= factor
        if scaling == "band":
            turns = context * f / (2 * math.pi)
            part = min(1.0, max(0.0, (turns - low) / (high - low)))
            f = part * f + (1 - part) * f / factor
        out.append(f)
    return torch.tensor(out, dtype=torch.float64), (0.1 * math.log(factor) + 1 if scaling == "band" else 1.0)


def turn(x, pos, freq, pairs, amp):
    """x [..][heads][hd] at positions pos [..], in fp64."""
    x = x.double()
    n = freq.numel()
    ang = (pos.double()[..., None] * freq.to(x.device))[..., None, :]
    c, s = amp * torch.cos(ang), amp * torch.sin(ang)
    y = x.clone()
    i = torch.arange(n, device=x.device)
    a, b = (2 * i, 2 * i + 1) if pairs else (i, i + n)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def codes(x, kind):
    """(codes as fp64 numbers, scales fp32) of rows x (fp64 values)."""
    top = 127.0 if kind == "int8" else 448.0
    scale = (x.abs().amax(-1) / top).float()
    y = torch.where(scale[..., None] > 0, x / scale.double()[..., None], torch.zeros_like(x))
    if kind == "int8":
        return y.round(), scale
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    e = torch.where(torch.exp2(e) > y.abs().clamp(min=2.0 ** -6), e - 1, e)
    step = torch.exp2(e - 3)
    return (y / step).round() * step, scale


def make_cache(kind, pages, kvh, page, hd, gen, device, junk=True, spread=0.3):
    """Random codes and scales; everything a test does not fill itself is junk
    (NaN, infinities) until `fill` puts numbers there."""
    c = {}
    for x in "kv":
        t = torch.randn(pages, kvh, page, hd, generator=gen, device=device)
        if kind == "bf16":
            c[x], c[x + "s"] = t.bfloat16(), None
        else:
            c[x] = (t * 32).round().clamp(-127, 127).to(torch.int8) if kind == "int8" \
                else (t * 112).clamp(-448, 448).to(torch.float8_e4m3fn)
            s = torch.exp(spread * torch.randn(pages, kvh, page, generator=gen, device=device))
            c[x + "s"] = s / (32.0 if kind == "int8" else 112.0)
    return c


def make_table(pages, B, cols, gen, device):
    perm = torch.randperm(pages, generator=gen, device=device)[:B * cols]
    return perm.view(B, cols).int().contiguous()


def junk_behind(c, table, lens, page, kind):
    """Rows behind each sequence's end become NaN, table entries behind it
    numbers of no page."""
    for b, n in enumerate(lens):
        cols = -(-n // page)
        if n % page:
            at = int(table[b, cols - 1])
            for x in "kv":
                if kind == "bf16":
                    c[x][at, :, n % page:] = float("nan")
                else:
                    c[x + "s"][at, :, n % page:] = float("nan")
        table[b, cols:] = torch.where(torch.arange(table.shape[1] - cols, device=table.device) % 2 == 0,
                                      -5, 2 ** 31 - 1).int()


def held(c, x, table, b, n, page):
    """Positions 0 .. n - 1 of sequence b, [kvh][n][hd] in fp64."""
    at = table[b, :-(-n // page)].long()
    t = c[x][at].float().double()
    if c[x + "s"] is not None:
        t = t * c[x + "s"][at].double()[..., None]
    return t.permute(1, 0, 2, 3).reshape(t.shape[1], -1, t.shape[3])[:, :n]


def attn(c, table, start, counts, q, scale, page):
    """(o, lse, sums of p |v| and what is left out of them, the largest sum of |q k| scale) in fp64, for the
    rows that are there; the others are NaN."""
    B, M, qh, hd = q.shape
    nan = float("nan")
    o = torch.full((B, M, qh, hd), nan, dtype=torch.float64, device=q.device)
    mag, lse, big = o.clone(), o[..., 0].clone(), torch.zeros((B, M, qh), dtype=torch.float64, device=q.device)
    for b in range(B):
        m = M if counts is None else counts[b]
        if m == 0:
            continue
        k, v = (held(c, x, table, b, start[b] + m, page) for x in "kv")
        rep = qh // k.shape[0]
        for i in range(m):
            n = start[b] + i + 1
            x = q[b, i].double().view(k.shape[0], rep, hd)
            s = scale * x @ k[:, :n].transpose(1, 2)
            p = torch.softmax(s, -1)
            o[b, i] = (p @ v[:, :n]).reshape(qh, hd)
            # the formula's sums, and what 8-bit caches and fp32 cannot see: weights
            # end 2^-37 below the largest weight times its row (8 bits), and at 2^-126
            # of a row's (any): in units of 2^-21, the smallest bound they meet
            rowmax = v[:, None, :n].abs().amax(-1)
            floor = n * (2.0 ** -37 * (p * rowmax).amax(-1) * (c["ks"] is not None) + 2.0 ** -126 * rowmax.amax(-1))
            mag[b, i] = (p @ v[:, :n].abs() + 2.0 ** 21 * floor[..., None]).reshape(qh, hd)
            lse[b, i] = torch.logsumexp(s, -1).flatten()
            big[b, i] = (abs(scale) * x.abs() @ k[:, :n].abs().transpose(1, 2)).amax(-1).flatten()
    return o, lse, mag, big


def attn_bounds(kind, dtype, hd, T, o, lse, mag, big):
    """What o and lse may be off by.

    Scores: sums of hd / 16 products in fp32 (each step 2^-23 of the sum of
    magnitudes `big`), the operands' cut 2^-22, scales, factor and the base-2
    exponent's rounding 4 x 2^-23; ex2.approx 2^-22.  A weight's relative error
    is that of its score; it enters the sum and the normaliser: twice.  The
    weights' cut: 2^-21 (bf16 tokens: on a bf16 cache two 8-bit parts, 2^-16, on an 8-bit
    one a single fp16, 2^-11);
    sums of T / 16 products over 8 warps and at most a few parts, in fp32, and
    the joins: (T / 128 + 40) 2^-23.  bf16 results: half a step, 2^-8, once."""
    d = (hd / 16 + 6) * 2.0 ** -23 * big + 2.0 ** -22
    tol = 2 * d + (T / 128 + 40) * 2.0 ** -23 + 2.0 ** -21
    if kind == "bf16" and dtype == "bf16":
        tol = tol + 2.0 ** -16
    if kind != "bf16" and dtype == "bf16":
        tol = tol + 2.0 ** -11
    bo = tol[..., None] * mag
    if dtype == "bf16":
        bo = bo * (1 + 2.0 ** -8) + 2.0 ** -8 * o.abs()
    return bo, d + (T / 128 + 40) * 2.0 ** -23 + 2.0 ** -22 * lse.abs()
