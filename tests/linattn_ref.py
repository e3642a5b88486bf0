"""Plain 64-bit forms of the linear-attention and 4-bit projection operators,
with the magnitudes that bound a 32-bit evaluation's error (the same sums
over absolute values).  Test infrastructure only."""

import torch

D = 128


def linattn(S, q, k, v, g, scale=1.0, lens=None, states=False):
    """Token by token in fp64: returns o, the final S and (states) the state
    after every token, each with its magnitude, as a dict."""
    S, q, k, v, g = (t.double() for t in (S, q, k, v, g))
    B, n, vh, _ = v.shape
    rep = vh // q.shape[2]
    mS = S.abs()
    o, mo, every = torch.zeros_like(v), torch.zeros_like(v), []
    for t in range(n):
        a = torch.exp(g if g.dim() == 1 else g[:, t]).expand(B, vh)[..., None, None]
        qt, kt = (x[:, t].repeat_interleave(rep, 1) for x in (q, k))
        vt = v[:, t]
        new = a * S + kt[..., :, None] * vt[..., None, :]
        mag = a * mS + kt.abs()[..., :, None] * vt.abs()[..., None, :]
        if lens is not None:
            on = (t < lens.to(S.device))[:, None, None, None]
            new, mag = torch.where(on, new, S), torch.where(on, mag, mS)
        S, mS = new, mag
        o[:, t] = scale * (S * qt[..., :, None]).sum(2)
        mo[:, t] = abs(scale) * (mS * qt.abs()[..., :, None]).sum(2)
        if states:
            every.append(S)
    out = {"S": S, "mS": mS, "o": o, "mo": mo}
    if states:
        out["states"] = torch.stack(every)
    return out


def weights(qw, scales):
    """The fp64 matrix [N][K] of packed codes and group scales."""
    lo, hi = (qw & 15).to(torch.int64), (qw >> 4).to(torch.int64)
    c = torch.stack([lo, hi], -1).reshape(qw.shape[0], -1)
    c = torch.where(c > 7, c - 16, c).double()
    return c * scales.double().repeat_interleave(c.shape[1] // scales.shape[1], 1)


def quant_linear(x, qw, scales):
    w = weights(qw, scales)
    return x.double() @ w.t(), x.double().abs() @ w.abs().t()


def make_linattn(seed, B, n, kh, vh, dtype=torch.float32, decay="token",
                 device="cuda", strong=False):
    """Seeded inputs: unit q and k rows, N(0, 1) values, a state of the
    layer's size; decays per head (2^-8h/vh) or per token (mild, or strong:
    down to e^-60 a token)."""
    gen = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=gen)

    def unit(x):
        return x / x.norm(dim=-1, keepdim=True)

    if decay == "head":
        g = -torch.exp2(-8.0 * torch.arange(1, vh + 1) / vh)
    else:
        g = -torch.nn.functional.softplus(2 * normal(B, n, vh)) * (10.0 if strong else 0.1)
    d = {"S": 0.1 * normal(B, vh, D, D), "q": unit(normal(B, n, kh, D)).to(dtype),
         "k": unit(normal(B, n, kh, D)).to(dtype), "v": normal(B, n, vh, D).to(dtype),
         "g": g}
    return {x: t.to(device) for x, t in d.items()}


def make_quant(seed, rows, N, K, group, dtype=torch.float32, device="cuda"):
    gen = torch.Generator().manual_seed(seed)
    qw = torch.randint(0, 256, (N, K // 2), generator=gen, dtype=torch.uint8)
    sc = torch.exp(0.3 * torch.randn(N, K // group, generator=gen)) / (4 * K ** 0.5)
    x = torch.randn(rows, K, generator=gen).to(dtype)
    return tuple(t.to(device) for t in (x, qw, sc.half()))


def half_step(dtype):
    """Largest relative error of one rounding to a 16-bit type; 0 for fp32."""
    return 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2


def assert_within(got, ref, tol, what):
    """|got - ref| <= tol elementwise, non-finite values alike."""
    got = got.double()
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = int(bad.flatten().nonzero()[0])
        raise AssertionError(
            f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance, first at "
            f"{i}: {got.flatten()[i].item():.9g} for {ref.flatten()[i].item():.9g}, "
            f"allowed {tol.flatten()[i].item():.3g}")
