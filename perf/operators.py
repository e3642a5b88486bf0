"""Cases of the linear-attention and 4-bit projection operators, with their
plain forms.

Three operators:

  step     M tokens of linear attention with a decay for each head, for B
           sequences; M = 1 is a decode step, M > 1 the verification of drafted
           tokens, with or without the state after every token kept:
               S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
  prefill  the same recurrence over whole prompts, some batches padded;
  q4       y = x W^T with W in 4 bits (two's complement, element 2j in the low
           half of byte j) and one fp16 scale per group of a row.

Shapes are those of the layer that the library serves: kh key heads shared by
vh value heads of 128 x 128 states, 2 kh 128 + vh 128 projected channels.
"""

import math

import torch

own = False

D = 128


# ------------------------------------------------------------------- cases

def _step(name, B, kh, vh, M, dtype, decay, ckpt=False):
    return {"name": name, "op": "step", "B": B, "kh": kh, "vh": vh, "M": M,
            "dtype": dtype, "decay": decay, "ckpt": ckpt}


def _prefill(name, B, kh, vh, T, dtype, decay, ragged=False):
    return {"name": name, "op": "prefill", "B": B, "kh": kh, "vh": vh, "T": T,
            "dtype": dtype, "decay": decay, "ragged": ragged}


def _q4(name, rows, N, K, group, dtype):
    return {"name": name, "op": "q4", "rows": rows, "N": N, "K": K,
            "group": group, "dtype": dtype}


def listed():
    return [
        # one user decoding: 48 heads, latency counts
        _step("step_1seq", 1, 16, 48, 1, "fp32", "head"),
        # a full decode batch; 201 MB of state, bound by HBM
        _step("step_64seq", 64, 16, 48, 1, "bf16", "token"),
        # verification of four drafted tokens with the states kept for rollback
        _step("verify_ckpt", 16, 16, 48, 4, "fp32", "token", True),
        # eight drafted tokens without checkpoints, as many key as value heads
        _step("verify_8tok", 27, 32, 32, 8, "bf16", "head"),
        # a batch of long prompts in the library's own precision
        _prefill("prompt_fp32", 8, 16, 48, 4096, "fp32", "token"),
        # the same batch as a served model holds it
        _prefill("prompt_bf16", 8, 16, 48, 4096, "bf16", "token"),
        # one very long prompt: too few heads to fill the GPU one by one
        _prefill("one_long", 1, 2, 8, 32701, "bf16", "head"),
        # many short prompts of different lengths in one padded batch
        _prefill("padded_short", 33, 16, 48, 111, "fp32", "head", True),
        # the gates' projection of one token: the smallest weight of the layer
        _q4("gates_1row", 1, 48, 5120, 32, "fp32"),
        # the layer's in-projection for one token
        _q4("in_proj_1row", 1, 10240, 5120, 128, "bf16"),
        # the same for eight drafted tokens
        _q4("in_proj_8row", 8, 10240, 5120, 128, "fp32"),
        # the out-projection of a decode batch
        _q4("out_proj_64row", 64, 5120, 6144, 64, "bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "prefill", "q4"])
    dtype = rng.choice(["fp32", "bf16"])
    if op == "q4":
        group = rng.choice([32, 64, 128])
        K = group * _log(rng, 1, 8192 // group)
        return {"op": op, "rows": _log(rng, 1, 64), "N": _log(rng, 1, 16384),
                "K": K, "group": group, "dtype": dtype}
    kh = rng.choice([1, 2, 3, 4, 8, 16])
    vh = kh * rng.choice([1, 2, 3, 4])
    decay = rng.choice(["head", "token"])
    if op == "step":
        M = rng.choice([1, 1, 1, 2, 3, 4, 5, 8])
        ckpt = M > 1 and rng.random() < 0.5
        B = _log(rng, 1, max(1, min(64, 4096 // (vh * (M if ckpt else 1)))))
        return {"op": op, "B": B, "kh": kh, "vh": vh, "M": M, "dtype": dtype,
                "decay": decay, "ckpt": ckpt}
    T = _log(rng, 1, 16384)
    B = _log(rng, 1, max(1, min(64, (1 << 20) // (T * vh))))
    return {"op": op, "B": B, "kh": kh, "vh": vh, "T": T, "dtype": dtype,
            "decay": decay, "ragged": B > 1 and rng.random() < 0.4}


# ------------------------------------------------------------------ inputs

_TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


def _inputs(case, seed):
    """The tensors of a case, from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFF)
    dt = _TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if case["op"] == "q4":
        rows, N, K, G = case["rows"], case["N"], case["K"], case["group"]
        # int4 codes of a rounded normal weight, scales around 1/(4 sqrt K)
        qw = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda",
                           dtype=torch.uint8)
        s = torch.exp(0.3 * normal(N, K // G)) / (4.0 * math.sqrt(K))
        return {"x": normal(rows, K).to(dt), "qw": qw, "scales": s.half(),
                "y": torch.empty(rows, N, device="cuda", dtype=dt)}
    B, kh, vh = case["B"], case["kh"], case["vh"]
    n = case["M"] if case["op"] == "step" else case["T"]

    def unit(x):
        return x / x.norm(dim=-1, keepdim=True)

    d = {"S": 0.02 * normal(B, vh, D, D), "q": unit(normal(B, n, kh, D)).to(dt),
         "k": unit(normal(B, n, kh, D)).to(dt), "v": normal(B, n, vh, D).to(dt),
         "scale": 1.0}
    if case["decay"] == "head":  # slopes from 1/2 down to 1/256, by head
        h = torch.arange(1, vh + 1, device="cuda", dtype=torch.float32)
        d["g"] = -torch.exp2(-8.0 * h / vh)
    else:  # data dependent, from none to a factor of e per token
        d["g"] = -0.1 * torch.nn.functional.softplus(2.0 * normal(B, n, vh))
    if case["op"] == "step":
        d["ckpt"] = torch.empty(n, B, vh, D, D, device="cuda") if case["ckpt"] else None
        d["o"] = torch.empty_like(d["v"])
    else:
        d["lens"] = None
        if case["ragged"]:
            d["lens"] = torch.randint(0, n + 1, (B,), generator=gen,
                                      device="cuda", dtype=torch.int32)
        # rows behind a prompt's end stay as they were
        d["o"] = torch.zeros_like(d["v"])
    return d


def prepare(case, seed):
    d = _inputs(case, seed)
    d["op"] = case["op"]
    if own and case["op"] == "prefill":
        import gated_deltanet_linear_gb300 as gdn
        n = gdn.gdn_linattn_prefill_workspace(case["B"], case["kh"], case["vh"],
                                              case["T"], dtype=d["q"].dtype)
        d["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return d


# ------------------------------------------------------------- plain forms

def _chunked(S, q, k, v, g, scale, C):
    """Chunks of C tokens: the states at the chunks' starts by one weighted
    sum over the earlier chunks, then each chunk for itself.  S [B][vh][D][D],
    q, k, v [B][vh][n C][D] in fp32, g [B][vh][n C] in fp64.  Returns o and
    the state at the end."""
    B, H, T, _ = v.shape
    n = T // C
    q, k, v = (t.view(B, H, n, C, D) for t in (q, k, v))
    G = g.view(B, H, n, C).cumsum(-1)               # decay from the chunk's start
    W = torch.cat([torch.zeros_like(G[..., :1, 0]), G[..., -1].cumsum(-1)], -1)
    end = torch.exp(G[..., -1:] - G).float()        # decay to the chunk's end
    local = (k * end[..., None]).transpose(-1, -2) @ v          # [B][H][n][D][D]
    hop = torch.exp((W[..., :, None] - W[..., None, 1:])
                    .masked_fill(~torch.ones(n + 1, n, device=v.device, dtype=torch.bool).tril(-1),
                                 -math.inf)).float()            # chunk j's sum at chunk i's start
    states = (hop @ local.view(B, H, n, D * D)).view(B, H, n + 1, D, D)
    states += torch.exp(W).float()[..., None, None] * S[:, :, None]
    mask = torch.ones(C, C, device=v.device, dtype=torch.bool).tril()
    L = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~mask, -math.inf)).float()
    o = torch.exp(G).float()[..., None] * (q @ states[:, :, :-1])
    o = (o + (L * (q @ k.transpose(-1, -2))) @ v) * scale
    return o.view(B, H, T, D), states[:, :, -1]


def _heads(t, rep):
    """[B][T][heads][D] as fp32 [B][heads * rep][T][D]."""
    return t.float().transpose(1, 2).repeat_interleave(rep, 1)


def _decay(s, B, n, vh):
    g = s["g"].double()
    return g[None, :, None].expand(B, vh, n) if g.dim() == 1 else g.transpose(1, 2)


def _plain_step(s):
    B, n, vh, _ = s["v"].shape
    rep = vh // s["q"].shape[2]
    q, k, v = _heads(s["q"], rep), _heads(s["k"], rep), _heads(s["v"], 1)
    S, g = s["S"], _decay(s, B, n, vh)
    if n == 1:
        S.mul_(torch.exp(g).float()[..., None]).add_(k.transpose(-1, -2) * v)
        o = (q @ S) * s["scale"]
        s["o"].copy_(o.transpose(1, 2))
        return
    G = g.cumsum(-1)
    mask = torch.ones(n, n, device=v.device, dtype=torch.bool).tril()
    L = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~mask, -math.inf)).float()
    A = torch.exp(G).float()
    o = A[..., None] * (q @ S) + (L * (q @ k.transpose(-1, -2))) @ v
    s["o"].copy_((o * s["scale"]).transpose(1, 2))
    if s["ckpt"] is not None:
        kv = (k[..., :, None] * v[..., None, :]).view(B, vh, n, D * D)
        every = (L @ kv).view(B, vh, n, D, D) + A[..., None, None] * S[:, :, None]
        s["ckpt"].copy_(every.permute(2, 0, 1, 3, 4))
        S.copy_(every[:, :, -1])
    else:
        S.mul_(A[..., -1, None, None]).add_((k * L[..., -1, :, None]).transpose(-1, -2) @ v)


def _plain_prefill(s):
    B, T, vh, _ = s["v"].shape
    rep = vh // s["q"].shape[2]
    C = 64
    pad = -T % C

    def padded(t):
        return torch.nn.functional.pad(t, (0, 0, 0, pad))

    q, k, v = _heads(s["q"], rep), _heads(s["k"], rep), _heads(s["v"], 1)
    g = torch.nn.functional.pad(_decay(s, B, T, vh), (0, pad))
    if s["lens"] is not None:  # behind the end: no decay, nothing added
        keep = (torch.arange(T, device=v.device) < s["lens"][:, None])[:, None, :, None]
        k, v = k.masked_fill(~keep, 0.0), v.masked_fill(~keep, 0.0)
        g = g.masked_fill(~torch.nn.functional.pad(keep[..., 0], (0, pad)), 0.0)
    o, S = _chunked(s["S"], padded(q), padded(k), padded(v), g, s["scale"], C)
    o = o[:, :, :T].transpose(1, 2)
    if s["lens"] is not None:
        o = torch.where(keep.transpose(1, 2), o, s["o"].float())
    s["o"].copy_(o)
    s["S"].copy_(S)


def _plain_q4(s):
    qw, sc = s["qw"], s["scales"]
    N, K = qw.shape[0], 2 * qw.shape[1]
    codes = torch.stack([qw & 15, qw >> 4], -1).view(N, K).to(torch.int8)
    w = (((codes ^ 8) - 8).float().view(N, sc.shape[1], -1) * sc.float()[..., None]).view(N, K)
    s["y"].copy_(s["x"].float() @ w.t())


def run(s):
    if s["op"] == "q4":
        if own:
            import gated_deltanet_linear_gb300 as gdn
            gdn.gdn_quant_linear(s["x"], s["qw"], s["scales"], s["y"])
        else:
            _plain_q4(s)
        return s["y"]
    if s["op"] == "step":
        if own:
            import gated_deltanet_linear_gb300 as gdn
            gdn.gdn_linattn_step_m(s["S"], s["S"], s["ckpt"], s["q"], s["k"],
                                   s["v"], s["g"], s["o"], scale=s["scale"])
        else:
            _plain_step(s)
        return {"S": s["S"], "o": s["o"], "ckpt": s["ckpt"]}
    if own:
        import gated_deltanet_linear_gb300 as gdn
        gdn.gdn_linattn_prefill(s["S"], s["q"], s["k"], s["v"], s["g"], s["o"],
                                scale=s["scale"], lens=s["lens"],
                                workspace=s["workspace"])
    else:
        _plain_prefill(s)
    return {"S": s["S"], "o": s["o"]}


# -------------------------------------------------------------------- work

def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "q4":
        r, N, K, G = case["rows"], case["N"], case["K"], case["group"]
        return {"bytes": N * K // 2 + 2 * N * (K // G) + e * r * (K + N),
                "flops": 2 * r * N * K}
    B, kh, vh = case["B"], case["kh"], case["vh"]
    n = case["M"] if case["op"] == "step" else case["T"]
    # a padded batch holds half of its rows on the average
    tokens = B * n * (0.5 if case.get("ragged") else 1.0)
    g = 4 * vh * (tokens if case["decay"] == "token" else 1)
    states = 2 + (n if case.get("ckpt") else 0)
    return {"bytes": states * B * vh * D * D * 4 + tokens * 2 * D * (kh + vh) * e + g,
            # S = a S + k v^T and S^T q: a multiply and two multiply-adds
            "flops": 5 * D * D * vh * tokens}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """Token by token (the product for q4), in fp64."""
    s = _inputs(case, seed)
    if case["op"] == "q4":
        low = s["qw"].to(torch.int32) & 15
        high = (s["qw"].to(torch.int32) >> 4) & 15
        w = torch.stack([low, high], 2).reshape(case["N"], case["K"])
        w = torch.where(w >= 8, w - 16, w).double()
        w = w * s["scales"].double().repeat_interleave(case["group"], 1)
        return torch.einsum("rk,nk->rn", s["x"].double(), w)
    rep = case["vh"] // case["kh"]
    S, g = s["S"].double(), s["g"].double()
    n = s["v"].shape[1]
    if n * S.numel() > 1.2e12:
        return None
    o = s["o"].double()
    states = []
    for t in range(n):
        a = torch.exp(g if g.dim() == 1 else g[:, t])
        q, k = (s[x][:, t].double().repeat_interleave(rep, 1) for x in "qk")
        v = s["v"][:, t].double()
        new = a.expand(S.shape[:2])[..., None, None] * S + k[..., :, None] * v[..., None, :]
        row = s["scale"] * torch.einsum("bhkv,bhk->bhv", new, q)
        if s.get("lens") is not None:
            on = (t < s["lens"])[:, None, None]
            row = torch.where(on, row, o[:, t])
            new = torch.where(on[..., None], new, S)
        S = new
        o[:, t] = row
        if s.get("ckpt") is not None:
            states.append(S)
    if case["op"] == "prefill":
        return {"S": S, "o": o}
    return {"S": S, "o": o, "ckpt": torch.stack(states) if case["ckpt"] else None}
