"""Cases of the attention layers' operators (rotary positions, the paged and
quantised key-value cache, attention of new tokens over it), with their plain
forms.

Four kinds of pass:

  rope   rows turned by their positions' angles, in pairs (i, i + rot / 2) or
         (2 i, 2 i + 1) of the first rot channels of a head;
  cache  M new tokens of B sequences: q and k turned, k and v rounded into the
         pages of the cache, and the new positions read back;
  read   positions of a cache that holds earlier tokens, as rows again;
  attn   M new tokens of B sequences against all positions of their own.

A cache is k, v [pages][kvh][page][hd] in bf16 or in 8 bits (int8, e4m3) with
one fp32 scale for each row; table [B][columns] names a sequence's pages.
"""

import math

import torch

own = False

# ------------------------------------------------------------------- cases


def _rope(name, rows, heads, hd, rot, layout, scaling, dtype, far):
    return {"name": name, "op": "rope", "rows": rows, "heads": heads, "hd": hd,
            "rot": rot, "layout": layout, "scaling": scaling, "dtype": dtype,
            "far": far}


def _cache(name, B, M, qh, kvh, hd, rot, layout, kind, page, dtype, ragged, far):
    return {"name": name, "op": "cache", "B": B, "M": M, "qh": qh, "kvh": kvh,
            "hd": hd, "rot": rot, "layout": layout, "scaling": "none",
            "kind": kind, "page": page, "dtype": dtype, "ragged": ragged,
            "far": far}


def _read(name, B, T, kvh, hd, kind, page, dtype, ragged):
    return {"name": name, "op": "read", "B": B, "T": T, "kvh": kvh, "hd": hd,
            "kind": kind, "page": page, "dtype": dtype, "ragged": ragged}


def _attn(name, B, M, T, qh, kvh, hd, kind, page, dtype, ragged):
    return {"name": name, "op": "attn", "B": B, "M": M, "T": T, "qh": qh,
            "kvh": kvh, "hd": hd, "kind": kind, "page": page, "dtype": dtype,
            "ragged": ragged}


def listed():
    return [
        # one user decoding behind a few thousand tokens: latency counts
        _attn("attn_1seq", 1, 1, 4099, 24, 4, 256, "int8", 64, "bf16", False),
        # a decode batch of all lengths up to 8192: 0.5 GB of cache
        _attn("attn_64seq", 64, 1, 8192, 32, 8, 128, "int8", 64, "bf16", True),
        # one very long sequence in the unquantised cache
        _attn("attn_long", 1, 1, 262001, 8, 2, 256, "bf16", 128, "bf16", False),
        # verification of four drafted tokens, in the library's own precision
        _attn("attn_verify", 16, 4, 8192, 24, 4, 256, "e4m3", 32, "fp32", True),
        # many short sequences, a key head for every query head, small pages
        _attn("attn_short", 33, 1, 300, 16, 16, 64, "bf16", 16, "fp32", True),
        # a decode batch's tokens into the cache, a quarter of the head turned
        _cache("cache_decode", 64, 1, 24, 4, 256, 64, "half", "int8", 64, "bf16", False, 1 << 18),
        # a padded batch of prompts
        _cache("cache_prompt", 8, 4096, 32, 8, 128, 128, "half", "e4m3", 64, "bf16", True, 4096),
        # an odd chunk of a few prompts, pairs side by side, small pages
        _cache("cache_chunk", 5, 333, 16, 4, 64, 32, "pairs", "bf16", 16, "fp32", True, 100000),
        # a cached prefix as rows, for a prompt that continues it
        _read("read_prefix", 1, 65531, 4, 256, "int8", 64, "bf16", False),
        # prefixes of several sequences in fp32
        _read("read_batch", 16, 1021, 8, 128, "e4m3", 16, "fp32", True),
        # the query heads of a decode batch, far out in a stretched context
        _rope("rope_decode", 64, 24, 256, 64, "half", "band", "fp32", 1 << 20),
        # the query heads of prompts, whole heads, pairs side by side
        _rope("rope_prompt", 32768, 32, 128, 128, "pairs", "linear", "bf16", 32768),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "cache", "read", "rope"])
    dtype = rng.choice(["fp32", "bf16"])
    hd = rng.choice([64, 128, 256])
    rot = 16 * rng.randint(1, hd // 16)
    layout = rng.choice(["half", "pairs"])
    if op == "rope":
        rows = _log(rng, 1, 32768)
        return {"op": op, "rows": rows,
                "heads": _log(rng, 1, max(1, min(48, (1 << 27) // (rows * hd)))),
                "hd": hd, "rot": rot, "layout": layout,
                "scaling": rng.choice(["none", "linear", "ntk", "band"]),
                "dtype": dtype, "far": _log(rng, 64, 1 << 20)}
    kvh = rng.choice([1, 2, 3, 4, 8])
    qh = kvh * rng.choice([1, 2, 3, 4, 5, 6, 8])
    kind = rng.choice(["bf16", "int8", "e4m3"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "cache":
        M = rng.choice([1, 2, 4, _log(rng, 1, 8192)])
        B = _log(rng, 1, max(1, min(64, (1 << 27) // (M * (qh + 2 * kvh) * hd))))
        return {"op": op, "B": B, "M": M, "qh": rng.choice([0, qh]), "kvh": kvh,
                "hd": hd, "rot": rng.choice([0, rot, rot]), "layout": layout,
                "scaling": rng.choice(["none", "linear", "ntk", "band"]),
                "kind": kind, "page": page, "dtype": dtype,
                "ragged": rng.random() < 0.5, "far": _log(rng, 64, 1 << 18)}
    T = _log(rng, 1, 65536)
    B = _log(rng, 1, max(1, min(64, (1 << 27) // (T * kvh * hd))))
    ragged = B > 1 and rng.random() < 0.6
    if op == "read":
        return {"op": op, "B": B, "T": T, "kvh": kvh, "hd": hd, "kind": kind,
                "page": page, "dtype": dtype, "ragged": ragged}
    return {"op": op, "B": B, "M": min(T, rng.choice([1, 1, 1, 2, 3, 4, 8])), "T": T,
            "qh": qh, "kvh": kvh, "hd": hd, "kind": kind, "page": page,
            "dtype": dtype, "ragged": ragged}


# ------------------------------------------------------------------ inputs

_TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
_KINDS = {"bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
# base, factor, context, low, high: a context of 8192 positions stretched by 16
_BASE, _FACTOR, _CONTEXT, _LOW, _HIGH = 1e6, 16.0, 8192.0, 1.0, 32.0


def _freqs(case):
    """Radians a position and the amplitude, in 64 bits on the host."""
    rot, scaling, base = case["rot"], case["scaling"], _BASE
    if scaling == "ntk":
        base = base * _FACTOR ** (rot / (rot - 2.0))
    f = base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    if scaling == "linear":
        f = f / _FACTOR
    if scaling == "band":
        w = ((_CONTEXT / (2.0 * math.pi) * f - _LOW) / (_HIGH - _LOW)).clamp(0.0, 1.0)
        f = f * (w + (1.0 - w) / _FACTOR)
        return f, 0.1 * math.log(_FACTOR) + 1.0
    return f, 1.0


def _pages(case, gen, most):
    """A cache with room for `most` positions of every sequence and a few
    pages more, and the table: pages in any order."""
    B, kvh, page, hd = case["B"], case["kvh"], case["page"], case["hd"]
    cols = -(-most // page)
    n = B * cols + 7
    every = torch.randperm(n, generator=gen, device="cuda")
    d = {"table": every[:B * cols].view(B, cols).int(), "spare": every[B * cols:]}
    for x in "kv":
        if case["op"] == "cache":
            d[x + "c"] = torch.zeros(n, kvh, page, hd, device="cuda", dtype=_KINDS[case["kind"]])
        else:
            t = torch.randn(n, kvh, page, hd, generator=gen, device="cuda", dtype=torch.bfloat16)
            if case["kind"] == "int8":
                t = (32.0 * t).round().clamp(-127, 127)
            if case["kind"] == "e4m3":
                t = (112.0 * t).clamp(-448, 448)
            d[x + "c"] = t.to(_KINDS[case["kind"]])
        d[x + "s"] = None
        if case["kind"] != "bf16":  # what rows of normal values have
            s = torch.exp(0.3 * torch.randn(n, kvh, page, generator=gen, device="cuda"))
            d[x + "s"] = s / (32.0 if case["kind"] == "int8" else 112.0)
    return d


def _inputs(case, seed):
    """The tensors of a case, from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFF)
    op, hd, dt = case["op"], case["hd"], _TYPES[case["dtype"]]

    def normal(*shape, dtype=dt):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)

    def whole(lo, hi, n):
        return torch.randint(lo, hi + 1, (n,), generator=gen, device="cuda", dtype=torch.int32)

    d = {}
    if case.get("rot"):
        f, d["amp"] = _freqs(case)
        d["freq"], d["layout"] = f.cuda(), case["layout"]
    if op == "rope":
        rows = case["rows"]
        d["x"] = normal(rows, case["heads"], hd)
        d["pos"] = whole(0, case["far"] - 1, rows)
        d["y"] = torch.empty_like(d["x"])
        return d
    B, kvh = case["B"], case["kvh"]
    d["counts"] = None
    if op == "cache":
        M, qh = case["M"], case["qh"]
        # positions of any sequence up to `far`; its pages hold the last ones
        d["start"] = whole(0, case["far"] - 1, B)
        first = (d["start"] // case["page"]).long()
        near = -(-(M + case["page"]) // case["page"])
        d.update(_pages(case, gen, near * case["page"]))
        cols = case["far"] // case["page"] + near + 1
        table = torch.full((B, cols), -1, device="cuda", dtype=torch.int32)
        at = first[:, None] + torch.arange(near, device="cuda")
        table.scatter_(1, at, d["table"][:, :near])
        d["table"] = table
        # the rows of a projection: q, k and v of a token side by side
        x = normal(B, M, (qh + 2 * kvh) * hd)
        d["q"] = x[..., :qh * hd].unflatten(-1, (qh, hd)) if qh else None
        d["k"] = x[..., qh * hd:(qh + kvh) * hd].unflatten(-1, (kvh, hd))
        d["v"] = x[..., (qh + kvh) * hd:].unflatten(-1, (kvh, hd))
        d["qo"] = torch.zeros(B, M, qh, hd, device="cuda", dtype=dt) if qh else None
        # read back in 16 bits: no more than 8 of them are in a cache
        d["ko"] = torch.zeros(B, M, kvh, hd, device="cuda", dtype=torch.bfloat16)
        d["vo"] = torch.zeros_like(d["ko"])
        if case["ragged"]:
            d["counts"] = whole(0, M, B)
        return d
    T = case["T"]
    d.update(_pages(case, gen, T))
    if op == "read":
        d["start"] = torch.zeros(B, device="cuda", dtype=torch.int32)
        if case["ragged"]:
            d["counts"] = whole(0, T, B)
        d["ko"] = torch.zeros(B, T, kvh, hd, device="cuda", dtype=dt)
        d["vo"] = torch.zeros_like(d["ko"])
        return d
    M = case["M"]
    d["start"] = whole(0, T - M, B) if case["ragged"] else torch.full_like(whole(0, 1, B), T - M)
    # queries of some weight: scores spread over several units
    d["q"] = normal(B, M, case["qh"], hd, dtype=torch.float32).mul_(2.0).to(dt)
    d["scale"] = hd ** -0.5
    d["o"] = torch.zeros_like(d["q"])
    d["lse"] = torch.zeros(B, M, case["qh"], device="cuda")
    return d


def prepare(case, seed):
    d = _inputs(case, seed)
    d["op"] = case["op"]
    if own:
        import gated_deltanet_linear_gb300 as gdn
        if "kc" in d:
            d["cache"] = gdn.KVCache(d["kc"], d["vc"], d["ks"], d["vs"])
        d["rope"] = None
        if "freq" in d:
            d["rope"] = gdn.Rope(d["freq"], gdn.GDN_ROPE_HALF if d["layout"] == "half"
                                 else gdn.GDN_ROPE_PAIRS, d["amp"])
        if case["op"] == "attn":
            n = gdn.gdn_attn_workspace(d["cache"], case["M"], case["qh"])
            d["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return d


# ------------------------------------------------------------- plain forms

def _turn(x, pos, s):
    """x [..][heads][hd] in fp32 at positions pos [..]."""
    if "freq" not in s:
        return x
    n = s["freq"].numel()
    a = pos.double()[..., None] * s["freq"]
    c, w = ((f(a) * s["amp"]).float()[..., None, :] for f in (torch.cos, torch.sin))
    y = x.clone()
    if s["layout"] == "half":
        p, q = x[..., :n], x[..., n:2 * n]
        y[..., :n], y[..., n:2 * n] = p * c - q * w, q * c + p * w
    else:
        p, q = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = p * c - q * w, q * c + p * w
    return y


def _plain_rope(s):
    s["y"].copy_(_turn(s["x"].float(), s["pos"], s))


def _places(s, T):
    """Page, row of the page and whether it is there, of the T positions from
    start on: [B][T] each.  What is not there goes to a page of nobody's."""
    t = torch.arange(T, device="cuda")
    pos = s["start"].long()[:, None] + t
    page = s["kc"].shape[2]
    col = (pos // page).clamp(max=s["table"].shape[1] - 1)
    at = s["table"].gather(1, col).long()
    if s["counts"] is None:
        return at, pos % page, None
    on = t < s["counts"][:, None]
    return torch.where(on, at, s["spare"][0]), pos % page, on


def _store(x, codes, scales, page, row):
    """x [B][M][kvh][hd] in fp32 into the rows of the cache."""
    at = (page[..., None], torch.arange(x.shape[2], device="cuda"), row[..., None])
    if scales is None:
        codes[at] = x.to(codes.dtype)
        return
    top = 127.0 if codes.dtype == torch.int8 else 448.0
    # (in 64 bits: which side of a border between two codes a value lies on)
    scale = (x.abs().amax(-1).double() / top).float()
    y = (x.double() / scale.double()[..., None]).clamp(-top, top)
    if codes.dtype == torch.int8:
        y = y.round()
    else:  # three bits behind the first, the last of them no smaller than 2^-9
        e = (y.abs().view(torch.int64) >> 52).clamp(min=1023 - 6)
        step = ((e - 3) << 52).view(torch.float64)
        y = (y / step).round() * step
    codes[at] = y.float().to(codes.dtype)
    scales[at] = scale


def _load(codes, scales, page, row):
    """Rows [B][T][kvh][hd] of the cache in fp32."""
    heads = torch.arange(codes.shape[1], device="cuda")
    at = (page[..., None], heads, row[..., None])
    x = codes[at].float()
    return x if scales is None else x * scales[at][..., None]


def _put(to, x, on):
    """Rows that are there; the others keep what they held."""
    to.copy_(x if on is None else torch.where(on[..., None, None], x, to.float()))


def _plain_read(s):
    page, row, on = _places(s, s["ko"].shape[1])
    for x, y in (("k", "ko"), ("v", "vo")):
        _put(s[y], _load(s[x + "c"], s[x + "s"], page, row), on)


def _plain_cache(s):
    M = s["k"].shape[1]
    page, row, on = _places(s, M)
    pos = s["start"].long()[:, None] + torch.arange(M, device="cuda")
    if s["q"] is not None:
        _put(s["qo"], _turn(s["q"].float(), pos, s), on)
    _store(_turn(s["k"].float(), pos, s), s["kc"], s["ks"], page, row)
    _store(s["v"].float(), s["vc"], s["vs"], page, row)
    _plain_read(s)


def _plain_attn(s):
    B, M, qh, hd = s["q"].shape
    kvh, page = s["kc"].shape[1], s["kc"].shape[2]
    at = s["table"].long()
    T = at.shape[1] * page

    def rows(x):  # [B][kvh][T][hd], by whole pages
        t = s[x + "c"][at].float()
        if s[x + "s"] is not None:
            t *= s[x + "s"][at][..., None]
        return t.transpose(1, 2).reshape(B, kvh, T, hd)

    q = s["q"].float().view(B, M, kvh, qh // kvh, hd).permute(0, 2, 1, 3, 4).reshape(B, kvh, -1, hd)
    w = (q * s["scale"]) @ rows("k").transpose(-1, -2)
    w = w.view(B, kvh, M, qh // kvh, T)
    seen = torch.arange(T, device="cuda") <= s["start"][:, None, None] + torch.arange(M, device="cuda")[:, None]
    w.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = w.amax(-1, keepdim=True)
    w = torch.exp(w.sub_(top))
    total = w.sum(-1, keepdim=True)
    o = (w.view(B, kvh, -1, T) @ rows("v")).view(B, kvh, M, qh // kvh, hd) / total
    s["o"].copy_(o.permute(0, 2, 1, 3, 4).reshape(B, M, qh, hd))
    s["lse"].copy_((top + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).reshape(B, M, qh))


def run(s):
    op = s["op"]
    if own:
        import gated_deltanet_linear_gb300 as gdn
        if op == "rope":
            gdn.gdn_rope_m(s["x"], s["pos"], s["rope"], s["y"])
        elif op == "attn":
            gdn.gdn_attn_step_m(s["cache"], s["q"], s["table"], s["start"], s["o"],
                                scale=s["scale"], lse=s["lse"], workspace=s["workspace"])
        else:
            if op == "cache":
                gdn.gdn_kv_write_m(s["cache"], s["k"], s["v"], s["table"], s["start"], rope=s["rope"],
                                   q=s["q"], q_out=s["qo"], counts=s["counts"])
            gdn.gdn_kv_read(s["cache"], s["table"], s["start"], s["ko"], s["vo"], counts=s["counts"])
    elif op == "rope":
        _plain_rope(s)
    elif op == "attn":
        _plain_attn(s)
    elif op == "cache":
        _plain_cache(s)
    else:
        _plain_read(s)
    if op == "rope":
        return {"y": s["y"]}
    if op == "attn":
        return {"o": s["o"], "lse": s["lse"]}
    return {"k": s["ko"], "v": s["vo"], "q": s.get("qo")}


# -------------------------------------------------------------------- work

def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    op, hd = case["op"], case["hd"]
    if op == "rope":
        n = case["rows"] * case["heads"]
        # a pair: four multiplications and two additions
        return {"bytes": 2 * n * hd * e + 4 * case["rows"], "flops": 3 * n * case["rot"]}
    ec, es = (2, 0) if case["kind"] == "bf16" else (1, 4)
    B, kvh = case["B"], case["kvh"]
    # a padded batch holds half of its rows on the average
    half = 0.5 if case["ragged"] else 1.0
    if op == "attn":
        M, qh = case["M"], case["qh"]
        keys = B * max(M, half * case["T"])
        return {"bytes": 2 * keys * kvh * (hd * ec + es) + B * M * qh * (2 * hd * e + 4),
                "flops": 4 * keys * M * qh * hd}
    if op == "read":
        rows = 2 * B * case["T"] * half * kvh
        return {"bytes": rows * (hd * (ec + e) + es), "flops": rows * hd}
    # tokens in and q out in their type, the cache's rows, and k and v again
    n = B * case["M"] * half
    return {"bytes": n * hd * (2 * case["qh"] + 2 * kvh) * e + 2 * n * kvh * (hd * (ec + 2) + es),
            "flops": n * (3 * (case["qh"] + kvh) * case["rot"] + 6 * kvh * hd)}


# ------------------------------------------------------------------- exact

def _exact_turn(x, pos, s, n):
    """Pairs as complex numbers, in fp64."""
    if not n:
        return x
    w = torch.polar(torch.full_like(pos, s["amp"], dtype=torch.float64)[..., None].expand(*pos.shape, n),
                    pos.double()[..., None] * s["freq"]).unsqueeze(-2)
    t = x[..., :2 * n]
    t = t.unflatten(-1, (2, n)).transpose(-1, -2) if s["layout"] == "half" else t.unflatten(-1, (n, 2))
    t = torch.view_as_real(torch.view_as_complex(t.contiguous()) * w)
    t = t.transpose(-1, -2) if s["layout"] == "half" else t
    return torch.cat([t.flatten(-2), x[..., 2 * n:]], -1)


def _exact_held(x, kind):
    """The values that rows of x have in the cache."""
    if kind == "bf16":
        return x.to(torch.bfloat16).double()
    top = 127.0 if kind == "int8" else 448.0
    scale = (x.abs().amax(-1, keepdim=True) / top).float().double()
    y = x / scale
    if kind == "int8":
        y = torch.round(y)
    else:  # steps of 1/8 of the power of two below, 2^-9 from 2^-6 down
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3.0)
        y = torch.round(y / step) * step
    return y * scale


def exact(case, seed):
    """The definitions in fp64, sequence by sequence."""
    s = _inputs(case, seed)
    op = case["op"]
    if op == "rope":
        return {"y": _exact_turn(s["x"].double(), s["pos"], s, case["rot"] // 2)}
    if op == "cache":
        M = case["M"]
        out = {"k": s["ko"].double(), "v": s["vo"].double(),
               "q": None if s["q"] is None else s["qo"].double()}
        for b in range(case["B"]):
            m = M if s["counts"] is None else int(s["counts"][b])
            pos = int(s["start"][b]) + torch.arange(m, device="cuda")
            if not m:
                continue
            out["k"][b, :m] = _exact_held(_exact_turn(s["k"][b, :m].double(), pos, s, case["rot"] // 2), case["kind"])
            out["v"][b, :m] = _exact_held(s["v"][b, :m].double(), case["kind"])
            if s["q"] is not None:
                out["q"][b, :m] = _exact_turn(s["q"][b, :m].double(), pos, s, case["rot"] // 2)
        return out

    def rows(x, b, n):  # the first n positions of sequence b, [kvh][n][hd]
        at = s["table"][b, :-(-n // case["page"])].long()
        t = s[x + "c"][at].float().double()
        if s[x + "s"] is not None:
            t = t * s[x + "s"][at].double().unsqueeze(-1)
        return torch.cat(list(t), 1)[:, :n] if t.shape[0] > 1 else t[0, :, :n]

    if op == "read":
        out = {"k": s["ko"].double(), "v": s["vo"].double(), "q": None}
        for b in range(case["B"]):
            n = case["T"] if s["counts"] is None else int(s["counts"][b])
            if n:
                out["k"][b, :n] = rows("k", b, n).transpose(0, 1)
                out["v"][b, :n] = rows("v", b, n).transpose(0, 1)
        return out
    o, lse = s["o"].double(), s["lse"].double()
    rep = case["qh"] // case["kvh"]
    for b in range(case["B"]):
        n = int(s["start"][b]) + case["M"]
        k, v = rows("k", b, n), rows("v", b, n)
        for m in range(case["M"]):
            t = n - case["M"] + m + 1
            q = s["q"][b, m].double().view(case["kvh"], rep, -1)
            w = torch.einsum("hgd,htd->hgt", q, k[:, :t]) * s["scale"]
            lse[b, m] = torch.logsumexp(w, -1).flatten()
            o[b, m] = torch.einsum("hgt,htd->hgd", torch.softmax(w, -1), v[:, :t]).flatten(0, 1)
    return {"o": o, "lse": lse}
