"""gdn_rope_m, gdn_kv_write_m and gdn_kv_read against 64-bit forms."""

import pytest
import torch

import gated_deltanet_linear_gb300 as gdn
from attn_ref import KINDS, TYPES, codes, freqs, turn

pytestmark = pytest.mark.gpu

SCALINGS = {"plain": gdn.GDN_ROPE_PLAIN, "linear": gdn.GDN_ROPE_LINEAR, "ntk": gdn.GDN_ROPE_NTK,
            "band": gdn.GDN_ROPE_BAND}
# A turned pair (x, y): two products of numbers within 2^-24 of themselves with
# cos and sin within 2^-22 (the angle's rounding pi 2^-24, sincospif 2^-23,
# times amp 2^-24), added once: below 2^-21 (|x| + |y|) amp.
TURN = 2.0 ** -21


def gen_of(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def empty_cache(kind, pages, kvh, page, hd):
    k = torch.full((pages, kvh, page, hd), 3, device="cuda").to(KINDS[kind])
    s = None if kind == "bf16" else torch.full((pages, kvh, page), 5.0, device="cuda")
    return gdn.KVCache(k, k.clone(), s, None if s is None else s.clone())


def near(x, pos, f, pairs, amp, dtype):
    """Turned in 64 bits, and what a result may be off by."""
    y = turn(x, pos, f, pairs, amp)
    a = x.double().abs()
    n = f.numel()
    i = torch.arange(n, device=x.device)
    p, q = (2 * i, 2 * i + 1) if pairs else (i, i + n)
    b = torch.zeros_like(a)
    b[..., p] = b[..., q] = TURN * abs(amp) * (a[..., p] + a[..., q])
    if dtype == "bf16":
        b = b * (1 + 2.0 ** -8) + 2.0 ** -8 * y.abs()
        b[..., 2 * n:] = 0
    return y, b


@pytest.mark.parametrize("hd,rot,pairs", [(64, 64, False), (64, 16, True), (128, 48, False), (128, 128, True),
                                          (256, 64, False), (256, 256, False), (256, 208, True)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,heads,scaling", [(1, 1, "plain"), (3, 40, "band"), (257, 5, "ntk"), (1000, 3, "linear")])
def test_rope(hd, rot, pairs, dtype, rows, heads, scaling):
    gen = gen_of(rot)
    f, amp = gdn.gdn_rope_freqs(rot, 1e6, SCALINGS[scaling], 8.0, 4096.0)
    rf, ramp = freqs(rot, 1e6, scaling, 8.0, 4096.0)
    assert ((f.cpu() - rf).abs() <= 1e-14 * rf).all() and abs(amp - ramp) <= 1e-7 * ramp
    x = torch.randn(rows, heads, hd, generator=gen, device="cuda").to(TYPES[dtype])
    pos = torch.randint(-2 ** 20, 2 ** 20, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    pos[-1] = 2 ** 31 - 1
    rope = gdn.Rope(f, gdn.GDN_ROPE_PAIRS if pairs else gdn.GDN_ROPE_HALF, amp)
    y = torch.empty_like(x)
    gdn.gdn_rope_m(x, pos, rope, y)
    ry, b = near(x, pos, f, pairs, amp, dtype)
    # (the frequency's rounding to a 64-bit float in turns, at the position)
    b = b + (pos.double().abs() * 2.0 ** -51)[:, None, None] * x.double().abs().amax(-1, keepdim=True) * amp * 2
    assert ((y.double() - ry).abs() <= b).all()
    assert torch.equal(y[..., rot:], x[..., rot:])
    z = x.clone()
    gdn.gdn_rope_m(z, pos, rope, z)               # in place
    assert torch.equal(z, y)
    wide = torch.full((rows, heads * hd + 24), float("nan"), device="cuda", dtype=x.dtype)
    wide[:, 8:8 + heads * hd] = x.flatten(1)
    gdn.gdn_rope_m(wide[:, 8:8 + heads * hd].unflatten(1, (heads, hd)), pos, rope, z.zero_())
    assert torch.equal(z, y)                      # rows with a stride
    # turned back (amp squared apart)
    back = gdn.Rope(-f, rope.layout, 1.0 / amp)
    gdn.gdn_rope_m(y, pos, back, z)
    tol = 4 * (TURN if dtype == "fp32" else 2.0 ** -7)
    lim = tol * 4 * x.double().abs().amax(-1, keepdim=True) + pos.double().abs()[:, None, None] * 2.0 ** -46
    assert ((z.double() - x.double()).abs() <= lim).all()


def test_rope_gradient():
    """The gradient of a sum w . turn(x) is w turned back: against the
    formula's and against differences in 64 bits."""
    gen = gen_of(3)
    f, _ = gdn.gdn_rope_freqs(32, device="cuda")
    x = torch.randn(5, 2, 64, generator=gen, device="cuda", dtype=torch.float64)
    w = torch.randn(5, 2, 64, generator=gen, device="cuda")
    pos = ints([0, 1, 77, 5000, 123456])
    g = torch.empty_like(w)
    gdn.gdn_rope_m(w, pos, gdn.Rope(-f), g)
    leaf = x.clone().requires_grad_()
    (turn_graph(leaf, pos, f) * w.double()).sum().backward()
    assert (g.double() - leaf.grad).abs().max() <= 2 * TURN * 4 * w.abs().max()
    e = torch.zeros_like(x)
    e[2, 1, 3] = 1e-3
    diff = ((turn(x + e, pos, f, False, 1.0) - turn(x - e, pos, f, False, 1.0)) * w.double()).sum() / 2e-3
    assert abs(diff - g[2, 1, 3].double()) <= 1e-5


def turn_graph(x, pos, f):
    n = f.numel()
    a = (pos.double()[:, None] * f)[:, None]
    p, q = x[..., :n], x[..., n:2 * n]
    return torch.cat([p * a.cos() - q * a.sin(), q * a.cos() + p * a.sin(), x[..., 2 * n:]], -1)


@pytest.mark.parametrize("kind", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("hd,kvh,qh,B,M,page", [(64, 3, 6, 5, 7, 16), (128, 2, 0, 9, 1, 64), (256, 4, 24, 3, 33, 32),
                                                (128, 1, 5, 2, 300, 256), (64, 40, 0, 1, 2, 16)])
def test_codes_are_the_nearest(kind, dtype, hd, kvh, qh, B, M, page):
    """Without a rotation codes and scales are those of 64 bits, to the bit;
    rows that are not the call's keep theirs."""
    gen = gen_of(hd + M)
    x = torch.randn(B, M, (qh + 2 * kvh) * hd, generator=gen, device="cuda").to(TYPES[dtype])
    q = x[..., :qh * hd].unflatten(-1, (qh, hd)) if qh else None
    k = x[..., qh * hd:(qh + kvh) * hd].unflatten(-1, (kvh, hd))
    v = x[..., (qh + kvh) * hd:].unflatten(-1, (kvh, hd))
    if M > 1:
        k[0, 0], v[0, 1, 0] = 0.0, 1e-42         # no scale; a scale of few bits
        v[-1, -1, :, : hd // 2] *= 1e30
    start = torch.randint(0, 3 * page, (B,), generator=gen, device="cuda", dtype=torch.int32)
    counts = torch.randint(0, M + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    counts[0] = M
    cols = 3 + -(-M // page) + 1
    table = torch.randperm(B * cols + 2, generator=gen, device="cuda")[:B * cols].view(B, cols).int()
    cache = empty_cache(kind, B * cols + 2, kvh, page, hd)
    want_k, want_v = cache.k.float().double(), cache.v.float().double()
    want_s = [None if s is None else s.clone() for s in (cache.k_scale, cache.v_scale)]
    q_out = None if q is None else torch.full((B, M, qh, hd), 9.0, device="cuda", dtype=x.dtype)
    err = ints([0])
    gdn.gdn_kv_write_m(cache, k, v, table, start, q=q, q_out=q_out, counts=counts, err_dev=err)
    assert int(err) == 0
    for b in range(B):
        n = int(counts[b])
        p = int(start[b]) + torch.arange(n, device="cuda")
        at, row = table[b][(p // page).long()].long(), (p % page).long()
        for src, want, i in ((k, want_k, 0), (v, want_v, 1)):
            y = src[b, :n].double()
            if kind == "bf16":
                want[at[:, None], torch.arange(kvh, device="cuda"), row[:, None]] = y.float().bfloat16().double()
                continue
            c, s = codes(y, kind)
            c = c.clamp(-127, 127) if kind == "int8" else c.clamp(-448, 448)
            want[at[:, None], torch.arange(kvh, device="cuda"), row[:, None]] = c
            want_s[i][at[:, None], torch.arange(kvh, device="cuda"), row[:, None]] = s
        if q is not None:
            assert torch.equal(q_out[b, :n], q[b, :n]) and bool((q_out[b, n:] == 9.0).all())
    for got, want, s, ws in ((cache.k, want_k, cache.k_scale, want_s[0]), (cache.v, want_v, cache.v_scale, want_s[1])):
        assert torch.equal(got.float().double(), want)
        assert s is None or torch.equal(s, ws)
    # read back: code * scale, and what is not asked for stays
    for out in ("fp32", "bf16"):
        ko = torch.full((B, M, kvh, hd), 9.0, device="cuda", dtype=TYPES[out])
        vo = ko.clone()
        gdn.gdn_kv_read(cache, table, start, ko, vo, counts=counts, err_dev=err)
        assert int(err) == 0
        for b in range(B):
            n = int(counts[b])
            p = int(start[b]) + torch.arange(n, device="cuda")
            at, row = table[b][(p // page).long()].long(), (p % page).long()
            for got, want, s in ((ko, want_k, want_s[0]), (vo, want_v, want_s[1])):
                y = want[at, :, row].float()
                if s is not None:
                    y = y * s[at, :, row][..., None]
                assert torch.equal(got[b, :n], y.to(got.dtype)) and bool((got[b, n:] == 9.0).all())


@pytest.mark.parametrize("kind", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("hd,rot,pairs,M", [(64, 32, True, 1), (128, 128, False, 19), (256, 64, False, 2), (256, 96, True, 70)])
def test_turned_rows(kind, dtype, hd, rot, pairs, M):
    gen = gen_of(rot + M)
    B, kvh, qh, page = 4, 2, 6, 32
    f, amp = gdn.gdn_rope_freqs(rot, 5e5, gdn.GDN_ROPE_BAND, 4.0, 8192.0)
    rope = gdn.Rope(f, gdn.GDN_ROPE_PAIRS if pairs else gdn.GDN_ROPE_HALF, amp)
    q, k, v = (torch.randn(B, M, h, hd, generator=gen, device="cuda").to(TYPES[dtype]) for h in (qh, kvh, kvh))
    start = ints([0, 9000, 77, 300])
    cols = (9000 + M) // page + 1
    pages = 4 * 20
    table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
    perm = torch.randperm(pages, generator=gen, device="cuda").int()
    for b in range(B):
        first = int(start[b]) // page
        table[b, first:first + 20] = perm[20 * b:20 * b + 20][:cols - first]
    cache = empty_cache(kind, pages, kvh, page, hd)
    q_out, err = torch.empty_like(q), ints([0])
    gdn.gdn_kv_write_m(cache, k, v, table, start, rope=rope, q=q, q_out=q_out, err_dev=err)
    assert int(err) == 0
    pos = start[:, None] + torch.arange(M, device="cuda")
    rq, bq = near(q, pos, f, pairs, amp, dtype)
    assert ((q_out.double() - rq).abs() <= bq).all()
    rk, bk = near(k, pos, f, pairs, amp, "fp32")
    ko = torch.empty(B, M, kvh, hd, device="cuda")
    vo = torch.empty_like(ko)
    gdn.gdn_kv_read(cache, table, start, ko, vo)
    top = rk.abs().amax(-1, keepdim=True)
    if kind == "bf16":      # half a step of the value
        held = 2.0 ** -8 * rk.abs()
    elif kind == "int8":    # half a code
        held = 0.5 * top / 127
    else:                   # half a step, or half of the smallest
        held = 2.0 ** -4 * rk.abs() + 2.0 ** -10 * top / 448
    lim = held * (1 + 2.0 ** -20) + bk + 2.0 ** -20 * top + bk.amax(-1, keepdim=True)
    assert ((ko.double() - rk).abs() <= lim).all()
    # v is not turned: its codes are those of a call without a rotation
    other = empty_cache(kind, pages, kvh, page, hd)
    gdn.gdn_kv_write_m(other, k, v, table, start)
    assert torch.equal(other.v.float(), cache.v.float())


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_rows_that_are_not_finite(kind):
    hd, page = 128, 16
    k = torch.randn(1, 4, 2, hd, device="cuda")
    v = torch.randn(1, 4, 2, hd, device="cuda")
    k[0, 1, 0, 7], k[0, 2, 1, 0], v[0, 3, 1, 127] = float("nan"), float("inf"), -float("inf")
    cache = empty_cache(kind, 1, 2, page, hd)
    gdn.gdn_kv_write_m(cache, k, v, ints([[0]]), ints([2]))
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    gdn.gdn_kv_read(cache, ints([[0]]), ints([2]), ko, vo)
    for x, y in ((k, ko), (v, vo)):
        fine = torch.isfinite(x).all(-1)
        assert torch.isnan(y[~fine]).all() and torch.isfinite(y[fine]).all()


def test_bad_pages_and_lengths_write_nothing():
    hd, page, kvh, M = 64, 16, 2, 3
    k = torch.randn(4, M, kvh, hd, device="cuda")
    cache = empty_cache("int8", 6, kvh, page, hd)
    before = cache.k.clone()
    err = ints([0])
    for start, counts, table in (([-1, 0, 0, 0], [3, 0, 0, 0], [[0, 1]] * 4), ([30, 0, 0, 0], [3, 0, 0, 0], [[0, 1]] * 4),
                                 ([0, 0, 0, 0], [4, 0, 0, 0], [[0, 1]] * 4), ([0, 0, 0, 0], [-1, 0, 0, 0], [[0, 1]] * 4),
                                 ([2, 0, 0, 0], [3, 0, 0, 0], [[6, 1]] * 4), ([2, 0, 0, 0], [3, 0, 0, 0], [[-1, 1]] * 4)):
        err.zero_()
        gdn.gdn_kv_write_m(cache, k, k.clone(), ints(table), ints(start), counts=ints(counts), err_dev=err)
        assert int(err) == 1 and torch.equal(cache.k, before)
        out = torch.full_like(k, 9.0)
        out2 = out.clone()
        err.zero_()
        gdn.gdn_kv_read(cache, ints(table), ints(start), out, out2, counts=ints(counts), err_dev=err)
        assert int(err) == 1 and bool((out == 9.0).all()) and bool((out2 == 9.0).all())
    # one bad page of two: the other's rows are written
    err.zero_()
    gdn.gdn_kv_write_m(cache, k[:1].clone(), k[:1].clone(), ints([[5, 9]]), ints([15]), err_dev=err)
    assert int(err) == 1 and not torch.equal(cache.k[5, :, 15], before[5, :, 15])
    before[5, :, 15] = cache.k[5, :, 15]
    assert torch.equal(cache.k, before)


def test_far_positions_and_far_pages():
    """The last positions of the longest table, in pages behind 2^32 bytes of
    a cache."""
    hd, page, kvh = 256, 256, 8
    pages = 2 ** 32 // (page * kvh * hd) + 5
    k = torch.zeros(pages, kvh, page, hd, dtype=torch.int8, device="cuda")
    cache = gdn.KVCache(k, torch.zeros_like(k), torch.zeros(pages, kvh, page, device="cuda"),
                        torch.zeros(pages, kvh, page, device="cuda"))
    cols = gdn.GDN_KV_MAX_POSITIONS // page
    table = torch.full((1, cols), -1, dtype=torch.int32, device="cuda")
    table[0, -1] = pages - 1
    gen = gen_of(21)
    x = torch.randn(1, 40, kvh, hd, generator=gen, device="cuda")
    f, _ = gdn.gdn_rope_freqs(64, 1e6)
    start = ints([gdn.GDN_KV_MAX_POSITIONS - 40])
    err = ints([0])
    gdn.gdn_kv_write_m(cache, x, x, table, start, rope=gdn.Rope(f), err_dev=err)
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    gdn.gdn_kv_read(cache, table, start, ko, vo, err_dev=err)
    assert int(err) == 0
    pos = start.long()[:, None] + torch.arange(40, device="cuda")
    rk, bk = near(x, pos, f, False, 1.0, "fp32")
    top = rk.abs().amax(-1, keepdim=True)
    # half a code, the turn's error, and the frequency's rounding at 2^30
    lim = 0.5 * top / 127 * (1 + 2.0 ** -20) + bk.amax(-1, keepdim=True) + 2.0 ** -19 * top
    assert ((ko.double() - rk).abs() <= lim).all()
    c, s = codes(x.double(), "int8")
    assert torch.equal(vo, c.float() * s[..., None])
    assert not bool(cache.k[:-1].any())
    gdn.gdn_kv_write_m(cache, x, x, table, start + 1, err_dev=err)     # one behind the end
    assert int(err) == 1


def test_calls_on_several_streams():
    """Writes of different sequences into one cache on three streams at once
    are those of one call."""
    gen = gen_of(22)
    B, M, hd, kvh, page = 9, 50, 128, 2, 16
    k, v = (torch.randn(B, M, kvh, hd, generator=gen, device="cuda") for _ in "kv")
    table = torch.randperm(B * 4, generator=gen, device="cuda").int().view(B, 4)
    start = ints([3] * B)
    one, many = empty_cache("int8", B * 4, kvh, page, hd), empty_cache("int8", B * 4, kvh, page, hd)
    gdn.gdn_kv_write_m(one, k, v, table, start)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for i, s in enumerate(streams):
        b = slice(3 * i, 3 * i + 3)
        gdn.gdn_kv_write_m(many, k[b], v[b], table[b], start[b], stream=s)
    torch.cuda.synchronize()
    for x in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(one, x), getattr(many, x))


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("kvh,hd,T", [(1, 64, 65003), (2, 128, 4003), (1, 256, 20003), (1, 128, 4003), (3, 64, 4003)])
def test_reads_of_few_heads(kind, kvh, hd, T):
    """Many positions of one to three heads, ends in the middle of what a group
    of lanes takes, a page that the cache has not."""
    gen = gen_of(24)
    page, B = 16, 5
    cols = -(-T // page)
    pages = B * cols
    k = torch.randn(pages, kvh, page, hd, generator=gen, device="cuda")
    k = (k * 30).round().clamp(-127, 127).to(torch.int8) if kind == "int8" else k.bfloat16()
    v = k.flip(0).contiguous()
    s = None if kind == "bf16" else torch.rand(pages, kvh, page, generator=gen, device="cuda")
    cache = gdn.KVCache(k, v, s, None if s is None else s.flip(0).contiguous())
    table = torch.randperm(pages, generator=gen, device="cuda").int().view(B, cols)
    counts = [T, 0, 1, 2001, T - 5]
    bad = table.clone()
    bad[3, 7] = pages
    err = ints([0])
    out = [torch.full((B, T, kvh, hd), 9.0, device="cuda") for _ in "kv"]
    gdn.gdn_kv_read(cache, bad, None, *out, counts=ints(counts), err_dev=err)
    assert int(err) == 1
    for got, c, sc in ((out[0], k, cache.k_scale), (out[1], v, cache.v_scale)):
        x = c[table.long()].float()
        if sc is not None:
            x = x * sc[table.long()][..., None]
        x = x.transpose(2, 3).reshape(B, -1, kvh, hd)[:, :T].clone()
        for b, n in enumerate(counts):
            x[b, n:] = 9.0
        x[3, 7 * page:8 * page] = 9.0
        assert torch.equal(got, x)
