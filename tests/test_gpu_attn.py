"""gdn_attn_step_m against a 64-bit form: every head size, cache type and
token type, lengths around the tiles' ends, rows that nothing may reach."""

import pytest
import torch

import gated_deltanet_linear_gb300 as gdn
from attn_ref import (KINDS, TYPES, attn, attn_bounds, held, junk_behind, make_cache, make_table)

pytestmark = pytest.mark.gpu


def gen_of(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def cache_of(c):
    return gdn.KVCache(c["k"], c["v"], c["ks"], c["vs"])


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def call(c, q, table, start, scale, counts=None, err=None, o=None, lse=None):
    """o and lse, with values of their own where the call writes nothing."""
    cache = cache_of(c)
    o = torch.full_like(q, 7.0) if o is None else o
    lse = torch.full(q.shape[:3], 7.0, device="cuda") if lse is None else lse
    ws = torch.empty(gdn.gdn_attn_workspace(cache, q.shape[1], q.shape[2]), dtype=torch.uint8, device="cuda")
    gdn.gdn_attn_step_m(cache, q, table, start, o, scale=scale, counts=counts, lse=lse, err_dev=err,
                        workspace=ws)
    return o, lse


def check(c, kind, dtype, q, table, start, counts, scale, page):
    hd = q.shape[3]
    o, lse = call(c, q, table, ints(start), scale, None if counts is None else ints(counts))
    ro, rl, mag, big = attn(c, table, start, counts, q, scale, page)
    T = max(s + q.shape[1] for s in start)
    bo, bl = attn_bounds(kind, dtype, hd, T, ro, rl, mag, big)
    there = ~torch.isnan(rl)
    assert bool((o[~there] == 7.0).all()) and bool((lse[~there] == 7.0).all())
    assert bool(torch.isfinite(o[there]).all())
    eo = ((o.double() - ro).abs() - bo)[there]
    el = ((lse.double() - rl).abs() - bl)[there]
    worst = ((o.double() - ro).abs() / bo.clamp(min=1e-300))[there].max().item()
    assert eo.max().item() <= 0, f"o at {worst:.2f} of its bound"
    assert el.max().item() <= 0
    return o, lse


LENS = [1, 2, 15, 16, 17, 31, 33, 64, 127, 128, 129, 255, 256, 257, 400, 513, 1000]


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("kind", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("M,kvh,group,page", [(1, 2, 4, 16), (1, 1, 8, 64), (2, 3, 1, 32), (1, 2, 13, 128),
                                              (4, 1, 6, 256), (3, 2, 5, 16), (7, 2, 3, 64), (5, 1, 9, 32)])
def test_against_64_bits(hd, kind, dtype, M, kvh, group, page):
    gen = gen_of(hd + M + group)
    lens = [n for n in LENS if n >= M]
    cols = -(-max(lens) // page) + 1
    B = len(lens)
    c = make_cache(kind, B * cols + 3, kvh, page, hd, gen, "cuda")
    table = make_table(B * cols + 3, B, cols, gen, "cuda")
    junk_behind(c, table, lens, page, kind)
    q = (2 * torch.randn(B, M, kvh * group, hd, generator=gen, device="cuda")).to(TYPES[dtype])
    check(c, kind, dtype, q, table, [n - M for n in lens], None, hd ** -0.5, page)


@pytest.mark.parametrize("hd,kind,dtype,kvh,group", [(128, "int8", "bf16", 1, 4), (256, "bf16", "fp32", 2, 8),
                                                     (64, "e4m3", "fp32", 3, 12)])
def test_long_sequences_split_over_many_ctas(hd, kind, dtype, kvh, group):
    gen = gen_of(5)
    lens, page = [40001, 3, 17777], 64
    cols = -(-max(lens) // page)
    c = make_cache(kind, 3 * cols, kvh, page, hd, gen, "cuda")
    table = make_table(3 * cols, 3, cols, gen, "cuda")
    junk_behind(c, table, lens, page, kind)
    q = (2 * torch.randn(3, 1, kvh * group, hd, generator=gen, device="cuda")).to(TYPES[dtype])
    check(c, kind, dtype, q, table, [n - 1 for n in lens], None, hd ** -0.5, page)


@pytest.mark.parametrize("kind", ["bf16", "int8", "e4m3"])
def test_counts_leave_rows_alone(kind):
    gen = gen_of(6)
    hd, page, M, B = 128, 16, 5, 7
    start, counts = [0, 40, 12, 100, 0, 7, 300], [5, 0, 1, 4, 1, 2, 3]
    lens = [s + n for s, n in zip(start, counts)]
    cols = -(-(max(lens) + M) // page)
    c = make_cache(kind, B * cols, 2, page, hd, gen, "cuda")
    table = make_table(B * cols, B, cols, gen, "cuda")
    junk_behind(c, table, lens, page, kind)
    q = torch.randn(B, M, 6, hd, generator=gen, device="cuda")
    check(c, kind, "fp32", q, table, start, counts, 0.1, page)


@pytest.mark.parametrize("kind", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("hd", [64, 256])
def test_rows_that_are_not_finite_stay_with_who_sees_them(kind, hd):
    """A later token's key or value holds NaN or infinities: earlier tokens of
    the call give the bits that they give without it."""
    gen = gen_of(7)
    page, M, start = 16, 6, 29
    c = make_cache(kind, 4, 1, page, hd, gen, "cuda")
    table = ints([[2, 0, 3]])
    q = torch.randn(1, M, 3, hd, generator=gen, device="cuda")
    clean, clean_lse = call(c, q, table, ints([start]), 0.2)
    for x in "kv":
        for bad in (float("nan"), float("inf")):
            d = {n: None if t is None else t.clone() for n, t in c.items()}
            p = start + 3  # seen by tokens 3, 4, 5
            page_of, row = int(table[0, p // page]), p % page
            if kind == "bf16":
                d[x][page_of, 0, row, 5] = bad
            else:
                d[x + "s"][page_of, 0, row] = float("nan")
            o, lse = call(d, q, table, ints([start]), 0.2)
            assert torch.equal(o[:, :3], clean[:, :3]) and torch.equal(lse[:, :3], clean_lse[:, :3])
            assert not bool(torch.isfinite(o[:, 3:, :, 5]).any())
    q2 = q.clone()
    q2[0, 1, 2, 9] = float("nan")
    o, _ = call(c, q2, table, ints([start]), 0.2)
    keep = torch.ones(1, M, 3, dtype=torch.bool, device="cuda")
    keep[0, 1, 2] = False
    assert torch.equal(o[keep], clean[keep]) and not bool(torch.isfinite(o[0, 1, 2]).any())


@pytest.mark.parametrize("hd,dtype", [(64, "bf16"), (128, "fp32"), (256, "fp32")])
@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_scales_of_any_size(hd, dtype, kind):
    """Value rows from 1e-25 to 1e25 beside each other, key rows from zeros up,
    queries from 1e-30 to 1e20: the bound goes by the weights' magnitudes."""
    gen = gen_of(8)
    page, lens = 32, [300, 77]
    cols = -(-max(lens) // page)
    c = make_cache(kind, 2 * cols, 2, page, hd, gen, "cuda")
    c["vs"] *= 10.0 ** (50 * torch.rand(c["vs"].shape, generator=gen, device="cuda") - 25)
    c["ks"] *= (torch.rand(c["ks"].shape, generator=gen, device="cuda") > 0.2)
    table = make_table(2 * cols, 2, cols, gen, "cuda")
    junk_behind(c, table, lens, page, kind)
    q = torch.randn(2, 1, 4, hd, generator=gen, device="cuda")
    q[0, 0, 1] *= 1e-30
    q[1, 0, 2] = 0
    check(c, kind, dtype, q.to(TYPES[dtype]), table, [n - 1 for n in lens], None, 0.3, page)
    c["ks"] *= 1e-20
    check(c, kind, dtype, (q * 1e20).to(TYPES[dtype]), table, [n - 1 for n in lens], None, 0.3, page)
    c["vs"].zero_()
    junk_behind(c, table.clone(), lens, page, kind)
    o, _ = call(c, q.to(TYPES[dtype]), table, ints([n - 1 for n in lens]), 0.3)
    assert bool((o == 0).all())


@pytest.mark.parametrize("kind", ["bf16", "int8", "e4m3"])
def test_one_key_takes_all(kind):
    """A score hundreds above the others, early or late: o is its value."""
    hd, page, n = 128, 64, 700
    gen = gen_of(9)
    for at in (0, 5, 350, 699):
        c = make_cache(kind, 12, 1, page, hd, gen, "cuda")
        table = make_table(12, 1, 11, gen, "cuda")
        q = torch.randn(1, 1, 2, hd, generator=gen, device="cuda")
        p, r = int(table[0, at // page]), at % page
        x = q[0, 0].sum(0)
        if kind == "int8":
            c["k"][p, 0, r] = (x / x.abs().max() * 127).round().to(torch.int8)
            c["ks"][p, 0, r] = 1.0
        elif kind == "e4m3":
            c["k"][p, 0, r] = (x / x.abs().max() * 448).to(torch.float8_e4m3fn)
            c["ks"][p, 0, r] = 0.3
        else:
            c["k"][p, 0, r] = (x * 40).bfloat16()
        o, _ = check(c, kind, "fp32", q, table, [n - 1], None, 0.2, page)
        v = held(c, "v", table, 0, n, page)[0, at]
        assert (o[0, 0].double() - v).abs().max() <= 2.0 ** -18 * v.abs().max()


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_bad_pages_and_lengths(kind):
    gen = gen_of(10)
    hd, page, B = 128, 16, 6
    c = make_cache(kind, 30, 2, page, hd, gen, "cuda")
    table = make_table(30, B, 5, gen, "cuda")
    q = torch.randn(B, 2, 4, hd, generator=gen, device="cuda")
    good, _ = call(c, q, table, ints([10, 20, 30, 40, 50, 60]), 0.1)
    err = ints([0])
    o, lse = call(c, q, table, ints([10, -1, 30, 79, 50, 60]), 0.1, counts=ints([2, 2, 3, 2, -1, 2]), err=err)
    assert int(err) == 1
    assert torch.equal(o[[0, 5]], good[[0, 5]])
    assert bool((o[1:5] == 7.0).all()) and bool((lse[1:5] == 7.0).all())
    for bad in (-1, 30, 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[2, 1] = bad
        err.zero_()
        o, lse = call(c, q, t, ints([10, 20, 30, 40, 50, 60]), 0.1, err=err)
        assert int(err) == 1
        assert torch.equal(o[[0, 1, 3, 4, 5]], good[[0, 1, 3, 4, 5]])
        assert not bool(torch.isfinite(o[2]).any()) and not bool(torch.isfinite(lse[2]).any())
    err.zero_()
    call(c, q, table, ints([10, 20, 30, 40, 50, 60]), 0.1, err=err)
    assert int(err) == 0


def test_same_bits_alone_and_again():
    """The same call twice, and on three streams at once with workspaces of
    their own."""
    gen = gen_of(11)
    hd, page, B, T = 128, 64, 5, 3000
    cols = -(-T // page)
    c = make_cache("int8", B * cols, 2, page, hd, gen, "cuda")
    table = make_table(B * cols, B, cols, gen, "cuda")
    start = ints([2999, 17, 640, 2000, 63])
    q = torch.randn(B, 1, 8, hd, generator=gen, device="cuda").bfloat16()
    first, lse = call(c, q, table, start, 0.1)
    cache = cache_of(c)
    n = gdn.gdn_attn_workspace(cache, 1, 8)
    runs = [(torch.cuda.Stream(), torch.zeros_like(q), torch.empty(n, dtype=torch.uint8, device="cuda"))
            for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, o, ws in runs:
            gdn.gdn_attn_step_m(cache, q, table, start, o, scale=0.1, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for _, o, _ in runs:
        assert torch.equal(o, first)


def test_captured_steps_follow_the_cursor():
    """One captured step, replayed while the host moves start and q."""
    gen = gen_of(12)
    hd, page, B = 64, 16, 3
    c = make_cache("e4m3", 3 * 20, 2, page, hd, gen, "cuda")
    table = make_table(3 * 20, B, 20, gen, "cuda")
    cache = cache_of(c)
    q = torch.zeros(B, 1, 4, hd, device="cuda")
    o, start = torch.zeros_like(q), ints([0, 0, 0])
    ws = torch.empty(gdn.gdn_attn_workspace(cache, 1, 4), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_attn_step_m(cache, q, table, start, o, workspace=ws)
    for n in ([0, 5, 300], [319, 15, 16], [100, 100, 0]):
        start.copy_(ints(n))
        q.copy_(torch.randn(q.shape, generator=gen, device="cuda"))
        graph.replay()
        want, _ = call(c, q, table, start, hd ** -0.5)
        assert torch.equal(o, want)


def test_offsets_beyond_32_bits():
    """Pages behind 2^31 elements and 2^32 bytes of a cache."""
    gen = gen_of(13)
    hd, page, kvh = 256, 256, 8
    pages = 2 ** 32 // (page * kvh * hd) + 40      # codes: 4.3 GB each
    k = torch.empty(pages, kvh, page, hd, dtype=torch.int8, device="cuda")
    v = torch.empty_like(k)
    s = torch.empty(pages, kvh, page, device="cuda")
    near = make_cache("int8", 8, kvh, page, hd, gen, "cuda")
    far = {"k": k, "v": v, "ks": s, "vs": s.clone()}
    at = [pages - 1, 0, pages - 3, 1, pages // 2, pages - 30, pages // 2 + 1, 3]
    for i, p in enumerate(at):
        for x in ("k", "v", "ks", "vs"):
            far[x][p] = near[x][i]
    q = torch.randn(1, 2, 16, hd, generator=gen, device="cuda")
    o1, _ = call(near, q, ints([list(range(8))]), ints([2040]), 0.1)
    o2, _ = call(far, q, ints([at]), ints([2040]), 0.1)
    assert torch.equal(o1, o2)
    k2 = torch.zeros(1, 2042, kvh, hd, device="cuda")
    v2 = torch.zeros_like(k2)
    gdn.gdn_kv_read(cache_of(far), ints([at]), None, k2, v2)
    k1, v1 = torch.zeros_like(k2), torch.zeros_like(k2)
    gdn.gdn_kv_read(cache_of(near), ints([list(range(8))]), None, k1, v1)
    assert torch.equal(k1, k2) and torch.equal(v1, v2)


@pytest.mark.parametrize("kind", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("scale", [0.0, -0.7, 3.0])
def test_scales_of_scores(kind, scale):
    """Zero (the mean of what is seen), negative and large ones, with masks."""
    gen = gen_of(14)
    hd, page, M, lens = 128, 32, 3, [3, 50, 259]
    c = make_cache(kind, 30, 2, page, hd, gen, "cuda")
    table = make_table(30, 3, 10, gen, "cuda")
    junk_behind(c, table, lens, page, kind)
    for group in (2, 5):
        q = torch.randn(3, M, 2 * group, hd, generator=gen, device="cuda")
        check(c, kind, "fp32", q, table, [n - M for n in lens], None, scale, page)


@pytest.mark.parametrize("B", [32, 33, 255, 256, 257, 700])
def test_batches_around_the_search(B):
    """Batches on both sides of the sizes that the lengths are searched by,
    with sequences left out at both ends and in the middle."""
    gen = gen_of(15)
    hd, page, cols = 64, 16, 5
    c = make_cache("int8", B * cols, 1, page, hd, gen, "cuda")
    table = make_table(B * cols, B, cols, gen, "cuda")
    start = torch.randint(0, cols * page - 2, (B,), generator=gen, device="cuda").tolist()
    counts = (torch.rand(B, generator=gen, device="cuda") > 0.3).long().mul(2).tolist()
    counts[0] = counts[-1] = 0
    counts[B // 2] = 2
    lens = [s + n for s, n in zip(start, counts)]
    junk_behind(c, table, lens, page, "int8")
    q = torch.randn(B, 2, 2, hd, generator=gen, device="cuda")
    check(c, "int8", "fp32", q, table, start, counts, 0.2, page)
    o, _ = call(c, q, table, ints(start), 0.2, counts=ints([0] * B))
    assert bool((o == 7.0).all())


@pytest.mark.parametrize("fill", [0, 0xff, 0x5a, None])
def test_workspaces_may_hold_anything(fill):
    """Joins over many CTAs with a workspace of zeros, ones, noise and what
    another call has left, four times each."""
    gen = gen_of(16)
    hd, page, T = 128, 64, 20000
    cols = -(-T // page)
    c = make_cache("int8", 2 * cols, 2, page, hd, gen, "cuda")
    table = make_table(2 * cols, 2, cols, gen, "cuda")
    start = ints([19999, 7000])
    q = torch.randn(2, 1, 8, hd, generator=gen, device="cuda")
    want, _ = call(c, q, table, start, 0.1)
    cache = cache_of(c)
    ws = torch.empty(gdn.gdn_attn_workspace(cache, 1, 8), dtype=torch.uint8, device="cuda")
    for _ in range(4):
        if fill is None:
            ws.copy_(torch.randint(0, 256, ws.shape, generator=gen, device="cuda", dtype=torch.uint8))
        else:
            ws.fill_(fill)
        for _ in range(2):
            o = torch.zeros_like(q)
            gdn.gdn_attn_step_m(cache, q, table, start, o, scale=0.1, workspace=ws)
            assert torch.equal(o, want)


@pytest.mark.parametrize("kind,hd,dtype", [("int8", 128, "bf16"), ("bf16", 256, "fp32"), ("e4m3", 256, "fp32"),
                                           ("bf16", 64, "bf16")])
@pytest.mark.parametrize("M,kvh,group", [(64, 1, 3), (33, 2, 1), (17, 1, 5)])
def test_many_tokens(kind, hd, dtype, M, kvh, group):
    """Up to 64 tokens: several row tiles, masks over several tiles of
    positions, and values that are not finite among the call's own."""
    gen = gen_of(17)
    page, lens = 16, [M, M + 1, 200]
    cols = -(-max(lens) // page)
    c = make_cache(kind, 3 * cols, kvh, page, hd, gen, "cuda")
    table = make_table(3 * cols, 3, cols, gen, "cuda")
    junk_behind(c, table, lens, page, kind)
    q = torch.randn(3, M, kvh * group, hd, generator=gen, device="cuda").to(TYPES[dtype])
    start = [n - M for n in lens]
    o, _ = check(c, kind, dtype, q, table, start, None, hd ** -0.5, page)
    p = lens[2] - M // 2                                 # seen by the later half
    if kind == "bf16":
        c["v"][int(table[2, p // page]), 0, p % page, 3] = float("inf")
    else:
        c["vs"][int(table[2, p // page]), 0, p % page] = float("nan")
    o2, _ = call(c, q, table, ints(start), hd ** -0.5)
    m = p - start[2]
    assert torch.equal(o2[:2], o[:2]) and torch.equal(o2[2, :m], o[2, :m])
    assert not bool(torch.isfinite(o2[2, m:, :group, 3]).any())


def test_many_heads():
    gen = gen_of(18)
    for kvh, group in ((300, 1), (2, 100), (1, 257)):
        c = make_cache("int8", 6, kvh, 16, 64, gen, "cuda")
        table = make_table(6, 2, 3, gen, "cuda")
        q = torch.randn(2, 1, kvh * group, 64, generator=gen, device="cuda")
        check(c, "int8", "fp32", q, table, [40, 3], None, 0.125, 16)


def test_negative_scales():
    """A cache filled elsewhere may hold them: they are numbers like others."""
    gen = gen_of(19)
    hd, page, n = 128, 32, 500
    c = make_cache("int8", 16, 2, page, hd, gen, "cuda")
    for x in ("ks", "vs"):
        c[x] *= torch.where(torch.rand(c[x].shape, generator=gen, device="cuda") < 0.5, -1.0, 1.0)
    c["vs"][:, :, ::3] *= 1e6
    table = make_table(16, 1, 16, gen, "cuda")
    q = torch.randn(1, 1, 8, hd, generator=gen, device="cuda")
    check(c, "int8", "fp32", q, table, [n - 1], None, 0.1, page)


def test_empty_batches_and_refusals():
    c = make_cache("int8", 4, 2, 16, 64, gen_of(20), "cuda")
    cache = cache_of(c)
    ws = torch.empty(gdn.gdn_attn_workspace(cache, 2, 4), dtype=torch.uint8, device="cuda")
    q = torch.zeros(0, 2, 4, 64, device="cuda")
    table = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    gdn.gdn_attn_step_m(cache, q, table, table[:, 0].contiguous(), torch.empty_like(q), workspace=ws)
    k = torch.zeros(0, 2, 2, 64, device="cuda")
    gdn.gdn_kv_write_m(cache, k, k, table, table[:, 0].contiguous())
    gdn.gdn_kv_read(cache, table, None, k, k)
    q = torch.zeros(1, 2, 4, 64, device="cuda")
    table = ints([[0, 1]])
    ok = dict(workspace=ws)
    call_ = gdn.gdn_attn_step_m
    o = torch.empty_like(q)
    call_(cache, q, table, ints([3]), o, **ok)
    for args, kw, status in (((q, table, ints([3]), q), ok, gdn.GDN_EALIAS),
                             ((q, table, ints([3]), o), dict(workspace=ws[:100]), gdn.GDN_ERANGE),
                             ((q, table, ints([3]), o), {}, gdn.GDN_EINVAL),
                             ((q, table, ints([3]), o), dict(workspace=o.view(torch.uint8)), gdn.GDN_ERANGE),
                             ((q.cpu(), table, ints([3]), o), ok, gdn.GDN_EPTR),
                             ((q, table.cpu(), ints([3]), o), ok, gdn.GDN_EPTR)):
        with pytest.raises(gdn.GDNError) as e:
            call_(cache, *args, **kw)
        assert e.value.status == status
    big = torch.empty(ws.numel() + o.numel() * 4, dtype=torch.uint8, device="cuda")
    inside = big[:o.numel() * 4].view(torch.float32).view(o.shape)
    with pytest.raises(gdn.GDNError) as e:
        call_(cache, q, table, ints([3]), inside, workspace=big)
    assert e.value.status == gdn.GDN_EALIAS
    with pytest.raises(gdn.GDNError) as e:                # a cache that is its own values
        gdn.gdn_kv_write_m(gdn.KVCache(c["k"], c["k"], c["ks"], c["vs"]), q[:, :, :2].contiguous(),
                           q[:, :, :2].contiguous(), table, ints([0]))
    assert e.value.status == gdn.GDN_EALIAS
    with pytest.raises(gdn.GDNError) as e:                # one row for all tokens
        gdn.gdn_kv_write_m(cache, q[:, :1, :2].expand(1, 2, 2, 64), q[:, :, :2].contiguous(), table, ints([0]))
    assert e.value.status == gdn.GDN_ESHAPE
    for bad in (dict(q=q.double()), dict(q=q[..., :32]), dict(table=table.long()), dict(start=ints([1, 2])),
                dict(o=o.bfloat16()), dict(o=o[:, :1])):
        a = dict(q=q, table=table, start=ints([3]), o=o)
        a.update(bad)
        with pytest.raises(ValueError):
            call_(cache, a["q"], a["table"], a["start"], a["o"], **ok)


@pytest.mark.parametrize("kind,hd,M,group", [("int8", 128, 1, 4), ("bf16", 256, 1, 8), ("e4m3", 256, 4, 6),
                                             ("int8", 64, 2, 5), ("bf16", 128, 3, 7)])
def test_nothing_outside_o_lse_and_the_workspace(kind, hd, M, group):
    """Guard bands around what a call writes, with joins over all CTAs."""
    gen = gen_of(23)
    page, T, kvh = 64, 60000, 2
    cols = -(-T // page)
    c = make_cache(kind, cols, kvh, page, hd, gen, "cuda")
    table = make_table(cols, 1, cols, gen, "cuda")
    cache = cache_of(c)
    n = gdn.gdn_attn_workspace(cache, M, kvh * group)
    room = torch.full((n + 8192,), 0xa5, dtype=torch.uint8, device="cuda")
    q = torch.randn(1, M, kvh * group, hd, generator=gen, device="cuda")
    out = torch.full((q.numel() + 512,), 7.0, device="cuda")
    o = out[256:256 + q.numel()].view(q.shape)
    ls = torch.full((M * kvh * group + 256,), 7.0, device="cuda")
    lse = ls[128:128 + M * kvh * group].view(1, M, -1)
    before = {x: None if c[x] is None else c[x].view(torch.uint8).clone() for x in ("k", "v", "ks", "vs")}
    gdn.gdn_attn_step_m(cache, q, table, ints([T - M]), o, scale=0.1, lse=lse, workspace=room[4096:4096 + n])
    assert bool((room[:4096] == 0xa5).all()) and bool((room[4096 + n:] == 0xa5).all())
    assert bool((out[:256] == 7.0).all()) and bool((out[-256:] == 7.0).all())
    assert bool((ls[:128] == 7.0).all()) and bool((ls[-128:] == 7.0).all())
    assert bool((o != 7.0).all()) and bool((lse != 7.0).all())
    for x, was in before.items():
        assert was is None or torch.equal(c[x].view(torch.uint8), was)
