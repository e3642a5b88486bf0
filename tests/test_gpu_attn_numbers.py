"""What gdn_attn_step_m keeps of its numbers."""

import math

import pytest
import torch

from attn_ref import TYPES, attn, attn_bounds, held, junk_behind, make_cache, make_table
from test_gpu_attn import call, check, gen_of, ints

pytestmark = pytest.mark.gpu


def bf16_steps(x):
    """The step between bf16 numbers at x (fp64)."""
    return torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -126))) - 7)


@pytest.mark.parametrize("kind", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("hd,group,M", [(64, 4, 1), (128, 4, 1), (256, 6, 1), (128, 5, 3), (256, 8, 3), (64, 4, 4)])
@pytest.mark.parametrize("T", [5, 40, 2000])
def test_bf16_results_are_rounded_once(kind, hd, group, M, T):
    """bf16 tokens get the fp32 result, rounded: every element is the rounding
    of a number within the bound of fp32 tokens, and few lie on the other side
    of a border.  A number that is off by d of its sum of magnitudes is rounded
    the other way with a chance of d mag / step, which moves it by a step; d =
    2^-21 (weights, their sum and the products' sums are each held to 2^-23),
    and twice that for chance."""
    gen = gen_of(hd + M + T)
    page, kvh, B = 16, 2, 48 if T < 100 else 3
    cols = -(-T // page)
    c = make_cache(kind, B * cols, kvh, page, hd, gen, "cuda")
    table = make_table(B * cols, B, cols, gen, "cuda")
    q = torch.randn(B, M, kvh * group, hd, generator=gen, device="cuda").bfloat16()
    start, scale = [T - M] * B, 0.3 * hd ** -0.5
    o, _ = call(c, q, table, ints(start), scale)
    ro, rl, mag, big = attn(c, table, start, None, q, scale, page)
    b, _ = attn_bounds(kind, "fp32", hd, T, ro, rl, mag, big)
    assert bool((o >= (ro - b).bfloat16()).all()) and bool((o <= (ro + b).bfloat16()).all())
    far = (o.double() - ro.bfloat16().double()).square().sum()
    lim = (2 * 2.0 ** -21 * mag * bf16_steps(ro)).sum()
    assert far <= lim, f"{(far / ro.square().sum()).sqrt().item():.2e} from the rounded result"


def sequences(kind, hd, page, scores, vs, gen):
    """A cache of one key head whose key rows give a query (1, 0, 0, ..) the scores
    [n][T], and whose value rows have the scales vs [n][T]; its table."""
    n, T = scores.shape
    cols = -(-T // page)
    c = make_cache(kind, n * cols, 1, page, hd, gen, "cuda", spread=0.0)
    table = make_table(n * cols, n, cols, gen, "cuda")
    at = (table.long().repeat_interleave(page, 1)[:, :T], 0, torch.arange(T, device="cuda").expand(n, T) % page)
    if kind == "bf16":
        k = torch.zeros(n, T, hd, device="cuda")
        k[..., 0] = scores
        c["k"][at] = k.bfloat16()
        c["v"][at] = (c["v"][at].float() * vs[..., None]).bfloat16()
    else:
        k = torch.zeros(n, T, hd, device="cuda")
        k[..., 0] = 1.0
        c["k"][at] = k.to(c["k"].dtype)
        c["ks"][at], c["vs"][at] = scores.float(), vs.float()
    return c, table


def check_many(c, table, kind, dtype, q, T, page, copies=48):
    """Every sequence `copies` times, so that one warp has many of its tiles,
    against 64 bits; q [n][M][qh][hd]."""
    n, M, _, hd = q.shape
    start = [T - M] * n
    o, lse = call(c, q.repeat(copies, 1, 1, 1), table.repeat(copies, 1), ints(start * copies), 1.0)
    ro, rl, mag, big = attn(c, table, start, None, q, 1.0, page)
    bo, bl = attn_bounds(kind, dtype, hd, T, ro, rl, mag, big)
    for x, r, b, name in ((lse, rl, bl, "lse"), (o, ro, bo, "o")):
        x = x.double().view(copies, *r.shape)
        assert bool(torch.isfinite(x).all()), name
        assert ((x - r).abs() <= b).all(), f"{name} at {((x - r).abs() / b.clamp(min=1e-300)).max().item():.3g} of its bound"
    return o, lse


LN2 = 0.6931471805599453
BEHIND = {"zeros, zeros 24 above, others": ((0, 0), (24, 0), (0, 1)),
          "zeros, others 40 above": ((0, 0), (40, 1), (3, 1)),
          "others, zeros 60 above": ((0, 1), (60, 0), (1, 1)),
          "others, zeros 110.5 above": ((0, 1), (110.5, 0), (0, 0)),
          "others, zeros 124 above": ((0, 1), (124, 0), (0, 0)),
          "others, zeros 130 above, others": ((0, 1), (130, 0), (130, 1)),
          "zeros, values of 2^40": ((0, 0), (0, 2.0 ** 40), (0, 0)),
          "values of 2^-60, 2^60, 2^-60": ((0, 2.0 ** -60), (0, 2.0 ** 60), (5, 2.0 ** -60)),
          "values of 2^-90": ((0, 2.0 ** -90), (10, 2.0 ** -90), (3, 2.0 ** -90)),
          "values of 2^100, zeros above": ((0, 2.0 ** 100), (90, 0), (0, 2.0 ** 90)),
          "zeros alone": ((0, 0), (30, 0), (90, 0))}


@pytest.mark.parametrize("name", BEHIND)
@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("hd,group,M,dtype", [(128, 4, 1, "bf16"), (64, 4, 1, "fp32"), (256, 6, 4, "fp32"), (128, 5, 2, "fp32")])
def test_scales_move_no_weights(name, kind, hd, group, M, dtype):
    """Rows of zeros have scale 0 and their weight all the same, whatever the
    scales of other rows and however far apart (scores in base 2, scales; each
    for a third of the positions, and mixed)."""
    gen = gen_of(hd)
    T, page, n = 960, 32, 4
    part = torch.arange(T, device="cuda").expand(n, T) * 3 // T
    part = torch.where(torch.arange(n, device="cuda")[:, None] < 2, part,
                       torch.randint(0, 3, (n, T), generator=gen, device="cuda"))
    sc, vs = (torch.tensor([float(p[i]) for p in BEHIND[name]], dtype=torch.float64, device="cuda")[part] for i in (0, 1))
    sc = (sc + torch.rand(n, T, generator=gen, device="cuda")) * LN2
    c, table = sequences(kind, hd, page, sc, vs, gen)
    q = torch.zeros(n, M, group, hd, device="cuda")
    q[..., 0] = 1.0
    q[:, :, 1::2, 0] = 0.75
    o, _ = check_many(c, table, kind, dtype, q.to(TYPES[dtype]), T, page)
    if name == "zeros alone":
        assert bool((o == 0).all())


@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 27, 2.0 ** 28.5, 2.0 ** 31, 2.0 ** 40, 2.0 ** 70, 2.0 ** 98, 1.2e30])
@pytest.mark.parametrize("kind,hd,group,M,dtype", [("int8", 128, 4, 1, "bf16"), ("e4m3", 64, 2, 1, "fp32"),
                                                   ("bf16", 128, 4, 1, "bf16"), ("bf16", 64, 1, 1, "fp32"),
                                                   ("int8", 256, 6, 4, "fp32"), ("bf16", 128, 7, 3, "fp32")])
def test_scores_of_any_size(size, kind, hd, group, M, dtype):
    """Scores up to 2^100 in base 2, of either sign or all far below zero: the
    largest takes all (the next is 2^-12 of it below, thousands in base 2 from
    2^27 on; at 2^20 some 300), equal ones share it.  o is within the cut of
    weights and sums of it, lse within six roundings, 2^-24 each, of the score."""
    gen = gen_of(int(math.log2(size)) + hd)
    T, page, n = 960, 32, 5
    step = torch.stack([torch.randperm(T, generator=gen, device="cuda") for _ in range(n)])
    sc = size * (1 - 2.0 * step / T)                         # from size down to -size
    sc[1] = size * (-0.8 - 0.15 * step[1] / T)               # all below zero
    sc[2] = -size * 0.9                                      # all the same
    sc[3] = torch.where(step[3] < 40, size, sc[3] / 2)       # 40 of them the same
    c, table = sequences(kind, hd, page, sc * LN2, torch.ones_like(sc), gen)
    q = torch.zeros(n, M, group, hd, device="cuda", dtype=TYPES[dtype])
    q[..., 0] = 1.0
    copies, start = 48, [T - M] * n
    o, lse = call(c, q.repeat(copies, 1, 1, 1), table.repeat(copies, 1), ints(start * copies), 1.0)
    for i in range(n):
        k, v = (held(c, x, table, i, T, page)[0] for x in "kv")
        for m in range(M):
            s = k[:T - M + m + 1, 0]
            top = s.max()
            best = s == top
            want, wl = v[:T - M + m + 1][best].mean(0), top + best.sum().double().log()
            tol = 2.0 ** -18 * v.abs().max() + (2.0 ** -8 * want.abs() if dtype == "bf16" else 0)
            assert ((o.view(copies, n, M, group, hd)[:, i, m].double() - want).abs() <= tol).all()
            assert ((lse.view(copies, n, M, group)[:, i, m].double() - wl).abs() <= 2.0 ** -21 * wl.abs()).all()


@pytest.mark.parametrize("kind,hd,group,M,dtype", [("int8", 128, 4, 2, "bf16"), ("e4m3", 64, 2, 4, "fp32"),
                                                   ("bf16", 128, 2, 3, "bf16"), ("bf16", 64, 3, 5, "fp32"),
                                                   ("int8", 256, 6, 4, "fp32"), ("bf16", 128, 8, 3, "fp32"),
                                                   ("e4m3", 256, 8, 2, "bf16")])
@pytest.mark.parametrize("copies", [1, 60])
def test_rows_of_padding_touch_no_other(kind, hd, group, M, dtype, copies):
    """The bits of a sequence's tokens, whatever the rows of tokens hold that it
    has not."""
    gen = gen_of(hd + M)
    page, T, n = 32, 1500, 3
    cols = -(-T // page)
    c = make_cache(kind, n * cols, 1, page, hd, gen, "cuda")
    table = make_table(n * cols, n, cols, gen, "cuda").repeat(copies, 1)
    q = 3 * torch.randn(n, M, group, hd, generator=gen, device="cuda")
    counts = [1, M - 1, M]
    start = ints([T - m for m in counts] * copies)
    have = torch.arange(M, device="cuda") < torch.tensor(counts, device="cuda")[:, None]

    def run(x):
        return call(c, x.to(TYPES[dtype]).repeat(copies, 1, 1, 1), table, start, 0.2, counts=ints(counts * copies))

    o, lse = run(torch.where(have[..., None, None], q, torch.zeros_like(q)))
    for junk in (1e30, float("nan"), -float("inf"), 5.0):
        o2, lse2 = run(torch.where(have[..., None, None], q, torch.full_like(q, junk)))
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kind,hd,group,M", [("int8", 128, 8, 3), ("e4m3", 128, 8, 3), ("bf16", 128, 8, 3),
                                             ("int8", 256, 8, 3), ("e4m3", 256, 6, 4), ("bf16", 256, 8, 2),
                                             ("int8", 64, 8, 2), ("int8", 128, 8, 2), ("int8", 128, 8, 1)])
def test_sums_do_not_drift(kind, hd, group, M):
    """Equal weights over values of one sign, in a batch that gives every warp
    a sequence's tiles of its own: o is their mean.  A tile's sum is cut off at
    most four times (2^-23 each) and its weights are held to 2^-22; n tiles are
    added to o and their weights to l, rounded, 2^-25 each, in either
    direction: 2 n^0.5 2^-25.  Sums that are cut off n times instead lose some
    n 2^-24."""
    gen = gen_of(hd + M)
    page, T, kvh, B = 64, 60000, 4, 40
    cols = -(-T // page)
    c = make_cache(kind, cols, kvh, page, hd, gen, "cuda", spread=0.0)
    c["v"] = (c["v"].float().abs() + 0.5).to(c["v"].dtype)
    table = make_table(cols, 1, cols, gen, "cuda").expand(B, cols).contiguous()
    q = torch.zeros(B, M, kvh * group, hd, device="cuda")
    o, _ = call(c, q, table, ints([T - M] * B), 1.0)
    v = held(c, "v", table, 0, T, page)
    n = T / 128
    for m in range(M):
        want = v[:, :T - M + m + 1].mean(1).repeat_interleave(group, 0)
        far = (o[:, m].double() - want).norm(dim=(1, 2)) / want.norm()
        assert far.max() <= 2.0 ** -21 + 2.0 ** -22 + 2 * n ** 0.5 * 2.0 ** -25


@pytest.mark.parametrize("kind,hd,group,M", [("bf16", 128, 4, 1), ("bf16", 64, 3, 3), ("bf16", 256, 2, 1), ("int8", 128, 4, 1)])
def test_queries_of_the_largest_floats(kind, hd, group, M):
    """fp32 queries up to 3.4028e38 over keys as small as that makes the scores
    ordinary; infinite ones make NaN of their row."""
    gen = gen_of(hd)
    T, page, n = 700, 16, 3
    sc = 20 * torch.rand(n, T, generator=gen, device="cuda", dtype=torch.float64) / 3.4e38
    c, table = sequences(kind, hd, page, sc, torch.ones_like(sc), gen)
    q = torch.zeros(n, M, group, hd, device="cuda")
    q[..., 0] = 3.4028234e38
    q[:, :, 1, 0] = -3.395e38
    check_many(c, table, kind, "fp32", q, T, page, copies=20)
    q[:, :, 0, 0] = float("inf")
    o, _ = call(c, q, table, ints([T - M] * n), 1.0)
    assert bool(o[:, :, 0].isnan().all()) and bool(torch.isfinite(o[:, :, 1:]).all())


@pytest.mark.parametrize("kind,hd,dtype,M,group", [("e4m3", 256, "fp32", 4, 6), ("int8", 256, "bf16", 3, 7), ("int8", 256, "fp32", 2, 8),
                                                   ("bf16", 128, "bf16", 3, 7), ("int8", 128, "fp32", 4, 6), ("e4m3", 64, "fp32", 4, 4),
                                                   ("bf16", 256, "fp32", 2, 8), ("bf16", 64, "bf16", 2, 7)])
def test_drafts_over_long_sequences(kind, hd, dtype, M, group):
    """9 to 24 rows a head over 60000 positions, joined from many CTAs, and
    shorter ones beside them."""
    gen = gen_of(hd + group)
    page, T = 64, [60000, 33, 20011]
    cols = -(-max(T) // page)
    c = make_cache(kind, 3 * cols, 2, page, hd, gen, "cuda")
    table = make_table(3 * cols, 3, cols, gen, "cuda")
    junk_behind(c, table, T, page, kind)
    q = (2 * torch.randn(3, M, 2 * group, hd, generator=gen, device="cuda")).to(TYPES[dtype])
    check(c, kind, dtype, q, table, [t - M for t in T], None, hd ** -0.5, page)


@pytest.mark.parametrize("name", BEHIND)
@pytest.mark.parametrize("kind,hd,group,M,dtype", [("int8", 128, 4, 1, "bf16"), ("e4m3", 256, 6, 4, "fp32"), ("int8", 64, 5, 2, "fp32")])
@pytest.mark.parametrize("copies", [1, 9])
def test_scales_move_no_weights_in_joins(name, kind, hd, group, M, dtype, copies):
    """The same over sequences that many CTAs share: parts with and without a
    unit of their own, joined by items and by CTAs."""
    gen = gen_of(hd + copies)
    T, page, n = 9000, 64, 4
    part = torch.arange(T, device="cuda").expand(n, T) * 3 // T
    part = torch.where(torch.arange(n, device="cuda")[:, None] < 2, part,
                       torch.randint(0, 3, (n, T), generator=gen, device="cuda"))
    sc, vs = (torch.tensor([float(p[i]) for p in BEHIND[name]], dtype=torch.float64, device="cuda")[part] for i in (0, 1))
    sc = (sc + torch.rand(n, T, generator=gen, device="cuda")) * LN2
    c, table = sequences(kind, hd, page, sc, vs, gen)
    q = torch.zeros(n, M, group, hd, device="cuda")
    q[..., 0] = 1.0
    q[:, :, 1::2, 0] = 0.75
    check_many(c, table, kind, dtype, q.to(TYPES[dtype]), T, page, copies)
