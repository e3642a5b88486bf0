"""Projections with 4-bit weights against a plain 64-bit product.

Tolerance, against the magnitude sum |x||w|: an element of x enters as it is
(bf16), as a sum of two 11-bit parts (fp32, few rows: 2^-22) or of three 8-bit
parts (fp32, many rows: exact), codes are exact, code * scale is exact in fp32,
and the fp32 sums run over at most K / 16 + 64 steps of 2^-23 (a tensor product
may truncate).  bf16 results add their own rounding.
"""

import pytest
import torch

import gated_deltanet_linear_gb300 as gdn
from linattn_ref import (assert_within, half_step, linattn, make_linattn, make_quant,
                         quant_linear, weights)

pytestmark = pytest.mark.gpu
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def tol(K, dtype, ref, mag):
    t = (K / 16 + 64) * 2.0 ** -23
    return t * mag + half_step(dtype) * (ref.abs() + t * mag)


def check(x, qw, sc):
    y = torch.full((x.shape[0] + 1, qw.shape[0]), -3.0, device="cuda", dtype=x.dtype)
    gdn.gdn_quant_linear(x, qw, sc, y[:-1])
    ref, mag = quant_linear(x, qw, sc)
    assert_within(y[:-1], ref, tol(x.shape[1], x.dtype, ref, mag), "y")
    assert (y[-1] == -3.0).all()
    return y[:-1]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,N,groups", [
    (1, 1, 1), (1, 48, 40), (1, 1000, 3), (2, 17, 5), (3, 129, 7), (4, 16, 64), (5, 300, 9),
    (7, 33, 2), (8, 2056, 20), (9, 64, 33), (13, 15, 3), (16, 500, 8), (17, 130, 11),
    (33, 257, 4), (64, 700, 21), (65, 40, 6), (130, 129, 3), (300, 20, 2)])
def test_product(dtype, group, rows, N, groups):
    check(*make_quant(rows * N + group, rows, N, groups * group, group, TYPES[dtype]))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 6, 40])
def test_codes_and_order(dtype, rows):
    """Every code at every position: x picks single elements, scales are
    powers of two, so results are exact."""
    K, N, group = 256, 64, 32
    qw = torch.arange(N * K // 2, device="cuda").mul(37).remainder(256).to(torch.uint8).view(N, K // 2)
    sc = torch.exp2((torch.arange(N * K // group, device="cuda") % 9 - 4).float()).half().view(N, -1)
    w = weights(qw, sc)
    for k0 in range(0, K, rows):
        k = torch.arange(k0, min(K, k0 + rows), device="cuda")
        x = torch.zeros(len(k), K, device="cuda", dtype=TYPES[dtype])
        x[torch.arange(len(k)), k] = 1.0
        y = torch.empty(len(k), N, device="cuda", dtype=TYPES[dtype])
        gdn.gdn_quant_linear(x, qw, sc, y)
        assert torch.equal(y.double(), w[:, k].t())


@pytest.mark.parametrize("rows", [1, 5, 40])
def test_ranges(rows):
    """Rows of very different size beside each other, elements far below
    their row's largest, scales down to fp16's subnormals."""
    x, qw, sc = make_quant(3, rows, 200, 512, 64)
    x *= torch.logspace(-20, 20, rows, device="cuda")[:, None]
    x[:, ::3] *= 2.0 ** -20
    x[:, 1::5] = 0.0
    sc = sc * 0 + torch.logspace(-7, 4, sc.numel(), device="cuda").view_as(sc).half()
    check(x, qw, sc)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 5, 40])
def test_small_codes(dtype, rows):
    """Rows of zeros give zeros; codes of -1, 0, 1 keep the accuracy that
    their own magnitude allows."""
    x, qw, sc = make_quant(8, rows, 90, 512, 64, TYPES[dtype])
    half = torch.tensor([0, 1, 15], device="cuda", dtype=torch.uint8)
    pick = torch.randint(0, 3, (2, *qw.shape), device="cuda",
                         generator=torch.Generator("cuda").manual_seed(1))
    qw = half[pick[0]] | half[pick[1]] << 4
    qw[::3] = 0
    y = check(x, qw, sc)
    assert (y[:, ::3] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 5, 40])
def test_large_elements(dtype, rows):
    """Elements of 2^112, the largest that every group's sum of code x (before
    its scale) is promised to stay finite for."""
    x, qw, sc = make_quant(5, rows, 60, 256, 128, TYPES[dtype])
    x.copy_(torch.where(x > 0, 2.0 ** 112, -2.0 ** 112))
    check(x, qw, sc)
    x.fill_(2.0 ** 112)
    check(x, qw, sc)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 5, 40])
def test_non_finite_rows_stay_apart(dtype, rows):
    x, qw, sc = make_quant(4, rows + 2, 100, 256, 64, TYPES[dtype])
    y0 = check(x, qw, sc)
    x[0, 5], x[-1, 7] = float("nan"), float("inf")
    y = torch.empty_like(y0)
    gdn.gdn_quant_linear(x, qw, sc, y)
    assert not torch.isfinite(y[0]).any() and torch.isnan(y[0]).all()
    code = weights(qw, sc)[:, 7] != 0
    assert not torch.isfinite(y[-1][code]).any()
    assert torch.equal(y[1:-1], y0[1:-1])
    x[0] = 0
    gdn.gdn_quant_linear(x, qw, sc, y)
    assert (y[0] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_many_rows_on_three_streams(dtype):
    """Clusters of several calls side by side, of each group size."""
    jobs = [make_quant(60 + g, rows, 2600, 2048, g, TYPES[dtype])
            for g, rows in ((32, 20), (64, 30), (128, 50), (32, 64))]
    ref = [torch.empty(x.shape[0], 2600, device="cuda", dtype=x.dtype) for x, _, _ in jobs]
    got = [[torch.empty_like(y) for y in ref] for _ in range(3)]
    for (x, qw, sc), y in zip(jobs, ref):
        gdn.gdn_quant_linear(x, qw, sc, y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in got]
    for turn in range(20):
        for i, (stream, ys) in enumerate(zip(streams, got)):
            j = (turn + i) % len(jobs)
            gdn.gdn_quant_linear(*jobs[j], ys[j], stream=stream)
    torch.cuda.synchronize()
    assert all(torch.equal(y, r) for ys in got for y, r in zip(ys, ref))
    assert gdn.gdn_wait_timeouts() == 0


def test_same_bits_and_graph():
    for rows in (1, 8, 50):
        x, qw, sc = make_quant(6, rows, 777, 1024, 128)
        y, y2 = (torch.empty(rows, 777, device="cuda") for _ in range(2))
        gdn.gdn_quant_linear(x, qw, sc, y)
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=stream):
            gdn.gdn_quant_linear(x, qw, sc, y2)
        y2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y2)


def test_weights_beyond_32_bits():
    """More than 2^32 weights: the last rows against their own product."""
    N, K, group = 300000, 16384, 128
    x, qw, sc = make_quant(8, 2, 1000, K, group)
    big, bs = qw.repeat(N // 1000, 1), sc.repeat(N // 1000, 1)
    y = torch.empty(2, N, device="cuda")
    gdn.gdn_quant_linear(x, big, bs, y)
    ref, mag = quant_linear(x, qw, sc)
    t = tol(K, x.dtype, ref, mag)
    for a in (0, N // 2, N - 1000):
        assert_within(y[:, a:a + 1000], ref, t, f"rows from {a}")


@pytest.mark.parametrize("rows", [1, 4])
def test_layer_run(rows):
    """In-projection, linear-attention steps, gated norm, out-projection: one
    layer step from hidden state to hidden state, against the same in fp64."""
    B, kh, vh, hidden = rows, 2, 4, 512
    conv = 2 * kh * 128 + vh * 128
    x, w_in, s_in = make_quant(1, B, conv, hidden, 64)
    z, w_out, s_out = make_quant(2, B, hidden, vh * 128, 64)
    d = make_linattn(3, B, 1, kh, vh, decay="head")
    w = torch.ones(128, device="cuda")
    proj = torch.empty(B, conv, device="cuda")
    gdn.gdn_quant_linear(x, w_in, s_in, proj)
    q, k, v = (t.contiguous() for t in proj.split([kh * 128, kh * 128, vh * 128], 1))
    S, o = d["S"].clone(), torch.empty(B, vh, 128, device="cuda")
    gdn.gdn_linattn_step(S, q.view(B, kh, 128), k.view(B, kh, 128), v.view(B, vh, 128), d["g"], o)
    y = torch.empty(B, 1, vh, 128, device="cuda")
    gdn.gdn_gated_rmsnorm_m(o.view(B, 1, vh, 128), z.view(B, 1, vh, 128), w, y)
    out = torch.empty(B, hidden, device="cuda")
    gdn.gdn_quant_linear(y.view(B, vh * 128), w_out, s_out, out)
    # fp64
    p, _ = quant_linear(x, w_in, s_in)
    q, k, v = p.split([kh * 128, kh * 128, vh * 128], 1)
    ref = linattn(d["S"], q.view(B, 1, kh, 128), k.view(B, 1, kh, 128), v.view(B, 1, vh, 128), d["g"])
    r = ref["o"] / (ref["o"].square().mean(-1, keepdim=True) + 1e-6).sqrt()
    zz = z.double().view(B, 1, vh, 128)
    r = (r * zz * torch.sigmoid(zz)).view(B, vh * 128)
    want, _ = quant_linear(r, w_out, s_out)
    # each stage is off by at most some 2^-17 of its magnitudes; the sums here
    # cancel by less than 2^5
    assert (out - want).norm() <= 2.0 ** -12 * want.norm()
    assert (S - ref["S"]).norm() <= 2.0 ** -12 * ref["S"].norm()


def test_refusals():
    x, qw, sc = make_quant(1, 2, 10, 128, 64)
    y = torch.empty(2, 10, device="cuda")
    with pytest.raises(ValueError):
        gdn.gdn_quant_linear(x.half(), qw, sc, y)
    with pytest.raises(ValueError):
        gdn.gdn_quant_linear(x, qw, sc.float(), y)
    with pytest.raises(ValueError):
        gdn.gdn_quant_linear(x, qw[:, :-1].contiguous(), sc, y)
    with pytest.raises(ValueError):
        gdn.gdn_quant_linear(x, qw, sc, y.t())
    with pytest.raises(gdn.GDNError) as e:
        gdn.gdn_quant_linear(x, qw, sc.repeat(1, 4)[:, :8].contiguous(), y)  # groups of 16
    assert e.value.status == gdn.GDN_ESHAPE
    big = torch.empty(64, 64, device="cuda")
    with pytest.raises(gdn.GDNError) as e:  # y over x
        gdn.gdn_quant_linear(big, torch.zeros(64, 32, device="cuda", dtype=torch.uint8),
                             torch.ones(64, 1, device="cuda").half(), big)
    assert e.value.status == gdn.GDN_EALIAS


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 5, 40])
@pytest.mark.parametrize("K", [32, 96, 288])
def test_infinite_scales(dtype, rows, K):
    """An infinite scale of the last group of a row whose length ends inside a
    block gives an infinity, and NaN stays with its row of weights."""
    x = torch.ones(rows, K, device="cuda", dtype=TYPES[dtype])
    qw = torch.full((7, K // 2), 0x11, device="cuda", dtype=torch.uint8)
    sc = torch.ones(7, K // 32, device="cuda", dtype=torch.float16)
    sc[2, -1], sc[4, -1], sc[5, -1] = float("inf"), -float("inf"), float("nan")
    y = torch.empty(rows, 7, device="cuda", dtype=TYPES[dtype])
    gdn.gdn_quant_linear(x, qw, sc, y)
    want = torch.full_like(y, K)
    want[:, 2], want[:, 4], want[:, 5] = float("inf"), -float("inf"), float("nan")
    assert torch.equal(y.isnan(), want.isnan())
    assert torch.equal(y.nan_to_num(1.5, 1e38, -1e38), want.nan_to_num(1.5, 1e38, -1e38))


@pytest.mark.parametrize("B,T", [(2, 90), (1, 300)])
def test_layer_run_after_a_prompt(B, T):
    """The same layer over a padded prompt, then one token: projections of all
    rows, prompt, token, gated norm, out-projection, against fp64."""
    kh, vh, hidden = 2, 4, 512
    conv = 2 * kh * 128 + vh * 128
    rows = B * (T + 1)
    x, w_in, s_in = make_quant(11, rows, conv, hidden, 64)
    z, w_out, s_out = make_quant(12, rows, hidden, vh * 128, 64)
    d = make_linattn(13, B, 1, kh, vh, decay="head")
    lens = torch.tensor([T - 17] + [T] * (B - 1), dtype=torch.int32, device="cuda")
    w = torch.ones(128, device="cuda")
    proj = torch.empty(rows, conv, device="cuda")
    gdn.gdn_quant_linear(x, w_in, s_in, proj)
    parts = proj.view(B, T + 1, conv).split([kh * 128, kh * 128, vh * 128], 2)
    q, k, v = (t.reshape(B, T + 1, -1, 128) for t in parts)
    S = d["S"].clone()
    o = torch.zeros(B, T + 1, vh, 128, device="cuda")
    n = gdn.gdn_linattn_prefill_workspace(B, kh, vh, T)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    po, to = torch.zeros(B, T, vh, 128, device="cuda"), torch.empty(B, vh, 128, device="cuda")
    gdn.gdn_linattn_prefill(S, *(t[:, :T].contiguous() for t in (q, k, v)), d["g"], po,
                            lens=lens, workspace=ws)
    gdn.gdn_linattn_step(S, *(t[:, T].contiguous() for t in (q, k, v)), d["g"], to)
    o[:, :T], o[:, T] = po, to
    y = torch.empty_like(o)
    gdn.gdn_gated_rmsnorm_m(o, z.view_as(o), w, y)
    out = torch.empty(rows, hidden, device="cuda")
    gdn.gdn_quant_linear(y.view(rows, vh * 128), w_out, s_out, out)
    # fp64
    p, _ = quant_linear(x, w_in, s_in)
    parts = p.view(B, T + 1, conv).split([kh * 128, kh * 128, vh * 128], 2)
    q, k, v = (t.reshape(B, T + 1, -1, 128) for t in parts)
    first = linattn(d["S"], q[:, :T], k[:, :T], v[:, :T], d["g"], lens=lens.long())
    token = linattn(first["S"], q[:, T:], k[:, T:], v[:, T:], d["g"])
    on = torch.arange(T, device="cuda") < lens[:, None]
    ref = torch.cat([first["o"] * on[..., None, None], token["o"]], 1)
    r = ref / (ref.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    zz = z.double().view_as(r)
    r = (r * zz * torch.sigmoid(zz)).view(rows, vh * 128)
    want, _ = quant_linear(r, w_out, s_out)
    # (as in test_layer_run)
    assert (out - want).norm() <= 2.0 ** -12 * want.norm()
    assert (S - token["S"]).norm() <= 2.0 ** -12 * token["S"].norm()
    pad = ~torch.cat([on, on.new_ones(B, 1)], 1).view(rows)
    assert (out[pad] == 0).all()
