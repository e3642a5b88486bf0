"""Linear attention with a decay for each head, against a plain 64-bit form.

Tolerances, all against the magnitude (the same recurrence over absolute
values, mS for the state and mo for an output):
  step   a token multiplies by exp(g) (CUDA's expf: 2 units in the last place,
         2^-22) and rounds a product and a multiply-add (2^-24 each), so n
         tokens give n (2^-22 + 2^-23) mS; o adds 8 multiply-adds, 4 sums
         and the scale, 13 roundings, and its own rounding to 16 bits.
  prompt the larger of that and of the chunked form's bound: operands as
         sums of two fp16 numbers (2^-22 of each, 2^-22 for the product of the
         two small parts), fp32 accumulation of at most 24 steps of a tensor
         product that may truncate (24 * 2^-23), the decays' exponentials, all
         below 2^-18 a chunk of 64, carried through n / 64 + 2 chunks:
         (n / 4 + 32) 2^-22.  With bf16 rows the products of o take the scores
         and the state rounded to fp16, 2^-11 of the magnitude each.
"""

import ctypes
import os
import subprocess
import sys

import pytest
import torch

import gated_deltanet_linear_gb300 as gdn
from linattn_ref import D, assert_within, half_step, linattn, make_linattn

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def step_tol(n):
    return n * 1.5 * 2.0 ** -22, (n * 6 + 14) * 2.0 ** -24


def check_steps(d, got_S, got_o, got_states=None, scale=1.0):
    n = d["v"].shape[1]
    ref = linattn(d["S"], d["q"], d["k"], d["v"], d["g"], scale, states=got_states is not None)
    ts, to = step_tol(n)
    assert_within(got_S, ref["S"], ts * ref["mS"], "S")
    h = half_step(d["v"].dtype)
    assert_within(got_o, ref["o"], to * ref["mo"] + h * (ref["o"].abs() + to * ref["mo"]), "o")
    if got_states is not None:
        # |S_m| <= m-th magnitude <= sum over the tokens so far
        mag = linattn_magnitudes(d)
        assert_within(got_states, ref["states"], ts * mag, "checkpoints")


def linattn_magnitudes(d):
    a = {x: d[x].abs() if x != "g" else d[x] for x in d}
    return linattn(a["S"], a["q"], a["k"], a["v"], a["g"], states=True)["states"]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("B,kh,vh,n,ckpt", [
    (1, 1, 1, 1, False), (3, 2, 6, 1, False), (2, 16, 48, 1, True), (5, 3, 3, 2, True),
    (2, 4, 8, 8, False), (1, 2, 2, 9, True), (1, 1, 3, 33, False)])
def test_steps(dtype, decay, B, kh, vh, n, ckpt):
    d = make_linattn(7 * B + n, B, n, kh, vh, TYPES[dtype], decay)
    S_out, o = torch.empty_like(d["S"]), torch.empty_like(d["v"])
    ck = torch.empty(n, *d["S"].shape, device="cuda") if ckpt else None
    keep = d["S"].clone()
    gdn.gdn_linattn_step_m(d["S"], S_out, ck, d["q"], d["k"], d["v"], d["g"], o, scale=0.75)
    check_steps(d, S_out, o, ck, scale=0.75)
    assert torch.equal(d["S"], keep)
    if ckpt:
        assert torch.equal(ck[-1], S_out)
    S = d["S"].clone()
    o2 = torch.empty_like(o)
    gdn.gdn_linattn_step_m(S, S, None, d["q"], d["k"], d["v"], d["g"], o2, scale=0.75)
    assert torch.equal(S, S_out) and torch.equal(o, o2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("B,n", [(2, 11), (70, 3)])
def test_many_tokens_are_single_tokens(dtype, decay, B, n):
    d = make_linattn(5, B, n, 4, 12, TYPES[dtype], decay)
    S_out, o = torch.empty_like(d["S"]), torch.empty_like(d["v"])
    ck = torch.empty(n, *d["S"].shape, device="cuda")
    gdn.gdn_linattn_step_m(d["S"], S_out, ck, d["q"], d["k"], d["v"], d["g"], o)
    S = d["S"].clone()
    for t in range(n):
        ot = torch.empty_like(o[:, 0])
        gdn.gdn_linattn_step(S, *(d[x][:, t].contiguous() for x in "qkv"),
                             d["g"] if decay == "head" else d["g"][:, t].contiguous(), ot)
        assert torch.equal(ot, o[:, t]) and torch.equal(S, ck[t])
    assert torch.equal(S, S_out)
    # the states are the library's: its rollback serves them
    m = torch.arange(B, device="cuda", dtype=torch.int32) % (n + 1)
    gdn.gdn_rollback_seq(S, n, m, d["S"], ck, 4)
    for b in range(B):
        want = d["S"][b] if m[b] == 0 else ck[int(m[b]) - 1, b]
        assert torch.equal(S[b], want)


def test_single_token_keeps_a_token_dimension():
    d = make_linattn(3, 2, 1, 2, 4)
    S, S2 = d["S"].clone(), d["S"].clone()
    o, o2 = torch.empty_like(d["v"]), torch.empty_like(d["v"])
    gdn.gdn_linattn_step(S, d["q"], d["k"], d["v"], d["g"], o)
    gdn.gdn_linattn_step_m(S2, S2, None, d["q"], d["k"], d["v"], d["g"], o2)
    assert torch.equal(S, S2) and torch.equal(o, o2)


@pytest.mark.parametrize("T", [1, 3, 70])
def test_decay_extremes(T):
    """g = -inf empties the state, g = 0 keeps it, and what one head holds
    (infinities, NaN) stays out of the others."""
    d = make_linattn(9, 2, T, 2, 4)
    g = torch.zeros_like(d["g"])
    g[:, 0, 1] = -float("inf")
    if T > 2:
        g[:, 2, 2] = -float("inf")
    g[:, T // 2, 3] = -200.0
    d["g"] = g
    d["S"][1, 0] = float("nan")
    ref = linattn(d["S"], d["q"], d["k"], d["v"], g)
    for call in ("step", "prefill"):
        S, o = d["S"].clone(), torch.empty_like(d["v"])
        run(call, S, d, o)
        assert torch.isnan(S[1, 0]).all() and torch.isnan(o[1, :, 0]).all()
        for x, r, m in ((S, ref["S"], ref["mS"]), (o.transpose(1, 2), ref["o"].transpose(1, 2),
                                                    ref["mo"].transpose(1, 2))):
            tol = prompt_tol(T)[0] * m
            assert_within(x[0], r[0], tol[0], call)
            assert_within(x[1, 1:], r[1, 1:], tol[1, 1:], call)


# ------------------------------------------------------------------ prompts

def workspace(d):
    B, T, vh, _ = d["v"].shape
    n = gdn.gdn_linattn_prefill_workspace(B, d["q"].shape[2], vh, T, dtype=d["v"].dtype)
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def run(call, S, d, o, **more):
    if call == "step":
        gdn.gdn_linattn_step_m(S, S, None, d["q"], d["k"], d["v"], d["g"], o, **more)
    else:
        gdn.gdn_linattn_prefill(S, d["q"], d["k"], d["v"], d["g"], o,
                                workspace=workspace(d), **more)


def prompt_tol(T, dtype=torch.float32):
    t = (1.5 * T + 32) * 2.0 ** -22
    return t, t + (2.0 ** -10 if dtype == torch.bfloat16 else 0.0)


def check_prompt(d, S, o, scale=1.0, lens=None, floor_S=0.0, floor_o=0.0):
    B, T, vh, _ = d["v"].shape
    clean = d
    if lens is not None:  # the plain form reads the rows behind a length as zeros
        on = (torch.arange(T, device="cuda") < lens[:, None])
        clean = {x: t if x == "S" or t.dim() == 1 else
                 torch.where(on.view(B, T, *[1] * (t.dim() - 2)), t, torch.zeros_like(t))
                 for x, t in d.items()}
    ref = linattn(clean["S"], clean["q"], clean["k"], clean["v"], clean["g"], scale, lens=lens)
    ts, to = prompt_tol(T, d["v"].dtype)
    assert_within(S, ref["S"], ts * ref["mS"] + floor_S, "S")
    tol = floor_o + to * ref["mo"] + half_step(d["v"].dtype) * (ref["o"].abs() + to * ref["mo"])
    if lens is not None:
        o = torch.where(on[..., None, None], o.double(), ref["o"])
    assert_within(o, ref["o"], tol, "o")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("B,kh,vh,T", [
    (1, 1, 1, 1), (2, 2, 6, 2), (1, 3, 3, 31), (1, 1, 2, 63), (2, 1, 1, 64), (1, 2, 2, 65),
    (1, 16, 48, 127), (3, 1, 4, 128), (1, 1, 1, 129), (1, 2, 4, 300), (1, 1, 2, 1000)])
def test_prompts(dtype, decay, B, kh, vh, T):
    d = make_linattn(T, B, T, kh, vh, TYPES[dtype], decay)
    S, o = d["S"].clone(), torch.empty_like(d["v"])
    run("prefill", S, d, o, scale=1.25)
    check_prompt(d, S, o, scale=1.25)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [50, 200])
def test_prompts_with_strong_decay(dtype, T):
    """Decays down to e^-60 a token: differences of sums of hundreds."""
    d = make_linattn(40 + T, 2, T, 1, 3, TYPES[dtype], strong=True)
    S, o = d["S"].clone(), torch.empty_like(d["v"])
    run("prefill", S, d, o)
    check_prompt(d, S, o)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 64, 90, 333])
def test_lengths(dtype, T):
    """Padded rows hold NaN and infinities; o behind a length keeps its
    values; a length outside 0..T leaves its sequence alone."""
    lens = torch.tensor([T, 0, 1, max(1, T // 2), T - 1, T + 1, -1], dtype=torch.int32,
                        device="cuda")
    B = lens.numel()
    d = make_linattn(11, B, T, 2, 4, TYPES[dtype])
    for b in range(B):
        n = int(lens[b]) if 0 <= lens[b] <= T else 0
        for x, bad in (("q", float("nan")), ("k", float("inf")), ("v", float("nan")),
                       ("g", float("nan"))):
            d[x][b, n:] = bad
    S, o = d["S"].clone(), torch.full_like(d["v"], 7.5)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    run("prefill", S, d, o, lens=lens, err_dev=err)
    assert int(err) == 1
    for b in range(B):
        n = int(lens[b]) if 0 <= lens[b] <= T else 0
        assert (o[b, n:] == 7.5).all()
        if n == 0:
            assert torch.equal(S[b], d["S"][b])
    good = slice(0, 5)
    check_prompt({x: t[good] for x, t in d.items()}, S[good], o[good], lens=lens[good].long())
    err.zero_()
    S5, o5 = d["S"][good].clone(), o[good].clone()
    d5 = {x: t[good].contiguous() for x, t in d.items()}
    run("prefill", S5, d5, o5, lens=lens[good].contiguous(), err_dev=err)
    assert int(err) == 0
    # (another batch size may cut the sequences elsewhere: not the same bits)
    check_prompt(d5, S5, o5, lens=lens[good].long())


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_of_very_different_size(dtype):
    """Key and value rows from 1e-6 to 1e6 within one chunk: a normwise error
    per row of the magnitude that the definition allows it."""
    d = make_linattn(21, 1, 150, 1, 2, TYPES[dtype])
    s = torch.logspace(-3, 3, 150, device="cuda")[torch.randperm(150, generator=torch.Generator().manual_seed(1))]
    d["k"] = (d["k"].float() * s[None, :, None, None]).to(TYPES[dtype])
    d["v"] = (d["v"].float() * s.flip(0)[None, :, None, None]).to(TYPES[dtype])
    S, o = d["S"].clone(), torch.empty_like(d["v"])
    run("prefill", S, d, o)
    check_prompt(d, S, o)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("decay", [0.0, -0.5, -1.1, -5.0])
@pytest.mark.parametrize("zero", ["q", "k", "v", "all"])
def test_zero_rows(dtype, decay, zero):
    """Rows of zeros at a prompt's start and within it (their scales are free),
    next to decays whose factors across a chunk span the range of a float."""
    T = 150
    d = make_linattn(23, 1, T, 1, 2, TYPES[dtype])
    d["g"].fill_(decay)
    for x in "qkv" if zero == "all" else zero:
        d[x][:, :40] = 0
        d[x][:, 70:75] = 0
        d[x][:, 128:] = 0
    S, o = d["S"].clone(), torch.empty_like(d["v"])
    run("prefill", S, d, o)
    # What the magnitudes of the terms do not cover:
    # e^-5 a token takes whole sums below fp32; a factor under the smallest normal
    # number, 2^-126, may read as 0.  It multiplies |k v| or |q.k v| of at most T
    # tokens, or |S0 q| summed over 128 rows: each below 16, as q and k are
    # (rounded) unit rows and |v|, |S0| are below 5.
    assert max(float(d[x].abs().max()) for x in ("v", "S")) < 5
    assert max(float(d[x].float().norm(dim=-1).max()) for x in "qk") < 2 ** 0.5
    under = (T + 128) * 16 * 2.0 ** -126
    # A score (q_t.k_s) e^{decay} is the sum of two fp16 numbers, the second
    # off by up to 2^-25 (half the spacing of fp16's smallest numbers), in units
    # of 2^22 (2^-14 |q_t|) (2^-14 2 w), |.| the largest element and w the row's
    # largest |k_s| e^{decay} <= |k|: by 2^-30 |q_t| |k|, times |v_s| of 64 tokens.
    # It shows where the tokens near t have v = 0 and the decays leave only
    # small weights for the others.
    top = {x: float(d[x].abs().max()) for x in "qkv"}
    score = 2.0 ** -30 * top["q"] * top["k"] * 64 * top["v"]
    check_prompt(d, S, o, floor_S=under, floor_o=under + score)


@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_then_tokens(dtype):
    """A prompt in two calls, then single tokens, is one longer sequence."""
    T, cut, B, kh, vh = 180, 97, 2, 2, 4
    d = make_linattn(31, B, T, kh, vh, TYPES[dtype])
    S, o = d["S"].clone(), torch.empty_like(d["v"])
    for a, z in ((0, cut), (cut, T - 3)):
        part = {x: (t if x == "S" else t[:, a:z].contiguous()) for x, t in d.items()}
        po = torch.empty_like(part["v"])
        run("prefill", S, part, po)
        o[:, a:z] = po
    for t in range(T - 3, T):
        ot = torch.empty_like(o[:, 0])
        gdn.gdn_linattn_step(S, *(d[x][:, t].contiguous() for x in "qkvg"), ot)
        o[:, t] = ot
    check_prompt(d, S, o)


@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_is_deterministic(dtype):
    """The same bits on every call."""
    d = make_linattn(17, 4, 140, 2, 6, TYPES[dtype])
    S, o = d["S"].clone(), torch.empty_like(d["v"])
    run("prefill", S, d, o)
    S2, o2 = d["S"].clone(), torch.empty_like(d["v"])
    run("prefill", S2, d, o2)
    assert torch.equal(S, S2) and torch.equal(o, o2)


@pytest.mark.parametrize("call,T", [("step", 2), ("prefill", 150)])
def test_graph_replay_and_streams(call, T):
    d = make_linattn(23, 2, T, 2, 4)
    S_ref, o_ref = d["S"].clone(), torch.empty_like(d["v"])
    run(call, S_ref, d, o_ref)
    run(call, S_ref, d, o_ref)
    S, o, ws = d["S"].clone(), torch.empty_like(d["v"]), workspace(d)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()

    def once():
        if call == "step":
            gdn.gdn_linattn_step_m(S, S, None, d["q"], d["k"], d["v"], d["g"], o)
        else:
            gdn.gdn_linattn_prefill(S, d["q"], d["k"], d["v"], d["g"], o, workspace=ws)

    with torch.cuda.graph(graph, stream=stream):
        once()
    S.copy_(d["S"])
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(S, S_ref) and torch.equal(o, o_ref)
    S.copy_(d["S"])
    o.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        once()
        once()
    stream.synchronize()
    assert torch.equal(S, S_ref) and torch.equal(o, o_ref)


def test_calls_at_once():
    """A prompt, tokens and projections on three streams at the same time, with
    workspaces of their own, against the same calls one after the other."""
    from linattn_ref import make_quant
    p = make_linattn(51, 3, 700, 2, 6)
    n = make_linattn(52, 9, 5, 2, 6, torch.bfloat16)
    xs = [make_quant(53 + r, r, 900, 1024, 64) for r in (3, 40)]
    ws = workspace(p)

    def outputs():
        return ([p["S"].clone(), torch.empty_like(p["v"]), n["S"].clone(), torch.empty_like(n["v"])]
                + [torch.empty(x.shape[0], 900, device="cuda") for x, _, _ in xs])

    def prompts(r, stream=None):
        for _ in range(6):
            gdn.gdn_linattn_prefill(r[0], p["q"], p["k"], p["v"], p["g"], r[1], workspace=ws,
                                    stream=stream)

    def tokens(r, stream=None):
        for _ in range(40):
            gdn.gdn_linattn_step_m(r[2], r[2], None, n["q"], n["k"], n["v"], n["g"], r[3],
                                   stream=stream)

    def projections(r, stream=None):
        for _ in range(30):
            for (x, qw, sc), y in zip(xs, r[4:]):
                gdn.gdn_quant_linear(x, qw, sc, y, stream=stream)

    ref, got = outputs(), outputs()
    for f in (prompts, tokens, projections):
        f(ref)
    torch.cuda.synchronize()
    for f in (prompts, tokens, projections):
        f(got, torch.cuda.Stream())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    assert gdn.gdn_wait_timeouts() == 0


def test_first_call_captured():
    """In a new process the first call of each entry is captured and replayed."""
    code = """
import sys; sys.path[:0] = [{root!r}, {tests!r}]
import torch, gated_deltanet_linear_gb300 as gdn
from linattn_ref import make_linattn, make_quant
p = make_linattn(1, 1, 600, 1, 2); n = make_linattn(2, 2, 3, 1, 2)
xs = [make_quant(r, r, 300, 512, 32) for r in (2, 30)]
ws = torch.empty(gdn.gdn_linattn_prefill_workspace(1, 1, 2, 600), dtype=torch.uint8, device="cuda")
def outs():
    return [p["S"].clone(), torch.empty_like(p["v"]), n["S"].clone(), torch.empty_like(n["v"])] + [
        torch.zeros(x.shape[0], 300, device="cuda") for x, _, _ in xs]
def calls(r):
    gdn.gdn_linattn_prefill(r[0], p["q"], p["k"], p["v"], p["g"], r[1], workspace=ws)
    gdn.gdn_linattn_step_m(r[2], r[2], None, n["q"], n["k"], n["v"], n["g"], r[3])
    for (x, qw, sc), y in zip(xs, r[4:]): gdn.gdn_quant_linear(x, qw, sc, y)
a, b = outs(), outs()
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph): calls(a)
graph.replay(); calls(b); torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(a, b))
""".format(root=os.path.dirname(HERE), tests=HERE)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_offsets_beyond_32_bits():
    """States and prompt rows behind 2^31 elements: the last sequence repeats
    the first one's bits."""
    vh, B = 512, 260                                  # 133,120 states: 2.18e9 elements
    d = make_linattn(2, 1, 1, 4, vh)
    S = torch.empty(B, vh, D, D, device="cuda")
    S[:] = d["S"]
    x = {n: d[n].expand(B, *d[n].shape[1:]).contiguous() for n in "qkvg"}
    o = torch.empty_like(x["v"])
    gdn.gdn_linattn_step_m(S, S, None, x["q"], x["k"], x["v"], x["g"], o)
    check_steps(d, S[:1], o[:1])
    assert torch.equal(S[-1], S[0]) and torch.equal(o[-1], o[0])
    del S, x, o
    B, T, kh, vh = 3, 65600, 1, 128                   # 2.5e9 elements of v
    d = make_linattn(3, 1, 128, kh, vh, torch.bfloat16)
    x = {n: torch.zeros(B, T, *d[n].shape[2:], device="cuda", dtype=d[n].dtype) for n in "qkvg"}
    for n in "qkvg":
        x[n][:, -128:] = d[n]
    S = torch.zeros(B, vh, D, D, device="cuda")
    o = torch.empty_like(x["v"])
    run("prefill", S, x, o)
    tail = {n: x[n][:1, -128:].contiguous() for n in "qkvg"}
    tail["S"] = torch.zeros(1, vh, D, D, device="cuda")
    check_prompt(tail, S[:1], o[:1, -128:])
    assert torch.equal(S[-1], S[0]) and torch.equal(o[-1, -128:], o[0, -128:])


def test_refusals():
    d = make_linattn(1, 2, 4, 2, 4)
    S, o = d["S"].clone(), torch.empty_like(d["v"])
    ok = (d["q"], d["k"], d["v"], d["g"])
    keep = S.clone()
    for bad in [dict(scale=float("nan")), dict(scale=float("inf"))]:
        with pytest.raises(gdn.GDNError) as e:
            gdn.gdn_linattn_step_m(S, S, None, *ok, o, **bad)
        assert e.value.status == gdn.GDN_EINVAL
    with pytest.raises(ValueError):  # a type of its own
        gdn.gdn_linattn_step_m(S, S, None, d["q"].half(), *ok[1:], o)
    with pytest.raises(ValueError):  # one tensor of another type
        gdn.gdn_linattn_step_m(S, S, None, d["q"].bfloat16(), *ok[1:], o)
    with pytest.raises(ValueError):  # strides
        gdn.gdn_linattn_step_m(S, S, None, d["q"].transpose(1, 2), *ok[1:], o)
    with pytest.raises(ValueError):  # a length too many
        gdn.gdn_linattn_prefill(S, *ok, o, lens=torch.zeros(3, dtype=torch.int32, device="cuda"),
                                workspace=workspace(d))
    for call in (lambda: gdn.gdn_linattn_step_m(S, S, None, *ok, d["v"]),
                 lambda: gdn.gdn_linattn_step_m(S, S, S[None].expand(1, *S.shape), *(t[:, :1].contiguous() for t in ok), o[:, :1].contiguous()),
                 lambda: gdn.gdn_linattn_prefill(S, *ok, d["v"], workspace=workspace(d))):
        with pytest.raises(gdn.GDNError) as e:  # o over v, the checkpoint over S
            call()
        assert e.value.status == gdn.GDN_EALIAS
    # misaligned and pageable pointers through the C ABI
    lib, sh = gdn.load(), gdn.Shape(2, 2, 4, 128, 128)
    ptr = [t.data_ptr() for t in (S, S)] + [None] + [t.data_ptr() for t in ok] + [o.data_ptr()]
    off = list(ptr)
    off[3] += 4
    call = lambda p: lib.gdn_linattn_step_m(ctypes.byref(sh), 4, 0, 0, 1.0, *p, None)
    assert call(off) == gdn.GDN_EALIGN
    cpu = torch.empty(1 << 16)
    off[3] = (cpu.data_ptr() + 15) & ~15
    assert call(off) == gdn.GDN_EPTR
    torch.cuda.synchronize()
    assert torch.equal(S, keep)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("what", ["q", "k", "v", "g"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_tokens_touch_only_later_rows(dtype, what, bad):
    """A token that is not finite leaves the rows before it, and (q: the rows
    after it; v: the other columns) what it has no part in, as they are."""
    if what == "g" and bad > 0:
        bad = float("nan")
    d = make_linattn(77, 1, 150, 1, 2, TYPES[dtype])
    clean = {x: t.clone() for x, t in d.items()}
    at = 37
    if what == "g":
        d["g"][0, at, 1] = bad
    else:
        d[what][0, at, -1, 5] = bad
    S, o = d["S"].clone(), torch.empty_like(d["v"])
    run("prefill", S, d, o)
    S0, o0 = clean["S"].clone(), torch.empty_like(d["v"])
    run("prefill", S0, clean, o0)
    touched = torch.zeros_like(o, dtype=torch.bool)
    if what == "q":
        touched[:, at] = True
        assert torch.isfinite(S).all()
    elif what == "k":
        touched[:, at:] = True
    elif what == "v":
        touched[:, at:, 1, 5] = True
        assert not torch.isfinite(S[0, 1, :, 5]).any()
    else:
        touched[:, at:, 1] = True
        assert torch.isnan(S[0, 1]).all()
    assert torch.isfinite(o[~touched]).all()
    tol = prompt_tol(150, TYPES[dtype])[1] + half_step(TYPES[dtype])
    ref = linattn(clean["S"], clean["q"], clean["k"], clean["v"], clean["g"])
    assert_within(o[~touched], ref["o"][~touched], (2 * tol * ref["mo"])[~touched], "o")
    if what != "q":
        assert not torch.isfinite(o[:, -1][touched[:, -1]]).any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,kh,vh,T", [(1, 1, 1, 700), (1, 1, 2, 2500), (2, 2, 4, 1500)])
def test_few_heads_long_prompts(dtype, B, kh, vh, T):
    """Sequences cut into segments, with lengths that end in any of them."""
    d = make_linattn(T, B, T, kh, vh, TYPES[dtype])
    S, o = d["S"].clone(), torch.empty_like(d["v"])
    run("prefill", S, d, o)
    check_prompt(d, S, o)
    for n in (0, 1, 65, T // 2, T - 1, T):
        lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
        S, o = d["S"].clone(), torch.full_like(d["v"], 7.5)
        run("prefill", S, d, o, lens=lens)
        assert (o[:, n:] == 7.5).all()
        check_prompt(d, S, o, lens=lens.long())
    assert gdn.gdn_wait_timeouts() == 0


def test_integer_buffers_stay_apart():
    """lens and err_dev over each other, over tensors and over the workspace."""
    d = make_linattn(1, 1, 4000, 1, 1)
    S, o, ws = d["S"].clone(), torch.zeros_like(d["v"]), workspace(d)
    args = (S, d["q"], d["k"], d["v"], d["g"], o)
    ints = lambda x: x.flatten()[:4].view(torch.int32)[:1]
    wsi = ws[:16].view(torch.int32)[:1]
    lens = torch.full((1,), 4000, dtype=torch.int32, device="cuda")
    for more in (dict(lens=lens, err_dev=lens), dict(err_dev=ints(d["q"])), dict(err_dev=ints(d["g"])),
                 dict(err_dev=ints(S)), dict(lens=ints(o)), dict(lens=wsi), dict(err_dev=wsi)):
        with pytest.raises(gdn.GDNError) as e:
            gdn.gdn_linattn_prefill(*args, workspace=ws, **more)
        assert e.value.status == gdn.GDN_EALIAS
    torch.cuda.synchronize()
    assert torch.equal(S, d["S"]) and int(lens) == 4000 and not o.any()


def test_workspace_refusals():
    d = make_linattn(1, 1, 4000, 1, 1)
    need = workspace(d).numel()
    assert need > 0
    S, o = d["S"].clone(), torch.empty_like(d["v"])
    args = (S, d["q"], d["k"], d["v"], d["g"], o)
    small = torch.empty(need - 1, dtype=torch.uint8, device="cuda")
    for ws, status in ((None, gdn.GDN_EINVAL), (small, gdn.GDN_ERANGE),
                       (torch.empty(need + 16, dtype=torch.uint8, device="cuda")[4:], gdn.GDN_EALIGN)):
        with pytest.raises(gdn.GDNError) as e:
            gdn.gdn_linattn_prefill(*args, workspace=ws)
        assert e.value.status == status
    over = torch.empty(need // 4 + S.numel(), device="cuda")
    Sin = over[-S.numel() - 256:][:S.numel()].view_as(S)
    with pytest.raises(gdn.GDNError) as e:  # the workspace reaches into S
        gdn.gdn_linattn_prefill(Sin, *args[1:], workspace=over[: need // 4 + 64])
    assert e.value.status == gdn.GDN_EALIAS
    assert torch.equal(S, d["S"])
