"""Prompts of linear attention where sizes, decays and rows of zeros meet:
against the plain 64-bit form, with the tolerances of test_gpu_linattn (t of the
magnitude, one rounding to 16 bits) and the floors that the interface names.
"""

import pytest
import torch

import gated_deltanet_linear_gb300 as gdn
from linattn_ref import assert_within, linattn, make_linattn
from test_gpu_linattn import TYPES, check_prompt, prompt_tol, run, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def prompt(d, **more):
    S, o = d["S"].clone(), torch.empty_like(d["v"])
    run("prefill", S, d, o, **more)
    return S, o


@pytest.mark.parametrize("decay", ["token", "head"])
@pytest.mark.parametrize("B,kh,vh,T", [(1, 1, 2, 70), (2, 2, 6, 200), (1, 1, 2, 900)])
def test_bf16_prompts_are_rounded_once(decay, B, kh, vh, T):
    """16-bit tokens ask for 16-bit tokens, not for fewer bits on the way: o is
    the rounding of an fp32 result.  With e the error before the rounding, o
    differs from the rounded 64-bit form by a whole step u_i <= 2^-7 |ref_i|
    where a border lies between the two, for the share |e_i| / u_i of the
    elements, so the expected square of the difference is the sum of u_i |e_i|,
    at most 2^-7 |ref| |e| in norms.  |e| <= 2^-19 |ref| (below) gives 2^-13;
    scores or states of 11 bits, |e| about 2^-12, would give 2^-9.5."""
    d = make_linattn(T, B, T, kh, vh, torch.bfloat16, decay)
    S, o = prompt(d)
    ref = linattn(d["S"], d["q"], d["k"], d["v"], d["g"])
    off = (o.double() - ref["o"].bfloat16().double()).norm()
    assert off <= 2.0 ** -13 * ref["o"].norm()
    assert (S - ref["S"]).norm() <= 2.0 ** -19 * ref["S"].norm()


def floors(d):
    """What the magnitudes do not cover.  Weights e^{sum of g} below 2^-126 may
    count as 0: at most |k v| (or |q.k v|, or |S0 q| over 128 rows) of T tokens
    times that.  A score is off by up to 2^-30 |q_t| |k| (the largest
    elements), times |v| of 64 tokens: it shows where the tokens near t have
    v = 0 (derived in test_gpu_linattn.test_zero_rows)."""
    top = {x: float(d[x].abs().max()) for x in "qkvS"}
    norm = {x: float(d[x].float().norm(dim=-1).max()) for x in "qk"}
    T = d["v"].shape[1]
    size = max(1.0, norm["q"]) * max(norm["k"] * top["v"], top["S"])
    return ((T + 128) * size * 2.0 ** -126,
            2.0 ** -30 * top["q"] * top["k"] * 64 * top["v"])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("what", ["k", "v", "columns"])
@pytest.mark.parametrize("decay", [-0.5, -1.0, -2.0])
@pytest.mark.parametrize("start,T", [(0, 64), (64, 150), (1344, 1500)])
def test_state_after_rows_of_zeros(dtype, what, decay, start, T):
    """The last rows of a chunk (and the chunks behind it) are zeros, and the
    decays leave small weights for the others: they are the whole state.
    (1500 tokens of 2 heads are cut into segments.)"""
    for keep in (16, 32, 48, 56):
        d = make_linattn(keep, 1, T, 1, 2, TYPES[dtype])
        assert (workspace(d).numel() > 0) == (T == 1500)
        d["S"].zero_()
        d["g"].fill_(decay)
        if what == "columns":  # of v, five of them
            d["v"][:, start + keep:, :, 7:12] = 0
        else:
            d[what][:, start + keep:] = 0
        S, o = prompt(d)
        under, score = floors(d)
        check_prompt(d, S, o, floor_S=under, floor_o=under + score)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("late", [False, True])
def test_state_of_small_rows(dtype, late):
    """Key rows 2^-40 of the others', the others with v = 0: they are the whole
    state; and values beside a zero key row do not count, whatever their
    size."""
    d = make_linattn(3, 1, 64, 1, 2, TYPES[dtype])
    d["S"].zero_()
    d["g"].zero_()
    small = slice(32, 64) if late else slice(0, 32)
    big = slice(0, 32) if late else slice(32, 64)
    d["k"][:, small] *= 2.0 ** -40
    d["v"][:, big] = 0
    S, _ = prompt(d)
    ref = linattn(d["S"], d["q"], d["k"], d["v"], d["g"])
    t = prompt_tol(64)[0]
    assert_within(S, ref["S"], t * ref["mS"], "S of small rows")
    d = make_linattn(4, 1, 64, 1, 2, TYPES[dtype])
    d["S"].zero_()
    d["k"][:, 60 if late else 5] = 0
    d["v"][:, 60 if late else 5] = 1e14
    S, _ = prompt(d)
    ref = linattn(d["S"], d["q"], d["k"], d["v"], d["g"])
    assert_within(S, ref["S"], t * ref["mS"], "S beside a zero key row")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("start,T", [(0, 150), (1344, 1500)])
@pytest.mark.parametrize("rows,decay", [
    (slice(10, 11), -200.0), (slice(10, 11), -float("inf")), (slice(20, 40), -12.0),
    (slice(20, 40), -50.0), (slice(44, 64), -12.0), (slice(0, 20), -50.0),
    (slice(63, 64), -float("inf"))])
def test_zero_key_rows_under_strong_decay(dtype, start, T, rows, decay):
    """Rows of zeros in k that carry strong decays, between ordinary rows."""
    d = make_linattn(31, 1, T, 1, 2, TYPES[dtype])
    d["g"].fill_(-0.05)
    at = slice(start + rows.start, start + rows.stop)
    d["g"][:, at] = decay
    d["k"][:, at] = 0
    S, o = prompt(d)
    assert torch.isfinite(o).all() and torch.isfinite(S).all()
    under, score = floors(d)
    check_prompt(d, S, o, floor_S=under, floor_o=under + score)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size", [dict(q=1e18, k=1e18), dict(v=2.0 ** 118, S=2.0 ** 118),
                                  dict(k=2.0 ** 100, q=2.0 ** -90), dict(S=2.0 ** 118, q=2.0 ** -60),
                                  dict(v=2.0 ** -110, S=2.0 ** -110, q=2.0 ** 50)])
def test_large_and_small_elements(dtype, size):
    """Elements whose products come near the range of a float, while o and S
    stay within it: as the token steps have them."""
    d = make_linattn(13, 1, 100, 1, 2, TYPES[dtype])
    if "S" in size:  # (make_linattn's state is 0.1 of its values)
        size = dict(size, S=10 * size["S"])
    for x, s in size.items():
        d[x] *= s
    S, o = prompt(d)
    # (products of fp32 numbers near 2^-126 are rounded to its subnormals)
    check_prompt(d, S, o, floor_S=64 * 2.0 ** -126, floor_o=64 * 2.0 ** -126)


@pytest.mark.parametrize("dtype", TYPES)
def test_large_scale(dtype):
    """The factor on o meets small rows before it could leave the floats."""
    d = make_linattn(14, 1, 100, 1, 2, TYPES[dtype])
    d["q"] *= 2.0 ** -40
    S, o = prompt(d, scale=2.9e38)
    check_prompt(d, S, o, scale=2.9e38)


@pytest.mark.parametrize("slow", [False, True])
@pytest.mark.parametrize("B,kh,vh,T", [(1, 1, 2, 90), (2, 2, 6, 190), (1, 1, 1, 700),
                                       (2, 2, 4, 1500), (1, 1, 2, 2500)])
def test_fp32_prompts_keep_fp32(slow, B, kh, vh, T):
    """Normwise error of every head's o and state, the same at any length: an
    operand that lost its second part is off by 2^-12 an element and by 2^-13
    to 2^-14 in norm; the operands as they should be, 2^-22 each, and the
    truncating sums of at most 8 steps, 2^-23 each, by 2^-20 if they all went
    one way.  2^-19 is between.  Slow decays, so that the start states of
    the segments (T >= 700) matter."""
    d = make_linattn(T, B, T, kh, vh)
    assert (workspace(d).numel() > 0) == (T >= 700)
    if slow:
        d["g"].mul_(0.01)
    S, o = prompt(d)
    ref = linattn(d["S"], d["q"], d["k"], d["v"], d["g"])
    off = (o - ref["o"]).norm(dim=(1, 3)) / ref["o"].norm(dim=(1, 3))
    assert float(off.max()) <= 2.0 ** -19
    off = (S - ref["S"]).norm(dim=(2, 3)) / ref["S"].norm(dim=(2, 3))
    assert float(off.max()) <= 2.0 ** -19


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [64, 150, 700])
@pytest.mark.parametrize("rate", [0.1, 0.86])
def test_growth_within_a_chunk(dtype, T, rate):
    """Factors above 1: up to e^(64 * 0.86), about 2^79, over a chunk's tokens and
    back in the next."""
    d = make_linattn(17, 1, T, 1, 2, TYPES[dtype])
    up = (torch.arange(T, device="cuda") // 64) % 2 == 0
    d["g"][:] = torch.where(up, rate, -rate)[None, :, None]
    S, o = prompt(d)
    under, score = floors(d)
    # (a score's error goes with its weight, up to 2^79 here)
    check_prompt(d, S, o, floor_S=under * 2.0 ** 79, floor_o=(under + score) * 2.0 ** 79)
    ref = linattn(d["S"], d["q"], d["k"], d["v"], d["g"])
    assert (S - ref["S"]).norm() <= 2.0 ** -19 * ref["S"].norm()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [111, 900])
def test_lengths_under_strong_decay(dtype, T):
    """Slopes of 1/2 and less a token over padded prompts that end anywhere in a
    chunk: the rows behind the end neither count nor scale."""
    ends = [1, 7, 56, 63, 64, 65, 100, T - 3, T]
    d = make_linattn(19, len(ends), T, 1, 2, TYPES[dtype], "head")
    d["g"] = torch.tensor([-0.5, -2.0], device="cuda")
    lens = torch.tensor(ends, dtype=torch.int32, device="cuda")
    for b, n in enumerate(ends):
        for x, bad in (("q", float("nan")), ("k", 1e30), ("v", float("inf"))):
            d[x][b, n:] = bad
    S, o = d["S"].clone(), torch.full_like(d["v"], 7.5)
    run("prefill", S, d, o, lens=lens)
    on = torch.arange(T, device="cuda") < lens[:, None]
    assert (o[~on] == 7.5).all()
    clean = {x: t if x in "Sg" else torch.where(on[..., None, None], t, torch.zeros_like(t))
             for x, t in d.items()}
    under, score = floors(clean)
    check_prompt(d, S, o, lens=lens.long(), floor_S=under, floor_o=under + score)
