"""Prompts of linear attention where sizes, decays and rows of zeros meet:
against the plain 64-bit form, with the tolerances of test_gpu_linattn (t of the
magnitude, one rounding to 16 bits) and the floors that the interface names.
"""

import pytest
import torch

import gated_deltanet_linear_gb300 as gdn
from linattn_ref import assert_within, half_step, linattn, make_linattn
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
