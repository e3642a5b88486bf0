"""What gdn_attn_step_m keeps of its numbers."""

import pytest
import torch

from attn_ref import attn, attn_bounds, make_cache, make_table
from test_gpu_attn import call, gen_of, ints

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
