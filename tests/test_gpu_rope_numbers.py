"""What gdn_rope_m keeps of its angles: far positions, frequencies of any size and
of either sign."""

from fractions import Fraction

import pytest
import torch

import gated_deltanet_linear_gb300 as gdn

pytestmark = pytest.mark.gpu

TWO_PI = Fraction(628318530717958647692528676655900576839433879875021, 10 ** 50)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


FREQS = [1.0, 0.7390851332151607, 1e-6, 3.3e-9, 1e-14, 2.5, 6.25, 1e-3] * 4
FREQS = [f * (1 + i / 37) for i, f in enumerate(FREQS)]
FAR = [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 1 << 20, 1, 0, -7, 123456789]


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_angles_of_far_positions(sign):
    """The angle of (1, 0) turned, against rational arithmetic: within 1e-7 and
    2^-53 of the whole angle, and what fp32 cosines and sines hold of it (2^-22)."""
    f = torch.tensor([sign * x for x in FREQS], dtype=torch.float64, device="cuda")
    n = f.numel()
    x = torch.zeros(len(FAR), 1, 64, device="cuda")
    x[..., :n] = 1.0
    y = torch.empty_like(x)
    gdn.gdn_rope_m(x, ints(FAR), gdn.Rope(f), y)
    got = torch.atan2(y[:, 0, n:].double(), y[:, 0, :n].double()).cpu()
    for i, p in enumerate(FAR):
        for j, v in enumerate(f.tolist()):
            whole = p * Fraction(v)
            off = (Fraction(got[i, j].item()) - whole) % TWO_PI
            off = float(min(off, TWO_PI - off))
            assert off <= 1e-7 + 2.0 ** -53 * abs(float(whole)) + 2.0 ** -22, (p, v, off)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_turning_back_is_the_mirror_image(pairs, dtype):
    """A pair (x, -y) turned on is that of (x, y) turned back with y negated, to
    the bit, at any position."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    f = torch.tensor(FREQS, dtype=torch.float64, device="cuda")
    n = f.numel()
    x = torch.randn(len(FAR), 3, 64, generator=gen, device="cuda").to(dtype)
    at = torch.arange(1, 2 * n, 2, device="cuda") if pairs else torch.arange(n, 2 * n, device="cuda")
    m = x.clone()
    m[..., at] = -m[..., at]
    layout = gdn.GDN_ROPE_PAIRS if pairs else gdn.GDN_ROPE_HALF
    on, back = torch.empty_like(x), torch.empty_like(x)
    gdn.gdn_rope_m(m, ints(FAR), gdn.Rope(f, layout, 1.25), on)
    gdn.gdn_rope_m(x, ints(FAR), gdn.Rope(-f, layout, 1.25), back)
    on[..., at] = -on[..., at]
    assert torch.equal(on, back)


@pytest.mark.parametrize("pairs", [False, True])
def test_frequencies_that_are_not_finite(pairs):
    """NaN in their pairs at every position, 0 among them, and nowhere else."""
    f = torch.tensor([0.5, float("nan"), 0.25, float("inf"), 1e-3, -float("inf"), 0.0, 2.0], dtype=torch.float64, device="cuda")
    x = torch.ones(4, 2, 64, device="cuda")
    y, z = torch.empty_like(x), torch.empty_like(x)
    layout = gdn.GDN_ROPE_PAIRS if pairs else gdn.GDN_ROPE_HALF
    gdn.gdn_rope_m(x, ints([0, 5, -3, 2 ** 30]), gdn.Rope(f, layout), y)
    gdn.gdn_rope_m(x, ints([0, 5, -3, 2 ** 30]), gdn.Rope(f.nan_to_num(0.0, 0.0, 0.0), layout), z)
    bad = torch.zeros(64, dtype=torch.bool, device="cuda")
    for i in (1, 3, 5):
        for at in ((2 * i, 2 * i + 1) if pairs else (i, i + 8)):
            bad[at] = True
    assert bool(y[..., bad].isnan().all()) and torch.equal(y[..., ~bad], z[..., ~bad])
