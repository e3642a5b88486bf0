"""gdn_rope_freqs: what is no number is refused."""

import pytest

import gated_deltanet_linear_gb300 as gdn
from gated_deltanet_linear_gb300 import _build


@pytest.mark.parametrize("kw", [dict(base=5e-324, rot=256), dict(base=5e-324, scaling=gdn.GDN_ROPE_NTK, factor=0.25),
                                dict(scaling=gdn.GDN_ROPE_LINEAR, factor=1e-320),
                                dict(scaling=gdn.GDN_ROPE_BAND, factor=1e-320, context=8192.0)])
def test_frequencies_beyond_the_floats_are_refused(kw):
    _build.build()
    with pytest.raises(gdn.GDNError) as e:
        gdn.gdn_rope_freqs(**{"rot": 64, "device": "cpu", **kw})
    assert e.value.status == gdn.GDN_EINVAL


def test_a_band_as_wide_as_the_floats():
    """Its blend is half of each everywhere."""
    _build.build()
    f, _ = gdn.gdn_rope_freqs(64, scaling=gdn.GDN_ROPE_BAND, factor=2.0, context=8192.0, low=-1.7e308, high=1.7e308, device="cpu")
    p, _ = gdn.gdn_rope_freqs(64, device="cpu")
    assert ((f / p - 0.75).abs() < 1e-14).all()
