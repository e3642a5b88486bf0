"""Scales of the scores whose product with log2 e is no float are refused."""

import ctypes

import pytest

import gated_deltanet_linear_gb300 as gdn
from test_attn_cpu import FAKE, attn_call, cache, lib  # noqa: F401


@pytest.mark.parametrize("scale,status", [(2.4e38, gdn.GDN_EINVAL), (-3e38, gdn.GDN_EINVAL), (2.3e38, gdn.GDN_OK), (-1e38, gdn.GDN_OK)])
def test_scales_at_the_end_of_the_floats(lib, scale, status):  # noqa: F811
    assert attn_call(lib, cache(), B=0, scale=scale, table=FAKE) == status


@pytest.mark.parametrize("scale,status", [(3e38, gdn.GDN_OK), (-2.9e38, gdn.GDN_OK), (float("inf"), gdn.GDN_EINVAL)])
def test_linear_attention_takes_them_as_before(lib, scale, status):  # noqa: F811
    shape = ctypes.byref(gdn.Shape(0, 2, 4, 128, 128))
    assert lib.gdn_linattn_step(shape, 0, 0, scale, *[None] * 7) == status
