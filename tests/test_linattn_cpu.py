"""The linear-attention and 4-bit projection entry points without a GPU: host
refusals, and the plain 64-bit forms the GPU tests use against closed forms."""

import ctypes

import pytest
import torch

import gated_deltanet_linear_gb300 as gdn
from gated_deltanet_linear_gb300 import _build
from linattn_ref import linattn, make_linattn, make_quant, quant_linear


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gdn.load()


NULLS = [None] * 8


def test_step_refusals(lib):
    ok = gdn.Shape(2, 2, 4, 128, 128)

    def call(sh=ok, M=1, dtype=0, decay=0, scale=1.0, ptrs=NULLS):
        return lib.gdn_linattn_step_m(ctypes.byref(sh) if sh else None, M, dtype, decay, scale,
                                      *ptrs, None)

    assert call(sh=None) == gdn.GDN_EINVAL
    for bad in [(2, 2, 4, 64, 128), (2, 2, 4, 128, 64), (2, 3, 4, 128, 128), (-1, 2, 4, 128, 128),
                (2, 0, 4, 128, 128), (2, 2, 0, 128, 128)]:
        assert call(sh=gdn.Shape(*bad)) == gdn.GDN_ESHAPE
    for M in (0, -1, gdn.GDN_MAX_TOKENS + 1):
        assert call(M=M) == gdn.GDN_ERANGE
    assert call(dtype=2) == gdn.GDN_EINVAL and call(dtype=-1) == gdn.GDN_EINVAL
    assert call(decay=2) == gdn.GDN_EINVAL
    for scale in (float("nan"), float("inf"), -float("inf")):
        assert call(scale=scale) == gdn.GDN_EINVAL
    assert call(sh=gdn.Shape(0, 2, 4, 128, 128)) == gdn.GDN_OK
    assert call() == gdn.GDN_EINVAL                       # NULL buffers
    fake = ctypes.c_void_p(0x1004)
    assert call(ptrs=[fake, fake, None] + [fake] * 5) == gdn.GDN_EALIGN
    assert lib.gdn_linattn_step(ctypes.byref(ok), 0, 0, 1.0, *[None] * 6, None) == gdn.GDN_EINVAL


def test_prefill_refusals(lib):
    ok = gdn.Shape(2, 2, 4, 128, 128)

    def call(sh=ok, T=8, dtype=0, decay=0):
        return lib.gdn_linattn_prefill(ctypes.byref(sh), T, dtype, decay, 1.0, *[None] * 9, 0, None)

    assert call(T=0) == gdn.GDN_ERANGE and call(T=gdn.GDN_MAX_TOKENS + 1) == gdn.GDN_ERANGE
    assert call(dtype=5) == gdn.GDN_EINVAL and call(decay=-1) == gdn.GDN_EINVAL
    assert call(sh=gdn.Shape(0, 2, 4, 128, 128)) == gdn.GDN_OK
    assert call(sh=gdn.Shape(2, 3, 4, 128, 128)) == gdn.GDN_ESHAPE
    assert call() == gdn.GDN_EINVAL
    size = lambda sh, T, dtype: lib.gdn_linattn_prefill_workspace(ctypes.byref(sh), T, dtype)
    assert size(ok, 0, 0) == 0 and size(ok, 8, 3) == 0
    assert size(gdn.Shape(2, 3, 4, 128, 128), 8, 0) == 0
    with pytest.raises(KeyError):
        gdn.gdn_linattn_prefill_workspace(1, 1, 1, 8, dtype=torch.float16)


def test_projection_refusals(lib):
    def call(rows=1, N=16, K=128, group=64, dtype=0, p=(None,) * 4):
        return lib.gdn_quant_linear(rows, N, K, group, dtype, *p, None)

    for bad in (dict(group=16), dict(group=0), dict(group=256), dict(K=0), dict(K=96),
                dict(K=-64), dict(rows=-1), dict(N=-1)):
        assert call(**bad) == gdn.GDN_ESHAPE
    top = gdn.GDN_QUANT_MAX_DIM
    assert call(N=top + 1) == gdn.GDN_ERANGE and call(K=top + 64) == gdn.GDN_ERANGE
    assert call(rows=gdn.GDN_MAX_TOKENS + 1) == gdn.GDN_ERANGE
    assert call(dtype=2) == gdn.GDN_EINVAL
    assert call(rows=0) == gdn.GDN_OK and call(N=0) == gdn.GDN_OK
    assert call() == gdn.GDN_EINVAL
    fake = ctypes.c_void_p(0x1008)
    assert call(p=(fake,) * 4) == gdn.GDN_EALIGN


def test_binding_refuses_cpu_tensors_and_shapes(lib):
    d = make_linattn(1, 1, 2, 1, 2, device="cpu")
    o = torch.empty_like(d["v"])
    with pytest.raises(ValueError):
        gdn.gdn_linattn_step_m(d["S"], d["S"], None, d["q"], d["k"], d["v"], d["g"], o)
    with pytest.raises(ValueError):
        gdn.gdn_linattn_step(d["S"], d["q"], d["k"], d["v"], d["g"], o)   # two tokens
    with pytest.raises(ValueError):
        gdn.gdn_linattn_prefill(d["S"], d["q"], d["k"], d["v"], d["g"], o)
    x, qw, sc = make_quant(1, 2, 4, 64, 32, device="cpu")
    with pytest.raises(ValueError):
        gdn.gdn_quant_linear(x, qw, sc, torch.empty(2, 4))
    with pytest.raises(ValueError):
        gdn.gdn_quant_linear(x, qw, sc[:, :0], torch.empty(2, 4))


def test_plain_form_closed_forms():
    """The token-by-token form is the explicit sum over earlier tokens."""
    d = make_linattn(4, 2, 7, 2, 4, device="cpu")
    got = linattn(d["S"], d["q"], d["k"], d["v"], d["g"], scale=0.5, states=True)
    q, k, v, S = (d[x].double() for x in ("q", "k", "v", "S"))
    G = d["g"].double().cumsum(1)
    for t in range(7):
        for h in range(4):
            for b in range(2):
                want = torch.exp(G[b, t, h]) * S[b, h]
                for s in range(t + 1):
                    want = want + torch.exp(G[b, t, h] - G[b, s, h]) * torch.outer(k[b, s, h // 2], v[b, s, h])
                assert torch.allclose(got["states"][t, b, h], want, rtol=1e-12, atol=1e-14)
                assert torch.allclose(got["o"][b, t, h], 0.5 * want.t() @ q[b, t, h // 2], rtol=1e-11, atol=1e-13)
    lens = torch.tensor([3, 0])
    cut = linattn(d["S"], d["q"], d["k"], d["v"], d["g"], lens=lens)
    assert torch.equal(cut["S"][0], got["states"][2, 0]) and torch.equal(cut["S"][1], S[1])


def test_plain_projection():
    x, qw, sc = make_quant(9, 3, 5, 64, 32, device="cpu")
    y, _ = quant_linear(x, qw, sc)
    for n in range(5):
        for r in range(3):
            s = 0.0
            for k in range(64):
                c = (int(qw[n, k // 2]) >> (4 * (k % 2))) & 15
                s += float(x[r, k]) * (c - 16 if c > 7 else c) * float(sc[n, k // 32])
            assert abs(s - float(y[r, n])) < 1e-12
