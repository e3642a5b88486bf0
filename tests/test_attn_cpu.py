"""The attention layers' entry points without a GPU: host refusals, the
frequencies, and the 64-bit forms of the GPU tests against closed forms."""

import ctypes
import math

import pytest
import torch

import gated_deltanet_linear_gb300 as gdn
from attn_ref import attn, codes, freqs, make_cache, make_table, turn
from gated_deltanet_linear_gb300 import _build, _Cache, _Rope


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gdn.load()


FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10004)


def cache(kind=1, pages=4, kvh=2, page=16, hd=128, k=0x10000, scale=0x20000):
    return ctypes.byref(_Cache(k, 0x30000, scale, 0x40000, kind, pages, kvh, page, hd))


def rope(rot=64, layout=0, amp=1.0, freq=0x50000):
    return ctypes.byref(_Rope(freq, rot, layout, amp))


def attn_call(lib, c, B=1, M=1, qh=4, dtype=0, scale=1.0, cols=2, q=None, ws=None, ws_bytes=1 << 40,
              table=FAKE, start=FAKE):
    return lib.gdn_attn_step_m(c, B, M, qh, dtype, scale, q, table, cols, start, None, q, None, None, ws,
                               ws_bytes, None)


def write_call(lib, c, B=1, M=1, qh=0, dtype=0, rp=None, q=None, qs=0, ks=256, vs=256, qo=None, cols=2,
               table=FAKE, start=FAKE):
    return lib.gdn_kv_write_m(c, B, M, qh, dtype, rp, q, qs, None, ks, None, vs, qo, table, cols, start,
                              None, None, None)


def read_call(lib, c, B=1, T=4, dtype=0, cols=2, table=FAKE):
    return lib.gdn_kv_read(c, B, T, dtype, table, cols, None, None, None, None, None, None)


BAD_CACHES = [(dict(kind=3), gdn.GDN_EINVAL), (dict(kind=-1), gdn.GDN_EINVAL), (dict(hd=32), gdn.GDN_ESHAPE),
              (dict(hd=192), gdn.GDN_ESHAPE), (dict(page=8), gdn.GDN_ESHAPE), (dict(page=48), gdn.GDN_ESHAPE),
              (dict(page=512), gdn.GDN_ESHAPE), (dict(page=0), gdn.GDN_ESHAPE), (dict(pages=0), gdn.GDN_ESHAPE),
              (dict(kvh=0), gdn.GDN_ESHAPE), (dict(kvh=5000), gdn.GDN_ESHAPE)]


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_caches_refused_by_every_call(lib, bad, status):
    for call in (attn_call, write_call, read_call):
        assert call(lib, cache(**bad)) == status
        assert call(lib, None) == gdn.GDN_EINVAL
    assert lib.gdn_attn_workspace(cache(**bad), 1, 4) == 0


def test_attn_refusals(lib):
    ok = cache()
    for kw, status in ((dict(B=-1), gdn.GDN_ESHAPE), (dict(qh=3), gdn.GDN_ESHAPE), (dict(qh=0), gdn.GDN_ESHAPE),
                       (dict(M=0), gdn.GDN_ERANGE), (dict(M=65), gdn.GDN_ERANGE), (dict(qh=4098), gdn.GDN_ERANGE),
                       (dict(B=1 << 28, M=64), gdn.GDN_ERANGE), (dict(dtype=2), gdn.GDN_EINVAL),
                       (dict(scale=math.nan), gdn.GDN_EINVAL), (dict(scale=math.inf), gdn.GDN_EINVAL),
                       (dict(cols=0), gdn.GDN_ESHAPE), (dict(cols=(1 << 26) + 1), gdn.GDN_ERANGE),
                       (dict(table=None), gdn.GDN_EINVAL), (dict(start=None), gdn.GDN_EINVAL),
                       (dict(), gdn.GDN_EINVAL), (dict(ws=FAKE, q=None), gdn.GDN_EINVAL),
                       (dict(ws=FAKE, ws_bytes=1000), gdn.GDN_ERANGE), (dict(ws=FAKE, q=ODD), gdn.GDN_EALIGN)):
        assert attn_call(lib, ok, **kw) == status, kw
    assert attn_call(lib, ok, B=0, table=None) == gdn.GDN_OK
    assert attn_call(lib, cache(scale=None), ws=FAKE, q=FAKE) == gdn.GDN_EINVAL
    size = lib.gdn_attn_workspace
    assert size(ok, 0, 4) == size(ok, 65, 4) == size(ok, 1, 3) == size(ok, 1, 0) == 0
    # two parts of 8 to 24 rows of 128 sums and 4 floats for each CTA, and 32 bytes
    assert size(ok, 1, 4) == 9728 + 2 * 304 * 8 * 132 * 4
    assert size(ok, 8, 4) == 9728 + 2 * 152 * 16 * 132 * 4
    assert size(ok, 10, 4) == size(cache(kind=0), 10, 4) == 9728 + 2 * 152 * 24 * 132 * 4
    assert size(cache(hd=64), 10, 4) == 9728 + 2 * 304 * 16 * 68 * 4


def test_write_and_read_refusals(lib):
    ok = cache()
    for kw, status in ((dict(B=-1), gdn.GDN_ESHAPE), (dict(qh=-1), gdn.GDN_ESHAPE), (dict(M=0), gdn.GDN_ERANGE),
                       (dict(M=(1 << 20) + 1), gdn.GDN_ERANGE), (dict(B=1 << 20, M=1 << 12), gdn.GDN_ERANGE),
                       (dict(dtype=7), gdn.GDN_EINVAL), (dict(qh=2), gdn.GDN_EINVAL), (dict(q=FAKE), gdn.GDN_EINVAL),
                       (dict(qo=FAKE), gdn.GDN_EINVAL), (dict(qh=2, q=FAKE, qo=FAKE, qs=255), gdn.GDN_ESHAPE),
                       (dict(qh=2, q=FAKE, qo=FAKE, qs=257), gdn.GDN_EALIGN), (dict(ks=255), gdn.GDN_ESHAPE),
                       (dict(ks=258), gdn.GDN_EALIGN), (dict(vs=260, dtype=1), gdn.GDN_EALIGN),
                       (dict(cols=0), gdn.GDN_ESHAPE), (dict(table=None), gdn.GDN_EINVAL),
                       (dict(start=None), gdn.GDN_EINVAL), (dict(), gdn.GDN_EINVAL)):
        assert write_call(lib, ok, **kw) == status, kw
    for kw, status in ((dict(rot=0), gdn.GDN_ESHAPE), (dict(rot=24), gdn.GDN_ESHAPE), (dict(rot=144), gdn.GDN_ESHAPE),
                       (dict(layout=2), gdn.GDN_EINVAL), (dict(amp=math.nan), gdn.GDN_EINVAL),
                       (dict(freq=None), gdn.GDN_EINVAL)):
        assert write_call(lib, ok, rp=rope(**kw)) == status, kw
        assert lib.gdn_rope_m(1, 1, 128, 0, rope(**kw), FAKE, 128, FAKE, FAKE, None) == status, kw
    assert write_call(lib, ok, B=0) == gdn.GDN_OK and read_call(lib, ok, B=0) == gdn.GDN_OK
    for kw, status in ((dict(B=-1), gdn.GDN_ESHAPE), (dict(T=0), gdn.GDN_ERANGE), (dict(B=3, T=1 << 30), gdn.GDN_ERANGE),
                       (dict(dtype=2), gdn.GDN_EINVAL), (dict(cols=-1), gdn.GDN_ESHAPE), (dict(table=None), gdn.GDN_EINVAL),
                       (dict(), gdn.GDN_EINVAL)):
        assert read_call(lib, ok, **kw) == status, kw
    rp = rope()
    call = lib.gdn_rope_m
    assert call(1, 1, 96, 0, rp, FAKE, 96, FAKE, FAKE, None) == gdn.GDN_ESHAPE
    assert call(-1, 1, 128, 0, rp, FAKE, 128, FAKE, FAKE, None) == gdn.GDN_ESHAPE
    assert call(1, 0, 128, 0, rp, FAKE, 128, FAKE, FAKE, None) == gdn.GDN_ESHAPE
    assert call(1, 5000, 128, 0, rp, FAKE, 5000 * 128, FAKE, FAKE, None) == gdn.GDN_ERANGE
    assert call(1, 1, 128, 3, rp, FAKE, 128, FAKE, FAKE, None) == gdn.GDN_EINVAL
    assert call(1, 1, 128, 0, None, FAKE, 128, FAKE, FAKE, None) == gdn.GDN_EINVAL
    assert call(1, 1, 128, 0, rp, FAKE, 120, FAKE, FAKE, None) == gdn.GDN_ESHAPE
    assert call(1, 1, 128, 0, rp, FAKE, 130, FAKE, FAKE, None) == gdn.GDN_EALIGN
    assert call(0, 1, 128, 0, rp, None, 128, None, None, None) == gdn.GDN_OK
    assert call(1, 1, 128, 0, rp, FAKE, 128, None, FAKE, None) == gdn.GDN_EINVAL


def test_binding_refusals(lib):
    """(ValueError before any CUDA call: these are CPU tensors)"""
    k = torch.zeros(4, 2, 16, 64, dtype=torch.int8)
    for args in ((k,), (k, k), (k.float(), k.float()), (k[0], k[0]), (k.bfloat16(), k.bfloat16(), torch.zeros(4, 2, 16))):
        with pytest.raises((ValueError, TypeError)):
            gdn.KVCache(*args)
    with pytest.raises(ValueError):
        gdn.Rope(torch.zeros(8, dtype=torch.float64))
    for kw in (dict(rot=3), dict(rot=0), dict(base=0.0), dict(base=math.inf), dict(scaling=4),
               dict(scaling=gdn.GDN_ROPE_LINEAR, factor=0.0), dict(rot=2, scaling=gdn.GDN_ROPE_NTK, factor=2.0),
               dict(scaling=gdn.GDN_ROPE_BAND, factor=2.0), dict(scaling=gdn.GDN_ROPE_BAND, factor=2.0, context=1.0, low=2.0, high=2.0)):
        with pytest.raises(gdn.GDNError):
            gdn.gdn_rope_freqs(**{"rot": 32, "device": "cpu", **kw})


@pytest.mark.parametrize("name,code", [("plain", 0), ("linear", 1), ("ntk", 2), ("band", 3)])
@pytest.mark.parametrize("rot", [4, 64, 256])
def test_frequencies(lib, name, code, rot):
    f, amp = gdn.gdn_rope_freqs(rot, 1e6, code, 16.0, 8192.0, 1.0, 32.0, device="cpu")
    rf, ramp = freqs(rot, 1e6, name, 16.0, 8192.0, 1.0, 32.0)
    assert ((f - rf).abs() <= 1e-14 * rf).all() and abs(amp - ramp) <= 1e-7 * ramp
    if name == "band":  # fast pairs as they were, slow ones stretched
        p = freqs(rot, 1e6)[0]
        assert f[0] == p[0] and (rot == 4 or abs(f[-1] * 16 / p[-1] - 1) < 1e-14)


def test_forms():
    """The tests' own forms: a turn keeps lengths and differences of positions,
    codes are nearest, attention of equal scores is the mean."""
    g = torch.Generator().manual_seed(1)
    x, y = torch.randn(6, 1, 64, generator=g), torch.randn(6, 1, 64, generator=g)
    f, _ = freqs(48)
    pos = torch.tensor([0, 1, 5, 100, 7, 9000])
    for pairs in (False, True):
        a, b = turn(x, pos, f, pairs, 1.0), turn(y, pos + 11, f, pairs, 1.0)
        c, d = turn(x, pos * 0, f, pairs, 1.0), turn(y, pos * 0 + 11, f, pairs, 1.0)
        assert torch.allclose((a * b).sum(-1), (c * d).sum(-1), rtol=0, atol=1e-11)
        assert torch.equal(a[0], x[0].double())
    v = torch.randn(50, 64, generator=g).double()
    c, s = codes(v, "int8")
    assert ((c * s.double()[:, None] - v).abs() <= 0.5 * s.double()[:, None] * (1 + 1e-6)).all()
    c, s = codes(v, "e4m3")
    fine = c.clamp(-448, 448)
    assert torch.equal(fine.float().to(torch.float8_e4m3fn).double(), fine)
    assert torch.equal(codes(torch.zeros(1, 64).double(), "int8")[0], torch.zeros(1, 64).double())
    for kind in ("bf16", "int8", "e4m3"):
        cache_ = make_cache(kind, 4, 1, 16, 64, g, "cpu")
        table = make_table(4, 1, 3, g, "cpu")
        q = torch.zeros(1, 2, 1, 64)
        o, lse, _, _ = attn(cache_, table, [20], None, q, 1.0, 16)
        assert torch.allclose(lse.flatten(), torch.tensor([21.0, 22.0]).log().double())
        at = table[0, :2].long()
        rows = cache_["v"][at].float().double()
        if kind != "bf16":
            rows = rows * cache_["vs"][at].double()[..., None]
        assert torch.allclose(o[0, 0, 0], rows[:, 0].reshape(-1, 64)[:21].mean(0))
