"""Host-side refusals of the rotary writes with several axes and of the span attentions: every call below fails its
validation (or has nothing to do) before any CUDA work."""
import ctypes

import pytest

vp, i32, i64, f32, szt = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
FAKE = 1 << 20   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from int4_token_head_kv_gb300._build import build_library
    return ctypes.CDLL(build_library())


@pytest.mark.parametrize("name", ["kv_int4_mrope_write", "kv_int8_mrope_write", "kv_int2_mrope_write"])
def test_mrope_write(lib, name):
    f, signs = getattr(lib, name), "8" not in name
    f.restype = ctypes.c_int
    f.argtypes = [vp, i64, i32, vp, i64, vp, i64, ctypes.c_int, i64, i32, i32, vp, i32, ctypes.c_char_p, vp, i64, i32, i32,
                  vp] + ([vp] if signs else []) + [vp, i64, vp, i64, i32, vp]
    axes = bytes([0] * 30 + [1] * 20 + [2] * 14)
    base = dict(q=FAKE, qs=1024, hq=8, k=FAKE, ks=256, v=FAKE, vs=256, dt=1, n=4, h=2, d=128, pos=FAKE, na=3, pa=axes, cs=FAKE,
                mp=64, rot=128, inter=0, slots=FAKE, signs=FAKE, qo=FAKE, qos=1024, cache=FAKE, nb=8, bs=16, st=None)
    if not signs:
        del base["signs"]

    def call(**kw):
        return f(*dict(base, **kw).values())

    assert call(na=0) == 1 and call(na=-2) == 1 and call(na=5) == 2
    assert call(pa=None) == 1 and call(na=2) == 1 and call(pa=axes[:63] + b"\xff") == 1   # an axis that is not there
    assert call(n=0, pa=None) == 1 and call(n=0, na=2) == 1
    assert call(d=96) == 2 and call(bs=32) == 2 and call(dt=2) == 2 and call(rot=24) == 2 and call(rot=144) == 2
    assert call(n=-1) == 1 and call(h=0) == 1 and call(hq=-1) == 1 and call(mp=0) == 1
    for x in ("q", "k", "v", "pos", "cs", "slots", "qo", "cache") + (("signs",) if signs else ()):
        assert call(**{x: None}) == 1, x
    assert call(ks=248) == 1 and call(qs=1016) == 1 and call(ks=260) == 3 and call(qos=1030) == 3
    for x in ("q", "k", "v", "cs", "qo", "cache"):
        assert call(**{x: FAKE + 8}) == 3, x
    assert call(n=1 << 29) == 2   # 32-bit vector index
    assert call(n=0, q=None, k=None, v=None) == 0


@pytest.mark.parametrize("name", ["kv_int4_span_attention", "kv_int8_span_attention", "kv_int2_span_attention"])
def test_span_attention(lib, name):
    f, signs = getattr(lib, name), "8" not in name
    f.restype = ctypes.c_int
    f.argtypes = [vp, ctypes.c_int, i64, i32, vp, i64, i32, i32, i32, vp, i32, vp, vp, i32, i32, i32, f32] + \
        ([vp] if signs else []) + [vp, vp, f32, vp, vp, ctypes.c_int, vp, szt, vp]
    base = dict(q=FAKE, qdt=1, n=12, hq=8, cache=FAKE, nb=8, h=2, d=128, bs=16, bt=FAKE, mb=4, lens=FAKE, qsl=FAKE, ns=3, mq=4,
                ms=64, scale=0.1, signs=FAKE, kb=FAKE, ke=None, cap=0.0, al=None, out=FAKE, odt=2, ws=FAKE, wsb=1 << 30, st=None)
    if not signs:
        del base["signs"]

    def call(**kw):
        return f(*dict(base, **kw).values())

    assert call(d=96) == 2 and call(bs=32) == 2 and call(qdt=2) == 2 and call(odt=3) == 2 and call(h=3, hq=6) == 2
    assert call(hq=6) == 2 and call(hq=32) == 2 and call(h=16, hq=16) == 2 and call(ns=65536) == 2 and call(n=1 << 31) == 2
    for x in ("n", "ns", "nb", "mq", "ms", "mb"):
        assert call(**{x: -1}) == 1, x
    assert call(cap=-1.0) == 1 and call(cap=float("inf")) == 1 and call(cap=float("nan")) == 1 and call(scale=float("nan")) == 1
    for x in ("q", "cache", "bt", "lens", "qsl", "out") + (("signs",) if signs else ()):
        assert call(**{x: None}) == 1, x
    assert call(mq=0) == 1 and call(mb=0) == 1
    for x in ("q", "cache", "out"):
        assert call(**{x: FAKE + 8}) == 3, x
    assert call(n=0, q=None) == 0 and call(ns=0) == 0


def test_span_workspace_refusals(lib):
    # 12 single tokens on up to 64000 keys: split, so the partials need their room
    need = lib.kv_int4_span_workspace_bytes
    need.restype, need.argtypes = szt, [i64, i32, i32, i32, i32, i32, i32]
    n = need(12, 8, 2, 128, 12, 1, 64000)
    assert n > 0
    f = lib.kv_int4_span_attention
    f.restype = ctypes.c_int
    f.argtypes = [vp, ctypes.c_int, i64, i32, vp, i64, i32, i32, i32, vp, i32, vp, vp, i32, i32, i32, f32, vp, vp, vp, f32,
                  vp, vp, ctypes.c_int, vp, szt, vp]

    def call(ws, size):
        return f(FAKE, 1, 12, 8, FAKE, 8, 2, 128, 16, FAKE, 4000, FAKE, FAKE, 12, 1, 64000, 0.1, FAKE, None, None, 0.0,
                 None, FAKE, 2, ws, size, None)

    assert call(None, n) == 4 and call(FAKE, n - 1) == 4 and call(FAKE, 0) == 4 and call(FAKE + 8, n) == 3


def test_span_workspace(lib):
    f = lib.kv_int4_span_workspace_bytes
    f.restype, f.argtypes = szt, [i64, i32, i32, i32, i32, i32, i32]
    for bad in ((0, 8, 2, 128, 3, 4, 64), (12, 8, 2, 128, 0, 4, 64), (12, 8, 0, 128, 3, 4, 64), (12, 0, 2, 128, 3, 4, 64),
                (12, 7, 2, 128, 3, 4, 64), (12, 8, 2, 0, 3, 4, 64), (-1, 8, 2, 128, 3, 4, 64), (12, 8, 2, 128, 3, -1, 64),
                (12, 8, 2, 128, 3, 4, -1)):
        assert f(*bad) == 0, bad
