"""Host-side refusals of the rotary writes, the read-back and the shared-prefix attention: every call
below fails its validation (or has nothing to do) before any CUDA work."""
import ctypes

import pytest

vp, i32, i64, f32, szt = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
FAKE = 1 << 20   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from int4_token_head_kv_gb300._build import build_library
    return ctypes.CDLL(build_library())


@pytest.mark.parametrize("name", ["kv_int4_rope_write", "kv_int8_rope_write", "kv_int2_rope_write"])
def test_rope_write(lib, name):
    f, signs = getattr(lib, name), "8" not in name
    f.restype = ctypes.c_int
    f.argtypes = [vp, i64, i32, vp, i64, vp, i64, ctypes.c_int, i64, i32, i32, vp, vp, i64, i32, i32, vp] + \
        ([vp] if signs else []) + [vp, i64, vp, i64, i32, vp]
    base = dict(q=FAKE, qs=1024, hq=8, k=FAKE, ks=256, v=FAKE, vs=256, dt=1, n=4, h=2, d=128, pos=FAKE, cs=FAKE, mp=64,
                rot=128, inter=0, slots=FAKE, signs=FAKE, qo=FAKE, qos=1024, cache=FAKE, nb=8, bs=16, st=None)
    if not signs:
        del base["signs"]

    def call(**kw):
        return f(*dict(base, **kw).values())

    assert call(d=96) == 2 and call(bs=32) == 2 and call(dt=2) == 2 and call(h=65, ks=65 * 128, vs=65 * 128) == 2
    assert call(rot=0) == 2 and call(rot=24) == 2 and call(rot=144) == 2 and call(hq=1025, qs=1 << 20, qos=1 << 20) == 2
    assert call(n=-1) == 1 and call(h=0) == 1 and call(hq=-1) == 1 and call(mp=-1) == 1 and call(rot=-16) == 1
    for x in ("q", "k", "v", "pos", "cs", "slots", "qo", "cache") + (("signs",) if signs else ()):
        assert call(**{x: None}) == 1, x
    assert call(ks=248) == 1 and call(vs=0) == 1 and call(qs=1016) == 1 and call(qos=8) == 1   # rows overlap
    assert call(ks=260) == 3 and call(vs=257) == 3 and call(qs=1028) == 3 and call(qos=1030) == 3
    for x in ("q", "k", "v", "cs", "qo", "cache"):
        assert call(**{x: FAKE + 8}) == 3, x
    assert call(n=1 << 29) == 2   # 32-bit vector index
    assert call(n=0, q=None, k=None, v=None) == 0
    assert call(n=0, d=96) == 2


@pytest.mark.parametrize("name", ["kv_int4_read", "kv_int8_read", "kv_int2_read"])
def test_read(lib, name):
    f, signs = getattr(lib, name), "8" not in name
    f.restype = ctypes.c_int
    f.argtypes = [vp, i64, i32, i32, i32, vp, i64] + ([vp] if signs else []) + [vp, vp, ctypes.c_int, vp]
    base = dict(cache=FAKE, nb=8, bs=16, h=2, d=64, slots=FAKE, n=4, signs=FAKE, ko=FAKE, vo=FAKE, dt=1, st=None)
    if not signs:
        del base["signs"]

    def call(**kw):
        return f(*dict(base, **kw).values())

    assert call(d=80) == 2 and call(bs=8) == 2 and call(dt=3) == 2 and call(h=65) == 2 and call(n=1 << 30) == 2
    assert call(n=-1) == 1 and call(h=0) == 1 and call(nb=-1) == 1
    for x in ("cache", "slots", "ko", "vo") + (("signs",) if signs else ()):
        assert call(**{x: None}) == 1, x
    for x in ("cache", "ko", "vo"):
        assert call(**{x: FAKE + 4}) == 3, x
    assert call(n=0, cache=None) == 0


def test_shared_prefix(lib):
    f = lib.kv_int4_shared_prefix_attention
    f.restype = ctypes.c_int
    f.argtypes = [vp, ctypes.c_int, i64, i32, vp, i64, i32, i32, i32, vp, i32, vp, i32, vp, vp, i32, i32, i32, f32, vp,
                  i32, vp, ctypes.c_int, vp, szt, vp, vp]
    base = dict(q=FAKE, qd=1, nq=4, hq=32, cache=FAKE, nb=64, h=8, d=128, bs=16, pb=FAKE, pl=4096, bt=FAKE, mb=260, sl=FAKE,
                qsl=FAKE, ns=4, mql=1, msl=4160, scale=0.088, signs=FAKE, seg=0, out=FAKE, od=2, ws=None, wsb=0, st=None, opts=None)

    def call(**kw):
        return f(*dict(base, **kw).values())

    from int4_token_head_kv_gb300 import AttnOptions
    for bad in (AttnOptions(-1, -1.0, None, None, 0), AttnOptions(-1, float("nan"), None, None, 0),
                AttnOptions(-1, 0.0, None, FAKE, 0)):
        assert call(opts=ctypes.addressof(bad)) == 1
    assert call(mql=2) == 2 and call(h=3, hq=24) == 2 and call(d=80) == 2 and call(seg=24) == 2 and call(od=5) == 2
    assert call(pl=-1) == 1 and call(pb=None) == 1 and call(pl=16 * 261) == 1 and call(q=None) == 1 and call(signs=None) == 1
    assert call(out=FAKE + 4) == 3
    assert call() == 4                                        # no workspace
    assert call(ws=FAKE, wsb=1000) == 4
    assert call(nq=0, pb=None) == 0 and call(ns=0, q=None) == 0
    w = lib.kv_int4_shared_prefix_workspace_bytes
    w.restype = szt
    w.argtypes = [i64, i32, i32, i32, i32, i32, i32, i32]
    plain = lib.kv_int4_attention_workspace_bytes
    plain.restype = szt
    plain.argtypes = [i32] * 6
    need = w(4, 32, 8, 128, 4, 4096, 4160, 0)
    suffix = plain(32, 8, 128, 4, 4160 - 4096, 0)
    # behind the suffix's workspace: per split and query row 128 fp32 outputs and a (max, sum) pair
    rows = need - (suffix + 255) // 256 * 256
    assert rows % (4 * 32 * (128 * 4 + 8)) == 0 and rows > 0
    assert call(ws=FAKE, wsb=need - 1) == 4
    assert w(4, 32, 8, 128, 4, 0, 320, 0) == plain(32, 8, 128, 4, 320, 0)    # nothing shared: the plain call's
    assert w(1, 32, 8, 128, 1, 4096, 4160, 0) == plain(32, 8, 128, 1, 4160, 0)  # one sequence
    assert w(4, 32, 8, 128, 4, 4080, 4160, 0) == plain(32, 8, 128, 4, 4160, 0)  # below 16 384 tokens in all
    assert w(2, 8, 2, 128, 2, 4096, 4160, 0) > plain(8, 2, 128, 2, 64, 0)       # 8 192 with few kv heads
    assert w(0, 32, 8, 128, 4, 256, 320, 0) == 0 and w(4, 30, 8, 128, 4, 256, 320, 0) == 0 and w(4, 32, 8, 128, 0, 256, 320, 0) == 0
    assert call(pl=(1 << 30) + 1, mb=1 << 27) == 2            # 32-bit key indices
    assert w(4, 32, 8, 128, 4, (1 << 30) + 1, 1 << 30, 0) == 0


@pytest.mark.parametrize("name", ["kv_int4_rope_write", "kv_int8_rope_write", "kv_int2_rope_write"])
def test_rope_write_in_place_needs_one_stride(lib, name):
    f = getattr(lib, name)
    f.restype = ctypes.c_int
    signs = [vp] if "8" not in name else []
    f.argtypes = [vp, i64, i32, vp, i64, vp, i64, ctypes.c_int, i64, i32, i32, vp, vp, i64, i32, i32, vp] + signs + \
        [vp, i64, vp, i64, i32, vp]
    head = (FAKE, 1024, 8, FAKE, 256, FAKE, 256, 1, 4, 2, 128, FAKE, FAKE, 64, 128, 0, FAKE) + (FAKE,) * len(signs)
    assert f(*head, FAKE, 2048, FAKE, 8, 16, None) == 1


@pytest.mark.parametrize("name", ["kv_int4_rope_write", "kv_int8_rope_write", "kv_int2_rope_write"])
def test_rope_write_needs_a_table_row(lib, name):
    """A table of no rows is refused whatever its pointer, unless there is no token either."""
    f = getattr(lib, name)
    f.restype = ctypes.c_int
    signs = [vp] if "8" not in name else []
    f.argtypes = [vp, i64, i32, vp, i64, vp, i64, ctypes.c_int, i64, i32, i32, vp, vp, i64, i32, i32, vp] + signs + \
        [vp, i64, vp, i64, i32, vp]

    def call(n):
        return f(FAKE, 1024, 8, FAKE, 256, FAKE, 256, 1, n, 2, 128, FAKE, FAKE, 0, 128, 0, FAKE, *(FAKE,) * len(signs), FAKE, 1024,
                 FAKE, 8, 16, None)

    assert call(4) == 1 and call(1) == 1 and call(0) == 0


def test_short_prefixes_take_the_plain_walk(lib):
    """However many sequences share them: the workspace is the plain call's."""
    w = lib.kv_int4_shared_prefix_workspace_bytes
    w.restype = szt
    w.argtypes = [i64, i32, i32, i32, i32, i32, i32, i32]
    plain = lib.kv_int4_attention_workspace_bytes
    plain.restype = szt
    plain.argtypes = [i32] * 6
    for Hq, H, least in ((8, 8, 32), (16, 8, 64), (32, 8, 128), (8, 1, 256), (32, 4, 384), (64, 8, 544)):
        for S in (1024, 8192):
            assert w(S, Hq, H, 128, S, least - 1, least + 100, 0) == plain(Hq, H, 128, S, least + 100, 0)
            shared = w(S, Hq, H, 128, S, least, least + 100, 0)
            assert shared > plain(Hq, H, 128, S, 100, 0) and shared != plain(Hq, H, 128, S, least + 100, 0)
    assert w(1024, 32, 8, 128, 1024, 16, 80, 0) == plain(32, 8, 128, 1024, 80, 0)
