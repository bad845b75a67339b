"""GPU parity of the rotary writes: cache bytes and rotated queries bit-exact against the rotary oracle
followed by each mode's write oracle, and the read-back within its roundings."""
import numpy as np
import pytest
import torch

import oracle
import workloads
from oracle import int2 as o2
from oracle import int8 as o8
from oracle import rope

pytestmark = pytest.mark.gpu

MODES = {4: oracle, 8: o8, 2: o2}


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from gpu_helpers import clear_status
    clear_status()


def _kv():
    import int4_token_head_kv_gb300 as kv
    return kv


def _call(bits, q, k, v, pos, tab, slots, signs, cache, **kw):
    kv = _kv()
    if bits == 8:
        return kv.kv_int8_rope_write(q, k, v, pos, tab, slots, cache, **kw)
    return (kv.kv_int4_rope_write if bits == 4 else kv.kv_int2_rope_write)(q, k, v, pos, tab, slots, signs, cache, **kw)


def _case(T, Hq, H, d, rot, dtype, seed, max_pos=512):
    r = np.random.default_rng(seed)
    x = torch.from_numpy(r.standard_normal((T, Hq + 2 * H, d)).astype(np.float32) * 3).to(dtype)
    nb = (T + 15) // 16 + 3
    return dict(x=x, pos=r.integers(0, max_pos, T), tab=rope.table(max_pos, rot), nb=nb,
                slots=r.permutation(nb * 16)[:T].astype(np.int64), signs=workloads.splitmix64_signs(d))


def _reference(bits, c, Hq, H, inter, fill):
    om, x = MODES[bits], c["x"]
    d = x.shape[2]
    ref = np.full(om.cache_shape(c["nb"], 16, H, d), fill, np.uint8)
    known = (c["pos"] >= 0) & (c["pos"] < c["tab"].shape[0])
    pos = np.where(known, c["pos"], 0)
    kr = rope.rotate(x[:, Hq:Hq + H], pos, c["tab"], inter)
    slots = np.where(known, c["slots"], -1)
    args = (kr, x[:, Hq + H:], slots) + (() if bits == 8 else (c["signs"],))
    bad = om.write(*args, ref)
    qr = torch.from_numpy(rope.rotate(x[:, :Hq], pos, c["tab"], inter)).to(x.dtype)
    return ref, qr, known, bad


def _check(bits, c, Hq, H, inter, fill=0xA5, fused=True):
    ref, qr, known, bad = _reference(bits, c, Hq, H, inter, fill)
    x = c["x"].cuda()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    cache = torch.full(ref.shape, fill, dtype=torch.uint8, device="cuda")
    out = torch.full(qr.shape, 7.0, dtype=x.dtype, device="cuda") if Hq else None
    got = _call(bits, q if Hq else None, k, v, torch.from_numpy(c["pos"]).cuda(), torch.from_numpy(c["tab"]).cuda(),
                torch.from_numpy(c["slots"]).cuda(), torch.from_numpy(c["signs"]).cuda(), cache, query_out=out,
                interleaved=inter)
    assert np.array_equal(cache.cpu().numpy(), ref), "cache bytes differ"
    if Hq:
        assert got is out
        g = got.cpu()
        assert torch.equal(g[known].view(torch.int16), qr[known].view(torch.int16)), "rotated queries differ"
        assert bool((g[~known] == 7.0).all()), "a skipped token's query row was written"
    else:
        assert got is None
    assert torch.equal(x.cpu(), c["x"]), "inputs were written"
    return bad


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d, rot", [(64, 64), (128, 128), (128, 48), (128, 96), (64, 16)])
@pytest.mark.parametrize("bits", [4, 8, 2])
def test_bit_exact(bits, d, rot, dtype, inter):
    _check(bits, _case(37, 8, 2, d, rot, dtype, seed=rot + bits), 8, 2, inter)


@pytest.mark.parametrize("bits", [4, 8, 2])
@pytest.mark.parametrize("T, Hq, H", [(1, 4, 4), (1, 64, 8), (3, 1, 1), (17, 24, 3), (5, 0, 8), (2, 16, 16), (9, 64, 64),
                                      (130, 20, 4)])
def test_head_and_token_counts(T, Hq, H, bits):
    c = _case(T, Hq, H, 128, 128, torch.bfloat16, seed=T + H)
    _check(bits, c, Hq, H, False, fused=T % 2 == 0)


@pytest.mark.parametrize("bits", [4, 8, 2])
def test_padding_and_bad_tokens(bits):
    from gpu_helpers import status
    c = _case(40, 8, 4, 64, 64, torch.bfloat16, seed=5, max_pos=100)
    c["slots"][[3, 9]] = -1                              # cached already: only the query is rotated
    c["slots"][11], c["pos"][11] = -1, -1                # padding token
    c["pos"][[20, 21]] = [100, -5]                       # outside the table
    c["slots"][30] = c["nb"] * 16                        # outside the cache
    assert _check(bits, c, 8, 4, False) == 1
    s = status()
    assert s["position_out_of_range"] == 2 and s["slot_out_of_range"] == 1


def test_many_tokens_and_in_place():
    c = _case(5000, 32, 8, 128, 128, torch.bfloat16, seed=8, max_pos=2048)
    ref, qr, _, _ = _reference(4, c, 32, 8, False, 0)
    x = c["x"].cuda()
    cache = torch.zeros(ref.shape, dtype=torch.uint8, device="cuda")
    q = x[:, :32]
    got = _kv().kv_int4_rope_write(q, x[:, 32:40], x[:, 40:], torch.from_numpy(c["pos"]).cuda(),
                                   torch.from_numpy(c["tab"]).cuda(), torch.from_numpy(c["slots"]).cuda(),
                                   torch.from_numpy(c["signs"]).cuda(), cache, query_out=q)
    assert got is q and torch.equal(x[:, :32].cpu(), qr)
    assert np.array_equal(cache.cpu().numpy(), ref)
    assert torch.equal(x[:, 32:].cpu(), c["x"][:, 32:])


def test_equals_a_rotation_of_position_zero():
    """At position 0 the rotation is the identity, so the bytes are the plain write's."""
    kv = _kv()
    c = _case(50, 4, 4, 128, 128, torch.bfloat16, seed=2)
    x, slots, signs = c["x"].cuda(), torch.from_numpy(c["slots"]).cuda(), torch.from_numpy(c["signs"]).cuda()
    a = torch.zeros(kv.kv_int4_cache_shape(c["nb"], 16, 4, 128), dtype=torch.uint8, device="cuda")
    b = torch.zeros_like(a)
    k, v = x[:, 4:8].contiguous(), x[:, 8:].contiguous()
    kv.kv_int4_write(k, v, slots, signs, a)
    kv.kv_int4_rope_write(None, k, v, torch.zeros(50, dtype=torch.int64, device="cuda"),
                          torch.from_numpy(c["tab"]).cuda(), slots, signs, b)
    assert torch.equal(a, b)


def test_captured_replays_and_other_stream():
    c = _case(24, 8, 2, 64, 64, torch.float16, seed=4)
    ref, qr, _, _ = _reference(4, c, 8, 2, True, 0)
    s = torch.cuda.Stream()
    x, pos, tab = c["x"].cuda(), torch.from_numpy(c["pos"]).cuda(), torch.from_numpy(c["tab"]).cuda()
    slots, signs = torch.from_numpy(c["slots"]).cuda(), torch.from_numpy(c["signs"]).cuda()
    cache = torch.zeros(ref.shape, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(x[:, :8].contiguous())
    torch.cuda.synchronize()
    args = (x[:, :8], x[:, 8:10], x[:, 10:], pos, tab, slots, signs, cache)
    with torch.cuda.stream(s):
        _kv().kv_int4_rope_write(*args, query_out=out, interleaved=True)   # first call: kernel attributes
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        _kv().kv_int4_rope_write(*args, query_out=out, interleaved=True)
    cache.zero_()
    out.zero_()
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(cache.cpu().numpy(), ref) and torch.equal(out.cpu(), qr)


def test_python_checks():
    kv = _kv()
    c = _case(4, 4, 2, 64, 64, torch.bfloat16, seed=1)
    x, pos, tab = c["x"].cuda(), torch.from_numpy(c["pos"]).cuda(), torch.from_numpy(c["tab"]).cuda()
    slots, signs = torch.from_numpy(c["slots"]).cuda(), torch.from_numpy(c["signs"]).cuda()
    cache = torch.zeros(kv.kv_int4_cache_shape(c["nb"], 16, 2, 64), dtype=torch.uint8, device="cuda")
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    ok = dict(query=q, key=k, value=v, positions=pos, cos_sin=tab, slot_mapping=slots, rht_signs=signs, kv_cache=cache)
    for bad in (dict(query=q.float()), dict(key=k.transpose(0, 1)), dict(positions=pos.int()), dict(cos_sin=tab.half()),
                dict(positions=pos[:3]), dict(slot_mapping=slots.cpu()), dict(rht_signs=signs[:32]),
                dict(kv_cache=cache[:, :, :, :1].contiguous()), dict(query=None, query_out=q.contiguous()),
                dict(query_out=q[:, :2]), dict(rht_signs=None), dict(value=v[:3])):
        with pytest.raises(ValueError):
            kv.kv_int4_rope_write(**{**ok, **bad})
    with pytest.raises(kv.KVInt4Error) as e:
        kv.kv_int4_rope_write(**{**ok, "cos_sin": tab[:, :24].contiguous()})   # 24 rotated dimensions
    assert e.value.status == 2
    assert not cache.any()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d, rot", [(128, 64), (64, 16), (128, 112)])
@pytest.mark.parametrize("bits", [4, 8, 2])
def test_dimensions_behind_the_rotated_ones_stay_whatever_they_hold(bits, d, rot, dtype, inter):
    """Infinities and NaN among them: at position 0, where the others are left too, the bytes are the plain
    write's; at any position an infinite element gives its row an infinite scale, as the definition does."""
    kv = _kv()
    c = _case(21, 4, 2, d, rot, dtype, seed=rot + bits)
    x = c["x"]
    plus, minus, nan = float("inf"), float("-inf"), float("nan")
    # (token, head of key or value, element): neighbours, first, last and several in one row
    for t, h, i, val in ((0, 4, rot, plus), (1, 5, rot + 1, minus), (2, 4, d - 1, plus), (3, 5, rot, nan), (4, 4, rot + 2, plus),
                         (4, 4, rot + 3, minus), (5, 6, rot, plus), (6, 2, rot + 5, plus), (7, 3, d - 2, nan)):
        x[t, h, i] = val
    gx, slots, signs = x.cuda(), torch.from_numpy(c["slots"]).cuda(), torch.from_numpy(c["signs"]).cuda()
    k, v = gx[:, 4:6].contiguous(), gx[:, 6:].contiguous()
    shape = {4: kv.kv_int4_cache_shape, 8: kv.kv_int8_cache_shape, 2: kv.kv_int2_cache_shape}[bits](c["nb"], 16, 2, d)
    want, got = (torch.full(shape, 0xA5, dtype=torch.uint8, device="cuda") for _ in range(2))
    if bits == 8:
        kv.kv_int8_write(k, v, slots, want)
    else:
        (kv.kv_int4_write if bits == 4 else kv.kv_int2_write)(k, v, slots, signs, want)
    tab = torch.from_numpy(c["tab"]).cuda()
    q = _call(bits, gx[:, :4], k, v, torch.zeros(21, dtype=torch.int64, device="cuda"), tab, slots, signs, got, interleaved=inter)
    assert torch.equal(got, want)
    assert torch.equal(q.contiguous().view(torch.int16), gx[:, :4].contiguous().view(torch.int16))
    pos = torch.from_numpy(c["pos"]).cuda()
    _call(bits, None, k, v, pos, tab, slots, signs, got, interleaved=inter)
    at = slots[[0, 1, 2]]
    scale = got[at // 16, 0, at % 16, torch.tensor([0, 1, 0], device="cuda"), -4:].contiguous().view(torch.int32)
    assert bool(((scale & ~15) == 0x7F800000).all())
