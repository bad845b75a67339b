"""GPU parity of the rotary writes with several position axes: cache bytes and rotated queries bit-exact against the
oracle's rotation followed by each mode's write oracle."""
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


def _call(bits, q, k, v, pos, tab, sections, slots, signs, cache, **kw):
    kv = _kv()
    if bits == 8:
        return kv.kv_int8_mrope_write(q, k, v, pos, tab, sections, slots, cache, **kw)
    return (kv.kv_int4_mrope_write if bits == 4 else kv.kv_int2_mrope_write)(q, k, v, pos, tab, sections, slots, signs, cache, **kw)


def _case(T, Hq, H, d, sections, dtype, seed, max_pos=512):
    r = np.random.default_rng(seed)
    x = torch.from_numpy(r.standard_normal((T, Hq + 2 * H, d)).astype(np.float32) * 3).to(dtype)
    nb = (T + 15) // 16 + 3
    return dict(x=x, pos=r.integers(0, max_pos, (len(sections), T)), tab=rope.table(max_pos, 2 * sum(sections)), nb=nb,
                slots=r.permutation(nb * 16)[:T].astype(np.int64), signs=workloads.splitmix64_signs(d), sections=sections)


def _reference(bits, c, Hq, H, mixed, inter, fill):
    om, x = MODES[bits], c["x"]
    ref = np.full(om.cache_shape(c["nb"], 16, H, x.shape[2]), fill, np.uint8)
    known = ((c["pos"] >= 0) & (c["pos"] < c["tab"].shape[0])).all(axis=0)
    pos = np.where(known, c["pos"], 0)
    kr = rope.rotate_axes(x[:, Hq:Hq + H], pos, c["tab"], c["sections"], mixed, inter)
    slots = np.where(known, c["slots"], -1)
    om.write(*((kr, x[:, Hq + H:], slots) + (() if bits == 8 else (c["signs"],))), ref)
    qr = torch.from_numpy(rope.rotate_axes(x[:, :Hq], pos, c["tab"], c["sections"], mixed, inter)).to(x.dtype)
    return ref, qr, known


def _check(bits, c, Hq, H, mixed, inter, fused=True):
    ref, qr, known = _reference(bits, c, Hq, H, mixed, inter, 0xA5)
    x = c["x"].cuda()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    cache = torch.full(ref.shape, 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full(qr.shape, 7.0, dtype=x.dtype, device="cuda") if Hq else None
    got = _call(bits, q if Hq else None, k, v, torch.from_numpy(c["pos"]).cuda(), torch.from_numpy(c["tab"]).cuda(),
                c["sections"], torch.from_numpy(c["slots"]).cuda(), torch.from_numpy(c["signs"]).cuda(), cache, query_out=out,
                interleaved=inter, mixed_sections=mixed)
    assert np.array_equal(cache.cpu().numpy(), ref), "cache bytes differ"
    if Hq:
        assert got is out
        g = got.cpu()
        assert torch.equal(g[known].view(torch.int16), qr[known].view(torch.int16)), "rotated queries differ"
        assert bool((g[~known] == 7.0).all()), "a skipped token's query row was written"
    else:
        assert got is None
    assert torch.equal(x.cpu(), c["x"]), "inputs were written"


@pytest.mark.parametrize("mixed, inter", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d, sections", [(128, (16, 24, 24)), (128, (24, 20, 20)), (64, (16, 16)), (128, (5, 3, 0, 16)),
                                         (64, (1, 7)), (128, (48,))])
@pytest.mark.parametrize("bits", [4, 8, 2])
def test_bit_exact(bits, d, sections, dtype, mixed, inter):
    _check(bits, _case(37, 8, 2, d, sections, dtype, seed=sum(sections) + bits), 8, 2, mixed, inter)


@pytest.mark.parametrize("bits", [4, 8, 2])
@pytest.mark.parametrize("T, Hq, H", [(1, 4, 4), (1, 64, 8), (3, 1, 1), (17, 24, 3), (5, 0, 8), (2, 16, 16), (9, 64, 64),
                                      (130, 20, 4), (3000, 8, 2)])
def test_head_and_token_counts(T, Hq, H, bits):
    _check(bits, _case(T, Hq, H, 128, (16, 24, 24), torch.bfloat16, seed=T + H), Hq, H, T % 3 == 0, False, fused=T % 2 == 0)


@pytest.mark.parametrize("bits", [4, 8, 2])
def test_padding_and_bad_tokens(bits):
    from gpu_helpers import status
    c = _case(40, 8, 4, 64, (10, 11, 11), torch.bfloat16, seed=5, max_pos=100)
    c["slots"][[3, 9]] = -1                              # cached already: only the query is rotated
    c["slots"][11], c["pos"][:, 11] = -1, -1             # padding token
    c["slots"][12], c["pos"][1, 12] = -1, -1             # not all of its positions are negative: counted
    c["pos"][0, 20], c["pos"][2, 21], c["pos"][1, 22] = 100, -5, 1 << 40   # outside the table on one axis
    c["pos"][:, 23] = -1                                 # no position, but a slot
    _check(bits, c, 8, 4, True, False)
    s = status()
    assert s["position_out_of_range"] == 5 and s["slot_out_of_range"] == 0


def test_equal_positions_give_the_one_axis_write():
    kv = _kv()
    c = _case(75, 8, 4, 128, (16, 24, 24), torch.bfloat16, seed=9)
    x, pos, tab = c["x"].cuda(), torch.from_numpy(c["pos"][0]).cuda(), torch.from_numpy(c["tab"]).cuda()
    slots, signs = torch.from_numpy(c["slots"]).cuda(), torch.from_numpy(c["signs"]).cuda()
    a = torch.zeros(kv.kv_int4_cache_shape(c["nb"], 16, 4, 128), dtype=torch.uint8, device="cuda")
    b = torch.zeros_like(a)
    qa = kv.kv_int4_rope_write(x[:, :8], x[:, 8:12], x[:, 12:], pos, tab, slots, signs, a)
    qb = kv.kv_int4_mrope_write(x[:, :8], x[:, 8:12], x[:, 12:], pos.expand(3, -1).contiguous(), tab, (16, 24, 24), slots, signs, b)
    assert torch.equal(a, b) and torch.equal(qa, qb)


@pytest.mark.parametrize("bits", [4, 8, 2])
def test_slots_past_32_bit_offsets(bits):
    """Slots whose rows lie more than 2^32 bytes into a cache: the bytes of the same slots of a small one."""
    c = _case(50, 8, 2, 64, (12, 10, 10), torch.bfloat16, 3)
    ref, _, _ = _reference(bits, c, 8, 2, False, False, 0)
    far = (1 << 32) // ref[0].size + 3
    cache = torch.zeros((far + c["nb"], *ref.shape[1:]), dtype=torch.uint8, device="cuda")
    x = c["x"].cuda()
    _call(bits, x[:, :8], x[:, 8:10], x[:, 10:], torch.from_numpy(c["pos"]).cuda(), torch.from_numpy(c["tab"]).cuda(), c["sections"],
          torch.from_numpy(c["slots"] + 16 * far).cuda(), torch.from_numpy(c["signs"]).cuda(), cache)
    assert np.array_equal(cache[far:].cpu().numpy(), ref)
    assert not bool(cache[:far].any())


def test_in_place_on_a_stream_and_replayed():
    c = _case(600, 32, 8, 128, (24, 20, 20), torch.float16, seed=8, max_pos=2048)
    ref, qr, _ = _reference(4, c, 32, 8, True, False, 0)
    s = torch.cuda.Stream()
    x = c["x"].cuda()
    pos, tab = torch.from_numpy(c["pos"]).cuda(), torch.from_numpy(c["tab"]).cuda()
    slots, signs = torch.from_numpy(c["slots"]).cuda(), torch.from_numpy(c["signs"]).cuda()
    cache = torch.zeros(ref.shape, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    q = x[:, :32]
    args = (x[:, 32:40], x[:, 40:], pos, tab, c["sections"], slots, signs, cache)
    got = _kv().kv_int4_mrope_write(q, *args, query_out=q, mixed_sections=True, stream=s)
    s.synchronize()
    assert got is q and torch.equal(q.cpu(), qr) and np.array_equal(cache.cpu().numpy(), ref)
    out = torch.empty_like(qr, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        _kv().kv_int4_mrope_write(q, *args, query_out=out, mixed_sections=True)
    x.copy_(c["x"])
    cache.zero_()
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), qr) and np.array_equal(cache.cpu().numpy(), ref)


def test_python_checks():
    kv = _kv()
    c = _case(4, 4, 2, 64, (16, 8, 8), torch.bfloat16, seed=1)
    x, pos, tab = c["x"].cuda(), torch.from_numpy(c["pos"]).cuda(), torch.from_numpy(c["tab"]).cuda()
    slots, signs = torch.from_numpy(c["slots"]).cuda(), torch.from_numpy(c["signs"]).cuda()
    cache = torch.zeros(kv.kv_int4_cache_shape(c["nb"], 16, 2, 64), dtype=torch.uint8, device="cuda")
    ok = dict(query=x[:, :4], key=x[:, 4:6], value=x[:, 6:], positions=pos, cos_sin=tab, sections=(16, 8, 8), slot_mapping=slots,
              rht_signs=signs, kv_cache=cache)
    for bad in (dict(sections=(16, 8)), dict(sections=(16, 8, 7)), dict(sections=(16, 16)), dict(sections=()),
                dict(positions=pos[0].contiguous()), dict(positions=pos.T.contiguous()), dict(positions=pos.T),
                dict(positions=pos.int()), dict(sections=(8, 8, 8, 4, 4)), dict(positions=pos.cpu())):
        with pytest.raises(ValueError):
            kv.kv_int4_mrope_write(**{**ok, **bad})
    assert not cache.any()
