"""GPU parity of the read-back: cached rows of the three modes as the oracles decode them in fp64.

Tolerances count roundings: half a step of the output type (and, below its normal range, half its
smallest step) for the last one, 2^-24 relative for each fp32 one before it.  INT4: c, s' c and the
product (the sums are exact integers).  INT8: the product.  INT2: the butterflies' sums round at
magnitudes of at most d times the largest centroid, log2(d) of them, then c and sigma."""
import numpy as np
import pytest
import torch

import oracle
import workloads
from oracle import int2 as o2
from oracle import int8 as o8

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SMALLEST = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133, torch.float32: 2.0 ** -149}


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from gpu_helpers import clear_status
    clear_status()


def _kv():
    import int4_token_head_kv_gb300 as kv
    return kv


def _read(bits, cache, slots, signs, **kw):
    kv = _kv()
    if bits == 8:
        return kv.kv_int8_read(cache, slots, **kw)
    return (kv.kv_int4_read if bits == 4 else kv.kv_int2_read)(cache, slots, signs, **kw)


def _random_cache(bits, nb, H, d, seed):
    """Any code bytes, scales over several magnitudes (INT4: any zero-point)."""
    r = np.random.default_rng(seed)
    om = {4: oracle, 8: o8, 2: o2}[bits]
    cache = r.integers(0, 256, om.cache_shape(nb, 16, H, d), dtype=np.uint8)
    s = (10.0 ** r.uniform(-3, 1, cache.shape[:-1])).astype("<f4").view(np.uint32)
    if bits == 4:
        s = (s & np.uint32(0xFFFFFFF0)) | r.integers(0, 16, s.shape, dtype=np.uint32)
    cache[..., -4:] = s[..., None].view(np.uint8).reshape(*s.shape, 4)
    return cache


def _decoded(bits, rows, signs):
    flat = rows.reshape(-1, rows.shape[-1])
    x = o8.decode_rows(flat) if bits == 8 else o2.decode_rows(flat, signs) if bits == 2 else oracle.decode_rows(flat, signs)
    return x.reshape(*rows.shape[:-1], -1)


def _check(bits, cache, slots, d, dtype, **kw):
    H = cache.shape[3]
    signs = workloads.splitmix64_signs(d)
    at = np.where((slots >= 0) & (slots < cache.shape[0] * 16), slots, 0)
    live = (slots >= 0) & (slots < cache.shape[0] * 16)
    rows = cache[at // 16, :, at % 16]                       # [T, 2, H, row]
    ref = _decoded(bits, rows, signs) * live[:, None, None, None]
    sigma = rows[..., -4:].copy().view("<f4")[..., 0].astype(np.float64)
    got = _read(bits, torch.from_numpy(cache).cuda(), torch.from_numpy(slots).cuda(), torch.from_numpy(signs).cuda(),
                dtype=dtype, **kw)
    half = torch.finfo(dtype).eps / 2
    for p in (0, 1):
        g = got[p].double().cpu().numpy()
        assert got[p].shape == (len(slots), H, d) and got[p].dtype == dtype
        r = ref[:, p]
        tol = np.abs(r) * (half + 4 * U) + SMALLEST[dtype] / 2
        if bits == 2:
            steps = np.log2(d) + 2
            tol = tol + (sigma[:, p] * live[:, None])[..., None] * 1.52 * np.sqrt(d) * steps * U
        assert np.all(np.abs(g - r) <= tol), f"plane {p}: worst {np.max(np.abs(g - r) - tol):.3g}"
        assert not np.any(g[~live]), "a row without a slot is not zero"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits", [4, 8, 2])
def test_any_codes(bits, d, dtype):
    cache = _random_cache(bits, 12, 4, d, seed=bits + d)
    slots = np.random.default_rng(1).permutation(12 * 16)[:101].astype(np.int64)
    _check(bits, cache, slots, d, dtype)


@pytest.mark.parametrize("bits", [4, 8, 2])
@pytest.mark.parametrize("T, H", [(1, 1), (1, 8), (7, 3), (33, 2), (40, 8), (5, 16), (3, 64), (50, 1)])
def test_head_and_token_counts(T, H, bits):
    nb = (T + 15) // 16 + 1
    cache = _random_cache(bits, nb, H, 128, seed=T * H)
    _check(bits, cache, np.random.default_rng(T).permutation(nb * 16)[:T].astype(np.int64), 128, torch.bfloat16)


@pytest.mark.parametrize("H", [8, 3])
@pytest.mark.parametrize("bits", [4, 8, 2])
def test_repeated_negative_and_outside_slots(bits, H):
    from gpu_helpers import status
    cache = _random_cache(bits, 2, H, 64, seed=3)
    # values that a dead row must not pick up from a neighbour: every code and scale is live
    slots = np.array([5, 5, -1, 31, 32, -7, 10 ** 12, 0, 5], np.int64)
    _check(bits, cache, slots, 64, torch.float32)
    assert status()["slot_out_of_range"] == 2


@pytest.mark.parametrize("bits", [4, 8, 2])
def test_many_rows(bits):
    cache = _random_cache(bits, 300, 8, 128, seed=9)
    _check(bits, cache, np.random.default_rng(2).permutation(4800).astype(np.int64), 128, torch.bfloat16)


def test_given_outputs_stream_and_empty():
    kv = _kv()
    cache = _random_cache(4, 4, 2, 64, seed=6)
    signs = torch.from_numpy(workloads.splitmix64_signs(64)).cuda()
    c, slots = torch.from_numpy(cache).cuda(), torch.arange(30, device="cuda")
    k = torch.full((30, 2, 64), 9.0, dtype=torch.float16, device="cuda")
    v = torch.full((30, 2, 64), 9.0, dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = kv.kv_int4_read(c, slots, signs, key_out=k, value_out=v, stream=s)
    s.synchronize()
    assert got[0] is k and got[1] is v
    want = kv.kv_int4_read(c, slots, signs, dtype=torch.float16)
    assert torch.equal(want[0], k) and torch.equal(want[1], v)
    e = kv.kv_int4_read(c, slots[:0], signs)
    assert e[0].shape == (0, 2, 64)
    for bad in (lambda: kv.kv_int4_read(c, slots.int(), signs), lambda: kv.kv_int4_read(c, slots, signs[:32]),
                lambda: kv.kv_int4_read(c, slots, None), lambda: kv.kv_int8_read(c[..., :20].contiguous(), slots),
                lambda: kv.kv_int4_read(c, slots, signs, key_out=k[:4]),
                lambda: kv.kv_int4_read(c, slots, signs, dtype=torch.int32)):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("bits", [4, 8, 2])
def test_write_then_read_keeps_the_vectors(bits):
    """A stored vector comes back within its quantiser's step (INT4: 1.5 s' in the rotated domain, so
    sqrt(d) 1.5 s' in the 2-norm; INT8: 0.51 s per element)."""
    kv = _kv()
    wl = workloads.random_write(60, 4, 128, seed=21)
    signs, slots = torch.from_numpy(wl.signs).cuda(), torch.from_numpy(wl.slot_mapping).cuda()
    k, v = wl.key.cuda(), wl.value.cuda()
    if bits == 8:
        cache = torch.zeros(kv.kv_int8_cache_shape(wl.num_blocks, 16, 4, 128), dtype=torch.uint8, device="cuda")
        kv.kv_int8_write(k, v, slots, cache)
    else:
        shape = kv.kv_int4_cache_shape if bits == 4 else kv.kv_int2_cache_shape
        cache = torch.zeros(shape(wl.num_blocks, 16, 4, 128), dtype=torch.uint8, device="cuda")
        (kv.kv_int4_write if bits == 4 else kv.kv_int2_write)(k, v, slots, signs, cache)
    gk, gv = _read(bits, cache, slots, signs, dtype=torch.float32)
    for g, x in ((gk, k.float()), (gv, v.float())):
        err = (g - x).norm(dim=-1)
        step = {4: 1.5 * (x.abs().sum(-1) / 128 ** 0.5 * 2).clamp(min=0) / 15, 8: 0.51 * x.abs().amax(-1) / 127}.get(bits)
        if bits == 2:
            assert bool((err < x.norm(dim=-1)).all())   # sigma and the centroids keep less than the norm lost
        else:
            assert bool((err <= 128 ** 0.5 * step).all())


@pytest.mark.parametrize("raw", [False, True])
def test_outputs_belong_to_the_stream_that_writes_them(raw):
    """Outputs allocated by a call on another stream and dropped while it has yet to run: the current stream
    must not be handed their memory."""
    kv = _kv()
    cache = torch.from_numpy(_random_cache(4, 4, 2, 64, seed=6)).cuda()
    signs, slots = torch.ones(64, device="cuda"), torch.arange(64, device="cuda").repeat(200)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(50_000_000)
    out = kv.kv_int4_read(cache, slots, signs, dtype=torch.float32, stream=s.cuda_stream if raw else s)
    shape = out[0].shape
    del out
    a, b = torch.zeros(shape, device="cuda"), torch.zeros(shape, device="cuda")
    torch.cuda.synchronize()
    assert not a.any() and not b.any()
    got = kv.kv_int4_read(cache, slots, signs, dtype=torch.float32, stream=0)   # the default stream's handle
    want = kv.kv_int4_read(cache, slots, signs, dtype=torch.float32)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_int4_rows_come_back_within_their_own_step():
    """A stored INT4 vector comes back within half a step of its row's own scale s' in every rotated dimension:
    code = N(y / s' + zp), and with elements of both signs no y / s' + zp lies further than half outside 0..15 (s' is
    short of (max - min) / 15 by less than 2^-19 of it).  So within sqrt(d) s' / 2 in the 2-norm, with 1e-4 for that
    and the fp32 butterflies; a read-back of zeros would not be."""
    kv = _kv()
    wl = workloads.random_write(60, 4, 128, seed=22)
    signs, slots = torch.from_numpy(wl.signs).cuda(), torch.from_numpy(wl.slot_mapping).cuda()
    k, v = wl.key.cuda(), wl.value.cuda()
    cache = torch.zeros(kv.kv_int4_cache_shape(wl.num_blocks, 16, 4, 128), dtype=torch.uint8, device="cuda")
    kv.kv_int4_write(k, v, slots, signs, cache)
    words = cache[slots // 16, :, slots % 16, :, -4:].contiguous().view(torch.int32)[..., 0]   # [T, 2, H]
    step = (words & -16).view(torch.float32)
    for p, (g, x) in enumerate(zip(kv.kv_int4_read(cache, slots, signs, dtype=torch.float32), (k.float(), v.float()))):
        bound = 128 ** 0.5 / 2 * step[:, p] * (1 + 1e-4)
        assert bool(((g - x).norm(dim=-1) <= bound).all())
        assert bool((x.norm(dim=-1) > bound).all())
