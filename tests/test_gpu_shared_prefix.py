"""GPU parity of the shared-prefix attention: against the oracle (which knows nothing of sharing), and on
larger batches against the plain decode call.  Batches of num_seqs x prefix >= 16 384 tokens take the
prefix kernel, smaller ones the plain walk; each case says which it means."""
import numpy as np
import pytest
import torch

import oracle
import workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from gpu_helpers import clear_status
    clear_status()


def _kv():
    import int4_token_head_kv_gb300 as kv
    return kv


class Batch:
    """A decode batch on a shared prefix: a written cache, tables and lengths (on the host and the GPU)."""

    def __init__(self, prefix, lens, Hq, H, d, dtype=torch.bfloat16, seed=0, query_lens=None, outliers=True, extra_q=0):
        r = np.random.default_rng(seed)
        S, shared = len(lens), prefix // 16
        mine = max(0, -(-max(lens) // 16) - shared)
        nb = shared + S * mine + 2
        ids = r.permutation(nb).astype(np.int32)
        self.prefix, self.prefix_blocks = prefix, ids[:shared].copy()
        self.tables = np.concatenate([np.tile(ids[:shared], (S, 1)), ids[shared:shared + S * mine].reshape(S, mine)], 1)
        if self.tables.shape[1] == 0:
            self.tables = np.zeros((S, 1), np.int32)
        self.lens = np.asarray(lens, np.int32)
        self.qlens = np.ones(S, np.int32) if query_lens is None else np.asarray(query_lens, np.int32)
        self.qsl = np.concatenate([[0], np.cumsum(self.qlens)]).astype(np.int32)
        g = torch.Generator(device="cuda").manual_seed(seed)
        k = torch.randn(nb * 16, H, d, generator=g, device="cuda")
        if outliers:
            k[:, :, :4] *= 10.0
        v = torch.randn(nb * 16, H, d, generator=g, device="cuda")
        self.signs = workloads.splitmix64_signs(d)
        self.gsigns = torch.from_numpy(self.signs).cuda()
        kv = _kv()
        self.cache = torch.zeros(kv.kv_int4_cache_shape(nb, 16, H, d), dtype=torch.uint8, device="cuda")
        kv.kv_int4_write(k.to(dtype), v.to(dtype), torch.arange(nb * 16, device="cuda"), self.gsigns, self.cache)
        self.q = torch.randn(int(self.qsl[-1]) + extra_q, Hq, d, generator=g, device="cuda").to(dtype)
        self.scale = d ** -0.5
        self.max_len = int(max(lens))

    def _args(self):
        return (torch.from_numpy(self.tables).cuda(), torch.from_numpy(self.lens).cuda(), torch.from_numpy(self.qsl).cuda())

    def shared(self, out_dtype=torch.float32, **kw):
        t, l, q = self._args()
        return _kv().kv_int4_shared_prefix_attention(self.q, self.cache, torch.from_numpy(self.prefix_blocks).cuda(),
                                                     self.prefix, t, l, q, self.scale, self.gsigns,
                                                     **{"max_seq_len": self.max_len, "out_dtype": out_dtype, **kw})

    def plain(self, out_dtype=torch.float32, **kw):
        t, l, q = self._args()
        return _kv().kv_int4_paged_attention(self.q, self.cache, t, l, q, self.scale, self.gsigns, max_query_len=1,
                                             max_seq_len=self.max_len, out_dtype=out_dtype, **kw)

    def is_shared(self):
        """Whether the call takes the prefix kernel: its workspace holds more than the plain walk's."""
        S, Hq, d = len(self.lens), self.q.shape[1], self.q.shape[2]
        H = self.cache.shape[3]
        kv = _kv()
        return kv.kv_int4_shared_prefix_workspace_bytes(self.q.shape[0], Hq, H, d, S, self.prefix, self.max_len) != \
            kv.kv_int4_attention_workspace_bytes(Hq, H, d, S, self.max_len)

    def oracle(self, seqs=None):
        return oracle.paged_attention(self.q, self.cache.cpu().numpy(), self.tables, self.lens, self.qsl, self.scale,
                                      self.signs, seqs=seqs)


def _check(b, shared=True, seqs=None, **kw):
    from gpu_helpers import assert_attention_close, status
    assert b.is_shared() == shared
    got = b.shared(**kw)
    assert_attention_close(got, b.oracle(seqs), "shared prefix")
    assert not any(status().values())
    return got


def _lens(prefix, S, most, seed):
    return list(prefix + np.random.default_rng(seed).integers(1, most + 1, S))


@pytest.mark.parametrize("Hq, H", [(1, 1), (4, 1), (8, 8), (8, 4), (8, 2), (16, 2), (64, 8)])
@pytest.mark.parametrize("d", [64, 128])
def test_head_layouts(Hq, H, d):
    _check(Batch(1024, _lens(1024, 16, 40, Hq), Hq, H, d, seed=Hq + d), seqs=range(0, 16, 3))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_types(dtype, out_dtype):
    _check(Batch(1000, _lens(1000, 17, 60, 1), 8, 2, 128, dtype=dtype, seed=2), out_dtype=out_dtype, seqs=range(0, 17, 4))


@pytest.mark.parametrize("prefix, S", [(128, 130), (129, 128), (144, 120), (205, 90), (256, 64), (391, 45), (640, 27),
                                       (1025, 16), (5000, 4), (4096, 2), (8200, 3)])
def test_prefix_lengths(prefix, S):
    _check(Batch(prefix, _lens(prefix, S, 50, S), 8, 2, 64, seed=prefix), seqs=range(0, S, max(1, S // 6)))


@pytest.mark.parametrize("prefix, S", [(0, 3), (15, 2), (16, 5), (256, 3), (1025, 15), (20000, 1), (4096, 1)])
def test_small_ones_take_the_plain_walk(prefix, S):
    b = Batch(prefix, _lens(prefix, S, 50, S), 8, 2, 64, seed=prefix)
    got = _check(b, shared=False)
    assert torch.equal(got, b.plain())


@pytest.mark.parametrize("Hq, H", [(1, 1), (2, 1), (4, 1), (8, 1)])
def test_batch_sizes_around_a_row_tile(Hq, H):
    tile = 128 // (Hq // H)
    for S in (tile - 1, tile, tile + 1, 2 * tile + 3):
        P = -(-16384 // S) + 20
        _check(Batch(P, _lens(P, S, 30, S), Hq, H, 64, seed=S), seqs=sorted({0, 1, tile - 2, min(tile, S - 1), S - 1}))


def test_lengths_inside_and_at_the_prefix():
    # padding rows, rows that end inside the prefix, at its end, and behind it
    lens = [0, 1, 128, 129, 1000, 2031, 2032, 2040, 2041, 2100, 0, 16]
    got = _check(Batch(2040, lens, 8, 2, 128, seed=3))
    assert not got[0].any() and not got[10].any()


def test_every_sequence_ends_inside_the_prefix():
    _check(Batch(4500, [4496, 4496, 100, 1, 0], 8, 4, 128, seed=4))


def test_a_batch_of_padding_rows():
    b = Batch(8192, [0, 8192, 0], 8, 2, 64, seed=14)
    b.lens[1] = 0
    assert b.is_shared() and not b.shared().any()


def test_sequences_without_a_query_and_rows_behind_the_last():
    from gpu_helpers import assert_attention_close
    r = np.random.default_rng(5)
    S, P = 70, 256
    qlens = (r.random(S) < 0.7).astype(np.int32)
    qlens[[0, 1, 2, S - 1]] = [0, 0, 1, 1]
    b = Batch(P, _lens(P, S, 40, 5), 8, 2, 64, seed=5, query_lens=qlens, extra_q=3)
    n = int(qlens.sum())
    assert b.is_shared()
    out = torch.full(b.q.shape, 5.0, device="cuda")
    got = b.shared(out=out)
    assert_attention_close(got[:n], b.oracle()[:n])
    assert bool((out[n:] == 5.0).all())


def test_bad_prefix_block_is_counted_and_skipped():
    from gpu_helpers import assert_attention_close, status
    b = Batch(2048, [2049, 2080, 2060, 2055, 2048, 2100, 2070, 2050], 8, 2, 64, seed=6)
    assert b.is_shared()
    b.prefix_blocks[3], b.prefix_blocks[9] = -7, 10 ** 6
    got = b.shared()
    assert status()["block_out_of_range"] > 0
    # the tokens of those blocks are no keys: the oracle on the sequences without them
    drop = np.ones(2048 // 16, bool)
    drop[[3, 9]] = False
    cols = np.concatenate([drop, np.ones(b.tables.shape[1] - 128, bool)])
    ref = oracle.paged_attention(b.q, b.cache.cpu().numpy(), b.tables[:, cols], b.lens - 32, b.qsl, b.scale, b.signs)
    assert_attention_close(got, ref)


def test_queries_of_very_different_magnitudes():
    """A CTA's rows share one prescale where they can: rows up to 2^100 apart, and rows of zeros."""
    b = Batch(2048, _lens(2048, 14, 20, 3), 8, 2, 128, seed=15, outliers=False)
    e = [0, -12, 0, -6, 0, 2, -12, -3, 0, 0, 1, -9, -100, -30]
    b.q *= (2.0 ** torch.tensor(e, device="cuda")).to(b.q.dtype)[:, None, None]
    b.q[8] = 0
    _check(b)
    b.q[0] *= 2.0 ** -70   # the row the shared exponent comes from
    _check(b)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 3e38])
@pytest.mark.parametrize("where", [0, 5])
def test_a_sequence_of_garbage_leaves_the_others_alone(where, bad):
    """A query that is not finite, or huge, reaches only its own sequence's output; a padding row's reaches none."""
    from gpu_helpers import assert_attention_close
    b = Batch(2048, _lens(2048, 12, 20, 4), 8, 2, 128, seed=16)
    ref = b.oracle()
    b.q[where, :, ::3] = bad
    got = b.shared()
    keep = [i for i in range(12) if i != where]
    assert_attention_close(got[keep], ref[keep])
    b.lens[where] = 0
    got = b.shared()
    assert_attention_close(got[keep], ref[keep])
    assert not got[where].any()


@pytest.mark.parametrize("scale", [0.0, -0.05, 1e-30, 3.0])
def test_softmax_scales(scale):
    b = Batch(2030, [2031, 2040, 1000, 2029, 5, 2032, 2050, 1999, 2047], 8, 2, 64, seed=17, outliers=False)
    b.scale = scale
    _check(b)


@pytest.mark.parametrize("opts", [dict(softcap=5.0), dict(window_left=900), dict(window_left=10), dict(alibi=True),
                                  dict(qq=True), dict(softcap=3.0, window_left=1500, alibi=True, qq=True)])
@pytest.mark.parametrize("Hq, H, d", [(8, 2, 128), (8, 1, 64)])
def test_options(Hq, H, d, opts):
    from gpu_helpers import assert_attention_close
    b = Batch(2030, [2031, 2040, 1000, 2029, 0, 2032, 2050, 1999, 2047, 15], Hq, H, d, seed=18, outliers=False)
    assert b.is_shared()
    o = {k: v for k, v in opts.items() if k in ("softcap", "window_left")}
    g = dict(o)
    if "alibi" in opts:
        o["alibi_slopes"] = np.float32(2.0) ** -np.arange(1, Hq + 1, dtype=np.float32)
        g["alibi_slopes"] = torch.from_numpy(o["alibi_slopes"]).cuda()
    if "qq" in opts:
        o["qq_bias"] = np.full((1, 1), 1.5, np.float32)
        g["qq_bias"] = torch.from_numpy(o["qq_bias"]).cuda()
    ref = oracle.paged_attention(b.q, b.cache.cpu().numpy(), b.tables, b.lens, b.qsl, b.scale, b.signs, **o)
    assert_attention_close(b.shared(**g), ref, str(opts))
    small = Batch(256, [260, 300, 257], Hq, H, d, seed=19)
    assert not small.is_shared() and torch.equal(small.shared(**g), small.plain(**g))


def test_heavy_tails_and_large_scales():
    b = Batch(2000, _lens(2000, 9, 90, 7), 16, 2, 128, seed=7)
    assert b.is_shared()
    kv = _kv()
    n = b.cache.shape[0] * 16
    g = torch.Generator(device="cuda").manual_seed(1)
    t3 = torch.randn(n, 2, 128, generator=g, device="cuda") / torch.rand(n, 2, 128, generator=g, device="cuda").clamp(min=0.02)
    mag = 10.0 ** (torch.rand(n, 1, 1, generator=g, device="cuda") * 4 - 2)
    kv.kv_int4_write((t3 * 0.5).bfloat16(), (t3.flip(0) * mag).bfloat16(), torch.arange(n, device="cuda"), b.gsigns, b.cache)
    ref = b.oracle()
    got = b.shared().double().cpu().numpy()
    # the weights are rounded to fp16 (2^-11 each) and the error of a row is at most that share of its
    # largest value magnitude; the values span four decades, so the bound is relative to the row's largest
    big = np.abs(ref).max(axis=2, keepdims=True)
    assert np.all(np.abs(got - ref) <= 1e-2 * np.abs(ref) + 1e-2 * big + 2e-3)


@pytest.mark.parametrize("S, prefix, Hq, H, d", [(64, 8192, 32, 8, 128), (100, 3000, 64, 8, 128), (40, 20000, 8, 1, 64),
                                                 (300, 700, 16, 4, 64)])
def test_larger_batches_match_the_plain_call(S, prefix, Hq, H, d):
    from gpu_helpers import ATOL, RTOL, status
    r = np.random.default_rng(S)
    b = Batch(prefix, list(prefix + r.integers(1, 600, S)), Hq, H, d, seed=S, outliers=False)
    a, c = b.shared().double(), b.plain().double()
    assert bool(((a - c).abs() <= 2 * (ATOL + RTOL * c.abs())).all())
    # far closer in the mean: both carry fp16 weights (a relative 2^-11 at most, independent per key)
    assert float((a - c).norm() / c.norm()) < 1e-3
    assert not any(status().values())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
def test_outputs_finer_than_bf16_are_not_rounded_by_the_weights(d, dtype):
    """fp16 and fp32 outputs carry the weights in two halves: the error against 64 bits, in the 2-norm, stays
    near the output's own rounding.  (fp32: Q' and the weights keep 22 bits, the products' sums are fp32 over
    128 dimensions and some thousand keys; a single fp16 weight would give about 2e-4.)"""
    b = Batch(2100, _lens(2100, 10, 30, 6), 8, 2, d, dtype=dtype, seed=20)
    assert b.is_shared()
    ref = torch.from_numpy(b.oracle())
    err = lambda out: float((out.double().cpu() - ref).norm() / ref.norm())
    assert err(b.shared(torch.float32)) < 2e-5
    # half a step is 2^-11 at most, its root mean square over the mantissas and signs about 0.42 of it
    assert err(b.shared(torch.float16)) < 0.5 * 2.0 ** -11


def test_same_bits_again_and_captured():
    b = Batch(1000, [1001 + 9 * i for i in range(20)], 32, 8, 128, seed=8)
    first = b.shared(out_dtype=torch.bfloat16)
    t, l, q = b._args()
    pb = torch.from_numpy(b.prefix_blocks).cuda()
    assert b.is_shared()
    need = _kv().kv_int4_shared_prefix_workspace_bytes(20, 32, 8, 128, 20, 1000, b.max_len)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(b.q)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        _kv().kv_int4_shared_prefix_attention(b.q, b.cache, pb, 1000, t, l, q, b.scale, b.gsigns, max_seq_len=b.max_len,
                                              out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)


def test_python_checks():
    kv = _kv()
    b = Batch(16384, [16390, 16384], 8, 2, 64, seed=9)
    with pytest.raises(ValueError):
        b.shared(workspace=torch.empty(1 << 20, dtype=torch.uint8))
    keep, b.prefix_blocks = b.prefix_blocks, b.prefix_blocks[:1023]
    with pytest.raises(ValueError):
        b.shared()
    b.prefix_blocks = keep
    with pytest.raises(kv.KVInt4Error) as e:
        b.shared(workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 4


def test_a_serving_step_as_it_runs():
    """Rotary append of the batch's new tokens, attention over the shared prefix with the rotated queries,
    and the new rows read back: one step after another on one stream, no synchronisation between."""
    from gpu_helpers import assert_attention_close
    from oracle import rope
    kv = _kv()
    S, P, Hq, H, d, steps = 24, 720, 32, 8, 128, 5
    b = Batch(P, [P + 1 + 3 * i + steps for i in range(S)], Hq, H, d, seed=10)
    assert b.is_shared()
    r = np.random.default_rng(0)
    tab = rope.table(1024, d)
    start = b.lens - steps
    gtab, gt = torch.from_numpy(tab).cuda(), torch.from_numpy(b.tables).cuda()
    pb, qsl = torch.from_numpy(b.prefix_blocks).cuda(), torch.from_numpy(b.qsl).cuda()
    xs, lens, slots, poss = [], [], [], []
    for i in range(steps):
        xs.append(torch.from_numpy(r.standard_normal((S, Hq + 2 * H, d)).astype(np.float32)).bfloat16())
        pos = (start + i).astype(np.int64)
        poss.append(pos)
        slots.append(b.tables[np.arange(S), pos // 16].astype(np.int64) * 16 + pos % 16)
        lens.append((start + i + 1).astype(np.int32))
    gx = [x.cuda() for x in xs]
    gl, gs, gp = ([torch.from_numpy(a).cuda() for a in z] for z in (lens, slots, poss))
    torch.cuda.synchronize()
    outs, rows = [], []
    for i in range(steps):
        q = kv.kv_int4_rope_write(gx[i][:, :Hq], gx[i][:, Hq:Hq + H], gx[i][:, Hq + H:], gp[i], gtab, gs[i], b.gsigns, b.cache)
        outs.append(kv.kv_int4_shared_prefix_attention(q, b.cache, pb, P, gt, gl[i], qsl, b.scale, b.gsigns,
                                                       max_seq_len=b.max_len, out_dtype=torch.float32))
        rows.append(kv.kv_int4_read(b.cache, gs[i], b.gsigns, dtype=torch.float32))
    torch.cuda.synchronize()
    cache = b.cache.cpu().numpy()   # later steps only added rows behind the earlier ones' lengths
    for i in (0, steps - 1):
        qr = torch.from_numpy(rope.rotate(xs[i][:, :Hq], poss[i], tab)).bfloat16()
        ref = oracle.paged_attention(qr, cache, b.tables, lens[i], b.qsl, b.scale, b.signs, seqs=range(0, S, 5))
        assert_attention_close(outs[i], ref, f"step {i}")
        want = oracle.decode_rows(cache[slots[i] // 16, 0, slots[i] % 16].reshape(S * H, -1), b.signs).reshape(S, H, d)
        assert np.allclose(rows[i][0].cpu().numpy(), want, rtol=1e-6, atol=1e-9)


def test_two_calls_at_once():
    """Calls on two streams, each with its own workspace, overlap and keep their bits."""
    a, b = Batch(4096, _lens(4096, 40, 300, 1), 32, 8, 128, seed=11), Batch(3000, _lens(3000, 30, 200, 2), 8, 1, 64, seed=12)
    want = a.shared(), b.shared()
    streams = [torch.cuda.Stream() for _ in range(2)]
    args = [(x.q, x.cache, torch.from_numpy(x.prefix_blocks).cuda(), x.prefix) + x._args() + (x.scale, x.gsigns, x.max_len)
            for x in (a, b)]   # alive until both streams are done
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            got[i].append(_kv().kv_int4_shared_prefix_attention(*args[i], out_dtype=torch.float32, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


def test_blocks_past_32_bit_offsets():
    """A cache of more than 4 GiB whose last blocks hold everything: rotary write, read-back and attention at
    byte offsets past 32 bits give the bits of the same rows in a small cache."""
    kv = _kv()
    b = Batch(1024, _lens(1024, 20, 30, 3), 32, 8, 128, seed=13)
    assert b.is_shared()
    small, nb = b.cache, b.cache.shape[0]
    far = (1 << 32) // (small.stride(0)) + 100
    big = torch.zeros((far + nb,) + tuple(small.shape[1:]), dtype=torch.uint8, device="cuda")
    assert far * small.stride(0) > 1 << 32
    r = np.random.default_rng(4)
    x = torch.from_numpy(r.standard_normal((nb * 16, 48, 128)).astype(np.float32)).bfloat16().cuda()
    tab = torch.from_numpy(r.uniform(-1, 1, (64, 128)).astype(np.float32)).cuda()
    pos, slots = torch.arange(nb * 16, device="cuda") % 64, torch.arange(nb * 16, device="cuda")
    for cache, off in ((small, 0), (big, far)):
        kv.kv_int4_rope_write(x[:, :32], x[:, 32:40], x[:, 40:], pos, tab, slots + 16 * off, b.gsigns, cache)
    assert torch.equal(big[far:], small) and not big[:far].any()
    want = kv.kv_int4_read(small, slots, b.gsigns)
    got = kv.kv_int4_read(big, slots + 16 * far, b.gsigns)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    want = b.shared()
    b.cache, b.tables, b.prefix_blocks = big, b.tables + np.int32(far), b.prefix_blocks + np.int32(far)
    assert torch.equal(b.shared(), want)


def test_calls_of_different_shapes_follow_each_other_on_one_workspace():
    """Shared and plain calls of different batch sizes and head layouts take turns on one stream with one
    workspace and nothing between them: each keeps the bits of a call by itself."""
    kv = _kv()
    batches = [Batch(1024, _lens(1024, 32, 300, 21), 32, 8, 128, seed=21), Batch(900, _lens(900, 64, 200, 22), 64, 8, 128, seed=22),
               Batch(2048, _lens(2048, 12, 900, 23), 8, 1, 64, seed=23), Batch(400, _lens(400, 200, 60, 24), 16, 4, 64, seed=24),
               Batch(64, _lens(64, 700, 30, 25), 4, 4, 64, seed=25)]
    calls = []
    for b in batches:
        t, l, q = b._args()
        pb = torch.from_numpy(b.prefix_blocks).cuda()
        calls.append(lambda ws, out, b=b, t=t, l=l, q=q, pb=pb: kv.kv_int4_shared_prefix_attention(
            b.q, b.cache, pb, b.prefix, t, l, q, b.scale, b.gsigns, max_seq_len=b.max_len, out=out, workspace=ws))
        calls.append(lambda ws, out, b=b, t=t, l=l, q=q: kv.kv_int4_paged_attention(
            b.q, b.cache, t, l, q, b.scale, b.gsigns, 1, b.max_len, out=out, workspace=ws))
    need = 0
    for b in batches:
        S, Hq, d, H = len(b.lens), b.q.shape[1], b.q.shape[2], b.cache.shape[3]
        need = max(need, kv.kv_int4_attention_workspace_bytes(Hq, H, d, S, b.max_len),
                   kv.kv_int4_shared_prefix_workspace_bytes(S, Hq, H, d, S, b.prefix, b.max_len))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(b.q) for b in batches for _ in range(2)]
    want = []
    for f, o in zip(calls, outs):
        torch.cuda.synchronize()
        want.append(f(ws, o).clone())
        torch.cuda.synchronize()
    order = list(np.random.default_rng(0).permutation(len(calls) * 8) % len(calls))
    got = [torch.empty_like(outs[i]) for i in order]
    torch.cuda.synchronize()
    for i, o in zip(order, got):
        calls[i](ws, o)
    torch.cuda.synchronize()
    bad = [(k, i) for k, (i, o) in enumerate(zip(order, got)) if not torch.equal(o, want[i])]
    assert not bad, bad


def test_outputs_are_the_next_calls_queries():
    """A call's output fed to the next call as its queries, with nothing between them on the stream."""
    b = Batch(1024, _lens(1024, 32, 200, 31), 32, 8, 128, seed=31)
    t, l, q = b._args()
    pb = torch.from_numpy(b.prefix_blocks).cuda()
    kv = _kv()

    def chain(sync):
        outs, x = [], b.q
        for i in range(12):
            if i % 3 == 2:
                x = kv.kv_int4_paged_attention(x, b.cache, t, l, q, b.scale, b.gsigns, 1, b.max_len)
            else:
                x = kv.kv_int4_shared_prefix_attention(x, b.cache, pb, b.prefix, t, l, q, b.scale, b.gsigns, max_seq_len=b.max_len)
            outs.append(x)
            if sync:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs

    want = chain(True)
    for _ in range(5):
        assert all(torch.equal(x, y) for x, y in zip(chain(False), want))


@pytest.mark.parametrize("Hq, H, d", [(8, 8, 64), (8, 4, 128), (8, 2, 128), (32, 8, 64)])
def test_bf16_outputs_are_the_fp32_ones_rounded(Hq, H, d):
    """With up to four query heads per kv head the weights keep two halves whatever the output, as the plain
    call's do: a bf16 output is the fp32 one with its last rounding."""
    b = Batch(2100, _lens(2100, 10, 30, 6), Hq, H, d, seed=32)
    assert b.is_shared()
    assert torch.equal(b.shared(torch.bfloat16), b.shared(torch.float32).bfloat16())


def test_bf16_outputs_of_eight_heads_stay_within_their_rounding():
    """Eight query heads per kv head and a bf16 output: one fp16 weight per key, as in the plain call.  Half a step
    of bf16 is 2^-8 at most, its root mean square about 0.42 of it; the weights' 2e-4 hardly adds to that."""
    b = Batch(2100, _lens(2100, 10, 30, 6), 16, 2, 128, seed=33)
    assert b.is_shared()
    ref = torch.from_numpy(b.oracle())
    assert float((b.shared(torch.bfloat16).double().cpu() - ref).norm() / ref.norm()) < 0.5 * 2.0 ** -8


@pytest.mark.parametrize("Hq, H, d", [(8, 2, 64), (32, 8, 128)])
def test_calls_agree_closely(Hq, H, d):
    """The two calls' fp32 outputs differ by the rounding of 22-bit weights and queries and of fp32 sums alone."""
    b = Batch(2000, _lens(2000, 40, 300, 34), Hq, H, d, seed=34, outliers=False)
    assert b.is_shared()
    x, y = b.shared().double(), b.plain().double()
    assert float((x - y).norm() / y.norm()) < 4e-5   # 2e-5 each, see the test of finer outputs


def test_more_than_512_sequences():
    b = Batch(300, [0 if i % 97 == 5 else 1 + i % 300 if i % 31 == 7 else 301 + i % 40 for i in range(700)], 8, 2, 64, seed=35)
    _check(b, seqs=range(0, 700, 23))
    _check(b, seqs=[5, 7, 38, 699])


@pytest.mark.parametrize("Hq, H", [(8, 8), (8, 4), (8, 2), (8, 1)])
def test_rows_never_written_count_as_in_the_plain_call(Hq, H):
    """A row of zeros (its token was skipped) is a key of logit 0 and a value of 0, whichever kernel reads it."""
    from gpu_helpers import assert_attention_close
    b = Batch(2048, [2049, 2100, 2048, 40, 16, 700, 2060, 2070, 33], Hq, H, 64, seed=36, outliers=False)
    assert b.is_shared()
    r = np.random.default_rng(36)
    tok = np.concatenate([np.arange(40), 40 + r.permutation(2008)[:900]])   # the first 40: all that some rows see
    blk = torch.from_numpy(b.prefix_blocks[tok // 16].astype(np.int64)).cuda()
    b.cache[blk, :, torch.from_numpy(tok % 16).cuda()] = 0
    b.cache[int(b.prefix_blocks[60]), 0, 3, H - 1] = 0        # a key alone, a value alone
    b.cache[int(b.prefix_blocks[61]), 1, 4, 0] = 0
    got, ref = b.shared(), b.oracle()
    assert_attention_close(got, ref)
    assert not got[[3, 4, 8]].any()
    c = b.plain().double()
    assert float((got.double() - c).norm() / c.norm()) < 1e-3


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 2 ** 31 - 1])
@pytest.mark.parametrize("Hq, H", [(8, 4), (8, 2)])
def test_any_block_id_outside_the_cache_is_counted(Hq, H, bad):
    from gpu_helpers import status
    b = Batch(2048, _lens(2048, 9, 40, 37), Hq, H, 64, seed=37)
    assert b.is_shared()
    good = b.shared()
    assert not any(status().values())
    b.prefix_blocks[100] = bad
    got = b.shared()
    assert status()["block_out_of_range"] > 0
    assert not torch.equal(got, good) and bool(torch.isfinite(got).all())


def test_a_dominant_key_leaves_the_small_weights_their_share():
    """65 536 keys some 24.5 binades below one of the first: 2^-8.5 of the softmax's mass, and all of the output,
    because the dominant key's value is zero.  A CTA's range holds all of them (19 row tiles of 8 kv heads are 152
    CTAs).  Each weight errs by half of fp16's smallest step at most, 2^-25, where the reference has 2^6: 2^16 keys
    together by 2^-15 of the value's size; a weight is the value's scale of 15 steps times its share."""
    S, P, Hq, H, d = 304, 65536, 64, 8, 64
    b = Batch(P, [P + 1 + i % 16 for i in range(S)], Hq, H, d, seed=38)
    kv, n = _kv(), b.cache.shape[0] * 16
    rows = S * Hq * (d * 4 + 8)   # bytes of one split's partials
    need = kv.kv_int4_shared_prefix_workspace_bytes(S, Hq, H, d, S, P, b.max_len)
    splits = (need - kv.kv_int4_attention_workspace_bytes(Hq, H, d, S, b.max_len - P)) // rows
    assert splits == 1 or torch.cuda.get_device_properties(0).multi_processor_count != 152
    g = torch.Generator(device="cuda").manual_seed(38)
    slot = int(b.prefix_blocks[0]) * 16 + 5
    k = torch.zeros(n, H, d, dtype=torch.bfloat16, device="cuda")
    k[slot] = 4.0
    v = (1.0 + 0.1 * torch.randn(n, H, d, generator=g, device="cuda")).bfloat16()
    v[slot] = 0.0
    kv.kv_int4_write(k, v, torch.arange(n, device="cuda"), b.gsigns, b.cache)
    b.q = torch.full_like(b.q, 24.5 / (4.0 * d * b.scale * 1.4427))
    got = b.shared().double()
    size = float(v.float().norm(dim=-1).max())
    for i in (0, 77, 303):
        tok = np.arange(int(b.lens[i]))
        slots = torch.from_numpy(b.tables[i, tok // 16].astype(np.int64) * 16 + tok % 16).cuda()
        kr, vr = (x.double() for x in kv.kv_int4_read(b.cache, slots, b.gsigns, dtype=torch.float32))
        for h in (0, 7):
            x = b.scale * kr[:, h] @ b.q[i, h * 8].double()
            assert 24.0 < float(x[5] - x[6]) * 1.442695 < 25.5
            ref = torch.softmax(x, 0) @ vr[:, h]
            err = float((got[i, h * 8] - ref).norm())
            assert err < 2.0 ** -15 * 2 * size + 2e-5 * float(ref.norm()), (err, float(ref.norm()))


@pytest.mark.parametrize("value", [float("inf"), 1e30, 1e6])
@pytest.mark.parametrize("Hq, H", [(8, 4), (8, 1)])
def test_values_behind_a_sequences_end_stay_out_of_it(Hq, H, value):
    """Sequences that end inside the prefix, before a token whose value vector is infinite or huge: in its tile and
    before it."""
    from gpu_helpers import assert_attention_close
    lens = [2041, 1500, 1499, 1490, 1409, 1408, 1400, 130, 2100, 1, 1501]
    b = Batch(2040, lens, Hq, H, 128, seed=39, outliers=False)
    assert b.is_shared()
    kv = _kv()
    at = torch.tensor([int(b.prefix_blocks[1500 // 16]) * 16 + 1500 % 16], device="cuda")
    x = torch.randn(1, H, 128, device="cuda").bfloat16()
    y = x.clone()
    y[:, :, 7] = value
    kv.kv_int4_write(x, y, at, b.gsigns, b.cache)
    before = [i for i, l in enumerate(lens) if l <= 1500]
    ref = b.oracle(seqs=before)
    for o in (torch.float32, torch.bfloat16):
        got, plain = b.shared(out_dtype=o), b.plain(out_dtype=o)
        assert_attention_close(got[before], ref[before])
        assert torch.equal(torch.isfinite(got), torch.isfinite(plain))
    for opts in (dict(window_left=1200), dict(softcap=30.0)):
        got, plain = b.shared(**opts), b.plain(**opts)
        assert_attention_close(got[before], plain[before].double().cpu().numpy())


@pytest.mark.parametrize("opts", [{}, dict(softcap=20.0)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_query_that_is_not_finite_shows(bad, opts):
    """Its outputs are not finite, wherever its sequence ends, as the plain call's are not."""
    b = Batch(2048, [2049, 100, 2048, 2100, 1500, 0, 16, 2060, 2070], 8, 2, 128, seed=40, outliers=False)
    assert b.is_shared()
    for i in range(9):
        b.q[i, :, 5 * i] = bad
    b.q[7] = 1.0
    got, plain = b.shared(**opts), b.plain(**opts)
    assert torch.equal(torch.isfinite(got), torch.isfinite(plain))
    assert not torch.isfinite(got[[0, 1, 2, 3, 4, 6, 8]]).any() and bool((got[5] == 0).all())


def test_a_key_that_is_not_finite_shows():
    """An infinite key of the prefix makes the outputs of the sequences that see it NaN, and no other's."""
    b = Batch(2048, [2049, 100, 2048, 2100, 700, 1500, 701, 2060, 2070], 8, 2, 128, seed=41, outliers=False)
    assert b.is_shared()
    at = torch.tensor([int(b.prefix_blocks[700 // 16]) * 16 + 700 % 16], device="cuda")
    x = torch.randn(1, 2, 128, device="cuda").bfloat16()
    x[:, 1, 9] = float("inf")
    _kv().kv_int4_write(x, x.nan_to_num(0, 0, 0), at, b.gsigns, b.cache)
    got, plain = b.shared(), b.plain()
    assert torch.equal(torch.isfinite(got), torch.isfinite(plain))
    assert bool(torch.isfinite(got[[1, 4]]).all()) and not torch.isfinite(got[0, 4:]).any()
