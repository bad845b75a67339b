"""GPU parity of the attention over key spans, for the three caches, against the oracle in 64 bits.

Tolerance, per row in the 2-norm, relative to size = sum_j w_j |v_j| (the un-rotation keeps the norm): the weights are
held in fp16 for a bf16 output, in two fp16 halves otherwise, an error of 2^-11 or 2^-21 of each weight.  An error
delta of the logits moves the weights by 2 delta: queries in two fp16 halves and fp32 sums of at most 128 products,
then a logit in log2 units rounded to fp32, 2^-18 of sum |q_i k_i| scale log2 e, which is below 2^4 for these
inputs: 2^-14, and twice that 2^-13.  The output's own rounding is eps / 2 of each value.
"""
import numpy as np
import pytest
import torch

import oracle
import workloads
from oracle import int2 as o2
from oracle import int8 as o8
from oracle import span as ospan

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


def _cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


class Batch:
    """Sequences with lens[b] cached tokens and qlens[b] queries, over a cache written by the library."""

    def __init__(self, bits, lens, qlens, hq, h, d, dtype=torch.bfloat16, seed=0, extra_q=0, outliers=True):
        r = np.random.default_rng(seed)
        kv = _kv()
        self.bits, self.h, self.d = bits, h, d
        self.lens, self.qsl = np.asarray(lens, np.int32), np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
        need = [-(-n // 16) for n in lens]
        nb = sum(need) + 2
        ids = r.permutation(nb).astype(np.int32)
        self.tables, at = np.full((len(lens), max(1, max(need))), -7, np.int32), 0   # entries past a sequence: no block
        for b, n in enumerate(need):
            self.tables[b, :n] = ids[at:at + n]
            at += n
        g = torch.Generator(device="cuda").manual_seed(seed)
        k = torch.randn(nb * 16, h, d, generator=g, device="cuda")
        if outliers:
            k[:, :, :2] *= 5.0
        v = torch.randn(nb * 16, h, d, generator=g, device="cuda")
        self.signs = workloads.splitmix64_signs(d)
        shape = {4: kv.kv_int4_cache_shape, 8: kv.kv_int8_cache_shape, 2: kv.kv_int2_cache_shape}[bits]
        self.cache = torch.zeros(shape(nb, 16, h, d), dtype=torch.uint8, device="cuda")
        slots = torch.arange(nb * 16, device="cuda")
        if bits == 8:
            kv.kv_int8_write(k.to(dtype), v.to(dtype), slots, self.cache)
        else:
            (kv.kv_int4_write if bits == 4 else kv.kv_int2_write)(k.to(dtype), v.to(dtype), slots, _cuda(self.signs), self.cache)
        self.q = torch.randn(int(self.qsl[-1]) + extra_q, hq, d, generator=g, device="cuda").to(dtype)
        self.scale = d ** -0.5
        self.mql, self.msl = int(max(qlens)), int(max(lens))

    def pos(self):
        """Position of every query row."""
        return np.concatenate([np.arange(n - (b - a), n) for a, b, n in zip(self.qsl[:-1], self.qsl[1:], self.lens)])

    def call(self, out_dtype=torch.float32, key_begin=None, key_end=None, alibi_slopes=None, **kw):
        kv = _kv()
        fn = {4: kv.kv_int4_span_attention, 8: kv.kv_int8_span_attention, 2: kv.kv_int2_span_attention}[self.bits]
        signs = () if self.bits == 8 else (_cuda(self.signs),)
        i32 = lambda x: None if x is None else _cuda(np.asarray(x, np.int32))
        return fn(self.q, self.cache, _cuda(self.tables), _cuda(self.lens), _cuda(self.qsl), self.scale, *signs,
                  **{"max_query_len": self.mql, "max_seq_len": self.msl, "out_dtype": out_dtype, "key_begin": i32(key_begin),
                     "key_end": i32(key_end), "alibi_slopes": None if alibi_slopes is None else _cuda(np.asarray(alibi_slopes, np.float32)),
                     **kw})

    def decode(self, rows):
        om = MODES[self.bits]
        return om.decode_rows(rows) if self.bits == 8 else om.decode_rows(rows, self.signs)

    def oracle(self, **kw):
        return ospan.attention(self.q, self.cache.cpu().numpy(), self.tables, self.lens, self.qsl, self.scale, self.decode, **kw)


def _close(got, want, size, what=""):
    step = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}[got.dtype]
    tol = 2.0 ** -13 + (2.0 ** -11 if got.dtype == torch.bfloat16 else 2.0 ** -21)
    got = got.double().cpu().numpy()
    rows = ~np.isnan(want).any(axis=(1, 2))
    assert rows.any()
    err = np.linalg.norm((got - want)[rows], axis=2)
    bound = tol * size[rows] + step * np.linalg.norm(want[rows], axis=2) + 1e-30
    worst = np.unravel_index(np.argmax(err / bound), err.shape)
    assert np.all(err <= bound), f"{what}: {err[worst] / bound[worst]:.3g} of the tolerance at {worst}"


def _check(b, out_dtype=torch.float32, out=None, **kw):
    from gpu_helpers import status
    got = b.call(out_dtype, out=out, **kw)
    _close(got, *b.oracle(**kw))
    assert not any(status().values()), status()
    return got


def _spans(kind, b, seed=0):
    """key_begin, key_end of every row for a mask of that kind."""
    r, pos = np.random.default_rng(seed), b.pos()
    if kind == "causal":
        return {}
    if kind == "window":
        return dict(key_begin=pos - 20)
    if kind == "prefix":
        prefix = np.repeat((b.lens * 0.6).astype(np.int32), np.diff(b.qsl))
        return dict(key_end=np.maximum(pos + 1, prefix))
    if kind == "all":
        return dict(key_end=np.full(len(pos), 1 << 30))
    if kind == "documents":
        cuts = np.unique(np.concatenate([[0], r.integers(1, max(2, b.msl), 9)]))
        return dict(key_begin=cuts[np.searchsorted(cuts, pos, side="right") - 1].clip(min=0))
    lo = r.integers(-5, b.msl + 3, len(pos))                     # any spans at all, some empty, some behind the end
    return dict(key_begin=lo, key_end=lo + r.integers(-3, max(4, b.msl // 2), len(pos)))


@pytest.mark.parametrize("kind", ["causal", "documents", "prefix", "any"])
@pytest.mark.parametrize("hq, h, d, dtype", [(8, 2, 64, torch.float16), (16, 2, 128, torch.bfloat16), (4, 4, 128, torch.float16),
                                             (2, 1, 64, torch.bfloat16), (32, 8, 128, torch.bfloat16), (8, 1, 128, torch.float16),
                                             (64, 8, 64, torch.bfloat16)])
@pytest.mark.parametrize("bits", [4, 8, 2])
def test_layouts_and_masks(bits, hq, h, d, dtype, kind):
    b = Batch(bits, (150, 37, 290), (70, 37, 1), hq, h, d, dtype, seed=hq + d)
    _check(b, **_spans(kind, b))


@pytest.mark.parametrize("bits", [4, 8, 2])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("softcap, alibi", [(0.0, False), (5.0, False), (0.0, True), (20.0, True)])
def test_capped_scores_and_distance_bias(bits, out_dtype, softcap, alibi):
    b = Batch(bits, (200, 65), (65, 1), 8, 2, 128, seed=3)
    slopes = 2.0 ** -np.arange(1.0, 9.0) if alibi else None
    for kind in ("causal", "prefix", "any"):
        _check(b, out_dtype, softcap=softcap, alibi_slopes=slopes, **_spans(kind, b))


@pytest.mark.parametrize("bits", [4, 8, 2])
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 1000])
def test_lengths(bits, L):
    """Contexts around the block and tile borders: single tokens, all of the context at once, and a few."""
    for qlen in sorted({1, min(L, 5), L}):
        b = Batch(bits, (L,), (qlen,), 4, 1, 128, seed=L)
        _check(b)
        _check(b, **_spans("any", b, L))
        _check(b, **_spans("all", b))


@pytest.mark.parametrize("bits", [4, 8, 2])
def test_single_tokens(bits):
    r = np.random.default_rng(5)
    lens = [1, 16, 0, 700, 33, 2048, 128, 129]
    for hq, h in ((64, 8), (8, 2), (1, 1), (4, 4)):
        b = Batch(bits, lens, [1] * 8, hq, h, 128, seed=h)
        _check(b)
        _check(b, key_begin=r.integers(-3, 600, 8), softcap=30.0)
        _check(b, key_begin=np.array(lens) - 1)
        _check(b, torch.bfloat16, key_end=np.array(lens) // 2, alibi_slopes=np.linspace(0, 0.5, hq))


def test_a_mixed_batch():
    """Single tokens, drafts, chunks, padding rows, sequences of no query, and rows of no sequence."""
    lens, qlens = [300, 0, 64, 513, 90, 40, 0, 1000], [1, 1, 64, 200, 0, 5, 0, 9]
    for bits in (4, 8, 2):
        b = Batch(bits, lens, qlens, 8, 2, 128, seed=bits, extra_q=7)
        out = torch.full(b.q.shape, 7.0, device="cuda")
        for kind in ("causal", "any", "documents"):
            got = _check(b, out=out, **{k: np.concatenate([v, [0] * 7]) for k, v in _spans(kind, b).items()})
            assert got is out and bool((out[-7:] == 7.0).all())
            assert not out[1].any()


@pytest.mark.parametrize("bits", [4, 8, 2])
def test_long_contexts(bits):
    """Few rows on many keys (work split over the keys), strong channels, fp16 outputs."""
    b = Batch(bits, (20000, 7001), (3, 40), 8, 2, 128, torch.float16, seed=9)
    for kind in ("causal", "prefix", "any"):
        _check(b, torch.float16, **_spans(kind, b))


@pytest.mark.parametrize("bits", [4, 8, 2])
def test_what_a_row_does_not_see_does_not_reach_it(bits):
    """Infinite and NaN scales, huge values and rows of ones in keys that a row's span leaves out; both planes."""
    b = Batch(bits, (260, 40), (130, 1), 8, 2, 128, seed=11)
    begin, end = np.full(131, 100), np.full(131, 200)
    begin[40:60], end[40:60] = 110, 113
    begin[130], end[130] = 3, 30
    want, size = b.oracle(key_begin=begin, key_end=end)
    clean = b.call(key_begin=begin, key_end=end)
    _close(clean, want, size)
    cache = b.cache
    hidden = [(0, j) for j in (*range(0, 100), *range(200, 260))] + [(1, j) for j in (0, 1, 2, *range(30, 40))]
    for word in (float("inf"), float("nan"), 3.0e38, -float("inf")):
        for s, j in hidden:
            row = cache[int(b.tables[s, j // 16]), :, j % 16]           # [2, H, bytes]
            row[..., -4:] = torch.tensor([word], device="cuda").view(torch.uint8)
        got = b.call(key_begin=begin, key_end=end)
        assert torch.equal(got, clean), word
    # rows of one sequence with different spans: a poisoned key reaches those that see it, no others
    row = cache[int(b.tables[0, 105 // 16]), :, 105 % 16]
    row[..., -4:] = torch.tensor([float("nan")], device="cuda").view(torch.uint8)
    got = b.call(key_begin=begin, key_end=end)
    sees = np.zeros(131, bool)
    sees[:130] = (begin[:130] <= 105) & (end[:130] > 105)
    assert torch.equal(got[torch.from_numpy(~sees).cuda()], clean[torch.from_numpy(~sees).cuda()])
    assert bool(torch.isnan(got[torch.from_numpy(sees).cuda()]).any(dim=2).all())


@pytest.mark.parametrize("bits", [4, 8, 2])
def test_queries_that_are_not_finite_show_in_their_own_rows(bits):
    b = Batch(bits, (150,), (40,), 8, 2, 128, seed=12)
    clean = b.call()
    b.q[7, 3, 5], b.q[20, 0, 0], b.q[33, 7, 127] = float("nan"), float("inf"), -float("inf")
    got = b.call()
    hit = torch.zeros(40, 8, dtype=torch.bool, device="cuda")
    hit[7, 3] = hit[20, 0] = hit[33, 7] = True
    assert bool(torch.isnan(got[hit]).any(dim=1).all())
    # the rows of a tile may share a power of two: last bits
    assert bool(((got - clean)[~hit].norm(dim=1) <= 2.0 ** -13 * clean[~hit].norm(dim=1).clamp(min=1e-3) * 4).all())


@pytest.mark.parametrize("bits", [4, 8, 2])
@pytest.mark.parametrize("size", [1e-20, 1e-3, 300.0, 3e4])
def test_queries_of_any_size(bits, size):
    """All of them, and some rows among others; the softmax scale keeps the logits where they are."""
    for qlen in (1, 9, 70):
        b = Batch(bits, (300, 140), (qlen, qlen), 8, 2, 128, seed=21)
        q = b.q.clone()
        b.q, b.scale = (q.float() * size).to(q.dtype), 128 ** -0.5 / size
        _check(b)
        b.q, b.scale = q.clone(), 128 ** -0.5
        b.q[::3, 1::2] = (q[::3, 1::2].float() * min(size, 0.01)).to(q.dtype)
        _check(b, **_spans("prefix", b))


@pytest.mark.parametrize("softcap", [1e-44, 1e-30, 1e-3, 0.5, 1e4, 3e38])
def test_caps_of_any_size(softcap):
    """Logits far beyond the cap, and far below it; a cap of next to nothing gives every visible key one weight."""
    for qlen in (1, 70):
        b = Batch(4, (200, 90), (qlen, qlen), 8, 2, 128, seed=22)
        b.cache[int(b.tables[0, 2])] = 0                     # rows of zeros: logits of 0
        _check(b, softcap=float(np.float32(softcap)))


@pytest.mark.parametrize("bits", [4, 8, 2])
def test_rows_of_zeros_are_keys(bits):
    b = Batch(bits, (90,), (30,), 8, 2, 128, seed=13)
    for j in (0, 5, 63, 64, 89):
        b.cache[int(b.tables[0, j // 16]), :, j % 16] = 0
    _check(b)
    b.cache.zero_()
    assert not b.call().any()


@pytest.mark.parametrize("bits", [4, 8, 2])
def test_bad_metadata_is_counted(bits):
    from gpu_helpers import clear_status, status
    b = Batch(bits, (150, 60, 33), (20, 1, 5), 8, 2, 128, seed=14)
    b.tables[0, 3] = -1
    b.tables[1, 1] = 1 << 20
    got = b.call()
    _close(got, *b.oracle())
    s = status()
    assert s["block_out_of_range"] >= 2 and s["bad_sequence"] == 0 and s["wait_timeout"] == 0
    clear_status()
    # a chunk longer than its sequence: its first queries lie before the sequence and see nothing
    b = Batch(bits, (150, 3), (20, 5), 8, 2, 128, seed=15)
    _close(b.call(), *b.oracle())
    assert status()["bad_sequence"] == 1
    clear_status()
    # queries past max_query_len are left, contexts past max_seq_len clamped
    b = Batch(bits, (150, 40), (20, 2), 8, 2, 128, seed=16)
    out = torch.full(b.q.shape, 7.0, device="cuda")
    end = np.full(22, 30)
    b.call(max_query_len=8, key_end=end, out=out)
    want, size = b.oracle(key_end=end)
    assert bool((out[8:20] == 7.0).all())
    _close(out[:8], want[:8], size[:8])
    _close(out[20:], want[20:], size[20:])
    assert status()["bad_sequence"] == 1
    clear_status()
    b.call(max_seq_len=100, key_end=end, out=out)
    _close(out, want, size)
    assert status()["bad_sequence"] == 1


def test_captured_calls_on_a_stream_of_their_own():
    """Two captured calls of different shapes, replayed in turn; the workspaces are theirs."""
    a, b = Batch(4, (500, 80), (90, 1), 8, 2, 128, seed=17), Batch(8, (3000,), (2,), 8, 2, 128, seed=18)
    wa, wb = a.call(**_spans("documents", a)), b.call()
    s = torch.cuda.Stream()
    args = []
    for x, kw in ((a, _spans("documents", a)), (b, {})):
        kv = _kv()
        fn = kv.kv_int4_span_attention if x.bits == 4 else kv.kv_int8_span_attention
        signs = (_cuda(x.signs),) if x.bits == 4 else ()
        need = kv.kv_int4_span_workspace_bytes(x.q.shape[0], x.q.shape[1], x.h, x.d, len(x.lens), x.mql, x.msl)
        args.append((fn, (x.q, x.cache, _cuda(x.tables), _cuda(x.lens), _cuda(x.qsl), x.scale, *signs),
                     dict(max_query_len=x.mql, max_seq_len=x.msl, out=torch.zeros(x.q.shape, device="cuda"),
                          workspace=torch.empty(max(need, 16), dtype=torch.uint8, device="cuda"),
                          **{k: _cuda(np.asarray(v, np.int32)) for k, v in kw.items()})))
    torch.cuda.synchronize()
    for fn, pos, kw in args:
        fn(*pos, stream=s, **kw)
    s.synchronize()
    assert torch.equal(args[0][2]["out"], wa) and torch.equal(args[1][2]["out"], wb)
    graphs = []
    for fn, pos, kw in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            fn(*pos, **kw)
        kw["out"].zero_()
        graphs.append(g)
    torch.cuda.synchronize()
    for i in (0, 1, 1, 0, 1):
        graphs[i].replay()
    torch.cuda.synchronize()
    assert torch.equal(args[0][2]["out"], wa) and torch.equal(args[1][2]["out"], wb)


@pytest.mark.parametrize("bits, hq, h, d", [(4, 8, 2, 128), (4, 16, 8, 64), (8, 4, 1, 128), (8, 8, 8, 64), (2, 4, 4, 128), (2, 8, 2, 64)])
def test_blocks_past_32_bit_offsets(bits, hq, h, d):
    """The same rows in blocks more than 2^32 bytes into a cache: the same bits."""
    b = Batch(bits, [700, 33, 1], [150, 33, 1], hq, h, d)
    want = b.call()
    one = b.cache[0].numel()
    far = (1 << 32) // one + 5
    cache = torch.empty((far + b.cache.shape[0], *b.cache.shape[1:]), dtype=torch.uint8, device="cuda")
    cache[far:] = b.cache
    b.cache, b.tables = cache, np.where(b.tables >= 0, b.tables + far, b.tables).astype(np.int32)
    assert torch.equal(b.call(), want)
    single = Batch(bits, [700, 33, 1], [1, 1, 1], hq, h, d)
    want = single.call()
    cache[far:] = single.cache
    single.cache, single.tables = cache, np.where(single.tables >= 0, single.tables + far, single.tables).astype(np.int32)
    assert torch.equal(single.call(), want)


@pytest.mark.parametrize("bits", [4, 8, 2])
def test_many_sequences(bits):
    """Thousands of sequences, most of them single tokens, some without any, and a few chunks."""
    r = np.random.default_rng(5)
    n = 2500
    qlens, lens = np.where(r.random(n) < 0.1, 0, 1), r.integers(1, 40, n)
    some = r.choice(n, 3, replace=False)
    qlens[some], lens[some] = (70, 200, 33), (70, 300, 400)
    b = Batch(bits, lens, qlens, 4, 2, 64, seed=5)
    _check(b, key_begin=b.pos() - 20)
    singles = Batch(bits, r.integers(0, 40, n), np.ones(n, int), 4, 2, 64, seed=6)
    _check(singles)


def test_the_same_call_gives_the_same_bits():
    b = Batch(4, (4000, 700), (200, 3), 32, 8, 128, seed=19)
    first = b.call(**_spans("any", b))
    for _ in range(3):
        assert torch.equal(b.call(**_spans("any", b)), first)


def test_python_checks():
    b = Batch(4, (40, 20), (4, 1), 8, 2, 64, seed=20)
    kv = _kv()
    ok = dict(query=b.q, kv_cache=b.cache, block_tables=_cuda(b.tables), seq_lens=_cuda(b.lens), query_start_loc=_cuda(b.qsl),
              softmax_scale=0.1, rht_signs=_cuda(b.signs), max_query_len=4, max_seq_len=40)
    ints = torch.zeros(5, dtype=torch.int32, device="cuda")
    kv.kv_int4_span_attention(**ok, key_begin=ints)
    for bad in (dict(key_begin=ints[:4]), dict(key_end=ints.long()), dict(key_end=ints.cpu()), dict(alibi_slopes=ints.float()),
                dict(query=b.q.float()), dict(rht_signs=None), dict(rht_signs=_cuda(b.signs[:32])), dict(seq_lens=ints),
                dict(kv_cache=b.cache[..., :-1].contiguous()), dict(out=torch.empty(4, 8, 64, device="cuda")),
                dict(block_tables=_cuda(b.tables[:1])), dict(query=b.q.transpose(0, 1))):
        with pytest.raises(ValueError):
            kv.kv_int4_span_attention(**{**ok, **bad})
    for bad in (dict(softcap=-1.0), dict(softcap=float("inf")), dict(softmax_scale=float("nan")), dict(max_query_len=0)):
        with pytest.raises(kv.KVInt4Error) as e:
            kv.kv_int4_span_attention(**{**ok, **bad})
        assert e.value.status == 1


def test_a_prompt_with_images_from_the_rotary_write_to_the_output():
    """A serving run: a packed prompt of text and images is rotated on three axes and written, attends under its mask,
    then a token is decoded; the cached rows read back give the same attention densely."""
    kv = _kv()
    T, hq, h, d = 200, 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    tab = torch.from_numpy(__import__("oracle.rope", fromlist=["table"]).table(512, d)).cuda()
    signs = _cuda(workloads.splitmix64_signs(d))
    cache = torch.zeros(kv.kv_int4_cache_shape(16, 16, h, d), dtype=torch.uint8, device="cuda")
    table = torch.randperm(16, generator=g, device="cuda").int()[None]
    slots = table[0].long().repeat_interleave(16) * 16 + torch.arange(256, device="cuda") % 16
    ends = torch.arange(1, T + 2, dtype=torch.int32, device="cuda")
    ends[30:94], ends[120:170] = 94, 170                                   # two images
    for start, n in ((0, T), (T, 1)):
        x = torch.randn(n, hq + 2 * h, d, generator=g, device="cuda").bfloat16()
        pos = torch.randint(0, 512, (3, n), generator=g, device="cuda")
        q = kv.kv_int4_mrope_write(x[:, :hq], x[:, hq:hq + h], x[:, hq + h:], pos, tab, (16, 24, 24),
                                   slots[start:start + n].contiguous(), signs, cache)
        out = kv.kv_int4_span_attention(q, cache, table, torch.tensor([start + n], dtype=torch.int32, device="cuda"),
                                        torch.tensor([0, n], dtype=torch.int32, device="cuda"), d ** -0.5, signs, max_query_len=n,
                                        max_seq_len=start + n, key_end=ends[start:start + n].contiguous(), out_dtype=torch.float32)
        kx, vx = kv.kv_int4_read(cache, slots[:start + n].contiguous(), signs, dtype=torch.float32)
        kx, vx = (t.double().repeat_interleave(hq // h, dim=1) for t in (kx, vx))
        s = torch.einsum("mhd,thd->hmt", q.double(), kx) * d ** -0.5
        hide = torch.arange(start + n, device="cuda") >= ends[start:start + n, None]
        w = torch.softmax(s.masked_fill(hide, float("-inf")), dim=-1)
        want, size = torch.einsum("hmt,thd->mhd", w, vx), torch.einsum("hmt,thd->mhd", w, vx.norm(dim=-1, keepdim=True))[..., 0]
        _close(out, want.cpu().numpy(), size.cpu().numpy())
