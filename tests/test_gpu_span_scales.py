"""The attention over key spans on rows that are not finite, at positions past 2^24, on values of very different
sizes, and the values themselves."""
import numpy as np
import pytest
import torch

from test_gpu_span import Batch, _close

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from gpu_helpers import clear_status
    clear_status()


def _row(b, seq, j):
    return b.cache[int(b.tables[seq, j // 16]), :, j % 16]   # [2, H, bytes]


def _set_scale(b, seq, j, plane, word):
    _row(b, seq, j)[plane, :, -4:] = torch.tensor([word], device="cuda").view(torch.uint8)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("plane", [0, 1])
@pytest.mark.parametrize("bits", [4, 8, 2])
def test_rows_that_are_not_finite_show(bits, plane, out_dtype):
    """A key, or a value, that is infinite or NaN leaves nothing finite in the rows that see it, and the others as
    they were; few rows and many, work split over the keys or not, with options and without, weights large and small."""
    for lens, qlens in (((260, 70), (130, 1)), ((9000,), (3,)), ((200, 33), (1, 1))):
        b = Batch(bits, lens, qlens, 8, 2, 128, seed=41)
        pos, seq = b.pos(), np.repeat(np.arange(len(lens)), qlens)
        at = 20
        begin = np.where(np.arange(len(pos)) % 5 == 1, at + 1, 0)       # every fifth row does not see it
        sees = torch.from_numpy((seq == 0) & (begin <= at) & (pos >= at)).cuda()
        for opts in ({}, dict(softcap=30.0), dict(alibi_slopes=np.full(8, 0.25))):
            kw = dict(key_begin=begin, **opts)
            clean, kept = b.call(out_dtype, **kw), _row(b, 0, at).clone()
            for word in (float("inf"), float("nan"), -float("inf")):
                _set_scale(b, 0, at, plane, word)
                got = b.call(out_dtype, **kw)
                assert not bool(torch.isfinite(got[sees]).any()), (opts, word)
                assert torch.equal(got[~sees], clean[~sees]), (opts, word)
            _row(b, 0, at).copy_(kept)


@pytest.mark.parametrize("bits", [4, 8, 2])
def test_written_infinities_show(bits):
    """A value (or key) with an infinite element as the write stores it: what sees it is not finite."""
    kv = __import__("int4_token_head_kv_gb300")
    write = {4: kv.kv_int4_write, 8: kv.kv_int8_write, 2: kv.kv_int2_write}[bits]
    for qlen in (1, 40):
        for bad_key in (False, True):
            b = Batch(bits, (150,), (qlen,), 8, 2, 128, seed=42)
            k, v = (torch.randn(1, 2, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
            (k if bad_key else v)[0, :, 7] = float("inf")
            slot = torch.tensor([int(b.tables[0, 2]) * 16 + 3], device="cuda")
            signs = () if bits == 8 else (torch.from_numpy(b.signs).cuda(),)
            write(k, v, slot, *signs, b.cache)
            if bool(torch.isfinite(_row(b, 0, 35)[0 if bad_key else 1, :, -4:].contiguous().view(torch.float32)).all()):
                continue   # (the write made a finite row of it)
            assert not bool(torch.isfinite(b.call()).any())


@pytest.mark.parametrize("far", [0, 1 << 24, 1 << 27])
@pytest.mark.parametrize("bits", [4, 8, 2])
def test_distances_in_long_contexts(bits, far):
    """The last keys of a context of millions of tokens, whose earlier blocks nothing sees: distances are exact there."""
    for qlen in (1, 3, 80):
        b = Batch(bits, (300,), (qlen,), 8, 2, 128, seed=43)
        slopes = np.linspace(0.1, 0.8, 8)
        begin, end = np.full(qlen, 140), np.full(qlen, 300)
        want = b.oracle(key_begin=begin, key_end=end, alibi_slopes=np.float32(slopes))
        b.tables = np.concatenate([np.zeros((1, far // 16), np.int32), b.tables], axis=1)
        b.lens = b.lens + np.int32(far)
        got = b.call(max_seq_len=300 + far, key_begin=begin + far, key_end=end + far, alibi_slopes=slopes)
        _close(got, *want)


# ------------------------------------------------------------------ values of very different sizes

def _steer(b, levels, sizes):
    """Sequence 0's keys with logits near levels (natural units) and values of these sizes, by the library's write."""
    kv = __import__("int4_token_head_kv_gb300")
    write = {4: kv.kv_int4_write, 8: kv.kv_int8_write, 2: kv.kv_int2_write}[b.bits]
    r = np.random.default_rng(44)
    u = r.choice([-1.0, 1.0], 128)
    b.q = (torch.from_numpy(u).cuda() + 0.05 * b.q.double()).to(b.q.dtype)
    b.scale = 1.0 / 128
    n, H = len(levels), b.cache.shape[3]
    k = np.repeat((np.asarray(levels)[:, None] * u)[:, None], H, 1)
    v = r.standard_normal((n, H, 128)) * np.asarray(sizes)[:, None, None]
    slots = torch.from_numpy(np.array([int(b.tables[0, j // 16]) * 16 + j % 16 for j in range(n)])).cuda()
    signs = () if b.bits == 8 else (torch.from_numpy(b.signs).cuda(),)
    write(*(torch.from_numpy(x).to(torch.bfloat16).cuda() for x in (k, v)), slots, *signs, b.cache)


def _far_apart(b, out_dtype, **kw):
    """Within the errors that the arithmetic has, for rows that see all keys of the one sequence:
    the logits', twice 2^-18 of the sums of magnitudes of their products (at most S, in log2 units), and the weights' own
    (2^-11 or 2^-21), both of sum w |v|; the output's rounding; and the weights' absolute error.  A weight times its scale
    w s is held in fp16 with the largest of a row, M, at 2^-2 or more (raised by 2^6, the exponent at most 8 binades above
    it), in steps of 2^-24: 2^-23 M of each, times the stored numbers |v| / s.  (M can belong to a row of next to no
    value: the writes give every row a scale of 1e-6 at least.)  Where the definition is not finite (scales past fp32),
    the output is not either."""
    got, (want, size) = b.call(out_dtype, **kw).double().cpu().numpy(), b.oracle(**kw)
    L, H = int(b.lens[0]), b.cache.shape[3]
    rows = b.cache.cpu().numpy()[np.asarray(b.tables[0])].transpose(0, 2, 3, 1, 4).reshape(-1, H, 2, b.cache.shape[4])[:L]
    flat = np.ascontiguousarray(rows.reshape(-1, rows.shape[-1]))
    x = b.decode(flat).reshape(L, H, 2, -1)
    words = flat[:, -4:].copy().view(np.uint32)[:, 0] & (0xFFFFFFF0 if b.bits == 4 else 0xFFFFFFFF)
    scale = words.astype(np.uint32).view(np.float32).astype(np.float64).reshape(L, H, 2)
    q = b.q.double().cpu().numpy()
    group = q.shape[1] // H
    step = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}[out_dtype]
    for g in range(q.shape[1]):
        k, v, s = x[:, g // group, 0], x[:, g // group, 1], scale[:, g // group, 1]
        logits = b.scale * q[:, g] @ k.T
        w = np.exp(logits - logits.max(axis=1, keepdims=True))
        w /= w.sum(axis=1, keepdims=True)
        S = (np.abs(q[:, g]) @ np.abs(k).T).max() * b.scale * 1.4427
        numbers = np.where(s > 0, np.linalg.norm(v, axis=1) / np.where(s > 0, s, 1), 0).sum()
        bound = (2.0 ** -17 * S + (2.0 ** -11 if out_dtype == torch.bfloat16 else 2.0 ** -21)) * size[:, g]
        bound = bound + step * np.linalg.norm(want[:, g], axis=1) + 2.0 ** -23 * (w * s).max(axis=1) * numbers
        err = np.linalg.norm(got[:, g] - want[:, g], axis=1)
        good = np.isfinite(want[:, g]).all(axis=1)
        assert not np.isfinite(got[:, g][~good]).all(axis=1).any()
        assert np.all(err[good] <= bound[good]), (err / bound)[good].max()


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("binades", [10, 24, 50, 90])
@pytest.mark.parametrize("bits", [4, 8, 2])
def test_values_of_very_different_sizes(bits, binades, out_dtype):
    """Large values of keys with next to no weight, a dominant key of small values, sizes that fall or rise as the logits
    rise: the rows keep their accuracy relative to what reaches the output.  Both orders of the key tiles."""
    n, big = 400, 2.0 ** binades
    j = np.arange(n)
    flat, one = np.zeros(n), np.ones(n)
    cases = []
    for at in (0, 130, 255, 399):
        hit = j == at
        cases.append((np.where(hit, -binades * 0.7 - 25.0, flat), np.where(hit, big, one)))     # large, no weight
        cases.append((np.where(hit, binades * 0.35 + 12.0, flat), np.where(hit, 1 / big, one)))   # dominant, small
    for up in (1.0, -1.0):
        level = binades * 0.69 * (j / n if up > 0 else 1 - j / n)
        cases.append((level * 1.2, 2.0 ** (-level / 0.69)))
        cases.append((level, 2.0 ** (level / 0.69)))
        cases.append((level, np.where(j % 7 == 3, big, one) * 2.0 ** (-level / 0.69)))
    for qlen in (1, 100):
        for levels, sizes in cases:
            b = Batch(bits, (n,), (qlen,), 8, 2, 128, seed=45)
            _steer(b, levels, sizes)
            end = np.full(qlen, n)
            _far_apart(b, out_dtype, key_end=end)
            _far_apart(b, out_dtype, key_end=end, alibi_slopes=np.zeros(8))


@pytest.mark.parametrize("bits", [4, 8, 2])
def test_rows_of_zeros_before_everything(bits):
    """Never written rows (logit 0, value 0) that hold nearly all of the weight: what the others add keeps its bits."""
    for level in (-5.0, -20.0, -40.0):
        for first in (0, 250):
            for qlen in (1, 100):
                b = Batch(bits, (400,), (qlen,), 8, 2, 128, seed=46)
                _steer(b, np.full(400, level), np.ones(400))
                for j in range(first, first + 50):
                    _row(b, 0, j).zero_()
                _far_apart(b, torch.float32, key_end=np.full(qlen, 400))


# ------------------------------------------------------------------ the values themselves

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits", [4, 8, 2])
def test_a_row_that_sees_one_key_gives_its_value(bits, d):
    """The output is the cached value as the read-back gives it, in the 2-norm within: the INT2 numbers in the tiles 2.5e-7,
    the weight's two halves 2^-23, the quotient by the sum and the factor of the rotation 3 2^-24, and the seven steps of the
    rotation 7 2^-24 of the norm: 1e-6."""
    for qlen in (1, 70):
        b = Batch(bits, (200, 90), (qlen, qlen), 8, 2, d, seed=47)
        got = b.call(key_begin=b.pos()).double().cpu().numpy()
        slots = np.concatenate([np.asarray(b.tables[i])[np.arange(n - qlen, n) // 16].astype(np.int64) * 16 + np.arange(n - qlen, n) % 16
                                for i, n in enumerate(b.lens)])
        rows = b.cache.cpu().numpy()[slots // 16, 1, slots % 16]
        want = b.decode(np.ascontiguousarray(rows.reshape(-1, rows.shape[-1]))).reshape(2 * qlen, 2, d).repeat(4, axis=1)
        assert (np.linalg.norm(got - want, axis=2) / np.linalg.norm(want, axis=2)).max() <= 1e-6
