"""The attention over key spans on rows that are not finite, and at positions past 2^24."""
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
