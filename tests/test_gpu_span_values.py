"""The attention over key spans at the edges of what its arithmetic holds: capped scores and what a row does not see, and the
accuracy of the cap."""
import numpy as np
import pytest
import torch

from test_gpu_span import Batch, _close, _cuda, _kv

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from gpu_helpers import clear_status
    clear_status()


def _scale_words(b, seq, keys, word, planes=slice(None)):
    """Put word into the scale words of these keys of a sequence."""
    for j in keys:
        b.cache[int(b.tables[seq, j // 16]), planes, j % 16, :, -4:] = torch.tensor([word], device="cuda").view(torch.uint8)


# ------------------------------------------------------------------ capped scores and what a row does not see

@pytest.mark.parametrize("alibi", [False, True])
@pytest.mark.parametrize("softcap", [0.0, 5.0, 50.0, 1e4, 1e8])
@pytest.mark.parametrize("bits", [4, 8, 2])
def test_hidden_keys_reach_no_bit_with_options(bits, softcap, alibi):
    """Large, infinite and NaN scales behind the spans, with a cap and a distance bias: the same bits as without them,
    for chunks and single tokens; what one row sees does not reach its neighbours."""
    b = Batch(bits, (260, 40), (130, 1), 8, 2, 128, seed=31)
    one = Batch(bits, (300, 90), (1, 1), 8, 2, 128, seed=32)
    begin, end = np.full(131, 100), np.full(131, 200)
    begin[40:60], end[40:60] = 110, 113
    begin[130], end[130] = 3, 30
    opts = dict(softcap=softcap, alibi_slopes=2.0 ** -np.arange(1.0, 9.0) if alibi else None)
    kw, one_kw = dict(key_begin=begin, key_end=end, **opts), dict(key_begin=[20, 0], key_end=[280, 75], **opts)
    clean, one_clean = b.call(**kw), one.call(**one_kw)
    _close(clean, *b.oracle(**kw))
    _close(one_clean, *one.oracle(**one_kw))
    for word in (1e3, 1e12, 3.0e38, float("inf"), float("nan"), -float("inf")):
        _scale_words(b, 0, (*range(0, 100), *range(200, 260)), word)
        _scale_words(b, 1, (0, 1, 2, *range(30, 40)), word)
        _scale_words(one, 0, (*range(0, 20), *range(280, 300)), word)
        _scale_words(one, 1, range(75, 90), word)
        assert torch.equal(b.call(**kw), clean) and torch.equal(one.call(**one_kw), one_clean), word
    hit = np.zeros(131, bool)
    hit[:130] = (begin[:130] <= 105) & (end[:130] > 105)
    for word in (1e3, float("nan")):
        _scale_words(b, 0, (105,), word)
        got = b.call(**kw)
        rest = torch.from_numpy(~hit).cuda()
        assert torch.equal(got[rest], clean[rest]), word


@pytest.mark.parametrize("softcap", [0.0, 5.0, 50.0, 1e8])
@pytest.mark.parametrize("bits", [4, 8, 2])
def test_other_rows_queries_reach_no_bit(bits, softcap):
    """Queries of another size in some rows: the others' bits stay."""
    for qlen in (1, 9, 130):
        b = Batch(bits, (300, 140), (qlen, qlen), 8, 2, 128, seed=33)
        clean = b.call(softcap=softcap)
        b.q[::2, 1::2] = b.q[::2, 1::2] * 30
        got = b.call(softcap=softcap)
        rest = torch.ones(2 * qlen, 8, dtype=torch.bool, device="cuda")
        rest[::2, 1::2] = False
        assert torch.equal(got[rest], clean[rest])


# ------------------------------------------------------------------ the accuracy of the cap

@pytest.mark.parametrize("qlen", [1, 70])
@pytest.mark.parametrize("softcap", [8.0, 50.0, 1e3, 1e5, 1e12, 3e38])
def test_capped_scores_keep_their_bits(softcap, qlen):
    """Logits of -3 .. 3 through caps from 8 on, the weights read off one by one: INT8 keys a_j e_0, values
    127 e_j and queries e_0 are exact, so the weight of key j is the output's element j over 127.

    Relative tolerance.  A logit s of at most 3: three roundings up to the product S s_K, the fit (1.2e-7, two
    roundings) and its last two roundings, 7 2^-24 of s: 1.26e-6.  Its exponent, below 16 in log2 units, is rounded when
    the offset is added and again when the reference moves: 2^-21 + 2^-22 log2 units at most, 0.5e-6.  A weight takes its
    own logit's error and, through the sum, those of the others: twice 1.76e-6.  Its exponential 2^-22, its two fp16 halves
    2^-22 (the weights lie above 2^-9 of the largest, which is raised to 2^6), scale, sum and quotient 3 2^-24: 0.7e-6.
    Together 4.2e-6."""
    kv = _kv()
    n, d = 96, 128
    k, v = torch.zeros(n, 1, d, device="cuda"), torch.zeros(n, 1, d, device="cuda")
    k[:, 0, 0] = torch.linspace(-3, 3, n, device="cuda")
    v[torch.arange(n), 0, torch.arange(n)] = 127.0
    cache = torch.zeros(kv.kv_int8_cache_shape(n // 16, 16, 1, d), dtype=torch.uint8, device="cuda")
    kv.kv_int8_write(k.half(), v.half(), torch.arange(n, device="cuda"), cache)
    q = torch.zeros(qlen, 1, d, device="cuda", dtype=torch.float16)
    q[:, 0, 0] = 1.0
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    out = kv.kv_int8_span_attention(q, cache, torch.arange(n // 16, dtype=torch.int32, device="cuda")[None], ints(n),
                                    ints(0, qlen), 1.0, max_query_len=qlen, max_seq_len=n, softcap=softcap,
                                    key_end=torch.full((qlen,), n, dtype=torch.int32, device="cuda"), out_dtype=torch.float32)
    from oracle import int8 as o8
    rows = cache.cpu().numpy()[:, 0].reshape(n, -1)
    s = o8.decode_rows(np.ascontiguousarray(rows)).astype(np.float64)[:, 0]
    assert abs(s).max() > 2.99
    cap = float(np.float32(softcap))
    s = cap * np.tanh(s / cap)
    w = np.exp(s - s.max())
    w /= w.sum()
    got = out.double().cpu().numpy()[:, 0, :n] / 127.0
    assert np.abs(got / w - 1).max() <= 4.3e-6
