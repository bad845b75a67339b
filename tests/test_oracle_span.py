"""Pins of the span-attention oracle, on the CPU."""
import numpy as np
import pytest

import oracle
import workloads
from oracle import int8 as o8
from oracle import span


def _batch(lens, qlens, hq, h, d, seed=0):
    r = np.random.default_rng(seed)
    nb = sum(-(-n // 16) for n in lens) + 2
    ids = r.permutation(nb).astype(np.int32)
    width = max(1, max(-(-n // 16) for n in lens))
    tables, at = np.zeros((len(lens), width), np.int32), 0
    for b, n in enumerate(lens):
        n = -(-n // 16)
        tables[b, :n] = ids[at:at + n]
        at += n
    signs = workloads.splitmix64_signs(d)
    cache = np.zeros(oracle.cache_shape(nb, 16, h, d), np.uint8)
    kv = r.standard_normal((2, nb * 16, h, d)).astype(np.float32)
    oracle.write(kv[0], kv[1], np.arange(nb * 16), signs, cache)
    qsl = np.concatenate([[0], np.cumsum(qlens)])
    q = r.standard_normal((qsl[-1], hq, d)).astype(np.float32)
    return q, cache, tables, np.array(lens), qsl, signs, (lambda rows: oracle.decode_rows(rows, signs))


def test_default_spans_are_the_causal_attention():
    q, cache, tables, lens, qsl, signs, dec = _batch((40, 7, 23), (5, 7, 1), 4, 2, 64)
    slopes = np.array([0.5, 0.25, 0.1, 0.0])
    want = oracle.paged_attention(q, cache, tables, lens, qsl, 0.2, signs, softcap=2.0, alibi_slopes=slopes)
    got, _ = span.attention(q, cache, tables, lens, qsl, 0.2, dec, softcap=2.0, alibi_slopes=slopes)
    assert np.allclose(got, want, rtol=1e-12, atol=1e-12)


def test_a_window_is_a_span():
    q, cache, tables, lens, qsl, signs, dec = _batch((40, 30), (40, 3), 2, 1, 64)
    pos = np.concatenate([np.arange(40), np.arange(27, 30)])
    want = oracle.paged_attention(q, cache, tables, lens, qsl, 0.2, signs, window_left=5)
    got, _ = span.attention(q, cache, tables, lens, qsl, 0.2, dec, key_begin=pos - 5)
    assert np.allclose(got, want, rtol=1e-12, atol=1e-12)


def test_documents_are_separate_sequences():
    """A packed prompt under its document mask gives what each document alone gives."""
    q, cache, tables, lens, qsl, signs, dec = _batch((48,), (48,), 2, 2, 64)
    begin = np.repeat([0, 16, 32], 16)
    got, _ = span.attention(q, cache, tables, lens, qsl, 0.3, dec, key_begin=begin)
    apart, _ = span.attention(q, cache, tables.T.copy(), [16, 16, 16], [0, 16, 32, 48], 0.3, dec)
    assert np.allclose(got, apart, rtol=1e-12, atol=1e-12)


def test_a_span_of_all_is_a_plain_softmax_and_an_empty_one_zero():
    q, cache, tables, lens, qsl, signs, dec = _batch((20,), (3,), 1, 1, 64)
    got, size = span.attention(q, cache, tables, lens, qsl, 0.2, dec, key_begin=[0, 4, 9], key_end=[20, 4, 10])
    rows = cache[tables[0, np.arange(20) // 16], :, np.arange(20) % 16, 0]
    k, v = dec(rows[:, 0]), dec(rows[:, 1])
    w = np.exp(0.2 * k @ q[0, 0])
    assert np.allclose(got[0, 0], w @ v / w.sum()) and not got[1].any() and np.allclose(got[2, 0], v[9])
    assert size[1, 0] == 0 and np.isclose(size[2, 0], np.linalg.norm(v[9]))


def test_hidden_blocks_rows_of_no_sequence_and_distance_behind_the_query():
    q, cache, tables, lens, qsl, signs, dec = _batch((33, 0), (2, 1), 1, 1, 64)
    tables[0, 1] = -1
    got, _ = span.attention(np.concatenate([q, q[:1]]), cache, tables, lens, qsl, 0.2, dec, key_end=[33, 33, 1, 1],
                            alibi_slopes=[0.5])
    assert np.isnan(got[3]).all() and not got[2].any()
    j = np.array([*range(16), 32])
    rows = cache[tables[0, j // 16], :, j % 16, 0]
    k, v = dec(rows[:, 0]), dec(rows[:, 1])
    w = np.exp(0.2 * k @ q[0, 0] - 0.5 * np.abs(31 - j))   # the first query's position is 31: key 32 lies behind it
    assert np.allclose(got[0, 0], w @ v / w.sum())


@pytest.mark.parametrize("lens", [(5,), (16, 17)])
def test_int8_rows(lens):
    r = np.random.default_rng(1)
    cache = np.zeros(o8.cache_shape(4, 16, 1, 64), np.uint8)
    kv = r.standard_normal((2, 64, 1, 64)).astype(np.float32)
    o8.write(kv[0], kv[1], np.arange(64), cache)
    tables = np.arange(4, dtype=np.int32).reshape(2, 2)[:len(lens)]
    q = r.standard_normal((len(lens), 2, 64)).astype(np.float32)
    qsl = np.arange(len(lens) + 1)
    want = o8.paged_attention(q, cache, tables, np.array(lens), qsl, 0.2)
    got, _ = span.attention(q, cache, tables, lens, qsl, 0.2, o8.decode_rows)
    assert np.allclose(got, want, rtol=1e-12, atol=1e-12)
