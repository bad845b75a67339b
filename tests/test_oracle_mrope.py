"""Pins of the oracle's rotary embedding with several position axes, on the CPU."""
import numpy as np
import pytest

from oracle import rope


def test_pair_axes_by_hand():
    assert rope.pair_axes((3, 1, 2)).tolist() == [0, 0, 0, 1, 2, 2]
    assert rope.pair_axes((3, 1, 2), True).tolist() == [0, 1, 2, 0, 2, 0]
    assert rope.pair_axes((0, 2), True).tolist() == [1, 1]


def test_the_binding_deals_the_same_axes():
    import int4_token_head_kv_gb300 as kv
    for sections in ((64,), (16, 24, 24), (24, 20, 20), (1, 0, 5, 2)):
        for mixed in (False, True):
            assert list(kv._pair_axes(sections, mixed)) == rope.pair_axes(sections, mixed).tolist()
    for bad in ((), (1, 2, 3, 4, 5), (4, -1), (2.0, 2)):
        with pytest.raises(ValueError):
            kv._pair_axes(bad, False)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("mixed", [False, True])
def test_complex_numbers(mixed, inter):
    """Every pair is multiplied by exp(i theta p) of its own axis, in 64 bits; two fp32 products and their sum, and
    the table's rounding, are 4 half steps of the pair's size at most."""
    r = np.random.default_rng(3)
    d, rot, sections = 64, 48, (5, 12, 7)
    x = r.standard_normal((9, 3, d)).astype(np.float32)
    pos = r.integers(0, 500, (3, 9))
    got = rope.rotate_axes(x, pos, rope.table(500, rot), sections, mixed, inter)
    axes = rope.pair_axes(sections, mixed)
    theta = 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    turn = np.exp(1j * pos[axes].T * theta)[:, None]
    a = np.arange(0, rot, 2) if inter else np.arange(rot // 2)
    b = a + 1 if inter else a + rot // 2
    z = (x[..., a].astype(np.float64) + 1j * x[..., b]) * turn
    bound = 4 * 2.0 ** -24 * np.abs(z) * 2 ** 0.5
    assert np.all(np.abs(got[..., a] - z.real) <= bound) and np.all(np.abs(got[..., b] - z.imag) <= bound)
    assert np.array_equal(got[..., rot:], x[..., rot:])


def test_equal_positions_are_one_axis():
    r = np.random.default_rng(4)
    x, pos = r.standard_normal((6, 2, 64)).astype(np.float32), r.integers(0, 90, 6)
    tab = rope.table(90, 64)
    assert np.array_equal(rope.rotate_axes(x, np.stack([pos] * 4), tab, (3, 9, 0, 20), True), rope.rotate(x, pos, tab))
