"""Pins of the rotary oracle: the complex product in fp64, position 0, norms, relative positions, the
two pairings, and the dimensions behind the rotated ones."""
import numpy as np
import pytest

from oracle import rope

U = 2.0 ** -24   # half a step of fp32


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d, rot", [(64, 64), (128, 128), (128, 32), (64, 16)])
def test_matches_the_complex_product(d, rot, interleaved):
    r = np.random.default_rng(1)
    x = r.standard_normal((5, 3, d)).astype(np.float32)
    pos = np.array([0, 1, 77, 1000, 4095])
    tab = rope.table(4096, rot)
    got = rope.rotate(x, pos, tab, interleaved).astype(np.float64)
    z = tab[pos, :rot // 2].astype(np.float64) + 1j * tab[pos, rot // 2:]
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    w = (x[..., ia].astype(np.float64) + 1j * x[..., ib]) * z[:, None]
    # two rounded products and a rounded sum: at most half a step each of |a| + |b| and of the result
    bound = (np.abs(x[..., ia]) + np.abs(x[..., ib])) * 2 * U * 1.01
    assert np.all(np.abs(got[..., ia] - w.real) <= bound) and np.all(np.abs(got[..., ib] - w.imag) <= bound)
    assert np.array_equal(got[..., rot:], x[..., rot:])
    assert np.array_equal(got[0], x[0])   # position 0


def test_scores_depend_on_relative_positions():
    r = np.random.default_rng(2)
    q, k = r.standard_normal((2, 1, 1, 128)).astype(np.float32)
    tab = rope.table(3000, 128)
    dots = [float((rope.rotate(q, [m + 40], tab).astype(np.float64) * rope.rotate(k, [m], tab)).sum()) for m in (0, 7, 2900)]
    assert np.ptp(dots) < 1e-4 * np.linalg.norm(q) * np.linalg.norm(k)


def test_pairings_are_one_permutation_apart():
    r = np.random.default_rng(3)
    x = r.standard_normal((4, 2, 64)).astype(np.float32)
    tab, pos = rope.table(100, 64), [3, 50, 99, 0]
    perm = np.concatenate([np.arange(0, 64, 2), np.arange(1, 64, 2)])   # neighbours -> halves
    assert np.array_equal(rope.rotate(x, pos, tab, True)[..., perm], rope.rotate(x[..., perm], pos, tab, False))
