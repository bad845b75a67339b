"""The sections of the rotary writes with several axes, on the host: what is refused does not depend on earlier calls."""
import numpy as np
import pytest

import int4_token_head_kv_gb300 as kv
from oracle import rope

GOOD = [(16, 24, 24), (3, 2, 2), (64,), (0, 5, 0, 1), (0, 0)]
BAD = [(16.0, 24, 24), (16, 24.5, 24), ("16", 24, 24), (), (1, 2, 3, 4, 5), (-1, 65), (None,), 64, "64", (1 << 40,), (np.float64(4), 4)]


def _kinds(sections):
    yield sections
    yield list(sections)
    yield tuple(np.int64(n) for n in sections)
    yield np.array(sections)
    yield np.array(sections, np.uint8)


@pytest.mark.parametrize("mixed", [False, True])
@pytest.mark.parametrize("sections", GOOD)
def test_integers_of_any_type(sections, mixed):
    want = bytes(rope.pair_axes(sections, mixed).astype(np.uint8))
    for _ in range(2):
        for kind in _kinds(sections):
            assert kv._pair_axes(kind, mixed) == want


def test_refusals_whatever_came_before():
    def refused():
        for bad in BAD:
            for mixed in (False, True):
                with pytest.raises(ValueError):
                    kv._pair_axes(bad, mixed)
    refused()
    for sections in GOOD + [(16, 24, 24), (4, 4)]:
        for mixed in (False, True):
            for kind in _kinds(sections):
                kv._pair_axes(kind, mixed)
    refused()
