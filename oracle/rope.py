"""CPU oracle of the rotary position embedding that the rotary cache writes apply.

TEST INFRASTRUCTURE ONLY.  The rotation is part of an encoding (the rotated keys' cache bytes must
match bit for bit), so it is stated as numpy fp32 steps: with the table row cs of a token's
position (rot/2 cosines, then rot/2 sines), each pair (a, b) of the first rot dimensions becomes
a' = fl(fl(a c) - fl(b s)), b' = fl(fl(b c) + fl(a s)); pairs are (x_i, x_{i + rot/2}), or
(x_{2i}, x_{2i+1}) when interleaved.
"""
from __future__ import annotations

import numpy as np


def table(max_position: int, rot: int, base: float = 10000.0) -> np.ndarray:
    """[max_position, rot] fp32: cos, then sin, of position * base^(-2i/rot), the angles in fp64."""
    inv = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    angle = np.arange(max_position, dtype=np.float64)[:, None] * inv
    return np.concatenate([np.cos(angle), np.sin(angle)], axis=1).astype(np.float32)


def rotate(x, positions, cos_sin: np.ndarray, interleaved: bool = False) -> np.ndarray:
    """x [T, heads, d] (any float type, upcast exactly) -> the rotated vectors, fp32."""
    x = x.detach().cpu().float().numpy() if hasattr(x, "detach") else np.asarray(x, np.float32)
    rot = cos_sin.shape[1]
    cs = cos_sin[np.asarray(positions)]
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = x[..., ia], x[..., ib]
    y = x.astype(np.float32).copy()
    y[..., ia] = (a * c).astype(np.float32) - (b * s).astype(np.float32)
    y[..., ib] = (b * c).astype(np.float32) + (a * s).astype(np.float32)
    return y
