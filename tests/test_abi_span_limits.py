"""Limits of the span attentions that are refused before any CUDA work."""
import ctypes

import pytest

vp, i32, i64, f32, szt = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
FAKE = 1 << 20   # never dereferenced


@pytest.mark.parametrize("name", ["kv_int4_span_attention", "kv_int8_span_attention", "kv_int2_span_attention"])
def test_contexts_of_2_31_tokens(name):
    """The kernel's positions are 32-bit up to the end of a tile of 128 keys."""
    from int4_token_head_kv_gb300._build import build_library
    f, signs = getattr(ctypes.CDLL(build_library()), name), "8" not in name
    f.restype = ctypes.c_int
    f.argtypes = [vp, ctypes.c_int, i64, i32, vp, i64, i32, i32, i32, vp, i32, vp, vp, i32, i32, i32, f32] + \
        ([vp] if signs else []) + [vp, vp, f32, vp, vp, ctypes.c_int, vp, szt, vp]

    def call(max_blocks, max_seq_len):   # with no queries: 0 unless refused
        return f(FAKE, 1, 0, 8, FAKE, 8, 2, 128, 16, FAKE, max_blocks, FAKE, FAKE, 3, 4, max_seq_len, 0.1,
                 *([FAKE] if signs else []), None, None, 0.0, None, FAKE, 2, FAKE, 1 << 30, None)

    top = (1 << 31) - 1
    assert call(1 << 27, top) == 2 and call(1 << 27, top - 127) == 2 and call(top, top) == 2
    assert call((1 << 27) - 8, top) == 2   # 2^31 - 128 tokens
    assert call(1 << 27, top - 128) == 0 and call(4, top) == 0 and call((1 << 27) - 9, top) == 0 and call(top, 100) == 0
