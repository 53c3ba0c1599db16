"""Strides whose products pass 64 bits: rows and heads that run into each other are refused (CPU only:
what is refused never reaches the GPU)."""
import ctypes as C

import pytest

import mxfp4_routed_expert_e2m1_amd as m
from test_attn_abi import A, STRIDE, attn, cache, rope

FAR = 1 << 40  # the largest stride that is taken


@pytest.mark.parametrize("rows", [2**23 + 1, 2**24 + 1])
def test_rows_and_heads_on_the_same_elements(rows):
    """ld = hs = 2^40: row 1 of head 0 is row 0 of head 1.  FAR * (rows - 1) is 2^63 and 2^64."""
    L = m.lib()
    assert L.moe_kv_write(cache(heads=2), A, FAR, FAR, A, FAR, FAR, 0, rows, A, None) == STRIDE
    assert L.moe_kv_read(cache(heads=2), A, rows, A, FAR, FAR, A, FAR, FAR, 0, None) == STRIDE
    assert L.moe_rope(rope(), A, 0, FAR, FAR, rows, 2, 64, A, rows, A, FAR, FAR, None) == STRIDE
    assert L.moe_attn_cache(attn(heads=2), cache(heads=1), A, 0, FAR, FAR, rows, A, 2, A, A, 8, 8, None,
                            C.c_void_p(0x200000), FAR, FAR, A, 1 << 30, None) == STRIDE


def test_the_least_strides_are_taken():
    """Heads of rows and rows of heads without a gap pass the strides' check and end at the next one
    (a misaligned list of slots); one element less does not."""
    L = m.lib()
    mis = C.c_void_p(0x100002)

    def write(rows, ld, hs):
        return L.moe_kv_write(cache(heads=3), A, ld, hs, A, ld, hs, 0, rows, mis, None)
    for rows in (2, 5, 1000):
        for ld, hs in ((3 * 64, 64), (64, 64 * rows)):
            assert write(rows, ld, hs) == -5
        for ld, hs in ((3 * 64 - 1, 64), (64, 64 * rows - 1), (2 * 70 + 63, 70), (70, 70 * (rows - 1) + 63)):
            assert write(rows, ld, hs) == STRIDE
        for ld, hs in ((2 * 70 + 64, 70), (70, 70 * (rows - 1) + 64)):
            assert write(rows, ld, hs) == -5
