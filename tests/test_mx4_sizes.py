"""Sizes whose tiles 64 bits cannot count are refused like others that are too large, before any launch. No GPU."""
import pytest

M63 = (1 << 63) - 1
HUGE = [(1 << 40, 1 << 40), (1 << 45, 1 << 20), (1 << 62, 1 << 62), (M63, 1), (1, M63), (M63, M63), (M63 - 200, 300),
        (1 << 36, (1 << 36) + 129), (1 << 42, 1 << 42)]


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    from zero_gradient_reduction_gb300 import build as zbuild
    zbuild.build()
    import zero_gradient_reduction_gb300 as z
    return z.lib()


@pytest.mark.parametrize("rows,cols", HUGE)
def test_too_large(L, rows, cols):
    for q, qt in ((16, 16), (16, None), (None, 16)):
        for dt in (0, 1, 2):
            assert L.zr_mx4_quantize(16, dt, rows, cols, cols, None, 0, q, qt, None) == 2
    assert L.zr_mx4_dequantize(16, rows, cols, 16, 2, cols, None) == 2
    assert b"too large" in L.zr_last_error()


def test_bytes(L):
    for rows, cols in HUGE:
        want = -(-rows // 128) * -(-cols // 256) * 17408
        assert L.zr_mx4_bytes(rows, cols) == (want if want <= M63 else -1)
    assert L.zr_mx4_bytes(M63, 0) == 0 and L.zr_mx4_bytes(0, M63) == 0
