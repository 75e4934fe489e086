"""Limits of the 4-bit and packed-attention entry points (no GPU): what does not fit their 32-bit
sizes is refused before anything is enqueued."""
import ctypes

import pytest

FAKE = 0x7f0000000000  # 16-byte aligned, never dereferenced
P = ctypes.c_void_p
G = 1 << 30
MOST_K = (1 << 31) - 256


@pytest.fixture(scope="module")
def m():
    import long_video_diffusion_b200 as mod
    return mod


@pytest.mark.parametrize("k", [MOST_K + 32, MOST_K + 160, (1 << 31) - 32])
def test_mx4_rows_that_end_behind_the_last_whole_step(m, k):
    """Behind 2^31 - 256 the number of tiles of a row would pass 2^31 on its way."""
    for dt in (0, 1, 2):
        assert m._lib.dp_mx4_quantize(P(FAKE), 1, k, dt, P(FAKE + 16 * G), P(FAKE + 32 * G), None) == m.ERR_UNSUPPORTED
        assert m._lib.dp_mx4_dequantize(P(FAKE + 16 * G), P(FAKE + 32 * G), 1, k, P(FAKE), dt, None) == m.ERR_UNSUPPORTED
        assert m._lib.dp_mx4_linear(P(FAKE), P(FAKE + 16 * G), P(FAKE + 32 * G), P(FAKE + 64 * G), None, 1, 8, k,
                                    P(FAKE + 80 * G), dt, None) == m.ERR_UNSUPPORTED
    with pytest.raises(m.DpError):
        m.mx4_scale_bytes(1, k)


def test_mx4_longest_row(m):
    assert m.mx4_scale_bytes(1, MOST_K) == MOST_K // 128 * 512
    assert m._lib.dp_mx4_quantize(P(0), 0, MOST_K, 1, P(0), P(0), None) == m.OK     # no rows: nothing is done
