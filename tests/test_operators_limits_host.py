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


def test_binding_refuses_sizes_that_32_bits_do_not_hold(m):
    """A size that the C call's int32_t cuts off must not come out as another one."""
    torch = pytest.importorskip("torch")

    def meta(*shape, dtype=torch.uint8):
        return torch.empty(*shape, dtype=dtype, device="meta")
    for rows, k in [(1, (1 << 32) + 32), (1, 64 - (1 << 33)), ((1 << 64) + 5, 32), (1 - (1 << 64), 32)]:
        with pytest.raises(m.DpError) as e:
            m.mx4_scale_bytes(rows, k)
        assert e.value.status == m.ERR_INVALID_ARG
    wide = (1 << 32) + 64
    codes, scales = meta(1, wide // 2), meta(wide * 4 + 4096)
    with pytest.raises(ValueError, match="2\\^31"):
        m.mx4_quantize(meta(1, wide, dtype=torch.bfloat16), codes, scales)
    with pytest.raises(ValueError, match="2\\^31"):
        m.mx4_dequantize(codes, scales, meta(1, wide, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="2\\^31"):
        m.mx4_linear(codes, scales, meta(8, wide // 2), meta(wide * 4 + 4096), None, meta(1, 8, dtype=torch.float32))
    many = (1 << 32) + 8
    with pytest.raises(ValueError, match="2\\^31"):
        m.mx4_linear(meta(1, 16), meta(512), meta(many, 16), meta(many * 4 + 4096), None, meta(1, many, dtype=torch.float32))
