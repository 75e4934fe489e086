"""GPU parity of the 4-bit product over the scales' whole range, and with scales that change along
a row.

A product of two elements is up to 36 times a power of two from 2^-256 to 2^254: exact in fp32
where it lies in [2^-126, 2^128); above, infinite; below, off by less than 2^-126.  With one product
per output its value is the output.  Sums: as in test_gpu_mx4.py."""
import numpy as np
import pytest
import torch

import oracle as O

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

# the least and the largest scale bytes, and enough between them to reach both of fp32's ends
BYTES = [0, 1, 2, 3, 30, 64, 100, 126, 127, 128, 129, 160, 200, 230, 250, 251, 252, 253, 254]
CODES = [1, 2, 7, 15]                                                     # 0.5, 1, 6, -6


def _held(rows, k, code, block, byte, other):
    """Rows of zeros with one element, code[r], in block `block` under byte[r]; the other blocks'
    scales are other[r]."""
    c = np.zeros((rows, k // 2), dtype=np.uint8)
    c[:, block * 16 + 5] = code << 4
    s = np.zeros(-(-rows // 128) * -(-k // 128) * 512, dtype=np.uint8)
    at = O.mx4_scale_index(rows, k)
    s[at] = other[:, None]
    s[at[:, block]] = byte
    return c, s


@pytest.mark.parametrize("k,block", [(32, 0), (256, 7), (288, 8)])
@pytest.mark.parametrize("m,n", [(16, 304), (31, 304), (64, 304), (300, 304), (1500, 6080)])
def test_products_over_the_scales_range(dp, m, n, k, block):
    pairs = np.array([(c, b) for b in BYTES for c in CODES], dtype=np.uint8)
    rng = np.random.default_rng(m + k)
    for first in range(0, len(pairs), m):                                 # every (code, scale) of a meets every one of w
        ia, iw = (np.arange(m) + first) % len(pairs), np.arange(n) % len(pairs)
        a = _held(m, k, pairs[ia, 0], block, pairs[ia, 1], rng.integers(0, 255, m).astype(np.uint8))
        w = _held(n, k, pairs[iw, 0], block, pairs[iw, 1], rng.integers(0, 255, n).astype(np.uint8))
        y = torch.full((m, n), 7.0, device="cuda")
        dp.mx4_linear(*(torch.from_numpy(t).cuda() for t in a + w), None, y)
        dp.device_status()
        want = O.mx4_values(*a)[:, 32 * block + 11, None] * O.mx4_values(*w)[None, :, 32 * block + 11]
        got = y.cpu().double().numpy()
        size = np.abs(want)
        normal, over = (size >= 2.0 ** -126) & (size < 2.0 ** 128), size >= 2.0 ** 128
        assert np.array_equal(got[normal], want[normal])
        assert np.array_equal(got[over], np.sign(want[over]) * np.inf)
        assert (np.abs(got - want)[~normal & ~over] < 2.0 ** -126).all()
        if m >= len(pairs):
            break


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", [(1, 64, 4096), (9, 520, 1120), (27, 264, 736), (64, 512, 2048), (257, 1000, 416), (700, 6152, 1056)])
def test_scales_that_change_along_a_row(dp, m, n, k, dtype):
    """Every block has a scale of its own, 2^-24 to 2^24, so that an exchanged one is off by more
    than the bound."""
    rng = np.random.default_rng(m + n + k)

    def held(rows):
        s = np.zeros(-(-rows // 128) * -(-k // 128) * 512, dtype=np.uint8)
        s[O.mx4_scale_index(rows, k)] = rng.integers(127 - 24, 127 + 25, (rows, k // 32))
        return rng.integers(0, 256, (rows, k // 2), dtype=np.uint8), s
    a, w = held(m), held(n)
    y = torch.empty(m, n, dtype=dtype, device="cuda")
    dp.mx4_linear(*(torch.from_numpy(t).cuda() for t in a + w), None, y)
    dp.device_status()
    va, vw = O.mx4_values(*a), O.mx4_values(*w)
    want, size = va @ vw.T, np.abs(va) @ np.abs(vw).T
    err = np.abs(y.cpu().double().numpy() - want)
    assert (err <= torch.finfo(dtype).eps / 2 * np.abs(want) + (k + 1) * 2.0 ** -24 * size * 1.01).all()
