"""GPU parity of packed attention where its promises are tightest: rows that see nothing beside
keys that hold anything.  Bounds: see test_gpu_packed_attention.py."""
import pytest
import torch

from test_gpu_packed_attention import BF16, F16, F32, _inputs, _run

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_len,k_len", [(3, 2), (8, 1), (40, 5), (300, 100), (200, 64), (640, 600)])
def test_rows_that_see_nothing_are_zeros(dp, q_len, k_len, d, dtype):
    """More queries than keys: the first q_len - k_len get out = 0 and lse = -infinity, whatever
    the keys and values that are hidden from them hold."""
    q, k, v = _inputs([q_len], [k_len], 4, 2, d, dtype)
    for bad in (float("nan"), float("inf")):
        k[:k_len], v[:k_len] = bad, bad
        out, lse = _run(dp, q, k, v, [q_len], [k_len])
        blind = q_len - k_len
        assert not bool(out[:blind].any())
        assert bool(torch.isneginf(lse[:blind]).all())
