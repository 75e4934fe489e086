"""GPU parity of packed attention where its promises are tightest: rows that see nothing beside
keys that hold anything, outputs and values at the types' ends, head groups whose cuts differ in
size, single tokens beside prompts on both sides of the rule that gives them a launch of their own.
Bounds: see test_gpu_packed_attention.py."""
import math

import numpy as np
import pytest
import torch

from test_gpu_packed_attention import BF16, F16, F32, _check, _inputs, _run

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


@pytest.mark.parametrize("q_len", [1, 40, 300])
@pytest.mark.parametrize("k_len", [64, 1024, 6000])
@pytest.mark.parametrize("d", [64, 128])
def test_f16_outputs_stay_finite(dp, d, q_len, k_len):
    """Values at f16's end under weights that all round up: an output is an average of values, so
    it is no larger than the largest.  Every 16th key has the score 0, the others one whose weight
    lies 0.5 above a tie (16392 of 32768) and rounds up by 7.5 / 16392.5: 15 of 16 of them move an
    output by 4.0e-4 of its value, beyond 65520, where f16 ends."""
    target = math.log(16392.5 / 32768)
    q = torch.zeros(q_len, 2, d)
    q[:, :, :2] = 1.0
    k = torch.zeros(k_len, 1, d)
    k[:, :, 0] = torch.tensor(target).to(F16).float()                     # and what that leaves, to 2^-22
    k[:, :, 1] = target - float(torch.tensor(target).to(F16))
    k[::16] = 0.0
    q, k = q.to(F16), k.to(F16)
    for top in (65504.0, -65504.0):
        v = torch.full((k_len, 1, d), top).to(F16)
        out, lse = _run(dp, q, k, v, [q_len], [k_len], causal=False, scale=1.0)
        _check(out, lse, q, k, v, [q_len], [k_len], None, False, scale=1.0)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("heads,kv_heads", [(129, 1), (258, 2), (387, 3)])
@pytest.mark.parametrize("q_lens,k_lens", [([70, 33, 1], [70, 33, 1]), ([2, 1], [5000, 300]), ([1], [9000])],
                         ids=lambda x: "_".join(map(str, x)))
def test_head_groups_cut_unevenly(dp, q_lens, k_lens, heads, kv_heads, dtype):
    """Groups of 129 heads are cut into 65 and 64: the second cut's tile reaches into the next
    k/v head's query heads, or behind the last; with many keys these are cut too."""
    for d in (64, 128):
        q, k, v = _inputs(q_lens, k_lens, heads, kv_heads, d, dtype)
        out, lse = _run(dp, q, k, v, q_lens, k_lens)
        _check(out, lse, q, k, v, q_lens, k_lens, None, True)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("heads,kv_heads,d", [(16, 16, 64), (8, 4, 64), (8, 4, 128), (8, 8, 128)])
def test_tokens_beside_prompts_in_one_launch_and_in_two(dp, heads, kv_heads, d, apart, dtype):
    """Sequences of at most 16 rows under a k/v head get a launch of their own from 40 tiles of 64
    keys per SM on: a fifth below that and a fifth above, so that neither side is missed."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rng = np.random.default_rng(heads + d)
    goal = 40 * sms * (1.2 if apart else 0.8) / kv_heads             # tiles of all tokens under one k/v head
    k_lens, q_lens = [], []
    while goal > 0:
        n = int(min(rng.integers(500, 4000), 64 * goal + 1))
        k_lens.append(n)
        q_lens.append(int(rng.integers(1, 1 + 16 * kv_heads // heads)))
        goal -= (n + 63) // 64
    tiles = sum((n + 63) // 64 for n in k_lens) * kv_heads
    assert (tiles >= 44 * sms) if apart else (tiles <= 36 * sms)
    for at, ql, kl in ((0, 140, 300), (1, 0, 70), (len(q_lens), 65, 65), (len(q_lens), 20, 5)):
        q_lens.insert(at, ql)
        k_lens.insert(at, kl)
    q, k, v = _inputs(q_lens, k_lens, heads, kv_heads, d, dtype)
    out, lse = _run(dp, q, k, v, q_lens, k_lens)
    _check(out, lse, q, k, v, q_lens, k_lens, None, True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("q_len", [1, 40, 300])
@pytest.mark.parametrize("grow", [0.0, 5.0])
def test_values_up_to_the_stated_size(dp, q_len, grow, dtype):
    """Values of up to 2^120 over the number of keys: with equal scores, and with scores that grow by
    up to 5 (7.2 in log2, less than what the running maximum may lag) along the keys."""
    n = 1000
    for d in (64, 128):
        q, k, v = _inputs([q_len], [n], 2, 1, d, dtype, spare=0)
        q[:], k[:] = 0.0, 0.0
        q[:, :, 0] = 1.0
        k[:, :, 0] = (torch.linspace(0.0, grow, n)[:, None]).to(dtype)
        v = (torch.sign(v.float()) * 2.0 ** 120 / n).to(dtype)
        v[:, :, ::2] = v[:, :, ::2].abs()
        out, lse = _run(dp, q, k, v, [q_len], [n], causal=False, scale=1.0)
        _check(out, lse, q, k, v, [q_len], [n], None, False, scale=1.0)


@pytest.mark.parametrize("q_len", [1, 40])
def test_a_captured_call_keeps_its_lengths(dp, q_len):
    """A replay answers for the lengths of the capture, on what the rows hold at the replay."""
    q, k, v = (t.cuda() for t in _inputs([q_len], [900], 4, 2, 64, BF16, spare=0))
    out, want = torch.zeros_like(q), torch.zeros_like(q)
    q_lens, k_lens, starts = [q_len], [500], [100]
    dp.packed_attention(q, k, v, q_lens, k_lens, out, k_starts=starts)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dp.packed_attention(q, k, v, q_lens, k_lens, out, k_starts=starts)
    q_lens[0], k_lens[0], starts[0] = 0, 800, 0
    k.mul_(-0.5)
    out.zero_()
    graph.replay()
    dp.packed_attention(q, k, v, [q_len], [500], want, k_starts=[100])
    torch.cuda.synchronize()
    assert torch.equal(out, want) and bool(out.any())
