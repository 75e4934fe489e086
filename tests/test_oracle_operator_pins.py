"""Pins of the 4-bit and packed-attention oracles: hand-worked cases and brute force."""
import math

import numpy as np
import pytest

import oracle as O


def test_mx4_hand_worked_block():
    """Largest magnitude 6.5: e = 2 - 2 = 0, so the codes are those of the values themselves."""
    x = np.zeros((1, 32))
    x[0, :15] = [6.5, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.26, -0.74, -5.1, 5.0001, -0.1, 4.9, -6.5]
    codes, scales = O.mx4_quantize(x)
    assert scales.shape == (512,) and scales[0] == 127 and not scales[1:].any()
    want = [6, 0, 1, 1, 2, 2, 4, 4, 0.5, -0.5, -6, 6, -0.0, 4, -6]      # ties to the even code, 6.5 saturates
    assert list(O.mx4_values(codes, scales)[0, :15]) == want
    assert codes[0, 0] == 7 and codes[0, 6] == (0b1000 | 6 << 4)       # low half first


@pytest.mark.parametrize("top,byte", [(1.0, 125), (1.999, 125), (2.0, 126), (7.999, 127), (2.0 ** -126, 0),
                                      (2.0 ** -140, 0), (0.0, 0), (3.0e38, 252), (math.inf, 255), (math.nan, 255)])
def test_mx4_scale_of_a_block(top, byte):
    x = np.zeros((1, 32))
    x[0, 5] = top
    codes, scales = O.mx4_quantize(x)
    assert scales[0] == byte
    v = O.mx4_values(codes, scales)
    assert np.isnan(v).all() if byte == 255 else np.isfinite(v).all()


def test_mx4_codes_are_nearest_and_scales_a_permutation():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((130, 160)) * np.exp2(rng.integers(-20, 20, (130, 1)))
    codes, scales = O.mx4_quantize(x)
    idx = O.mx4_scale_index(130, 160)
    assert idx.max() < scales.size == 2 * 2 * 512 and len(np.unique(idx)) == idx.size
    assert (idx[0, 0], idx[1, 0], idx[32, 0], idx[0, 3], idx[0, 4], idx[128, 0]) == (0, 16, 4, 3, 512, 1024)
    s = np.exp2(scales[idx].astype(float) - 127).repeat(32, axis=1)
    grid = np.concatenate([O.mx4.MAGNITUDES, -O.mx4.MAGNITUDES])
    best = np.abs((x / s)[..., None] - grid).min(axis=-1)
    assert np.array_equal(np.abs(x - O.mx4_values(codes, scales)) / s, best)


def test_packed_attention_brute_force_and_masks():
    rng = np.random.default_rng(1)
    q_lens, k_lens, starts = [3, 0, 2, 4], [5, 2, 0, 2], [7, 0, 3, 1]
    q, k, v = rng.standard_normal((9, 4, 8)), rng.standard_normal((12, 2, 8)), rng.standard_normal((12, 2, 8))
    for causal in (True, False):
        out, lse, _ = O.packed_attention(q, k, v, q_lens, k_lens, starts, causal)
        at = 0
        for ql, kl, ks in zip(q_lens, k_lens, starts):
            for t in range(ql):
                for h in range(4):
                    seen = [j for j in range(kl) if not causal or j <= kl - ql + t]
                    e = [math.exp(sum(q[at + t, h, c] * k[ks + j, h // 2, c] for c in range(8)) / math.sqrt(8)) for j in seen]
                    want = sum(x * v[ks + j, h // 2] for x, j in zip(e, seen)) / sum(e) if seen else np.zeros(8)
                    assert np.allclose(out[at + t, h], want, rtol=0, atol=1e-12)
                    assert lse[at + t, h] == pytest.approx(math.log(sum(e)), abs=1e-12) if seen else lse[at + t, h] == -math.inf
            at += ql
    assert not O.packed_attention(q, k, v, q_lens, k_lens, starts, True)[0][5:7].any()   # 4 queries, 2 keys: two see none


def test_packed_attention_of_one_sequence_is_window_attention():
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal((6, 2, 4)) for _ in range(3))
    flat = [a.reshape(6, 8) for a in (q, k, v)]
    none = np.zeros((0, 8))
    want = O.window_attention(*flat, none, none, 0, [0, 6], [np.zeros((3, 8))], 2, 4, mod_q=False, gate_out=False)
    out, _, weight = O.packed_attention(q, k, v, [6], [6], causal=False)
    assert np.allclose(out.reshape(6, 8), want, atol=1e-12)
    assert (weight >= np.abs(out) - 1e-12).all()
