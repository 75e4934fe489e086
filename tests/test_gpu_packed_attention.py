"""GPU parity of the attention over packed sequences against the float64 oracle.

Bounds, for a row with n keys, u the type's half step (eps / 2), W = sum_j p_j |v_j|:
  a score is a fp32 sum of d products, off by at most e = d * 2^-24 * sum_c |q_c k_c| * scale,
  which moves a softmax weight by the factor exp(+-2 e) (its own exponent and the sum's); the
  exponentials are within 1e-5 of their values (log2 units times a rounding included in e), and
  a weight in 16 bits rounds by u; the sums of n terms add n * 2^-24; the store rounds by u:
    |out - exact| <= u |exact| + W (u [16-bit types] + 2 e + 2e-5 + n 2^-23)
    |lse - exact| <= e + 1e-5 + n 2^-24 + 2^-22 |exact|
with e taken at its largest over the keys.  Every buffer holds NaN where no sequence has rows:
none of it may reach a result, and what lies behind the last sequence stays as it was."""
import numpy as np
import pytest
import torch

import oracle as O

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _inputs(q_lens, k_lens, heads, kv_heads, d, dtype, k_starts=None, spare=3, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed + sum(q_lens) + 7 * sum(k_lens) + d)
    nq = sum(q_lens)
    starts = list(np.cumsum([0] + list(k_lens))[:-1]) if k_starts is None else k_starts
    nk = max([s + n for s, n in zip(starts, k_lens)] + [0])
    q = torch.full((nq + spare, heads, d), float("nan"))
    k, v = (torch.full((nk + spare, kv_heads, d), float("nan")) for _ in range(2))
    q[:nq] = torch.randn(nq, heads, d, generator=g) * std
    for s, n in zip(starts, k_lens):
        k[s:s + n] = torch.randn(n, kv_heads, d, generator=g) * std
        v[s:s + n] = torch.randn(n, kv_heads, d, generator=g)
    return q.to(dtype), k.to(dtype), v.to(dtype)


def _check(got, lse, q, k, v, q_lens, k_lens, k_starts, causal, scale=None):
    nq, (heads, d) = sum(q_lens), q.shape[1:]
    args = [t.double().numpy() for t in (q, k, v)]
    want, want_lse, weight = O.packed_attention(*args, q_lens, k_lens, k_starts, causal, scale)
    dtype = q.dtype
    u = torch.finfo(dtype).eps / 2
    qa, ka = args[0][:nq], np.nan_to_num(args[1])
    sc = d ** -0.5 if scale is None else scale
    # sum_c |q_c k_c| <= |q| |k| (Cauchy-Schwarz), the longest key of all
    e = d * 2.0 ** -24 * np.linalg.norm(qa, axis=2) * np.linalg.norm(ka, axis=2).max(initial=0.0) * sc
    n = max(list(k_lens) + [1])
    bound = u * np.abs(want) + weight * ((0 if dtype == F32 else u) + 2 * e[..., None] + 2e-5 + n * 2.0 ** -23) + 1e-30
    if dtype == F16:
        bound = bound + 2.0 ** -24
    g = got[:nq].double().cpu().numpy()
    assert np.isfinite(g).all()
    err = np.abs(g - want)
    assert (err <= bound).all(), float((err / bound).max())
    empty = np.isinf(want_lse)
    assert not g[empty].any()
    if lse is not None:
        gl = lse[:nq].double().cpu().numpy()
        assert np.array_equal(np.isneginf(gl), empty)
        le = np.abs(gl[~empty] - want_lse[~empty])
        assert (le <= e[~empty] + 1e-5 + n * 2.0 ** -24 + 2.0 ** -22 * np.abs(want_lse[~empty])).all(), float(le.max())


def _run(dp, q, k, v, q_lens, k_lens, k_starts=None, causal=True, scale=0.0, stream=None):
    out = torch.full(q.shape, 3.25, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 4.5, device="cuda")
    dp.packed_attention(q.cuda(), k.cuda(), v.cuda(), q_lens, k_lens, out, k_starts=k_starts, causal=causal, lse=lse,
                        softmax_scale=scale, stream=stream)
    dp.device_status(stream)
    nq = sum(q_lens)
    assert bool((out[nq:] == 3.25).all()) and bool((lse[nq:] == 4.5).all())
    return out, lse


PROMPTS = [[1], [2], [64], [65], [77], [128, 1, 127], [129, 0, 3, 257], [300, 64, 63, 1, 1, 511], [1000]]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", PROMPTS, ids=lambda x: "_".join(map(str, x)))
def test_causal_prompts(dp, lens, d, dtype):
    q, k, v = _inputs(lens, lens, 4, 2, d, dtype)
    out, lse = _run(dp, q, k, v, lens, lens)
    _check(out, lse, q, k, v, lens, lens, None, True)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 3), (3, 1), (5, 1), (14, 2), (8, 1), (40, 8), (130, 1)])
def test_head_groups(dp, heads, kv_heads, dtype):
    lens = [70, 33, 1]
    for d in (64, 128):
        q, k, v = _inputs(lens, lens, heads, kv_heads, d, dtype)
        out, lse = _run(dp, q, k, v, lens, lens)
        _check(out, lse, q, k, v, lens, lens, None, True)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("q_lens,k_lens", [
    ([1], [1]), ([1], [4097]), ([1, 1, 1], [1, 63, 700]), ([1] * 5, [129, 0, 2000, 64, 128]), ([5], [1000]),
    ([128, 17], [640, 17]), ([300, 9], [100, 2]), ([64], [0]), ([0, 4, 0], [9, 5, 0]), ([200], [2300]), ([3, 200], [1, 199])],
    ids=lambda x: "_".join(map(str, x)))
def test_chunks_and_single_tokens(dp, q_lens, k_lens, dtype, causal):
    """More keys than queries, fewer (rows that see nothing), none; the tail of a tile of keys."""
    for d in (64, 128):
        q, k, v = _inputs(q_lens, k_lens, 8, 2, d, dtype)
        out, lse = _run(dp, q, k, v, q_lens, k_lens, None, causal)
        _check(out, lse, q, k, v, q_lens, k_lens, None, causal)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_padded_cache_and_shared_prefix(dp, dtype):
    """Sequences over a padded cache whose padding holds NaN; two that share their keys; any order."""
    q_lens, k_lens, starts = [1, 1, 2, 1], [200, 77, 77, 511], [1000, 20, 20, 300]
    q, k, v = _inputs(q_lens, k_lens, 8, 2, 128, dtype, starts)
    out, lse = _run(dp, q, k, v, q_lens, k_lens, starts)
    _check(out, lse, q, k, v, q_lens, k_lens, starts, True)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_columns_of_one_buffer(dp, dtype):
    """q, k, v as column ranges of one buffer, out as one of another: the columns between stay."""
    lens, heads, kv, d = [150, 1, 99], 6, 2, 64
    g = torch.Generator().manual_seed(5)
    buf = torch.randn(sum(lens), (heads + 2 * kv + 1) * d, generator=g).to(dtype).cuda().view(sum(lens), -1, d)
    q, k, v = buf[:, :heads], buf[:, heads:heads + kv], buf[:, heads + kv:heads + 2 * kv]
    wide = torch.full((sum(lens), heads + 4, d), 2.5, dtype=dtype, device="cuda")
    lse = torch.empty(sum(lens), heads, device="cuda")
    dp.packed_attention(q, k, v, lens, lens, wide[:, 1:1 + heads], lse=lse)
    dp.device_status()
    _check(wide[:, 1:1 + heads], lse, q.cpu(), k.cpu(), v.cpu(), lens, lens, None, True)
    assert bool((wide[:, 0] == 2.5).all()) and bool((wide[:, 1 + heads:] == 2.5).all())


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("std", [0.02, 6.0])
def test_flat_and_peaked_softmax(dp, dtype, std):
    lens = [500, 130]
    q, k, v = _inputs(lens, lens, 4, 1, 128, dtype, std=std)
    out, lse = _run(dp, q, k, v, lens, lens)
    _check(out, lse, q, k, v, lens, lens, None, True)


@pytest.mark.parametrize("q_lens,k_lens", [([1], [200]), ([1, 1], [4000, 300]), ([90], [700]), ([20], [5000])])
@pytest.mark.parametrize("d", [64, 128])
def test_small_weights_keep_their_bits(dp, d, q_lens, k_lens):
    """One key has all but some 2^-15 of the weight and a value of 0 in half the columns, where the
    output is what the other keys' small weights give: f16 ones under 2^-14 would lose bits."""
    for dtype in (F16, BF16, F32):
        q, k, v = _inputs(q_lens, k_lens, 4, 2, d, dtype, spare=0, std=0.2)
        q[:, :, 0] = 1.0
        k[:, :, 0] = 0.0
        at = 0
        for n in k_lens:
            k[at + n // 2, :, 0] = 15 * float(np.log(2)) + float(np.log(n))  # 2^15 times all the others
            v[at + n // 2, :, ::2] = 0.0
            at += n
        out, lse = _run(dp, q, k, v, q_lens, k_lens, causal=False, scale=1.0)
        _check(out, lse, q, k, v, q_lens, k_lens, None, False, scale=1.0)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_scores_that_grow_and_fall_along_the_keys(dp, dtype):
    """The running maximum moves at every tile of keys (growing) or never after the first."""
    n, d = 1100, 64
    g = torch.Generator().manual_seed(1)
    for sign in (1.0, -1.0):
        q = torch.ones(3, 2, d)
        k = (sign * torch.linspace(-4, 4, n)[:, None, None] + torch.randn(n, 1, d, generator=g) * 0.1)
        v = torch.randn(n, 1, d, generator=g)
        q, k, v = q.to(dtype), k.to(dtype), v.to(dtype)
        out, lse = _run(dp, q, k, v, [3], [n])
        _check(out, lse, q, k, v, [3], [n], None, True)


def test_softmax_scale_and_no_lse(dp):
    lens = [90, 40]
    q, k, v = _inputs(lens, lens, 2, 2, 64, BF16)
    out, lse = _run(dp, q, k, v, lens, lens, scale=0.5)
    _check(out, lse, q, k, v, lens, lens, None, True, scale=0.5)
    alone = torch.empty_like(out)
    dp.packed_attention(q.cuda(), k.cuda(), v.cuda(), lens, lens, alone, softmax_scale=0.5)
    assert torch.equal(alone[:130], out[:130])


def test_another_sequence_does_not_matter(dp):
    """Rows of a sequence are the same bits whatever the others hold, NaN and infinities included."""
    lens = [100, 70, 130]
    q, k, v = _inputs(lens, lens, 4, 2, 128, BF16)
    ref, _ = _run(dp, q, k, v, lens, lens)
    for bad in (float("nan"), float("inf"), -3e38):
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        for t in (q2, k2, v2):
            t[100:170] = bad
        got = torch.empty(q.shape, dtype=BF16, device="cuda")
        dp.packed_attention(q2.cuda(), k2.cuda(), v2.cuda(), lens, lens, got)
        assert torch.equal(got[:100], ref[:100]) and torch.equal(got[170:300], ref[170:300])


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("q_len,k_len,n", [(1, 200, 70), (3, 64, 64), (40, 70, 70), (150, 600, 9), (70, 3000, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_bad_values_show(dp, d, q_len, k_len, n, dtype):
    """Sequence i's key at about i k_len / n is spoilt: the queries that see it get NaN, those that do
    not what they get without it; a spoilt query likewise."""
    heads, group = 4, 2
    q_lens, k_lens = [q_len] * n, [k_len] * n
    q, k, v = _inputs(q_lens, k_lens, heads, heads // group, d, dtype, spare=0)
    clean, clean_lse = (torch.empty(q.shape, dtype=dtype, device="cuda"), torch.empty(q.shape[:2], device="cuda"))
    dp.packed_attention(q.cuda(), k.cuda(), v.cuda(), q_lens, k_lens, clean, lse=clean_lse)
    places = [min(k_len - 1, max(0, k_len - n) // 2 + i if n >= 64 else i * k_len // n + 5) for i in range(n)]
    for bad in (float("nan"), float("inf")):
        k2, q2 = k.clone(), q.clone()
        hit = torch.zeros(q.shape[:2], dtype=torch.bool)
        for i, j in enumerate(places):
            k2[i * k_len + j, 1, 3] = bad
            for t in range(q_len):  # its queries are its last rows; the second k/v head's query heads
                if j > k_len - q_len + t:
                    continue
                for h in (2, 3):
                    # the score is bad * q[3] + finite: NaN, or an infinity of q[3]'s sign
                    hit[i * q_len + t, h] = bad != bad or q[i * q_len + t, h, 3] >= 0
        q2[q_len - 1, 0, 7] = float("nan")
        hit[q_len - 1, 0] = True
        out, lse = torch.empty_like(clean), torch.empty_like(clean_lse)
        dp.packed_attention(q2.cuda(), k2.cuda(), v.cuda(), q_lens, k_lens, out, lse=lse)
        assert torch.equal(torch.isnan(out).all(dim=2).cpu(), hit)
        assert torch.equal(torch.isnan(out).any(dim=2).cpu(), hit)
        assert torch.equal(torch.isnan(lse).cpu(), hit)
        # a score of -infinity is a weight of 0: not the clean result, the others are
        same = torch.ones(q.shape[:2], dtype=torch.bool)
        for i, j in enumerate(places):
            for t in range(q_len):
                if j <= k_len - q_len + t:
                    same[i * q_len + t, 2:] = False
        same[q_len - 1, 0] = False
        assert torch.equal(out.cpu()[same], clean.cpu()[same]) and torch.equal(lse.cpu()[same], clean_lse.cpu()[same])


def test_no_score_above_minus_infinity(dp):
    for q_lens, k_lens in (([1], [40]), ([1], [9000]), ([30], [60]), ([200], [5000])):
        for dtype in (BF16, F16, F32):
            for d in (64, 128):
                q, k, v = _inputs(q_lens, k_lens, 2, 1, d, dtype, spare=0)
                q[:, 0, 0], k[:, 0, 0] = 1.0, -float("inf")
                q[:, 1, 0] = -1.0  # and these scores +infinity
                out = torch.empty(q.shape, dtype=dtype, device="cuda")
                dp.packed_attention(q.cuda(), k.cuda(), v.cuda(), q_lens, k_lens, out, causal=False)
                assert torch.isnan(out).all()


@pytest.mark.parametrize("tokens", [1, 3])
@pytest.mark.parametrize("n,heads,kv_heads,keys,d", [(3, 8, 8, 2000, 64), (12, 16, 16, 2100, 64), (40, 8, 4, 2500, 128)])
def test_tokens_beside_prompts(dp, n, heads, kv_heads, keys, d, tokens):
    """Single tokens and drafts over a cache in one call with chunks of prompts, in any order, few
    enough keys to be taken along and enough for a launch of their own."""
    rng = np.random.default_rng(n)
    k_lens = [int(x) for x in rng.integers(keys // 2, keys + keys // 2, n)]
    q_lens = [tokens] * n
    for at, ql, kl in ((0, 140, 300), (n // 2, 0, 70), (n, 65, 65), (n + 3, 20, 5)):
        q_lens.insert(at, ql)
        k_lens.insert(at, kl)
    for dtype in (BF16, F16):
        q, k, v = _inputs(q_lens, k_lens, heads, kv_heads, d, dtype)
        out, lse = _run(dp, q, k, v, q_lens, k_lens)
        _check(out, lse, q, k, v, q_lens, k_lens, None, True)


@pytest.mark.parametrize("n", [33, 1000, 1024])
def test_many_sequences(dp, n):
    rng = np.random.default_rng(n)
    lens = [int(x) for x in rng.integers(0, 9, n)]
    k_lens = [int(x) for x in rng.integers(0, 40, n)]
    for dtype in (BF16, F32):
        q, k, v = _inputs(lens, k_lens, 2, 1, 64, dtype)
        out, lse = _run(dp, q, k, v, lens, k_lens)
        _check(out, lse, q, k, v, lens, k_lens, None, True)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_more_items_than_blocks_fit(dp, d, causal):
    """Far more (tile, k/v head) items than the SMs hold blocks, so that blocks go on from one to
    the next: sequences without keys, of one token and with every tail of a key tile among them."""
    rng = np.random.default_rng(d)
    lens = [int(x) for x in rng.integers(0, 90, 150)] + [0, 1, 400, 17]
    k_lens = [int(x) for x in rng.integers(0, 200, 150)] + [5, 0, 700, 64]
    q, k, v = _inputs(lens, k_lens, 12, 4, d, F16)
    out, lse = _run(dp, q, k, v, lens, k_lens, None, causal)
    _check(out, lse, q, k, v, lens, k_lens, None, causal)
    again, _ = _run(dp, q, k, v, lens, k_lens, None, causal)
    assert torch.equal(out[:sum(lens)], again[:sum(lens)])


@pytest.mark.parametrize("q_lens,k_lens", [([1] * 9, [700, 3000, 5, 64, 1, 2000, 4100, 0, 129]), ([300, 40, 777], [300, 900, 777])])
def test_calls_one_behind_the_other_on_the_same_buffers(dp, q_lens, k_lens):
    """The output of one call is the query of the next, and its keys change between calls."""
    for d, dtype in ((64, F16), (128, BF16), (128, F32)):
        q, k, v = (t.cuda() for t in _inputs(q_lens, k_lens, 8, 2, d, dtype, spare=0))
        a, b = q.clone(), torch.empty_like(q)

        def run(wait):
            a.copy_(q)
            kk, seen = k.clone(), []
            for i in range(10):
                for src, dst in ((a, b), (b, a)):
                    dp.packed_attention(src, kk, v, q_lens, k_lens, dst)
                    if wait:
                        torch.cuda.synchronize()
                kk.mul_(-0.9)
                a.add_(q)
                seen.append(a.clone())
            torch.cuda.synchronize()
            return seen
        for x, y in zip(run(True), run(False)):
            assert torch.equal(x, y)


def test_calls_of_two_threads(dp):
    """Two threads, a stream each, several calls under way: no call depends on another."""
    import threading
    lens, k_lens = [1, 40, 200], [3000, 900, 200]
    q, k, v = (t.cuda() for t in _inputs(lens, k_lens, 8, 2, 128, BF16, spare=0))
    ref, _ = _run(dp, q, k, v, lens, k_lens)
    torch.cuda.synchronize()
    outs = [[torch.zeros_like(ref) for _ in range(20)] for _ in range(2)]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for o in outs[i]:
                dp.packed_attention(q, k, v, lens, k_lens, o)
            torch.cuda.current_stream().synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(torch.equal(o, ref) for side in outs for o in side)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_long_sequence_last_rows(dp, dtype):
    """A 9000-token prompt: its last and first rows against the oracle, the whole finite and repeatable."""
    n = 9000
    q, k, v = _inputs([n], [n], 2, 1, 128, dtype, spare=0)
    out, lse = _run(dp, q, k, v, [n], [n])
    again, _ = _run(dp, q, k, v, [n], [n])
    assert torch.equal(out, again) and bool(torch.isfinite(out).all())
    _check(out[:200], lse[:200], q[:200], k, v, [200], [200], None, True)
    _check(out[-150:], lse[-150:], q[-150:], k, v, [150], [n], None, True)


@pytest.mark.parametrize("dtype,q_lens,k_lens", [
    (BF16, [300, 1, 90], [300, 700, 1100]), (F16, [1, 3], [900, 1200]), (F32, [40, 1], [500, 300])])
def test_offsets_behind_32_bits(dp, dtype, q_lens, k_lens):
    """Rows 2^20 elements apart, the last sequences' behind 2^32 elements (fp32: 2^31)."""
    heads, kv, d, pitch = 4, 2, 64, 1 << 20
    rows = 4200 if dtype != F32 else 2300
    starts = [0] * (len(k_lens) - 1) + [rows - k_lens[-1]]
    q_all, k_all = list(q_lens), list(k_lens)
    if sum(q_lens) > 40:  # an empty-handed sequence in front: its queries see no key
        q_all, k_all, starts = [rows - sum(q_lens)] + q_all, [0] + k_all, [0] + starts
    q, k, v = _inputs(q_all, k_all, heads, kv, d, dtype, k_starts=starts, spare=0)
    nq = sum(q_all)
    held, res = (torch.empty(rows, pitch, dtype=dtype, device="cuda") for _ in range(2))
    parts = held[:, :(heads + 2 * kv) * d].unflatten(1, (-1, d))
    parts[:nq, :heads].copy_(q)
    parts[:, heads:].copy_(torch.cat([k, v], dim=1))
    out = res[:nq, 256:256 + heads * d].unflatten(1, (-1, d))
    lse = torch.empty(nq, heads, device="cuda")
    dp.packed_attention(parts[:nq, :heads], parts[:, heads:heads + kv], parts[:, heads + kv:], q_all, k_all, out,
                        k_starts=starts, lse=lse)
    dp.device_status()
    _check(out, lse, q, k, v, q_all, k_all, starts, True)


def test_side_stream_and_two_captured_graphs(dp):
    lens = [1, 1, 40]
    k_lens = [900, 3000, 40]
    q, k, v = (t.cuda() for t in _inputs(lens, k_lens, 8, 2, 128, BF16, spare=0))
    ref, _ = _run(dp, q, k, v, lens, k_lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = _run(dp, q, k, v, lens, k_lens, stream=side)
    assert torch.equal(got, ref)
    outs, graphs = [torch.zeros_like(ref) for _ in range(2)], [torch.cuda.CUDAGraph() for _ in range(2)]
    torch.cuda.synchronize()
    for o, gr in zip(outs, graphs):
        with torch.cuda.graph(gr):
            dp.packed_attention(q, k, v, lens, k_lens, o)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref)
    q.mul_(0.5)
    graphs[0].replay()
    torch.cuda.synchronize()
    half, _ = _run(dp, q, k, v, lens, k_lens)
    assert torch.equal(outs[0], half)


def test_nothing_to_do_leaves_everything(dp):
    q = torch.zeros(4, 2, 64, dtype=BF16, device="cuda")
    k = torch.zeros(0, 1, 64, dtype=BF16, device="cuda")
    out = torch.full_like(q, 2.0)
    dp.packed_attention(q, k, k, [0], [0], out)
    torch.cuda.synchronize()
    assert bool((out == 2.0).all())
    dp.packed_attention(q, k, k, [3], [0], out)            # no keys at all
    torch.cuda.synchronize()
    assert not bool(out[:3].any()) and bool((out[3] == 2.0).all())


def test_binding_refuses_what_does_not_match(dp):
    q = torch.zeros(8, 4, 64, dtype=BF16, device="cuda")
    k = torch.zeros(8, 2, 64, dtype=BF16, device="cuda")
    out = torch.empty_like(q)
    with pytest.raises(ValueError):
        dp.packed_attention(q, k, k, [8], [8, 1], out)
    with pytest.raises(ValueError):
        dp.packed_attention(q, k, k[:7], [8], [8], out)
    with pytest.raises(ValueError):
        dp.packed_attention(q.transpose(0, 1), k, k, [4], [4], out)
    with pytest.raises(TypeError):
        dp.packed_attention(q, k.float(), k.float(), [8], [8], out)
    with pytest.raises(ValueError):
        dp.packed_attention(q, k, k, [8], [8], out, lse=torch.empty(8, 3, device="cuda"))
    for bad in (dict(q_lens=[9], k_lens=[8]), dict(q_lens=[8], k_lens=[9]), dict(q_lens=[-1], k_lens=[8]),
                dict(q_lens=[8], k_lens=[8], k_starts=[1]), dict(q_lens=[8], k_lens=[8], k_starts=[-1])):
        with pytest.raises(dp.DpError) as e:
            dp.packed_attention(q, k, k, out=out, **bad)
        assert e.value.status == dp.ERR_INVALID_ARG
    with pytest.raises(dp.DpError):
        dp.packed_attention(q, k, k, [8], [8], q)           # in place


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_a_layer_in_four_bits(dp, dtype):
    """A packed batch through a layer as it is served: pre-norm, q/k/v product in 4 bits, causal
    attention on the product's column ranges, output product in 4 bits; each stage checked from
    the stage before as the GPU left it."""
    lens, heads, kv, d, hidden = [40, 1, 130, 77], 6, 2, 128, 768
    n, width = sum(lens), (heads + 2 * kv) * d
    g = torch.Generator().manual_seed(11)
    x = torch.randn(n, hidden, generator=g).to(BF16).cuda()
    table = torch.tanh(torch.randn(4, 3, hidden, generator=g)).cuda()
    w_qkv = (torch.randn(width, hidden, generator=g) * hidden ** -0.5).cuda()
    w_out = (torch.randn(hidden, heads * d, generator=g) * (heads * d) ** -0.5).to(F16).cuda()
    bias = torch.randn(width, generator=g).cuda()
    wq, wo = dp.mx4_empty(width, hidden), dp.mx4_empty(hidden, heads * d)
    dp.mx4_quantize(w_qkv, *wq)
    dp.mx4_quantize(w_out, *wo)
    h = torch.empty_like(x)
    dp.ln_modulate(x, h, dp.blocks_from_table(table, [0, 1, 2, 3], lens))
    hq = dp.mx4_empty(n, hidden)
    dp.mx4_quantize(h, *hq)
    qkv = torch.empty(n, width, dtype=dtype, device="cuda")
    dp.mx4_linear(*hq, *wq, bias, qkv)
    rows = qkv.view(n, heads + 2 * kv, d)
    q, k, v = rows[:, :heads], rows[:, heads:heads + kv], rows[:, heads + kv:]
    o = torch.empty(n, heads, d, dtype=dtype, device="cuda")
    lse = torch.empty(n, heads, device="cuda")
    dp.packed_attention(q, k, v, lens, lens, o, lse=lse)
    oq = dp.mx4_empty(n, heads * d)
    dp.mx4_quantize(o.view(n, -1), *oq)
    y = torch.empty(n, hidden, device="cuda")
    dp.mx4_linear(*oq, *wo, None, y)
    dp.device_status()

    def values(pair):
        return O.mx4_values(pair[0].cpu().numpy(), pair[1].cpu().numpy())
    codes, scales = O.mx4_quantize(h.cpu().double().numpy())
    assert np.array_equal(hq[0].cpu().numpy(), codes) and np.array_equal(hq[1].cpu().numpy(), scales)
    a, w = values(hq), values(wq)
    want, size = a @ w.T + bias.cpu().double().numpy(), np.abs(a) @ np.abs(w).T + bias.cpu().double().abs().numpy()
    u = torch.finfo(dtype).eps / 2
    assert (np.abs(qkv.cpu().double().numpy() - want) <= u * np.abs(want) + 770 * 2.0 ** -24 * size + 2.0 ** -24).all()
    _check(o, lse, q.cpu(), k.cpu(), v.cpu(), lens, lens, None, True)
    a, w = values(oq), values(wo)
    assert (np.abs(y.cpu().double().numpy() - a @ w.T) <= 2.0 ** -24 * np.abs(a @ w.T) + 770 * 2.0 ** -24 * (np.abs(a) @ np.abs(w).T)).all()
