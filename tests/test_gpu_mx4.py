"""GPU parity of the microscaled 4-bit operators against the float64 oracle.

Bounds: the quantisation is exact up to its one rounding, so codes and scales equal the
oracle's bit for bit, and so do the values in bf16 and f32 (powers of two times e2m1).  The
product's terms are exact in fp32; k of them summed in fp32 are within k * 2^-24 times the sum
of their magnitudes, and the store rounds by half a step: eps / 2 of the value."""
import numpy as np
import pytest
import torch

import oracle as O

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _quantize(dp, x):
    codes, scales = dp.mx4_empty(*x.shape)
    codes.fill_(0xAA)
    scales.fill_(0xFF)
    dp.mx4_quantize(x, codes, scales)
    return codes, scales


def _rows(rows, k, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, k, generator=g) * torch.exp2(torch.randint(-9, 9, (rows, k // 32), generator=g).float()).repeat_interleave(32, 1)
    return x.to(dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,k", [(1, 32), (1, 1536), (129, 160), (33, 4096), (300, 96), (128, 128), (257, 1120)])
def test_quantize_equals_oracle(dp, rows, k, dtype):
    x = _rows(rows, k, dtype, rows * k)
    codes, scales = _quantize(dp, x.cuda())
    want_codes, want_scales = O.mx4_quantize(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), want_scales)
    assert np.array_equal(codes.cpu().numpy(), want_codes)


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_edge_blocks(dp, dtype):
    """Ties, saturation, signed zeros, denormals, the type's extremes, infinities and NaN, one per block."""
    top = torch.finfo(dtype)
    tiny = torch.tensor([1], dtype=torch.int16 if top.bits == 16 else torch.int32).view(dtype).item()   # least denormal
    x = torch.zeros(10, 64, dtype=torch.float64)
    x[0, :12] = torch.tensor([6.0, .25, .75, 1.25, 1.75, 2.5, 3.5, 5.0, -.25, -0.0, 7.0, -5.0])
    x[1, :4] = torch.tensor([top.max, -top.max, top.max / 2, 1.0])
    x[2, :3] = torch.tensor([tiny, -tiny, 0.0])
    x[3, :3] = torch.tensor([7 * tiny, 3 * tiny, tiny])
    x[4, 7], x[5, 8], x[6, 9] = float("inf"), float("-inf"), float("nan")
    x[7, :2] = torch.tensor([top.smallest_normal, top.smallest_normal * 1.5])
    x[8, 32:] = 1.0
    x = x.to(dtype)
    codes, scales = _quantize(dp, x.cuda())
    want_codes, want_scales = O.mx4_quantize(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), want_scales)
    bad = want_scales[O.mx4_scale_index(10, 64)].repeat(16, axis=1) == 255    # codes under a NaN scale say nothing
    assert np.array_equal(np.where(bad, 0, codes.cpu().numpy()), np.where(bad, 0, want_codes))
    y = torch.empty(10, 64, device="cuda")
    dp.mx4_dequantize(codes, scales, y)
    assert np.array_equal(y.cpu().double().numpy(), O.mx4_values(want_codes, want_scales), equal_nan=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,k", [(1, 32), (130, 288), (5, 4128)])
def test_dequantize_any_codes(dp, rows, k, dtype):
    rng = np.random.default_rng(rows)
    codes = rng.integers(0, 256, (rows, k // 2), dtype=np.uint8)
    scales = np.zeros(dp.mx4_scale_bytes(rows, k), dtype=np.uint8)
    scales[O.mx4_scale_index(rows, k)] = rng.integers(0, 256, (rows, k // 32))
    y = torch.empty(rows, k, dtype=dtype, device="cuda")
    dp.mx4_dequantize(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), y)
    want = torch.from_numpy(O.mx4_values(codes, scales))
    if dtype == torch.float16:
        want = want.clamp(-65504, 65504)
    assert torch.equal(torch.nan_to_num(y.cpu(), nan=7.0), torch.nan_to_num(want.to(dtype), nan=7.0))


def _check_product(dp, m, n, k, bias, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + m + n + k)
    a = torch.randn(m, k, generator=g).cuda()
    w = (torch.randn(n, k, generator=g) * torch.exp2(torch.randint(-6, 2, (n, 1), generator=g).float())).cuda()
    b = torch.randn(n, generator=g).cuda() if bias else None
    qa, qw = _quantize(dp, a), _quantize(dp, w)
    guard = torch.full((m + 2, n), 3.5, dtype=dtype, device="cuda")
    y = guard[1:m + 1]
    dp.mx4_linear(*qa, *qw, b, y)
    dp.device_status()
    va, vw = (torch.from_numpy(O.mx4_values(c.cpu().numpy(), s.cpu().numpy())) for c, s in (qa, qw))
    want = va @ vw.T + (b.cpu().double() if bias else 0.0)
    # the bias is one more term, with its own rounding
    size = va.abs() @ vw.abs().T + (b.cpu().double().abs() if bias else 0.0)
    bound = torch.finfo(dtype).eps / 2 * want.abs() + (k + 1) * 2.0 ** -24 * size * 1.01 + 1e-30
    if dtype == torch.float16:
        want = want.clamp(-65504, 65504)
        bound = bound + 2.0 ** -25  # half the least denormal
    err = (y.cpu().double() - want).abs()
    assert bool((err <= bound).all()), (err / bound).max().item()
    assert bool((guard[0] == 3.5).all()) and bool((guard[-1] == 3.5).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k,bias", [
    (1, 8, 32, False), (1, 4096, 4096, True), (2, 136, 96, True), (16, 128, 256, False), (17, 1024, 1536, True),
    (33, 264, 544, False), (64, 512, 2048, True), (65, 72, 64, True), (100, 640, 224, False), (128, 256, 1024, True),
    (129, 264, 160, True), (255, 1000, 288, False), (256, 4608, 1536, True), (257, 120, 4128, True),
    (300, 2048, 512, False), (513, 776, 1120, True), (1000, 520, 192, True), (32, 2056, 736, True), (448, 1160, 352, True),
    (700, 6152, 96, False), (257, 20000, 64, True)])
def test_linear_within_rounding(dp, m, n, k, bias, dtype):
    _check_product(dp, m, n, k, bias, dtype)


@pytest.mark.parametrize("m,n,k", [(4500, 1536, 4096), (2711, 6144, 2048), (8, 11008, 8192), (12480, 64, 512)])
def test_linear_many_tiles(dp, m, n, k):
    _check_product(dp, m, n, k, True, torch.bfloat16)


def test_offsets_behind_32_bits(dp):
    """More than 2^32 elements quantised, read back and multiplied: the last rows are the oracle's."""
    rows, k, n, last = 530000, 8192, 8200, 300
    x = torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda")
    tail = _rows(last, k, torch.bfloat16, 5)
    x[-last:] = tail.cuda()
    codes, scales = _quantize(dp, x)
    want, want_scales = O.mx4_quantize(tail.double().numpy())
    assert np.array_equal(codes[-last:].cpu().numpy(), want)
    back = x
    dp.mx4_dequantize(codes, scales, back)
    values = O.mx4_values(want, want_scales)
    assert torch.equal(back[-last:].cpu().double(), torch.from_numpy(values)) and not bool(back[:1000].any())
    del x, back
    w = _rows(n, 64, torch.bfloat16, 6)
    a = torch.zeros(rows, 64, dtype=torch.bfloat16, device="cuda")
    a[-last:] = _rows(last, 64, torch.bfloat16, 7).cuda()
    qa, qw = _quantize(dp, a), _quantize(dp, w.cuda())
    y = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    dp.mx4_linear(*qa, *qw, None, y)
    dp.device_status()
    va = O.mx4_values(*O.mx4_quantize(a[-last:].cpu().double().numpy()))
    vw = O.mx4_values(*O.mx4_quantize(w.double().numpy()))
    exact, size = va @ vw.T, np.abs(va) @ np.abs(vw).T
    err = np.abs(y[-last:].cpu().double().numpy() - exact)
    assert (err <= 2.0 ** -8 * np.abs(exact) + 65 * 2.0 ** -24 * 1.01 * size + 1e-30).all()
    assert not bool(y[:1000].any())


@pytest.mark.parametrize("m", [3, 700])
def test_linear_nan_block_reaches_its_row_only(dp, m):
    """A block that was quantised from a NaN makes its row NaN and no other; a f16 output saturates."""
    g = torch.Generator().manual_seed(m)
    a, w = torch.randn(m, 416, generator=g), torch.randn(136, 416, generator=g)
    a[1, 410] = float("nan")
    a[2] = 6000.0
    w[3] = 6000.0
    qa, qw = _quantize(dp, a.cuda()), _quantize(dp, w.cuda())
    y = torch.empty(m, 136, dtype=torch.float16, device="cuda")
    dp.mx4_linear(*qa, *qw, None, y)
    dp.device_status()
    got = y.cpu()
    assert bool(torch.isnan(got[1]).all()) and not bool(torch.isnan(got[torch.arange(m) != 1]).any())
    assert got[2, 3].item() == 65504.0 and not bool(torch.isinf(got).any())


def test_linear_is_the_same_every_time_and_on_another_stream(dp):
    a, w = _rows(77, 2080, torch.bfloat16, 1).cuda(), _rows(1032, 2080, torch.bfloat16, 2).cuda()
    qw = _quantize(dp, w)
    outs = []
    side = torch.cuda.Stream()
    for i in range(3):
        codes, scales = dp.mx4_empty(77, 2080)
        y = torch.empty(77, 1032, device="cuda")
        torch.cuda.synchronize()
        s = side if i else None
        dp.mx4_quantize(a, codes, scales, stream=s)
        dp.mx4_linear(codes, scales, *qw, None, y, stream=s)
        torch.cuda.synchronize()
        outs.append(y)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("m", [1, 40, 600])
def test_captured_and_replayed_with_new_inputs(dp, m):
    k, n = 1536, 512
    w = _quantize(dp, _rows(n, k, torch.bfloat16, 3).cuda())
    x = _rows(m, k, torch.bfloat16, 4).cuda()
    codes, scales = dp.mx4_empty(m, k)
    y = torch.empty(m, n, device="cuda", dtype=torch.bfloat16)

    def layer():
        dp.mx4_quantize(x, codes, scales)
        dp.mx4_linear(codes, scales, *w, None, y)
    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for seed in (5, 6):
        x.copy_(_rows(m, k, torch.bfloat16, seed))
        layer()
        want = y.clone()
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("m,k,n", [(3, 1536, 512), (700, 2080, 4360), (9000, 512, 64)])
def test_calls_one_behind_the_other_on_the_same_buffers(dp, m, k, n):
    """Kernels may start before the ones ahead of them have ended: results are those of a stream
    that is waited for after every call, other libraries' kernels between them included."""
    w = _quantize(dp, _rows(n, k, torch.bfloat16, 1).cuda())
    x = _rows(m, k, torch.bfloat16, 2).cuda()
    codes, scales = dp.mx4_empty(m, k)
    y = torch.empty(m, n, device="cuda")
    back = torch.empty(m, k, dtype=torch.bfloat16, device="cuda")

    def run(wait):
        x.copy_(_rows(m, k, torch.bfloat16, 2))
        seen = []
        for i in range(12):
            for call in (lambda: dp.mx4_quantize(x, codes, scales), lambda: dp.mx4_linear(codes, scales, *w, None, y),
                         lambda: dp.mx4_dequantize(codes, scales, back), lambda: dp.mx4_quantize(back, codes, scales),
                         lambda: dp.mx4_dequantize(codes, scales, back)):
                call()
                if wait:
                    torch.cuda.synchronize()
            seen += [y.clone(), back.clone()]
            x.mul_(1.25)
            x.add_(back, alpha=-0.5)
        torch.cuda.synchronize()
        return seen
    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)


def test_first_call_of_a_thread(dp):
    """A thread that has made no CUDA call yet."""
    import threading
    c, w = (_quantize(dp, _rows(n, 512, torch.bfloat16, n).cuda()) for n in (70, 264))
    ys = [torch.zeros(70, 264, device="cuda") for _ in range(2)]
    dp.mx4_linear(*c, *w, None, ys[0])
    torch.cuda.synchronize()
    t = threading.Thread(target=lambda: dp.mx4_linear(*c, *w, None, ys[1]))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert torch.equal(*ys)


def test_no_rows_do_nothing(dp):
    codes, scales = dp.mx4_empty(0, 64)
    x = torch.empty(0, 64, device="cuda")
    dp.mx4_quantize(x, codes, scales)
    dp.mx4_dequantize(codes, scales, x)
    w = _quantize(dp, torch.randn(8, 64, device="cuda"))
    dp.mx4_linear(codes, scales, *w, None, torch.empty(0, 8, device="cuda"))
    torch.cuda.synchronize()


def test_binding_refuses_what_does_not_match(dp):
    x = torch.randn(4, 64, device="cuda")
    codes, scales = dp.mx4_empty(4, 64)
    w = _quantize(dp, torch.randn(8, 64, device="cuda"))
    y = torch.empty(4, 8, device="cuda")
    with pytest.raises(ValueError):
        dp.mx4_quantize(x[:, ::2], codes, scales)
    with pytest.raises(ValueError):
        dp.mx4_quantize(x, codes[:3], scales)
    with pytest.raises(ValueError):
        dp.mx4_quantize(x, codes, scales[:511])
    with pytest.raises(ValueError):
        dp.mx4_quantize(x.cpu(), codes, scales)
    with pytest.raises(ValueError):
        dp.mx4_quantize(x, codes.cpu(), scales)
    with pytest.raises(TypeError):
        dp.mx4_quantize(x.double(), codes, scales)
    with pytest.raises(ValueError):
        dp.mx4_linear(codes, scales, *w, None, y.T)
    with pytest.raises(ValueError):
        dp.mx4_linear(codes, scales, *w, torch.zeros(7, device="cuda"), y)
    with pytest.raises(dp.DpError) as e:
        dp.mx4_quantize(torch.randn(4, 48, device="cuda"), torch.empty(4, 24, dtype=torch.uint8, device="cuda"), scales)
    assert e.value.status == dp.ERR_UNSUPPORTED
