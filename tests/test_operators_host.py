"""Argument checks of the 4-bit and packed-attention entry points (no GPU): every call fails its
checks, or has nothing to do, before anything is enqueued."""
import ctypes

import pytest

FAKE = 0x7f0000000000  # 16-byte aligned, never dereferenced
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def m():
    import long_video_diffusion_b200 as mod
    return mod


def test_mx4_scale_bytes(m):
    assert m.mx4_scale_bytes(1, 32) == 512 and m.mx4_scale_bytes(128, 128) == 512
    assert m.mx4_scale_bytes(129, 160) == 2048 and m.mx4_scale_bytes(0, 32) == 0
    for rows, k in [(-1, 32), (1, 0), (1, 33), (1, -32), (1 << 31, 32)]:
        with pytest.raises(m.DpError):
            m.mx4_scale_bytes(rows, k)


def test_mx4_quantize_checks(m):
    for fn in ("dp_mx4_quantize", "dp_mx4_dequantize"):
        def call(x=FAKE, n=64, k=64, dt=1, codes=FAKE + (1 << 20), scales=FAKE + (2 << 20)):
            f = getattr(m._lib, fn)
            return f(P(x), n, k, dt, P(codes), P(scales), None) if fn == "dp_mx4_quantize" else \
                f(P(codes), P(scales), n, k, P(x), dt, None)
        assert call(n=0, x=0) == m.OK
        assert call(dt=9) == m.ERR_INVALID_ARG
        assert call(n=-1) == m.ERR_INVALID_ARG and call(n=1 << 31) == m.ERR_INVALID_ARG
        assert call(k=0) == m.ERR_INVALID_ARG and call(k=48) == m.ERR_UNSUPPORTED
        assert call(x=0) == m.ERR_INVALID_ARG and call(codes=0) == m.ERR_INVALID_ARG and call(scales=0) == m.ERR_INVALID_ARG
        assert call(x=FAKE + 8) == m.ERR_INVALID_ARG and call(scales=FAKE + (2 << 20) + 4) == m.ERR_INVALID_ARG
        assert call(codes=FAKE + 64 * 64 * 2 - 16) == m.ERR_INVALID_ARG        # overlaps the last row
        assert call(scales=FAKE) == m.ERR_INVALID_ARG


def test_mx4_linear_checks(m):
    M = 1 << 20

    def call(a=FAKE, sa=FAKE + M, w=FAKE + 2 * M, sw=FAKE + 3 * M, b=FAKE + 4 * M, rows=64, n=64, k=64, y=FAKE + 5 * M, dt=1):
        return m._lib.dp_mx4_linear(P(a), P(sa), P(w), P(sw), P(b), rows, n, k, P(y), dt, None)
    assert call(rows=0, a=0) == m.OK
    assert call(dt=3) == m.ERR_INVALID_ARG
    assert call(rows=-5) == m.ERR_INVALID_ARG and call(n=0) == m.ERR_INVALID_ARG and call(k=-32) == m.ERR_INVALID_ARG
    assert call(n=60) == m.ERR_UNSUPPORTED and call(k=40) == m.ERR_UNSUPPORTED
    for name in ("a", "sa", "w", "sw", "y"):
        assert call(**{name: 0}) == m.ERR_INVALID_ARG
        assert call(**{name: FAKE + 8 * M + 8}) == m.ERR_INVALID_ARG
    assert call(b=FAKE + 4) == m.ERR_INVALID_ARG
    for at in (0, 1, 2, 3, 4):
        assert call(y=FAKE + at * M) == m.ERR_INVALID_ARG                      # overlaps an input


def test_packed_attention_checks(m):
    M = 1 << 20

    def call(q=FAKE, k=FAKE + M, v=FAKE + 2 * M, out=FAKE + 3 * M, lse=FAKE + 4 * M, ql=(8, 4), kl=(8, 4), ks=None, qr=12,
             kr=12, H=4, G=2, d=64, ld=None, scale=0.0, flags=1, dt=1, n=None):
        i64 = ctypes.c_int64
        lq, lk, lv, lo = ld or (H * d, G * d, G * d, H * d)
        arr = lambda x: None if x is None else (i64 * max(len(x), 1))(*x)
        return m._lib.dp_packed_attention(P(q), lq, P(k), lk, P(v), lv, P(out), lo, P(lse), qr, kr, arr(ql), arr(kl), arr(ks),
                                          len(ql or (0,)) if n is None else n, H, G, d, scale, flags, dt, None)
    bad = m.ERR_INVALID_ARG
    assert call(ql=(0, 0), q=0, out=0) == m.OK                                 # no query rows
    assert call(dt=4) == bad and call(flags=2) == bad
    assert call(H=5) == bad and call(G=0) == bad and call(H=0) == bad and call(d=0) == bad
    assert call(d=96) == m.ERR_UNSUPPORTED and call(d=32) == m.ERR_UNSUPPORTED
    assert call(scale=float("nan")) == bad and call(scale=float("inf")) == bad
    assert call(ql=None) == bad and call(kl=None) == bad
    assert call(n=0) == bad and call(ql=(1,) * 1025, kl=(0,) * 1025, qr=2000) == bad
    assert call(ql=(8, 5)) == bad and call(kl=(8, 5)) == bad and call(ql=(-1, 4)) == bad and call(kl=(8, -4)) == bad
    assert call(ks=(0, 9)) == bad and call(ks=(-1, 0)) == bad and call(ks=(0, 1 << 40)) == bad
    assert call(ql=(1 << 62, 1 << 62)) == bad and call(kl=(1 << 62, 1 << 62)) == bad
    assert call(qr=-1) == bad and call(kr=1 << 31) == bad
    assert call(ld=(255, 128, 128, 256)) == bad and call(ld=(256, 127, 128, 256)) == bad
    assert call(ld=(260, 128, 128, 256)) == bad                                # 520 bytes: no multiple of 16
    assert call(ld=(256, 1 << 29, 128, 256)) == bad
    for name in ("q", "k", "v", "out"):
        assert call(**{name: 0}) == bad
        assert call(**{name: FAKE + 8 * M + 8}) == bad
    assert call(lse=FAKE + 4 * M + 4) == bad
    assert call(out=FAKE) == bad and call(out=FAKE + M) == bad and call(out=FAKE + 2 * M + 16) == bad
    for at in (0, 1, 2, 3):
        assert call(lse=FAKE + at * M) == bad
    assert b"overlaps" in m._lib.dp_last_error_detail()
