"""CPU checks of the gated feed-forward operators: argument errors come back
before anything is launched, and the derivative the backward pass uses is the
derivative of the forward formula."""
import ctypes as C

import numpy as np
import pytest

import bit_block_scaled_amd as bbs
from gated_ref import act64, act_slope64

L = bbs.lib
P = C.c_void_p


def fp4(rows=32, cols=64, tile2d=0, per_row=0, codes=0x1000):
    return bbs.Fp4Desc(codes, 0x2000, 0x3000, rows, cols, tile2d, per_row)


def mx8(rows=32, cols=64, codes=0x1000, scales=0x2000):
    return bbs.Mx8Desc(codes, scales, rows, cols)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_slope_is_the_derivative(act):
    g = np.concatenate([np.linspace(-12, 12, 4801), [-80.0, -30.0, 30.0, 80.0]])
    h = 1e-5
    d = (act64(act, g + h) - act64(act, g - h)) / (2 * h)
    # a central difference is off by h^2 / 6 of the third derivative (below 8
    # here) and by the rounding of the two values over 2 h
    assert np.all(np.abs(d - act_slope64(act, g)) <= 8 * h * h / 6 + 4 * 2.0 ** -53 * (np.abs(g) + 1) / h)


def gated(A=None, Wg=None, Wu=None, act=0, H=0x4000, dt=1, ldh=48, g8=None, u8=None):
    A = fp4() if A is None else A
    Wg = fp4(48) if Wg is None else Wg
    Wu = fp4(48) if Wu is None else Wu
    ref = [C.byref(d) if d is not None else None for d in (g8, u8)]
    return L.nvfp4_gated_gemm(C.byref(A), C.byref(Wg), C.byref(Wu), act, P(H), dt, ldh, *ref, None)


def test_gated_gemm_errors():
    assert L.nvfp4_gated_gemm(None, None, None, 0, P(0x4000), 1, 48, None, None, None) == bbs.BBS_EINVAL
    assert gated(A=fp4(30)) == bbs.BBS_EINVAL
    assert gated(A=fp4(0)) == bbs.BBS_EINVAL
    assert gated(A=fp4(32, 32)) == bbs.BBS_EINVAL                    # K differs
    assert gated(Wu=fp4(32)) == bbs.BBS_EINVAL                       # shapes differ
    assert gated(Wu=fp4(48, tile2d=1)) == bbs.BBS_ENOTSUP
    assert gated(Wg=fp4(48, per_row=1)) == bbs.BBS_ENOTSUP
    assert gated(act=2) == bbs.BBS_EINVAL
    assert gated(act=-1) == bbs.BBS_EINVAL
    assert gated(dt=2) == bbs.BBS_EINVAL
    assert gated(H=None) == bbs.BBS_EINVAL
    assert gated(H=0x4008) == bbs.BBS_EINVAL
    assert gated(ldh=32) == bbs.BBS_EINVAL                           # shorter than a row
    assert gated(ldh=52) == bbs.BBS_EINVAL                           # 104 bytes
    assert b"H must be" in L.bbs_last_error()
    W64 = fp4(64)
    assert gated(Wg=W64, Wu=fp4(64), ldh=64, g8=mx8(32, 64)) == bbs.BBS_EINVAL
    assert b"together" in L.bbs_last_error()
    assert gated(Wg=W64, Wu=fp4(64), ldh=64, g8=mx8(32, 64), u8=mx8(32, 32)) == bbs.BBS_EINVAL
    assert gated(Wg=W64, Wu=fp4(64), ldh=64, g8=mx8(16, 64), u8=mx8(16, 64)) == bbs.BBS_EINVAL
    assert gated(Wg=W64, Wu=fp4(64), ldh=64, g8=mx8(32, 64, codes=0x1008), u8=mx8()) == bbs.BBS_EINVAL
    # 48 columns hold no whole number of 32-blocks
    assert gated(g8=mx8(32, 48), u8=mx8(32, 48)) == bbs.BBS_EINVAL


def bwd(dY=None, Wt=None, g8=None, u8=None, act=0, dG=0x4000, dU=0x5000, dt=1, ld=96):
    dY = mx8(24, 64) if dY is None else dY
    Wt = mx8(96, 64) if Wt is None else Wt
    g8 = mx8(24, 96) if g8 is None else g8
    u8 = mx8(24, 96) if u8 is None else u8
    return L.mxfp8_gemm_gated_bwd(C.byref(dY), C.byref(Wt), C.byref(g8), C.byref(u8), act, P(dG), P(dU), dt, ld,
                                  None)


def test_k_of_2_to_the_25():
    """Row offsets inside a tile are 32 bits wide."""
    K = 1 << 25
    W = fp4(48, K)
    assert gated(A=fp4(32, K), Wg=W, Wu=fp4(48, K)) == bbs.BBS_ENOTSUP
    assert bwd(dY=mx8(24, K), Wt=mx8(96, K)) == bbs.BBS_ENOTSUP


def test_gated_bwd_errors():
    assert L.mxfp8_gemm_gated_bwd(None, None, None, None, 0, P(0x4000), P(0x5000), 1, 96, None) == bbs.BBS_EINVAL
    assert bwd(dY=mx8(0, 64)) == bbs.BBS_EINVAL
    assert bwd(dY=mx8(24, 48)) == bbs.BBS_EINVAL                     # K % 32
    assert bwd(dY=mx8(24, 32)) == bbs.BBS_EINVAL                     # K differs
    assert bwd(g8=mx8(24, 64)) == bbs.BBS_EINVAL
    assert bwd(u8=mx8(32, 96)) == bbs.BBS_EINVAL
    assert bwd(u8=mx8(24, 96, scales=None)) == bbs.BBS_EINVAL
    assert bwd(act=5) == bbs.BBS_EINVAL
    assert bwd(dG=None) == bbs.BBS_EINVAL
    assert bwd(dU=None) == bbs.BBS_EINVAL
    assert bwd(dU=0x5004) == bbs.BBS_EINVAL
    assert bwd(dt=3) == bbs.BBS_EINVAL
    assert bwd(ld=64) == bbs.BBS_EINVAL
    assert bwd(ld=97) == bbs.BBS_EINVAL
    assert b"dG must be" in L.bbs_last_error()


def gemv(fmt=0, x=0x1000, T=1, ldx=64, W=None, y=0x4000, dt=1, ldy=48):
    W = fp4(48) if W is None else W
    return L.nvfp4_gemv(fmt, P(x), T, ldx, C.byref(W), P(y), dt, ldy, None)


def test_gemv_errors():
    for T in (0, -1, 65):
        assert gemv(T=T) == bbs.BBS_EINVAL
        assert b"tokens" in L.bbs_last_error()
    assert gemv(x=None) == bbs.BBS_EINVAL
    assert gemv(x=0x1008) == bbs.BBS_EINVAL
    assert gemv(y=None) == bbs.BBS_EINVAL
    assert gemv(y=0x4001) == bbs.BBS_EINVAL
    assert gemv(y=0x4002, dt=0) == bbs.BBS_EINVAL
    assert gemv(ldx=56) == bbs.BBS_EINVAL
    assert gemv(ldx=68) == bbs.BBS_EINVAL
    assert gemv(ldy=47) == bbs.BBS_EINVAL
    assert gemv(dt=2) == bbs.BBS_EINVAL
    assert gemv(fmt=1) == bbs.BBS_EINVAL
    assert gemv(W=fp4(40)) == bbs.BBS_EINVAL
    assert gemv(W=fp4(48, per_row=1)) == bbs.BBS_ENOTSUP
    assert gemv(fmt=2, W=bbs.Mx4Desc(0x1000, 0x2000, 48, 48)) == bbs.BBS_EINVAL
    assert gemv(fmt=2, W=bbs.Mx4Desc(0x1000, None, 48, 64)) == bbs.BBS_EINVAL
    assert L.nvfp4_gemv(0, P(0x1000), 1, 64, None, P(0x4000), 1, 48, None) == bbs.BBS_EINVAL


def test_gated_gemv_errors():
    def call(Wg, Wu, act=0, fmt=0, T=1):
        return L.nvfp4_gated_gemv(fmt, P(0x1000), T, 64, C.byref(Wg) if Wg else None,
                                  C.byref(Wu) if Wu else None, act, P(0x4000), 1, 48, None)
    assert call(fp4(48), None) == bbs.BBS_EINVAL
    assert call(None, fp4(48)) == bbs.BBS_EINVAL
    assert call(fp4(48), fp4(32)) == bbs.BBS_EINVAL
    assert call(fp4(48), fp4(48, tile2d=1)) == bbs.BBS_ENOTSUP
    assert call(fp4(48), fp4(48, per_row=1)) == bbs.BBS_ENOTSUP
    assert call(fp4(48), fp4(48), act=2) == bbs.BBS_EINVAL
    assert call(fp4(48), fp4(48), T=65) == bbs.BBS_EINVAL
    a, b = bbs.Mx4Desc(0x1000, 0x2000, 48, 64), bbs.Mx4Desc(0x1000, 0x2000, 32, 64)
    assert call(a, b, fmt=2) == bbs.BBS_EINVAL
