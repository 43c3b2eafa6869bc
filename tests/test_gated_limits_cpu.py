"""Sizes past what one launch of the gated kernels can cover come back as
BBS_ENOTSUP before anything is launched."""
import ctypes as C

import pytest

import bit_block_scaled_amd as bbs

P = C.c_void_p


def fp4(rows, cols=64):
    return bbs.Fp4Desc(0x1000, 0x2000, 0x3000, rows, cols, 0, 0)


def mx8(rows, cols):
    return bbs.Mx8Desc(0x1000, 0x2000, rows, cols)


@pytest.mark.parametrize("M,F", [(1 << 32, 48), (1 << 30, 256), ((1 << 28) + 16, 1008), (1 << 44, 16), (16, 1 << 30)])
def test_gated_gemm_tiles(M, F):
    W = fp4(F)
    s = bbs.lib.nvfp4_gated_gemm(C.byref(fp4(M)), C.byref(W), C.byref(fp4(F)), 0, P(0x4000), 1, F, None, None, None)
    assert s == bbs.BBS_ENOTSUP and b"2^24 tiles of 256 x 64" in bbs.lib.bbs_last_error()


@pytest.mark.parametrize("M,F", [(1 << 31, 32), ((1 << 30) + 1, 192), (1, 1 << 31), (1 << 44, 32)])
def test_gated_bwd_tiles(M, F):
    s = bbs.lib.mxfp8_gemm_gated_bwd(C.byref(mx8(M, 64)), C.byref(mx8(F, 64)), C.byref(mx8(M, F)), C.byref(mx8(M, F)),
                                     0, P(0x4000), P(0x5000), 1, F, None)
    assert s == bbs.BBS_ENOTSUP and b"2^24 tiles of 128 x 128" in bbs.lib.bbs_last_error()
