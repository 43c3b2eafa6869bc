"""Sizes past what a launch of the linear layer's operators holds: they are refused
before anything is launched.  A launch of 2^32 threads or more in a dimension is cut
off without an error."""
import ctypes as C

import pytest

pytest.importorskip("torch")

import bit_block_scaled_amd as bbs                                          # noqa: E402

L = bbs.lib
P = C.c_void_p


def bwd(cols, db):
    """The backward pass of one row; without dZ and db it is refused for that alone."""
    return L.mxfp8_bias_act_bwd(P(0x1000), 1, cols, 1 << 31, None, bbs.ACT_NONE, None, 0, P(db), 0, P(0x6000), None)


def test_bwd_columns():
    """A workgroup of 256 threads takes 128 columns: 2^24 of them are 2^32 threads."""
    for cols in ((1 << 31) - 112, (1 << 31) - 16, 1 << 31, 1 << 40):
        assert bwd(cols, None) == bbs.BBS_ENOTSUP, cols
        assert bwd(cols, 0x5000) == bbs.BBS_ENOTSUP, cols
    assert bwd((1 << 31) - 128, None) == bbs.BBS_EINVAL
    assert b"neither" in L.bbs_last_error()
