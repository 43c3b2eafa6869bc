"""CPU checks of the expert layer for a few tokens: argument errors come back
before anything is launched, from the C ABI and from the Python call."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")

import bit_block_scaled_amd as bbs                                          # noqa: E402
from test_gated_bindings_cpu import bf, mx8, refused                        # noqa: E402
from test_gated_cpu import fp4                                              # noqa: E402

L = bbs.lib
P = C.c_void_p
EINVAL, ENOTSUP = bbs.BBS_EINVAL, bbs.BBS_ENOTSUP


def mx4(rows, cols, scales=0x2000):
    return bbs.Mx4Desc(0x1000, scales, rows, cols)


# four experts, 64 features in, 32 hidden, 48 out
def call(fmt=0, x=0x1000, T=2, ldx=64, ids=0x1000, w=0x1000, k=2, E=4, Wg=None, Wu=None, Wd=None, gated=True, act=0,
         r=None, ldr=48, ws=0x1000, y=0x4000, dt=1, ldy=48):
    Wg, Wu, Wd = (d if d is not None else n for d, n in ((Wg, fp4(128)), (Wu, fp4(128)), (Wd, fp4(192, 32))))
    return L.nvfp4_moe_gemv(fmt, P(x), T, ldx, P(ids), P(w), k, E, C.byref(Wg) if gated else None,
                            C.byref(Wu) if Wu else None, C.byref(Wd) if Wd else None, act, P(r), ldr, P(ws), P(y), dt, ldy,
                            None)


def test_errors():
    for name in ("x", "ids", "ws", "y"):
        assert call(**{name: None}) == EINVAL
    assert call(x=0x1008) == EINVAL
    assert call(ws=0x1008) == EINVAL
    assert call(ids=0x1002) == EINVAL
    assert call(w=0x1002) == EINVAL
    assert call(y=0x4001) == EINVAL
    assert call(y=0x4002, dt=0) == EINVAL
    assert call(dt=2) == EINVAL
    assert call(ldy=47) == EINVAL
    assert call(r=0x5000, ldr=47) == EINVAL
    assert call(r=0x5001) == EINVAL
    for T in (0, 65):
        assert call(T=T) == EINVAL
    for k in (0, 33):
        assert call(k=k) == EINVAL
    for E in (0, -4, 1025):
        assert call(E=E) == EINVAL
    assert call(ldx=56) == EINVAL
    assert call(ldx=68) == EINVAL
    for act in (-1, 2, 3):                                              # gated experts need an activation
        assert call(act=act) == EINVAL
    assert call(act=3, gated=False) == EINVAL
    assert call(fmt=1) == EINVAL
    assert call(Wu=False) == EINVAL
    assert call(Wd=False) == EINVAL
    assert call(E=3) == EINVAL                                          # 128 rows among three experts
    assert call(E=16) == EINVAL                                         # 8 rows each
    assert call(Wg=fp4(192)) == EINVAL                                  # shapes differ
    assert call(Wu=fp4(128, 32), Wg=fp4(128, 64)) == EINVAL
    assert call(Wd=fp4(192, 64)) == EINVAL                              # not the hidden rows
    assert b"hidden rows" in L.bbs_last_error()
    assert call(Wu=fp4(128, per_row=1)) == ENOTSUP
    assert call(Wg=fp4(128, tile2d=1)) == ENOTSUP
    assert call(Wd=fp4(192, 32, tile2d=1)) == ENOTSUP
    n = 1 << 24
    assert call(Wg=fp4(4 * n), Wu=fp4(4 * n), Wd=fp4(192, n)) == ENOTSUP
    assert call(Wg=fp4(128, n), Wu=fp4(128, n), ldx=n) == ENOTSUP
    assert call(Wd=fp4(4 * n, 32), ldy=n, ldr=n) == ENOTSUP
    m = dict(fmt=2, Wg=mx4(128, 64), Wu=mx4(128, 64), Wd=mx4(192, 32))
    assert call(**{**m, "Wu": mx4(128, 64, scales=None)}) == EINVAL
    assert call(**{**m, "Wd": mx4(190, 32)}) == EINVAL
    assert call(**{**m, "Wu": mx4(128, 48)}) == EINVAL


def test_workspace_size():
    size = L.nvfp4_moe_ws_bytes
    assert size(1, 8, 64, 1536, 4096) >= 3 * 8 * 1536 * 2
    assert size(64, 32, 1024, 1536, 4096) % 4 == 0
    for a in ((0, 8, 64, 64, 64), (65, 8, 64, 64, 64), (1, 0, 64, 64, 64), (1, 33, 64, 64, 64), (1, 8, 0, 64, 64),
              (1, 8, 1025, 64, 64), (1, 8, 64, 0, 64), (1, 8, 64, 1 << 24, 64), (1, 8, 64, 64, 0), (1, 8, 64, 64, 1 << 24)):
        assert size(*a) == EINVAL
    assert bbs.moe_workspace(2, 2, 4, 32, 48, "cpu").numel() == size(2, 2, 4, 32, 48)
    with pytest.raises(bbs.BbsError):
        bbs.moe_workspace(65, 2, 4, 32, 48, "cpu")


T, k, E, K, F, N = 3, 2, 4, 64, 32, 48


def stack(rows, cols, scales=E):
    return bbs.NVFP4Tensor.empty(E * rows, cols, device="cpu", n_scales=scales)


def test_python_call():
    def moe(match, x=None, ids=None, w=None, Wg=None, Wu=None, Wd=None, y=None, dt=1, fmt=0, experts=E, **kw):
        refused(match, bbs.nvfp4_moe_gemv, fmt, bf(T, K) if x is None else x,
                torch.zeros((T, k), dtype=torch.int32) if ids is None else ids, torch.zeros((T, k)) if w is None else w, experts,
                stack(F, K) if Wg is None else Wg, stack(F, K) if Wu is None else Wu, stack(N, F) if Wd is None else Wd,
                bf(T, N) if y is None else y, dt, **kw)
    moe("GPU")
    moe("experts must", experts=0)
    moe("experts must", experts=1025)
    moe("^x must", x=torch.zeros((T, K)))
    moe("^x must", x=bf(T, K - 16))
    moe("^x must", x=bf(T, 2 * K)[:, ::2])
    moe("ids must", ids=torch.zeros((T, k), dtype=torch.int64))
    moe("ids must", ids=torch.zeros((T + 1, k), dtype=torch.int32))
    moe("ids must", ids=torch.zeros((k, T), dtype=torch.int32).t())
    moe("ids must", ids=torch.zeros((T,), dtype=torch.int32))
    moe("weights must", w=torch.zeros((T, k), dtype=torch.bfloat16))
    moe("weights must", w=torch.zeros((T, k + 1)))
    moe("weights must", w=torch.zeros((k, T)).t())
    moe("decode scale", Wu=stack(F, K, 1))
    moe("decode scale", Wd=stack(N, F, E + 1))
    moe("format", fmt=2)
    moe("format", Wd=mx8(E * N, F))
    moe("format", Wg=bbs.MXFP4Tensor.empty(E * F, K, device="cpu"))
    moe("y must", y=bf(T, N - 1))
    moe("y must", dt=0)
    moe("residual must", residual=torch.zeros((T, N)))
    moe("residual must", residual=bf(T - 1, N))
    moe("ws must", ws=torch.empty(16, dtype=torch.uint8))
    moe("ws must", ws=torch.empty(1 << 16))
