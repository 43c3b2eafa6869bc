"""CPU checks of the linear layer's operators: argument errors come back before
anything is launched, from the C ABI and from the Python calls."""
import ctypes as C

import pytest

torch = pytest.importorskip("torch")

import bit_block_scaled_amd as bbs                                          # noqa: E402
from test_gated_bindings_cpu import bf, mx8, nv, refused                    # noqa: E402
from test_gated_cpu import fp4, mx8 as mx8_desc                             # noqa: E402

L = bbs.lib
P = C.c_void_p
EINVAL, ENOTSUP = bbs.BBS_EINVAL, bbs.BBS_ENOTSUP


def gemm(A=None, B=None, bias=None, bias_dtype=0, act=2, r=None, ldr=48, z8=None, out=0x4000, dt=1, ldc=48):
    A = fp4() if A is None else A
    B = fp4(48) if B is None else B
    return L.nvfp4_gemm_bias_act(C.byref(A), C.byref(B), P(bias), bias_dtype, act, P(r), ldr,
                                 C.byref(z8) if z8 is not None else None, P(out), dt, ldc, None)


def test_gemm_errors():
    assert L.nvfp4_gemm_bias_act(None, None, None, 0, 2, None, 0, None, P(0x4000), 1, 48, None) == EINVAL
    assert gemm(A=fp4(30)) == EINVAL
    assert gemm(A=fp4(0)) == EINVAL
    assert gemm(A=fp4(32, 32)) == EINVAL                                # K differs
    assert gemm(B=fp4(48, per_row=1)) == ENOTSUP
    for act in (-1, 3):
        assert gemm(act=act) == EINVAL
    assert gemm(dt=2) == EINVAL
    assert gemm(out=None) == EINVAL
    assert gemm(out=0x4008) == EINVAL
    assert gemm(ldc=32) == EINVAL
    assert gemm(ldc=52) == EINVAL
    assert gemm(bias=0x5008) == EINVAL
    assert b"bias not aligned" in L.bbs_last_error()
    assert gemm(bias=0x5000, bias_dtype=2) == EINVAL
    assert gemm(r=0x6008) == EINVAL
    assert gemm(r=0x6000, ldr=40) == EINVAL
    assert gemm(r=0x6000, ldr=52) == EINVAL
    assert b"residual must be" in L.bbs_last_error()
    assert gemm(z8=mx8_desc(32, 48)) == EINVAL                          # no whole number of 32-blocks
    assert gemm(B=fp4(64), ldc=64, z8=mx8_desc(16, 64)) == EINVAL
    assert gemm(B=fp4(64), ldc=64, z8=mx8_desc(32, 64, codes=0x1008)) == EINVAL
    K = 1 << 25
    assert gemm(A=fp4(32, K), B=fp4(48, K)) == ENOTSUP
    n = 1 << 27
    assert gemm(A=fp4(n), B=fp4(n), ldc=n) == ENOTSUP                   # 2^39 tiles


def bwd(dY=0x1000, rows=24, cols=96, ldy=96, z8=None, act=0, dZ=0x4000, ldz=96, db=0x5000, dt=0, ws=0x6000):
    z8 = mx8_desc(24, 96) if z8 is None else z8
    return L.mxfp8_bias_act_bwd(P(dY), rows, cols, ldy, C.byref(z8) if z8 else None, act, P(dZ), ldz, P(db), dt,
                                P(ws), None)


def test_bwd_errors():
    assert bwd(dY=None) == EINVAL
    assert bwd(dY=0x1008) == EINVAL
    assert bwd(rows=0) == EINVAL
    assert bwd(cols=0) == EINVAL
    assert bwd(cols=90) == EINVAL
    assert bwd(rows=1 << 31) == ENOTSUP
    assert bwd(act=3) == EINVAL
    assert bwd(act=-1) == EINVAL
    assert bwd(ldy=88) == EINVAL
    assert bwd(ldy=100) == EINVAL
    assert bwd(z8=False) == EINVAL
    assert bwd(z8=mx8_desc(24, 64)) == EINVAL
    assert bwd(z8=mx8_desc(32, 96)) == EINVAL
    assert bwd(z8=mx8_desc(24, 96, scales=None)) == EINVAL
    assert bwd(dZ=0x4008) == EINVAL
    assert bwd(ldz=90) == EINVAL
    assert bwd(db=0x5002) == EINVAL
    assert bwd(db=0x5001, dt=1) == EINVAL
    assert bwd(dt=2) == EINVAL
    assert bwd(ws=None) == EINVAL
    assert bwd(dZ=None, db=None) == EINVAL
    assert b"neither" in L.bbs_last_error()


def gemv(fmt=0, x=0x1000, T=1, ldx=64, W=None, bias=None, bias_dtype=0, act=2, r=None, ldr=48, y=0x4000, dt=1, ldy=48):
    W = fp4(48) if W is None else W
    return L.nvfp4_gemv_bias_act(fmt, P(x), T, ldx, C.byref(W), P(bias), bias_dtype, act, P(r), ldr, P(y), dt, ldy, None)


def test_gemv_errors():
    for T in (0, 65):
        assert gemv(T=T) == EINVAL
    assert gemv(act=3) == EINVAL
    assert gemv(act=-1) == EINVAL
    assert gemv(x=0x1008) == EINVAL
    assert gemv(y=0x4001) == EINVAL
    assert gemv(fmt=1) == EINVAL
    assert gemv(W=fp4(48, per_row=1)) == ENOTSUP
    assert gemv(bias=0x5001, bias_dtype=1) == EINVAL
    assert gemv(bias=0x5002) == EINVAL
    assert gemv(bias=0x5000, bias_dtype=7) == EINVAL
    assert gemv(r=0x6000, ldr=47) == EINVAL
    assert gemv(r=0x6001) == EINVAL
    assert gemv(r=0x6002, dt=0) == EINVAL


M, N, K = 32, 64, 96


def test_python_gemm():
    def call(match, out=None, dt=1, **kw):
        refused(match, bbs.nvfp4_gemm_bias_act, nv(M, K), nv(N, K), bf(M, N) if out is None else out, dt, **kw)
    call("GPU")
    call("GPU", bias=torch.zeros(N), residual=bf(M, N), z_ckpt=mx8(M, N))
    call("out must", dt=0)
    call("out must", out=bf(M, N - 8))
    call("out must", out=bf(N, M).t())
    call("out must", ldo=N + 8)
    call("bias must", bias=torch.zeros(N - 1))
    call("bias must", bias=torch.zeros(N + 1))
    call("bias must", bias=torch.zeros(N, dtype=torch.float16))
    call("bias must", bias=torch.zeros(2 * N)[::2])
    call("bias must", bias=torch.zeros((1, N)))
    call("residual must", residual=torch.zeros((M, N)))
    call("residual must", residual=bf(M - 1, N))
    call("residual must", residual=bf(1, N).expand(M, N)[:, ::2])
    call("residual must", residual=bf(M, N), ldr=N + 8)
    call("z_ckpt must", z_ckpt=mx8(M, N + 32))
    call("z_ckpt must", z_ckpt=nv(M, N))


def test_python_bwd():
    def call(match, dY=None, z8=None, act=0, **kw):
        refused(match, bbs.mxfp8_bias_act_bwd, bf(M, N) if dY is None else dY, mx8(M, N) if z8 is None else z8, act, **kw)
    call("GPU", dZ=bf(M, N), dbias=torch.zeros(N))
    call("dY must", dY=torch.zeros((M, N)))
    call("dY must", dY=bf(N, M).t())
    call("dZ must", dZ=bf(M, N - 8))
    call("dZ must", dZ=torch.zeros((M, N)))
    call("z_ckpt must", z8=mx8(M, N + 32), dZ=bf(M, N))
    call("dbias must", dbias=torch.zeros(N + 1))
    call("dbias must", dbias=torch.zeros(N, dtype=torch.float64))
    call("ws must", dbias=torch.zeros(N), ws=torch.zeros(bbs.BIAS_PARTS * N - 1))
    call("ws must", dbias=torch.zeros(N), ws=torch.zeros(bbs.BIAS_PARTS * N, dtype=torch.bfloat16))
    refused("needs z_ckpt", bbs.mxfp8_bias_act_bwd, bf(M, N), None, 0, bf(M, N))


def test_python_gemv():
    def call(match, x=None, y=None, dt=1, **kw):
        refused(match, bbs.nvfp4_gemv_bias_act, 0, bf(4, K) if x is None else x, nv(N, K), bf(4, N) if y is None else y,
                dt, **kw)
    call("GPU")
    call("^x must", x=torch.zeros((4, K)))
    call("output must", y=bf(4, N - 1))
    call("output must", dt=0)
