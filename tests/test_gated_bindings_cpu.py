"""The Python calls of the gated and the few-token operators, and their layers,
refuse tensors that the C ABI would take for something else: host memory,
another type, shapes too small, elements of a row that are not adjacent,
weights of another format.  Nothing is launched."""
import pytest

torch = pytest.importorskip("torch")

import bit_block_scaled_amd as bbs                                          # noqa: E402
from bit_block_scaled_amd import layer                                      # noqa: E402

M, F, K = 32, 64, 96


def nv(rows, cols, device="cpu"):
    return bbs.NVFP4Tensor.empty(rows, cols, device=device)


def mx8(rows, cols):
    return bbs.MXFP8Tensor.empty(rows, cols, device="cpu")


def refused(match, f, *a, **kw):
    with pytest.raises(ValueError, match=match):
        f(*a, **kw)


def bf(rows, cols):
    return torch.zeros((rows, cols), dtype=torch.bfloat16)


@pytest.mark.parametrize("gated", [False, True])
def test_few_token_calls(gated):
    def call(match, x=None, y=None, dt=1, W=None, fmt=0, **kw):
        x, y, W = bf(4, K) if x is None else x, bf(4, F) if y is None else y, nv(F, K) if W is None else W
        if gated:
            refused(match, bbs.nvfp4_gated_gemv, fmt, x, W, W, y, dt, **kw)
        else:
            refused(match, bbs.nvfp4_gemv, fmt, x, W, y, dt, **kw)
    call("GPU")                                                             # host memory
    call("^x must", x=torch.zeros((4, K)))
    call("^x must", x=torch.zeros((4, K), dtype=torch.float16))
    call("^x must", x=bf(4, K - 16))
    call("^x must", x=bf(4, 2 * K)[:, :K - 16])                             # rows far enough apart, but short
    call("unpack", x=torch.zeros(K, dtype=torch.bfloat16)[None, None])
    call("unpack", x=torch.zeros(K, dtype=torch.bfloat16))
    call("^x must", x=bf(4, 2 * K)[:, ::2])
    call("^x must", x=bf(K, 4).t())
    call("output must", y=torch.zeros((4, F)))
    call("output must", dt=0)
    call("output must", y=torch.zeros((4, F), dtype=torch.float16))
    call("output must", y=bf(3, F))
    call("output must", y=bf(4, F - 1))
    call("output must", y=bf(4, 2 * F)[:, ::2])
    call("output must", **{"ldh" if gated else "ldy": F + 1})
    call("format", fmt=2)
    call("format", W=bbs.MXFP4Tensor.empty(F, K, device="cpu"))
    call("format", W=mx8(F, K))
    call("format", W=mx8(F, K), fmt=bbs.FMT_MXFP8)
    if gated:
        refused("format", bbs.nvfp4_gated_gemv, 0, bf(4, K), nv(F, K), mx8(F, K), bf(4, F), 1)


def test_gated_gemm():
    def call(match, H=None, dt=1, **kw):
        refused(match, bbs.nvfp4_gated_gemm, nv(M, K), nv(F, K), nv(F, K), bf(M, F) if H is None else H, dt, **kw)
    call("GPU")
    call("GPU", g_ckpt=mx8(M, F), u_ckpt=mx8(M, F))
    call("H must", dt=0)
    call("H must", H=torch.zeros((M, F)))
    call("H must", H=bf(M - 1, F))
    call("H must", H=bf(M, F - 8))
    call("H must", H=bf(F, M).t())
    call("H must", ldh=F + 8)


def test_gated_bwd():
    def call(match, dG=None, dU=None, dt=1, **kw):
        refused(match, bbs.mxfp8_gemm_gated_bwd, mx8(M, K), mx8(F, K), mx8(M, F), mx8(M, F),
                bf(M, F) if dG is None else dG, bf(M, F) if dU is None else dU, dt, **kw)
    call("GPU")
    call("dG must", dt=0)
    call("dU must", dU=torch.zeros((M, F)))
    call("dG must", dG=bf(M - 1, F))
    call("dU must", dU=bf(M, F - 8))
    call("dU must", dU=bf(M, 2 * F)[:, ::2])
    call("row stride", dU=bf(M, 2 * F)[:, :F])
    call("dU must", dG=bf(M, F + 8), ld=F + 8)


def test_layers():
    b = layer.QGatedMLP(64, 96, device="cpu")
    refused("GPU", b, bf(32, 64))
    refused("GPU", b.inference)
    refused("GPU", layer.QGatedMLPInference, b.w_gate_up.detach(), b.w_down.detach())


def test_packed_descriptors():
    for t in (nv(F, K), bbs.NVFP4Tensor.empty(F, K, tile2d=True, device="cpu"),
              bbs.NVFP4Tensor.empty(F, K, device="cpu", sdec_per_row=True),
              bbs.MXFP4Tensor.empty(F, K, device="cpu")):
        assert t.packed() == bytes(t.desc())
