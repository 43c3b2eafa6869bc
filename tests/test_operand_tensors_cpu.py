"""The tensors that an operand of the linear layer's operators and of the expert layer
consists of: all of them are on the GPU of the call, and a checkpoint's hold its rows.  A
kernel that is given host memory, or less memory than its sizes say, faults."""
import pytest

torch = pytest.importorskip("torch")

import bit_block_scaled_amd as bbs                                          # noqa: E402
from test_gated_bindings_cpu import bf, mx8, nv, refused                    # noqa: E402

M, N, K, E = 32, 64, 96, 4


class Looked(Exception):
    pass


@pytest.fixture
def looked(monkeypatch):
    """The tensors whose device a call looks at; it ends there."""
    seen = []

    def on_current(stream, *tensors):
        seen.extend(id(t) for t in tensors)
        raise Looked

    monkeypatch.setattr(bbs, "_on_current", on_current)
    return seen


def parts(*operands):
    return [t for q in operands for t in (q.codes, q.scales, getattr(q, "s_dec", None)) if t is not None]


def check(looked, tensors, call, *a, **kw):
    with pytest.raises(Looked):
        call(*a, **kw)
    assert {id(t) for t in tensors} <= set(looked)


def test_gemm_operands(looked):
    A, W, z8, b, r, y = nv(M, K), nv(N, K), mx8(M, N), torch.zeros(N), bf(M, N), bf(M, N)
    check(looked, [*parts(A, W, z8), b, r, y], bbs.nvfp4_gemm_bias_act, A, W, y, 1, bias=b, residual=r, z_ckpt=z8)


def test_bwd_operands(looked):
    z8, dy, dz, db, ws = mx8(M, N), bf(M, N), bf(M, N), torch.zeros(N), torch.zeros(bbs.BIAS_PARTS * N)
    check(looked, [*parts(z8), dy, dz, db, ws], bbs.mxfp8_bias_act_bwd, dy, z8, 0, dz, db, ws)


@pytest.mark.parametrize("fmt", [bbs.FMT_NVFP4, bbs.FMT_MXFP4])
def test_moe_operands(looked, fmt):
    def stack(rows, cols):
        if fmt == bbs.FMT_MXFP4:
            return bbs.MXFP4Tensor.empty(E * rows, cols, device="cpu")
        return bbs.NVFP4Tensor.empty(E * rows, cols, device="cpu", n_scales=E)

    F, T = 32, 3
    W = [stack(F, K), stack(F, K), stack(N, F)]
    x, ids, w, y, r = bf(T, K), torch.zeros((T, 2), dtype=torch.int32), torch.zeros((T, 2)), bf(T, N), bf(T, N)
    ws = bbs.moe_workspace(T, 2, E, F, N, "cpu")
    check(looked, [*parts(*W), x, ids, w, y, r, ws], bbs.nvfp4_moe_gemv, fmt, x, ids, w, E, *W, y, 1, residual=r, ws=ws)


class OnDevice:
    """A weight's tensor that says where it is."""

    def __init__(self, device):
        self.device = device

    def get_device(self):
        return self.device


@pytest.mark.parametrize("part", ["codes", "scales", "s_dec"])
def test_gemv_operands(monkeypatch, part):
    W = nv(N, K)
    for name in ("codes", "scales", "s_dec"):
        setattr(W, name, OnDevice(-1 if name == part else 0))
    x, y = bf(2, K), bf(2, N)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(bbs, "_device", lambda: 0)
    monkeypatch.setattr(bbs, "_raw_stream", lambda dev: 0)
    refused("one GPU", bbs.nvfp4_gemv_bias_act, 0, x, W, y, 1)


def test_checkpoint_holds_its_rows():
    def ckpt(codes=None, scales=None):
        t = mx8(M, N)
        return bbs.MXFP8Tensor(t.codes if codes is None else codes, t.scales if scales is None else scales, M, N)

    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)                       # noqa: E731
    for bad in (ckpt(codes=u8(M - 1, N)), ckpt(codes=u8(M, 2 * N)[:, :N]), ckpt(codes=torch.zeros(M, N)),
                ckpt(scales=u8(M, N // 32 - 1)), ckpt(scales=u8(M, N // 16)[:, ::2]), ckpt(scales=torch.zeros(M, N // 32))):
        refused("z_ckpt must", bbs.nvfp4_gemm_bias_act, nv(M, K), nv(N, K), bf(M, N), 1, z_ckpt=bad)
        refused("z_ckpt must", bbs.mxfp8_bias_act_bwd, bf(M, N), bad, 0, bf(M, N))
    e4m3 = ckpt(codes=torch.zeros((M, N), dtype=torch.float8_e4m3fn), scales=u8(M * N // 32 + 5))
    for good in (ckpt(), e4m3, ckpt(codes=u8(2 * M, N))):                   # larger ones, and any type of a byte
        refused("GPU", bbs.nvfp4_gemm_bias_act, nv(M, K), nv(N, K), bf(M, N), 1, z_ckpt=good)
        refused("GPU", bbs.mxfp8_bias_act_bwd, bf(M, N), good, 0, bf(M, N))


@pytest.mark.parametrize("bad", [lambda: torch.zeros(E, dtype=torch.float64), lambda: torch.zeros(2 * E)[::2]])
def test_moe_decode_scales(bad):
    F, T = 32, 3
    W = [bbs.NVFP4Tensor.empty(E * r, c, device="cpu", n_scales=E) for r, c in ((F, K), (F, K), (N, F))]
    for i in range(3):
        mine = list(W)
        mine[i] = bbs.NVFP4Tensor(W[i].codes, W[i].scales, bad(), W[i].rows, W[i].cols, False)
        refused("decode scale", bbs.nvfp4_moe_gemv, 0, bf(T, K), torch.zeros((T, 2), dtype=torch.int32), None, E, *mine,
                bf(T, N), 1)
