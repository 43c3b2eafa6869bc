"""What QGatedMLP makes and keeps for its backward pass, by which gradients are
wanted.  The kernels are replaced by recorders, so nothing runs on a GPU."""
import pytest

torch = pytest.importorskip("torch")

from bit_block_scaled_amd import layer as L                                 # noqa: E402

M, K, F = 64, 96, 128


@pytest.fixture
def calls(monkeypatch):
    """Transposed copies made (their rows) and checkpoints written."""
    seen = {"copies": [], "ckpt": 0}

    def quantize(x, row=None, col=None, *a, col_rht=False, **kw):
        assert col_rht == (col is not None)
        if col is not None:
            seen["copies"].append(col.rows)

    def gated(A, Wg, Wu, H, dt, act=0, g_ckpt=None, u_ckpt=None):
        assert (g_ckpt is None) == (u_ckpt is None)
        seen["ckpt"] += g_ckpt is not None
        H.zero_()

    monkeypatch.setattr(L, "nvfp4_quantize", quantize)
    monkeypatch.setattr(L, "nvfp4_gated_gemm", gated)
    monkeypatch.setattr(L, "nvfp4_gemm", lambda fmt, A, B, C, dt: C.zero_())
    monkeypatch.setattr(L, "mxfp8_requantize_t", lambda *a: None)
    monkeypatch.setattr(L, "mxfp8_gemm_gated_bwd", lambda *a, **kw: None)
    monkeypatch.setattr(L, "_on_current", lambda *a: 0)
    return seen


def block():
    return L.QGatedMLP(K, F, device="cpu")


def test_no_grad_makes_nothing_for_a_backward_pass(calls):
    b, x = block(), torch.zeros((M, K), dtype=torch.bfloat16)
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            y = b(x)
        assert not y.requires_grad and calls == {"copies": [], "ckpt": 0}
    for p in b.parameters():
        p.requires_grad_(False)
    assert not b(x).requires_grad and calls == {"copies": [], "ckpt": 0}


@pytest.mark.parametrize("need_x", [False, True])
@pytest.mark.parametrize("need_gu", [False, True])
@pytest.mark.parametrize("need_d", [False, True])
def test_only_what_the_gradients_read_is_kept(calls, need_x, need_gu, need_d):
    if not (need_x or need_gu or need_d):
        return
    b = block()
    b.w_gate_up.requires_grad_(need_gu)
    b.w_down.requires_grad_(need_d)
    x = torch.zeros((M, K), dtype=torch.bfloat16, requires_grad=need_x)
    y = b(x)
    assert calls["copies"] == [K] * need_gu + [F] * need_d
    assert calls["ckpt"] == (need_x or need_gu)
    kept = [t is not None for t in y.grad_fn.saved_tensors]
    h = need_x or need_gu
    assert kept == [need_gu] * 3 + [need_x] * 3 + [need_d] * 3 + [h] * 3 + [h] * 4
    y.backward(torch.zeros_like(y))
    assert [t.grad is not None for t in (x, b.w_gate_up, b.w_down)] == [need_x, need_gu, need_d]


def test_function_without_the_grad_argument(calls):
    """Seven arguments, as an own autograd graph may call it."""
    b = block()
    leaves = [t.detach().requires_grad_() for t in (torch.zeros((M, K), dtype=torch.bfloat16), *b.parameters())]
    y = L.QGatedMLPFn.apply(*leaves, 0, 1, 2, 3)
    g = torch.autograd.grad(y, leaves, torch.zeros_like(y))
    assert calls["ckpt"] == 1 and [t.shape for t in g] == [t.shape for t in leaves]
