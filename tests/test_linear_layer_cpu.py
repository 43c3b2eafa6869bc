"""What QLinear makes and keeps for its backward pass, by which gradients are
wanted, and what the layers on the linear and the expert operators refuse.  The
kernels are replaced by recorders, so nothing runs on a GPU."""
import pytest

torch = pytest.importorskip("torch")

from bit_block_scaled_amd import layer as L                                 # noqa: E402

M, K, N = 64, 96, 128


@pytest.fixture
def calls(monkeypatch):
    seen = {"copies": 0, "ckpt": 0, "plain": 0, "bwd": []}

    def quantize(x, row=None, col=None, row_mx8=None, *a, col_rht=False, **kw):
        assert col_rht == (col is not None)
        seen["copies"] += col is not None and row is not None

    def fused(A, B, out, dt, bias=None, act=2, residual=None, z_ckpt=None):
        seen["ckpt"] += z_ckpt is not None
        out.zero_()

    def bwd(dy, z8, act, dz=None, db=None):
        seen["bwd"].append((z8 is not None, dz is not None, db is not None))
        for t in (dz, db):
            if t is not None:
                t.zero_()

    def gemm(fmt, A, B, C, dt):
        seen["plain"] += 1
        C.zero_()

    for name, f in (("nvfp4_quantize", quantize), ("nvfp4_gemm_bias_act", fused), ("mxfp8_bias_act_bwd", bwd),
                    ("nvfp4_gemm", gemm), ("mxfp8_requantize_t", lambda *a: None), ("_on_current", lambda *a: 0)):
        monkeypatch.setattr(L, name, f)
    return seen


def bf(*shape, grad=False):
    return torch.zeros(shape, dtype=torch.bfloat16, requires_grad=grad)


def test_plain_layer_takes_the_plain_product(calls):
    L.QLinear(K, N, device="cpu")(bf(M, K))
    assert calls["plain"] == 1 and calls["ckpt"] == 0
    assert set(dict(L.QLinear(K, N, device="cpu").named_parameters())) == {"weight"}


def test_no_grad_makes_nothing_for_a_backward_pass(calls):
    m = L.QLinear(K, N, device="cpu", bias=True, act="gelu")
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            assert not m(bf(M, K)).requires_grad
    assert calls["copies"] == calls["ckpt"] == 0


@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("need", range(1, 16))
def test_only_what_the_gradients_read_is_kept(calls, act, need):
    need_x, need_w, need_b, need_r = (bool(need >> i & 1) for i in range(4))
    m = L.QLinear(K, N, device="cpu", bias=True, act=act, dtype=torch.float32)
    m.weight.requires_grad_(need_w), m.bias.requires_grad_(need_b)
    x, r = bf(M, K, grad=need_x), torch.zeros((M, N), requires_grad=need_r)
    y = m(x, r)
    z = act is not None and (need_x or need_w or need_b)
    assert calls["copies"] == need_w and calls["ckpt"] == z
    assert [t is not None for t in y.grad_fn.saved_tensors] == [need_w] * 3 + [need_x] * 3 + [z] * 2
    y.backward(torch.zeros_like(y))
    assert [t.grad is not None for t in (x, m.weight, m.bias, r)] == [need_x, need_w, need_b, need_r]
    assert all(t.grad is None or t.grad.dtype == t.dtype for t in (x, m.weight, m.bias, r))
    dz = act is not None and (need_x or need_w)
    assert calls["bwd"] == ([(act is not None, dz, need_b)] if dz or need_b else [])


def test_refusals(calls):
    for kw in ({"act": "relu"}, {"act": ""}):
        with pytest.raises(ValueError):
            L.QLinear(K, N, device="cpu", **kw)
    m = L.QLinear(K, N, device="cpu", act="silu")
    for a in ((bf(M, K), bf(M, K)), (bf(M, K), bf(1, M, N)), (bf(0, K),), (bf(30, K),), (bf(M, K + 32),)):
        with pytest.raises(ValueError):
            m(*a)
    for a in ((bf(N, K + 8),), (bf(N, K), bf(K)), (bf(N, K), None, "relu"), (bf(N),)):
        with pytest.raises(ValueError):
            L.QLinearInference(*a)
    E, F = 4, 32
    good = bf(E, F, K), bf(E, F, K), bf(E, N, F)
    for a in ((good[0], good[1], bf(E, F, N)), (good[0], good[1], bf(3, N, F)), (bf(E, F, 32), *good[1:]),
              (*good, "relu"), (*good, None), (None, bf(E, F, 40), bf(E, N, F)), (None, bf(0, F, K), bf(0, N, F))):
        with pytest.raises(ValueError):
            L.QMoEInference(*a)
    f = L.QMoEInference(*good)
    ids, x = torch.zeros((5, 2), dtype=torch.int64), bf(5, K)
    for a in ((bf(5, N), ids), (x, ids[:4]), (x, ids, torch.zeros(5, 3)), (x, ids.float()), (x, ids.bool()),
              (x, ids, None, bf(5, K))):
        with pytest.raises(ValueError):
            f(*a)


def test_refusals_of_host_memory():
    with pytest.raises(ValueError, match="GPU"):
        L.QLinear(K, N, device="cpu", bias=True)(bf(M, K))
    with pytest.raises(ValueError, match="GPU"):
        L.QLinearInference(bf(N, K))
    with pytest.raises(ValueError, match="GPU"):
        L.QMoEInference(None, bf(4, 32, K), bf(4, N, 32))
