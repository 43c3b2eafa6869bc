"""The gated feed-forward block (bit_block_scaled_amd.layer.QGatedMLP and
QGatedMLPInference): the operators in their training and serving sequence."""
import numpy as np
import pytest

import oracle as O
from gated_ref import act64, act_slope64
from gpu_util import announce, bf16_bits_to_f64, dev, host, to_dev
from workloads import synth

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

SEED, SIGNS = 0x77A1, 0x5A3C


@pytest.fixture(scope="module")
def L():
    import bit_block_scaled_amd.layer as m
    return m


def _block(L, M, K, F, act, dtype=torch.bfloat16, step=0):
    b = L.QGatedMLP(K, F, act=act, seed=SEED, rht_signs=SIGNS, device=dev(), dtype=dtype)
    wb, db, xb, gb = (synth.normal(2 * F, K, 1, K ** -0.5), synth.normal(K, F, 2, F ** -0.5),
                      synth.normal_with_outliers(M, K, 3), synth.laplace(M, K, 4, 1e-2))
    with torch.no_grad():
        b.w_gate_up.copy_(to_dev(wb).view(torch.bfloat16))
        b.w_down.copy_(to_dev(db).view(torch.bfloat16))
    b.step = step
    x = to_dev(xb).view(torch.bfloat16).reshape(2, M // 2, K).requires_grad_(True)
    dy = to_dev(gb).view(torch.bfloat16).reshape(2, M // 2, K)
    return b, x, dy, [bf16_bits_to_f64(v) for v in (wb, db, xb, gb)]


def _f64(t):
    return host(t.detach().double())


@pytest.mark.parametrize("M,K,F,act,dtype", [(64, 96, 160, "gelu", torch.bfloat16),
                                             (256, 512, 384, "silu", torch.bfloat16),
                                             (128, 256, 256, "silu", torch.float32)])
def test_block_against_the_unquantized_block(L, M, K, F, act, dtype):
    """Output and gradients against the same block in 64 bits.  Each NVFP4 operand
    is off by about 10% of its norm (14% stochastic, as the published figures),
    each MXFP8 one by 4%, independently: a product of two NVFP4 operands by 14%,
    H by both products (20%) and Y, with H and Wd quantized again, by 25%; dW, of
    two stochastic copies whose own inputs are off by up to 25%, by 35%.  Twice
    that is far from what a wrong formula gives (a missing factor: 100%)."""
    announce(f"QGatedMLP {M}x{K}x{F} {act} {dtype}")
    b, x, dy, (w, d, xv, gv) = _block(L, M, K, F, act, dtype)
    y = b(x)
    y.backward(dy)
    torch.cuda.synchronize()
    assert b.step == 1 and y.shape == x.shape and y.dtype == torch.bfloat16
    assert x.grad.shape == x.shape and b.w_gate_up.grad.dtype == dtype and b.w_down.grad.dtype == dtype
    g, u = xv @ w[:F].T, xv @ w[F:].T
    h = act64(act, g) * u
    dh = gv @ d
    dgu = np.concatenate([dh * u * act_slope64(act, g), dh * act64(act, g)], 1)
    for name, got, ref, tol in (("y", y.reshape(M, K), h @ d.T, 0.5), ("dx", x.grad.reshape(M, K), dgu @ w, 0.5),
                                ("dw_down", b.w_down.grad, gv.T @ h, 0.7),
                                ("dw_gate_up", b.w_gate_up.grad, dgu.T @ xv, 0.7)):
        err = O.rel_fro(_f64(got), ref)
        print(f"  {name}: {err:.3f}", flush=True)
        assert err <= tol, name


def test_block_is_the_sequence_of_the_operators(L):
    """Bit for bit the public calls in their order, with Philox streams 8t .. 8t + 7."""
    import bit_block_scaled_amd as bbs
    announce("QGatedMLP as the sequence of calls")
    M, K, F, t = 128, 256, 288, 5
    b, x, dy, _ = _block(L, M, K, F, "silu", step=t)
    y = b(x)
    y.backward(dy)
    new4 = lambda r, c, tile=False: bbs.NVFP4Tensor.empty(r, c, tile2d=tile, device=dev())   # noqa: E731
    new8 = lambda r, c: bbs.MXFP8Tensor.empty(r, c, device=dev())                            # noqa: E731
    bf = lambda r, c: torch.empty((r, c), dtype=torch.bfloat16, device=dev())                # noqa: E731
    bits = lambda v: v.detach().reshape(-1, v.shape[-1]).view(torch.int16)                   # noqa: E731
    xq, xc, wq, hq, hc, dq = new4(M, K), new4(K, M), new4(2 * F, K, True), new4(M, F), new4(F, M), new4(K, F, True)
    kw = dict(col_round=1, col_rht=True, rht_signs=SIGNS)
    bbs.nvfp4_quantize(bits(x), xq, xc, col_rng=(SEED, 8 * t), **kw)
    bbs.nvfp4_quantize(bits(b.w_gate_up), wq, tile2d=True)
    bbs.nvfp4_quantize(bits(b.w_down), dq, tile2d=True)
    gate = bbs.NVFP4Tensor(wq.codes[:F], wq.scales[:F // 16], wq.s_dec, F, K, True)
    up = bbs.NVFP4Tensor(wq.codes[F:], wq.scales[F // 16:], wq.s_dec, F, K, True)
    h, g8, u8 = bf(M, F), new8(M, F), new8(M, F)
    bbs.nvfp4_gated_gemm(xq, gate, up, h, 1, g_ckpt=g8, u_ckpt=u8)
    bbs.nvfp4_quantize(bits(h), hq, hc, col_rng=(SEED, 8 * t + 1), **kw)
    yy = bf(M, K)
    bbs.nvfp4_gemm(0, hq, dq, yy, 1)
    yc, ym, wdt, dgu = new4(K, M), new8(M, K), new8(F, K), bf(M, 2 * F)
    bbs.nvfp4_quantize(bits(dy), None, yc, ym, col_rng=(SEED, 8 * t + 2), mx8_round=1, mx8_rng=(SEED, 8 * t + 3), **kw)
    bbs.mxfp8_requantize_t(dq, wdt, 1, (SEED, 8 * t + 4))
    bbs.mxfp8_gemm_gated_bwd(ym, wdt, g8, u8, dgu[:, :F], dgu[:, F:], 1)
    gc, gm, wt = new4(2 * F, M), new8(M, 2 * F), new8(K, 2 * F)
    bbs.nvfp4_quantize(bits(dgu), None, gc, gm, col_rng=(SEED, 8 * t + 5), mx8_round=1, mx8_rng=(SEED, 8 * t + 6), **kw)
    bbs.mxfp8_requantize_t(wq, wt, 1, (SEED, 8 * t + 7))
    dx, dwd, dwgu = bf(M, K), bf(K, F), bf(2 * F, K)
    bbs.nvfp4_gemm(1, gm, wt, dx, 1)
    bbs.nvfp4_gemm(0, yc, hc, dwd, 1)
    bbs.nvfp4_gemm(0, gc, xc, dwgu, 1)
    torch.cuda.synchronize()
    for name, a, c in (("y", y, yy), ("dx", x.grad, dx), ("dw_down", b.w_down.grad, dwd),
                       ("dw_gate_up", b.w_gate_up.grad, dwgu)):
        assert torch.equal(a.detach().reshape(c.shape), c), name


def test_block_without_some_gradients(L):
    """Frozen weights and inputs: the other gradients are the same bits."""
    announce("QGatedMLP partial gradients")
    M, K, F = 64, 128, 96
    full, x, dy, _ = _block(L, M, K, F, "silu")
    full(x).backward(dy)
    part, xp, dyp, _ = _block(L, M, K, F, "silu")
    part.w_gate_up.requires_grad_(False)
    xp = xp.detach()
    y = part(xp)
    y.backward(dyp)
    assert part.w_gate_up.grad is None and torch.equal(part.w_down.grad, full.w_down.grad)
    with torch.no_grad():
        part.step = 0
        assert torch.equal(part(xp), y.detach())


@pytest.mark.parametrize("T", [0, 1, 5, 16, 33, 64, 65, 100, 160])
def test_inference(L, T):
    """Any number of tokens against the block in 64 bits over the quantized weights:
    with BF16 activations only H and Y are rounded (2^-9 each, times the norms'
    share of cancellation); beyond 64 tokens X and H are NVFP4 too (10% each, X
    twice)."""
    announce(f"QGatedMLPInference {T} tokens")
    K, F = 224, 320
    b, _, _, (w, d, _, _) = _block(L, 64, K, F, "gelu")
    inf = b.inference()
    with torch.no_grad():
        b.w_gate_up.zero_()                                  # the object has its own weights
    xb = synth.normal_with_outliers(max(T, 1), K, 9)[:T]
    x = to_dev(xb).view(torch.bfloat16).reshape(T, 1, K)
    y = inf(x)
    torch.cuda.synchronize()
    assert y.shape == (T, 1, K) and y.dtype == torch.bfloat16
    if T == 0:
        return
    xv = bf16_bits_to_f64(xb)
    wq = O.nvfp4_quantize(synth.normal(2 * F, K, 1, K ** -0.5), tile2d=True).dequant_f64()
    dq = O.nvfp4_quantize(synth.normal(K, F, 2, F ** -0.5), tile2d=True).dequant_f64()
    ref = (act64("gelu", xv @ wq[:F].T) * (xv @ wq[F:].T)) @ dq.T
    err = O.rel_fro(_f64(y).reshape(T, K), ref)
    print(f"  rel {err:.2e}", flush=True)
    assert err <= (4 * 2.0 ** -9 if T <= 64 else 0.4)


def test_block_and_inference_in_a_graph(L):
    """Forward and backward passes of one training step, and the inference form
    with few and with many tokens, captured and replayed: the eager bits, with
    other eager work between the replays."""
    announce("QGatedMLP captured")
    M, K, F = 96, 256, 288
    b, x, dy, _ = _block(L, M, K, F, "silu")
    inf = b.inference()
    xs = [x.detach().reshape(-1, K)[:T].clone() for T in (7, 80)]

    def run(out):
        with torch.no_grad():
            out["inf"] = [inf(v) for v in xs]
        leaves = [t.detach().requires_grad_() for t in (x, b.w_gate_up, b.w_down)]
        y = L.QGatedMLPFn.apply(*leaves, 0, SEED, 3, SIGNS)
        out["train"] = [y.detach(), *torch.autograd.grad(y, leaves, dy)]

    eager, cap = {}, {}
    run(eager)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run({})
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(cap)
    for r in range(4):
        with torch.no_grad():
            x.copy_(torch.roll(x, 1, -1))
            for v in xs:
                v.copy_(torch.roll(v, 3, -1))
        graph.replay()
        run(eager)
        torch.cuda.synchronize()
        for k in eager:
            assert all(torch.equal(p, q) for p, q in zip(eager[k], cap[k])), (r, k)


def test_block_with_an_expanded_gradient_and_a_padded_input(L):
    """dy of one element (y.sum()), x a slice of a wider tensor: the bits of the dense tensors."""
    announce("QGatedMLP strides")
    M, K, F = 64, 128, 96
    got = []
    for dense in (True, False):
        b, x, _, _ = _block(L, M, K, F, "gelu")
        wide = torch.zeros((*x.shape[:-1], K + 16), dtype=x.dtype, device=x.device)
        wide[..., :K] = x.detach()
        xi = x.detach().clone().requires_grad_() if dense else wide[..., :K].requires_grad_()
        y = b(xi)
        one = torch.ones((), dtype=y.dtype, device=y.device).expand(y.shape)
        y.backward(one.contiguous() if dense else one)
        got.append((y.detach(), xi.grad, b.w_gate_up.grad, b.w_down.grad))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(*got))


def test_refusals(L):
    with pytest.raises(ValueError):
        L.QGatedMLP(64, 48, device=dev())
    with pytest.raises(ValueError):
        L.QGatedMLP(64, 64, act="relu", device=dev())
    b = L.QGatedMLP(64, 64, device=dev())
    for shape in ((32, 32), (16, 64), (0, 64)):
        with pytest.raises(ValueError):
            b(torch.zeros(shape, dtype=torch.bfloat16, device=dev()))
    with pytest.raises(ValueError):
        L.QGatedMLPInference(b.w_gate_up.detach(), b.w_down.detach()[:, :32])
    with pytest.raises(ValueError):
        b.inference()(torch.zeros((3, 48), dtype=torch.bfloat16, device=dev()))
