"""The layers on the linear and the expert operators: QLinear with bias, activation
and residual, QLinearInference and QMoEInference."""
import numpy as np
import pytest

import oracle as O
from gated_ref import act64, act_slope64
from gpu_util import announce, bf16_bits_to_f64, dev, host, to_dev
from test_gpu_gated import nv64, within
from test_gpu_linear import activated, normal, product_t, with_bias
from test_gpu_moe import layer64
from workloads import synth

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

SEED, SIGNS = 0x77A1, 0x5A3C


@pytest.fixture(scope="module")
def L():
    import bit_block_scaled_amd.layer as m
    return m


def make(L, M, K, N, act, bias, dtype=torch.bfloat16, step=0):
    m = L.QLinear(K, N, seed=SEED, rht_signs=SIGNS, device=dev(), dtype=dtype, bias=bias, act=act)
    wb, xb, gb = synth.normal(N, K, 1, K ** -0.5), synth.normal_with_outliers(M, K, 2), synth.laplace(M, N, 3, 1e-2)
    bb, rb = synth.normal(1, N, 4, 0.5), synth.normal(M, N, 5, 1.0)
    bits = lambda b: to_dev(b).view(torch.bfloat16)                      # noqa: E731
    with torch.no_grad():
        m.weight.copy_(bits(wb))
        if bias:
            m.bias.copy_(bits(bb)[0])
    m.step = step
    x = bits(xb).reshape(2, M // 2, K).requires_grad_(True)
    r = bits(rb).reshape(2, M // 2, N).requires_grad_(True)
    dy = bits(gb).reshape(2, M // 2, N)
    return m, x, r, dy, [bf16_bits_to_f64(v) for v in (wb, xb, gb, bb, rb)]


@pytest.mark.parametrize("M,K,N,act,bias,res,dtype", [
    (64, 96, 160, "gelu", True, True, torch.bfloat16), (256, 512, 384, "silu", True, False, torch.bfloat16),
    (128, 256, 256, None, True, True, torch.float32), (96, 128, 64, "gelu", False, True, torch.float32),
    (1024, 512, 4096, None, False, True, torch.bfloat16)])
def test_layer_against_the_unquantized_layer(L, M, K, N, act, bias, res, dtype):
    """Output and gradients against the same layer in 64 bits.  Each NVFP4 operand is
    off by about 10% of its norm (14% stochastic), each MXFP8 one by 4%,
    independently: a product of two NVFP4 operands by 14%, dW, of two stochastic
    copies whose own inputs are off by up to 14%, by 25%; db is a sum of exact dY
    times slopes at an argument that is off by 14%.  Twice that is far from what a
    wrong formula gives (a missing factor: 100%)."""
    announce(f"QLinear {M}x{K}x{N} {act} bias={bias} residual={res} {dtype}")
    m, x, r, dy, (w, xv, g, b, rv) = make(L, M, K, N, act, bias, dtype)
    y = m(x, r) if res else m(x)
    y.backward(dy)
    torch.cuda.synchronize()
    assert m.step == 1 and y.shape == dy.shape and y.dtype == torch.bfloat16
    z = xv @ w.T + (b if bias else 0)
    dz = g * act_slope64(act, z) if act else g
    v = act64(act, z) if act else z
    got = [("y", y.reshape(M, N), v + (rv if res else 0), 0.3), ("dx", x.grad.reshape(M, K), dz @ w, 0.3),
           ("dw", m.weight.grad, dz.T @ xv, 0.5)]
    if bias:
        assert m.bias.grad.dtype == dtype
        got.append(("db", m.bias.grad, dz.sum(0), 0.3))
    if res:
        assert torch.equal(r.grad, dy)
    for name, a, ref, tol in got:
        err = O.rel_fro(host(a.detach().double()), ref)
        print(f"  {name}: {err:.3f}", flush=True)
        assert err <= tol, name


@pytest.mark.parametrize("act,bias,res", [("gelu", True, True), (None, True, False), ("silu", False, False),
                                          (None, False, True)])
def test_layer_is_the_sequence_of_the_operators(L, act, bias, res):
    """Bit for bit the public calls in their order, with Philox streams 4t .. 4t + 3."""
    import bit_block_scaled_amd as bbs
    announce(f"QLinear as the sequence of calls {act} bias={bias} residual={res}")
    M, K, N, t = 128, 256, 288, 5
    m, x, r, dy, _ = make(L, M, K, N, act, bias, step=t)
    y = m(x, r) if res else m(x)
    y.backward(dy)
    code = {None: bbs.ACT_NONE, "silu": bbs.ACT_SILU, "gelu": bbs.ACT_GELU}[act]
    new4 = lambda a, c, tile=False: bbs.NVFP4Tensor.empty(a, c, tile2d=tile, device=dev())   # noqa: E731
    new8 = lambda a, c: bbs.MXFP8Tensor.empty(a, c, device=dev())                            # noqa: E731
    bf = lambda a, c: torch.empty((a, c), dtype=torch.bfloat16, device=dev())                # noqa: E731
    bits = lambda v: v.detach().reshape(-1, v.shape[-1]).view(torch.int16)                   # noqa: E731
    kw = dict(col_round=1, col_rht=True, rht_signs=SIGNS)
    xq, xc, wq = new4(M, K), new4(K, M), new4(N, K, True)
    bbs.nvfp4_quantize(bits(x), xq, xc, col_rng=(SEED, 4 * t), **kw)
    bbs.nvfp4_quantize(bits(m.weight), wq, tile2d=True)
    yy, z8 = bf(M, N), new8(M, N) if act else None
    bbs.nvfp4_gemm_bias_act(xq, wq, yy, 1, bias=m.bias.detach() if bias else None, act=code,
                            residual=r.detach().reshape(M, N) if res else None, z_ckpt=z8)
    g, db = dy.reshape(M, N), torch.empty((N,), dtype=torch.bfloat16, device=dev())
    dz = bf(M, N) if act else g
    bbs.mxfp8_bias_act_bwd(g, z8, code, dz if act else None, db)
    gc, gm, wt = new4(N, M), new8(M, N), new8(K, N)
    bbs.nvfp4_quantize(bits(dz), None, gc, gm, col_rng=(SEED, 4 * t + 1), mx8_round=1, mx8_rng=(SEED, 4 * t + 2), **kw)
    bbs.mxfp8_requantize_t(wq, wt, 1, (SEED, 4 * t + 3))
    dx, dw = bf(M, K), bf(N, K)
    bbs.nvfp4_gemm(1, gm, wt, dx, 1)
    bbs.nvfp4_gemm(0, gc, xc, dw, 1)
    torch.cuda.synchronize()
    pairs = [("y", y, yy), ("dx", x.grad, dx), ("dw", m.weight.grad, dw)] + ([("db", m.bias.grad, db)] if bias else [])
    for name, a, c in pairs:
        assert torch.equal(a.detach().reshape(c.shape), c), name


def test_plain_layer_keeps_its_bits(L):
    """A layer without bias, activation and residual and one whose bias is zero: the same gradients."""
    announce("QLinear without and with a zero bias")
    M, K, N = 1024, 256, 4096                                           # both products on the large tiles
    a, x, _, dy, _ = make(L, M, K, N, None, False)
    b, x2, _, _, _ = make(L, M, K, N, None, True)
    with torch.no_grad():
        b.bias.zero_()
    y, z = a(x), b(x2)
    y.backward(dy), z.backward(dy)
    assert torch.equal(y, z) and torch.equal(x.grad, x2.grad) and torch.equal(a.weight.grad, b.weight.grad)


def test_layer_without_some_gradients(L):
    """Frozen inputs and parameters: the other gradients are the same bits."""
    announce("QLinear partial gradients")
    M, K, N = 64, 128, 96
    m, x, r, dy, _ = make(L, M, K, N, "silu", True)
    m(x, r).backward(dy)
    want = {"x": x.grad, "w": m.weight.grad, "b": m.bias.grad, "r": r.grad}
    for mask in range(1, 16):
        m, x, r, dy, _ = make(L, M, K, N, "silu", True)
        leaves = {"x": x, "w": m.weight, "b": m.bias, "r": r}
        for i, t in enumerate(leaves.values()):
            t.requires_grad_(bool(mask >> i & 1))
        m(x, r).backward(dy)
        for i, (k, t) in enumerate(leaves.items()):
            assert (t.grad is None) if not mask >> i & 1 else torch.equal(t.grad, want[k]), (mask, k)
    with torch.no_grad():
        assert not m(x, r).requires_grad


def test_layer_with_an_expanded_gradient_and_a_strided_residual(L):
    announce("QLinear: sum().backward(), strided residual")
    M, K, N = 64, 128, 96
    m, x, r, _, _ = make(L, M, K, N, "gelu", True)
    wide = torch.zeros((2, M // 2, N + 5), dtype=torch.bfloat16, device=dev())
    wide[..., 3:3 + N] = r.detach()
    y = m(x, wide[..., 3:3 + N])
    m.step = 0
    x2 = x.detach().requires_grad_(True)
    z = m(x2, r)
    assert torch.equal(y, z)
    y.sum().backward()
    z.backward(torch.ones_like(z))
    assert torch.equal(x.grad, x2.grad)
    flat = torch.zeros(M * N + 1, dtype=torch.bfloat16, device=dev())   # contiguous, two bytes off its alignment
    flat[1:] = r.detach().flatten()
    m.step = 0
    assert torch.equal(m(x, flat[1:].view(2, M // 2, N)), z)


@pytest.mark.parametrize("T", [0, 1, 5, 64, 65, 200])
@pytest.mark.parametrize("act,bias,res", [("gelu", True, True), (None, True, False), ("silu", False, True)])
def test_linear_inference(L, T, act, bias, res):
    announce(f"QLinearInference {T} tokens {act} bias={bias} residual={res}")
    M, K, N = 32, 272, 208
    w, b = normal((N, K), torch.bfloat16, 1, K ** -0.5), normal((N,), torch.float32, 2) if bias else None
    f = L.QLinearInference(w, b, act)
    x, r = normal((T, K), torch.float32, 3), normal((T, N), torch.float32, 4) if res else None
    y = f(x, r)
    assert y.shape == (T, N) and y.dtype == torch.bfloat16
    if not T:
        return
    xb = x.bfloat16()
    if T > 64:
        import bit_block_scaled_amd as bbs
        rows = (T + 15) // 16 * 16
        q = bbs.NVFP4Tensor.empty(rows, K, device=dev())
        bbs.nvfp4_quantize(torch.nn.functional.pad(xb, (0, 0, 0, rows - T)), q)
        xv = nv64(q)[:T]
    else:
        xv = xb.double()
    z, Ez = with_bias(*product_t(xv, nv64(f.weight)), b)
    within(y, *activated(act or "", z, Ez, r.bfloat16() if res else None, True), True, "y")
    if b is not None:                                                   # later changes of the bias do not reach it
        b.zero_(), w.zero_()
        assert torch.equal(f(x, r), y)


def test_layer_inference(L):
    announce("QLinear.inference")
    m, x, r, _, _ = make(L, 64, 128, 96, "gelu", True)
    f = m.inference()
    import bit_block_scaled_amd as bbs
    y = torch.empty((32, 96), dtype=torch.bfloat16, device=dev())
    bbs.nvfp4_gemv_bias_act(0, x.detach()[0], f.weight, y, 1, bias=m.bias.detach(), act=bbs.ACT_GELU, residual=r.detach()[0])
    assert torch.equal(f(x.detach()[0], r.detach()[0]), y)


@pytest.mark.parametrize("T", [0, 1, 7, 64, 150])
@pytest.mark.parametrize("gated,act,kind", [(True, "silu", torch.int64), (False, "gelu", torch.int32),
                                            (False, None, torch.int64)])
def test_moe_inference(L, T, gated, act, kind):
    announce(f"QMoEInference {T} tokens gated={gated} {act}")
    E, k, F, K, N = 9, 3, 48, 80, 112
    wg, wu = (normal((E, F, K), torch.bfloat16, s, K ** -0.5) for s in (1, 2))
    wd = normal((E, N, F), torch.bfloat16, 3, F ** -0.5)
    wd[4] *= 7                                                          # an expert of another range
    f = L.QMoEInference(wg if gated else None, wu, wd, act)
    x = normal((T, K), torch.bfloat16, 4).reshape(T, 1, K)
    ids = torch.randint(-1, E + 1, (T, 1, k), generator=torch.Generator().manual_seed(5)).to(dev()).to(kind)
    if kind == torch.int64 and T:
        ids[0, 0, 0] = (1 << 32) + 2                                    # no expert, although its lower half is one
    w = torch.softmax(normal((T, 1, k), torch.float32, 6), -1)
    r = normal((T, 1, N), torch.bfloat16, 7)
    y = f(x, ids, w, r)
    assert y.shape == (T, 1, N) and y.dtype == torch.bfloat16
    if not T:
        return
    ref, err = layer64(__import__("bit_block_scaled_amd"), x[:, 0], ids[:, 0], w[:, 0], E, f.gate, f.up, f.down, act or "",
                       r[:, 0], True)
    within(y[:, 0], ref, err, True, "y")
    # each expert's weight is a tensor of its own
    one = O.nvfp4_quantize(host(wd[4].view(torch.int16)).view(np.uint16), tile2d=True)
    assert np.array_equal(host(f.down.codes).reshape(E, N, -1)[4], one.codes)
    assert np.array_equal(host(f.down.scales).reshape(E, N // 16, -1)[4], one.scales)


def test_layers_in_a_graph(L):
    """A training step's forward and backward pass and the two inference layers, captured and replayed."""
    announce("linear layers: graph")
    M, K, N, E, k = 64, 128, 96, 6, 2
    m, x, r, dy, _ = make(L, M, K, N, "gelu", True)
    f = m.inference()
    moe = L.QMoEInference(normal((E, 48, N), torch.bfloat16, 1), normal((E, 48, N), torch.bfloat16, 2),
                          normal((E, K, 48), torch.bfloat16, 3))
    ids = torch.randint(0, E, (5, k), generator=torch.Generator().manual_seed(1)).to(dev())
    xs, rs, gs = x.detach().clone(), r.detach().clone(), dy.clone()

    def step():
        m.step = 3
        leaves = [xs.detach().requires_grad_(True), m.weight, m.bias]
        y = m(leaves[0], rs)
        grads = torch.autograd.grad(y, leaves, gs)
        t = f(xs[0, :5], rs[0, :5])
        return [y.detach(), *grads, t, moe(t, ids)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = step()
    for i in range(4):
        xs.copy_(torch.roll(xs, 1, 2)), rs.copy_(torch.roll(rs, 1, 1)), gs.copy_(torch.roll(gs, 1, 1))
        ids.copy_((ids + 1) % E)
        graph.replay()
        torch.cuda.synchronize()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(cap, eager)), i


def test_refusals(L):
    m = L.QLinear(64, 96, device=dev(), bias=True, act="gelu")
    x = torch.zeros((32, 64), dtype=torch.bfloat16, device=dev())
    for bad in (lambda: m(x[:, :32]), lambda: m(x[:16]), lambda: m(x[:0]), lambda: m(x, x),
                lambda: m(x, torch.zeros((32, 96), dtype=torch.bfloat16)), lambda: m(x.cpu()),
                lambda: m.inference()(x.cpu()), lambda: m.inference()(x, x)):
        with pytest.raises(ValueError):
            bad()


def test_inputs_at_any_address(L):
    """Contiguous inputs and gradients that begin between two 16-byte addresses."""
    announce("layers: inputs at any address")

    def moved(t):
        flat = torch.empty((t.numel() + 1,), dtype=t.dtype, device=t.device)
        flat[1:] = t.detach().reshape(-1)
        return flat[1:].view(t.shape)

    m, x, r, dy, _ = make(L, 64, 96, 160, "gelu", True)
    want = m(x, r)
    want.backward(dy)
    grads = [t.grad.clone() for t in (x, r, m.weight, m.bias)]
    m.weight.grad = m.bias.grad = None
    m.step = 0
    x2, r2 = moved(x).requires_grad_(True), moved(r).requires_grad_(True)
    y = m(x2, r2)
    y.backward(moved(dy))
    assert torch.equal(y, want)
    assert all(torch.equal(a, b.grad) for a, b in zip(grads, (x2, r2, m.weight, m.bias)))
    q = m.inference()
    for T in (5, 64 * 2):
        v = normal((T, 96), torch.bfloat16, 7)
        assert torch.equal(q(v), q(moved(v)))
    W = [normal((4, a, b), torch.bfloat16, 8) for a, b in ((64, 96), (64, 96), (32, 64))]
    e = L.QMoEInference(*W)
    v, ids = normal((70, 96), torch.bfloat16, 9), torch.arange(140, device=dev()).reshape(70, 2) % 4
    assert torch.equal(e(v, ids), e(moved(v), ids))


def test_moe_inference_ids_of_every_type(L):
    """More experts than a narrow type counts: the same answer from ids of every integer type."""
    announce("QMoEInference: types of the ids")
    E, k, F, K, N, T = 200, 3, 32, 48, 64, 6
    f = L.QMoEInference(*(normal((E, a, b), torch.bfloat16, s, b ** -0.5) for s, a, b in ((1, F, K), (2, F, K), (3, N, F))))
    x = normal((T, K), torch.bfloat16, 4)
    ids = torch.randint(0, 128, (T, k), generator=torch.Generator().manual_seed(5)).to(dev())
    want = f(x, ids)
    assert bool((want.abs().amax(1) > 0).all())
    for kind in (torch.int8, torch.uint8, torch.int16, torch.uint16, torch.int32, torch.uint32, torch.uint64):
        assert torch.equal(f(x, ids.to(kind)), want), kind
