"""A linear layer's product with bias, activation and residual (nvfp4_gemm_bias_act),
its backward pass (mxfp8_bias_act_bwd) and its form for a few tokens
(nvfp4_gemv_bias_act) against their definition in 64 bits.

A sum of K exact products in FP32 is off by at most (K + 32) 2^-24 sum |a b|, the
bias adds one rounding of z, the residual one of the result; the activation's
own error is bounded in gated_ref.py (its form for BF16 outputs rounds the
exponent's product once more, at most |z| 2^-24 of e^-z, which the factor 1.4
on that bound covers), and its slope lies in [-0.13, 1.13]."""
import numpy as np
import pytest

from gated_ref import ULP
from gpu_util import announce, dev
from test_gpu_gated import SENTINEL, act_t, checkpoint_within, mx64, nv64, product_t, random_mx, random_nv, within

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

ACTS = {"": 2, "silu": 0, "gelu": 1}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def bbs():
    import bit_block_scaled_amd as b
    return b


def gen(seed):
    return torch.Generator(device=dev()).manual_seed(seed)


def normal(shape, dtype, seed, std=1.0):
    return (torch.randn(shape, generator=gen(seed), device=dev()) * std).to(dtype)


def framed(rows, cols, dtype, pad):
    """A sentinel-filled output with `pad` columns behind each row and a row behind the last."""
    words = 1 if dtype == torch.bfloat16 else 2
    full = torch.full((rows + 1, (cols + pad) * words), SENTINEL, dtype=torch.int16, device=dev()).view(dtype)
    return full, full[:rows, :cols]


def untouched(full, rows, cols, what):
    raw = full.view(torch.int16).view(rows + 1, -1)
    w = cols * (1 if full.dtype == torch.bfloat16 else 2)
    assert bool((raw[rows] == SENTINEL).all()) and bool((raw[:rows, w:] == SENTINEL).all()), f"{what}: wrote outside"


def with_bias(z, Ez, b):
    if b is None:
        return z, Ez
    b = b.double()
    return z + b, Ez + 2 * ULP * (z.abs() + b.abs() + Ez)


def activated(act, z, Ez, r, bf16):
    """act(z) + r and its bound, z off by Ez."""
    if act:
        v, _, ea, _ = act_t(act, z)
        E = 1.13 * Ez + (1.4 if bf16 else 1.0) * ea
    else:
        v, E = z, Ez
    if r is not None:
        v = v + r.double()
        E = E + 2 * ULP * (v.abs() + E)
    return v, E


# rows, features, K, 16x16 weight scales, A scales, act, bias, residual, output, checkpoint, padding, scale shift:
# the small tiles with four and two groups of waves, the large tiles and their
# halves, and 256-row tiles (many tiles where K % 128 != 0 or scales are off
# their alignment), at whole and partial slabs
CASES = [
    (16, 16, 16, False, "", "", "", False, "f32", False, 0, 0),
    (16, 16, 16, True, "", "gelu", "f32", True, "bf16", False, 8, 0),
    (32, 32, 16, False, "", "silu", "bf16", True, "f32", True, 8, 1),
    (48, 112, 272, False, "rows", "silu", "f32", False, "bf16", False, 24, 2),
    (64, 320, 128, True, "tiles", "gelu", "bf16", True, "bf16", True, 0, 0),
    (272, 1568, 1184, False, "", "gelu", "bf16", True, "bf16", True, 0, 0),
    (528, 336, 1552, False, "", "", "f32", True, "f32", False, 16, 3),
    (256, 512, 1024, True, "rows", "silu", "bf16", False, "f32", True, 0, 0),
    (16, 1536, 4096, True, "", "gelu", "bf16", True, "f32", False, 0, 0),
    (1040, 288, 256, True, "", "silu", "", True, "bf16", True, 8, 0),
    (1040, 4160, 128, True, "", "silu", "bf16", True, "bf16", True, 0, 0),
    (1040, 4160, 256, False, "tiles", "gelu", "f32", True, "f32", True, 8, 0),
    (1040, 4160, 384, True, "rows", "gelu", "f32", False, "bf16", True, 16, 0),
    (1040, 4160, 1024, False, "", "", "bf16", True, "bf16", False, 0, 0),
    (1040, 4160, 1024, True, "", "silu", "f32", False, "f32", True, 8, 0),
    (1040, 4160, 1024, False, "", "gelu", "f32", True, "f32", True, 0, 3),
    (1040, 4160, 144, True, "", "", "", False, "f32", True, 0, 1),
    (1040, 4160, 272, False, "", "gelu", "bf16", True, "bf16", True, 8, 0),
    (1040, 4144, 16, False, "rows", "silu", "bf16", True, "f32", False, 0, 0),
    (4112, 3088, 640, True, "", "gelu", "bf16", True, "bf16", False, 8, 0),
    (272, 16400, 256, False, "", "", "f32", True, "bf16", False, 0, 0),
]


@pytest.mark.parametrize("M,N,K,tile2d,scales,act,bias,res,out,ckpt,pad,shift", CASES)
def test_gemm_bias_act(bbs, M, N, K, tile2d, scales, act, bias, res, out, ckpt, pad, shift):
    announce(f"linear {M} x {N} x {K} tile2d={tile2d} A {scales} {act} bias={bias} residual={res} {out} ckpt={ckpt} "
             f"shift={shift}")
    A = random_nv(bbs, M, K, scales == "tiles", 1, shift)
    if scales == "rows":
        d = (1.0 + torch.arange(M, device=dev()) % 7) * 0.25 / K ** 0.5
        A = bbs.NVFP4Tensor(A.codes, A.scales, d.float(), M, K, False, sdec_per_row=True)
    W = random_nv(bbs, N, K, tile2d, 2, shift)
    W.s_dec.fill_(0.5)
    dtype = DTYPES[out]
    b = normal((N,), DTYPES[bias], 3, 0.5) if bias else None
    r = normal((M, N + pad), dtype, 4)[:, :N] if res else None
    full, y = framed(M, N, dtype, pad)
    c = bbs.MXFP8Tensor.empty(M, N, device=dev()) if ckpt else None
    bbs.nvfp4_gemm_bias_act(A, W, y, int(out == "bf16"), bias=b, act=ACTS[act], residual=r, z_ckpt=c)
    z, Ez = with_bias(*product_t(nv64(A), nv64(W)), b)
    v, E = activated(act, z, Ez, r, out == "bf16")
    within(y, v, E, out == "bf16", "y")
    untouched(full, M, N, "y")
    if ckpt:
        checkpoint_within(c, z, Ez, "z")


@pytest.mark.parametrize("M,N,K", [(272, 1568, 1184), (1040, 4160, 256), (1040, 4160, 272)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_residual_in_place(bbs, M, N, K, out):
    """The residual may be the output itself: the same bits as with one of its own."""
    announce(f"linear in place {M} x {N} x {K} {out}")
    A, W, b = random_nv(bbs, M, K, False, 1), random_nv(bbs, N, K, True, 2), normal((N,), torch.float32, 3)
    r = normal((M, N), DTYPES[out], 4)
    y = torch.empty_like(r)
    kind = int(out == "bf16")
    bbs.nvfp4_gemm_bias_act(A, W, y, kind, bias=b, act=bbs.ACT_GELU, residual=r)
    bbs.nvfp4_gemm_bias_act(A, W, r, kind, bias=b, act=bbs.ACT_GELU, residual=r)
    assert torch.equal(y, r)


def test_plain_epilogue_is_the_plain_product(bbs):
    """Without bias, activation and residual the large tiles give nvfp4_gemm's bits."""
    announce("linear without an epilogue")
    M, N, K = 1040, 4160, 512
    A, W = random_nv(bbs, M, K, False, 1), random_nv(bbs, N, K, True, 2)
    for kind, dtype in ((0, torch.float32), (1, torch.bfloat16)):
        y, z = (torch.empty((M, N), dtype=dtype, device=dev()) for _ in range(2))
        bbs.nvfp4_gemm_bias_act(A, W, y, kind)
        bbs.nvfp4_gemm(bbs.FMT_NVFP4, A, W, z, kind)
        assert torch.equal(y, z)


@pytest.mark.parametrize("act", ["", "silu", "gelu"])
def test_nan_and_infinite_values_stay_where_they_are(bbs, act):
    """A NaN bias or an infinite residual reaches its column or its element alone."""
    announce(f"linear: NaN and infinities {act}")
    for M, N, K in ((80, 272, 144), (1040, 4160, 256)):
        A, W = random_nv(bbs, M, K, False, 1), random_nv(bbs, N, K, True, 2)
        b, r = normal((N,), torch.float32, 3), normal((M, N), torch.float32, 4)
        b[130] = float("nan")
        r[33, 5] = float("inf")
        y = torch.empty_like(r)
        bbs.nvfp4_gemm_bias_act(A, W, y, 0, bias=b, act=ACTS[act], residual=r)
        want = torch.zeros_like(y, dtype=torch.bool)
        want[:, 130] = True
        assert torch.equal(torch.isnan(y), want)
        want.zero_()[33, 5] = True
        assert torch.equal(torch.isinf(y), want)


def test_output_beyond_32_bits(bbs):
    """More than 2^31 outputs: the last rows, with a residual and a checkpoint."""
    announce("linear past 2^31 outputs")
    M, N, K = 65552, 32800, 128
    A, W = random_nv(bbs, M, K, False, 1), random_nv(bbs, N, K, True, 2)
    b, y = normal((N,), torch.bfloat16, 3), torch.empty((M, N), dtype=torch.bfloat16, device=dev())
    y[-48:] = normal((48, N), torch.bfloat16, 4)
    r = y[-48:].clone()
    c = bbs.MXFP8Tensor.empty(M, N, device=dev())
    bbs.nvfp4_gemm_bias_act(A, W, y, 1, bias=b, act=bbs.ACT_SILU, residual=y, z_ckpt=c)
    z, Ez = with_bias(*product_t(nv64(A)[-48:], nv64(W)), b)
    within(y[-48:], *activated("silu", z, Ez, r, True), True, "y")
    checkpoint_within(bbs.MXFP8Tensor(c.codes[-48:], c.scales[-48:], 48, N), z, Ez, "z")
    dz = torch.empty_like(y)
    bbs.mxfp8_bias_act_bwd(y, c, bbs.ACT_SILU, dz)
    check_bwd("silu", y[-48:], bbs.MXFP8Tensor(c.codes[-48:], c.scales[-48:], 48, N), dz[-48:], None)


# ---------------------------------------------------------------------------
# Backward pass
# ---------------------------------------------------------------------------

def check_bwd(act, dy, z8, dz, db):
    g = dy.double()
    if act:
        _, slope, _, es = act_t(act, mx64(z8))
        ref, E = g * slope, g.abs() * (1.4 * es + 2 * ULP * slope.abs()) + 2.0 ** -125
    else:
        ref, E = g, torch.zeros_like(g)
    if dz is not None:
        within(dz, ref, E, True, "dZ")
    if db is not None:
        s = ref.sum(0)
        Es = E.sum(0) + (len(ref) + 8) * ULP * (ref.abs() + E).sum(0)
        within(db, s, Es, db.dtype == torch.bfloat16, "dbias")


BWD = [
    (1, 32, "silu", "f32", 0), (1, 16, "", "bf16", 8), (15, 96, "gelu", "f32", 8), (16, 160, "silu", "bf16", 0),
    (17, 2048, "gelu", "bf16", 0), (64, 128, "", "f32", 0), (65, 4000, "silu", "f32", 16), (272, 1568, "silu", "bf16", 0),
    (1000, 288, "gelu", "f32", 8), (5003, 32, "gelu", "f32", 0), (2111, 14336, "gelu", "bf16", 0), (4096, 1040, "", "f32", 8),
    (20011, 64, "silu", "f32", 0),
]


@pytest.mark.parametrize("M,N,act,bias,pad", BWD)
def test_bias_act_bwd(bbs, M, N, act, bias, pad):
    announce(f"linear bwd {M} x {N} {act} dbias {bias}")
    dy = normal((M, N + pad), torch.bfloat16, 1, 1e-3)[:, :N]
    z8 = random_mx(bbs, M, N, 2, 122) if act else None
    full, dz = framed(M, N, torch.bfloat16, pad)
    db = torch.full((N + 8,), 7.0, dtype=DTYPES[bias], device=dev())
    bbs.mxfp8_bias_act_bwd(dy, z8, ACTS[act], dz, db[:N])
    check_bwd(act, dy, z8, dz, db[:N])
    untouched(full, M, N, "dZ")
    assert bool((db[N:] == 7).all())
    # either output alone, and dZ over dY, give the same bits
    dz2, db2 = torch.empty_like(dz), torch.empty_like(db[:N])
    bbs.mxfp8_bias_act_bwd(dy, z8, ACTS[act], dz2)
    bbs.mxfp8_bias_act_bwd(dy, z8, ACTS[act], None, db2)
    assert torch.equal(dz2, dz) and torch.equal(db2, db[:N])
    bbs.mxfp8_bias_act_bwd(dy, z8, ACTS[act], dy, db2)
    assert torch.equal(dy, dz) and torch.equal(db2, db[:N])


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_bwd_of_every_checkpoint_value(bbs, act):
    """Every finite E4M3 code at scales from the smallest to the largest: finite slopes."""
    announce(f"linear bwd over the checkpoint's range {act}")
    codes = torch.arange(256, dtype=torch.int32, device=dev())
    codes = codes[(codes & 0x7F) != 0x7F]
    codes = torch.cat([codes, codes[:2]]).to(torch.uint8).repeat(246, 1).contiguous()      # 256 columns
    scales = torch.arange(0, 246, dtype=torch.uint8, device=dev()).view(-1, 1).repeat(1, 8).contiguous()
    z8 = bbs.MXFP8Tensor(codes, scales, 246, 256)
    dy = torch.ones((246, 256), dtype=torch.bfloat16, device=dev())
    dz = torch.empty_like(dy)
    bbs.mxfp8_bias_act_bwd(dy, z8, ACTS[act], dz)
    z = mx64(z8)
    near = z.clamp(-30, 30)                                             # beyond, act is 0 or the identity
    _, slope, _, es = act_t(act, near)
    within(dz, slope, 1.4 * es + 2 * ULP + 1e-10, True, "slope")


def test_bwd_is_the_gradient_of_the_forward_pass(bbs):
    """dZ and dbias against differences of the forward pass at the checkpointed z:
    sum(dY act(z + h e)) over h, with z given by the bias alone."""
    announce("linear bwd against differences")
    M, N, K, h = 32, 64, 16, 2.0 ** -6
    A, W = random_nv(bbs, M, K, False, 1), random_nv(bbs, N, K, False, 2)
    A.codes.zero_()                                                     # z is the bias
    g = torch.linspace(-6, 6, 97, device=dev())
    g = g[(g.abs() * 16 % 1 == 0)]                                      # values the checkpoint holds exactly
    b = torch.cat([torch.tensor([0.0, 1, -1, 2, -2, 4, -4, 0.5, -0.5, 1.5, -1.5, 3, -3, 6, -6, 0.25], device=dev())] * 4)
    dy = normal((M, N), torch.bfloat16, 3)
    for act in ("silu", "gelu"):
        z8 = bbs.MXFP8Tensor.empty(M, N, device=dev())
        y = [torch.empty((M, N), device=dev()) for _ in range(3)]
        for t, d in zip(y, (-h, h, 0.0)):
            bbs.nvfp4_gemm_bias_act(A, W, t, 0, bias=b + d, act=ACTS[act], z_ckpt=z8)
        assert torch.equal(mx64(z8), b.double().expand(M, N))
        dz, db = torch.empty((M, N), dtype=torch.bfloat16, device=dev()), torch.empty((N,), device=dev())
        bbs.mxfp8_bias_act_bwd(dy, z8, ACTS[act], dz, db)
        diff = (y[1].double() - y[0].double()) / (2 * h) * dy.double()
        # h^2 / 6 of the third derivative (below 8) and the rounding of two values
        off = dy.double().abs() * (8 * h * h / 6 + 32 * ULP * (1 + b.double().abs()) / h)
        assert bool(((dz.double() - diff).abs() <= off + (diff.abs() + off) * 2.0 ** -8).all())
        assert bool(((db.double() - diff.sum(0)).abs() <= off.sum(0) + 64 * ULP * dy.double().abs().sum(0)).all())


# ---------------------------------------------------------------------------
# A few tokens
# ---------------------------------------------------------------------------

def random_mx4(bbs, rows, cols, seed):
    g = gen(seed)
    codes = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, device=dev(), generator=g)
    scales = torch.randint(120, 126, (rows, cols // 32), dtype=torch.uint8, device=dev(), generator=g)
    return bbs.MXFP4Tensor(codes, scales, rows, cols)


def mx4_64(t):
    n = torch.stack((t.codes & 15, t.codes >> 4), 2).flatten(1).long()
    v = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=dev())[n]
    return v * torch.exp2(t.scales.double() - 127).repeat_interleave(32, 1)


GEMV = [
    (1, 16, 16, "nvfp4", False, "gelu", "bf16", True, "f32", 0), (1, 1, 32, "mxfp4", False, "", "f32", True, "bf16", 0),
    (1, 1536, 4096, "nvfp4", True, "gelu", "bf16", False, "bf16", 0), (2, 5, 96, "mxfp4", False, "silu", "f32", True, "bf16", 3),
    (3, 48, 272, "nvfp4", False, "", "", True, "f32", 1), (4, 1536, 528, "nvfp4", True, "silu", "f32", True, "bf16", 8),
    (5, 4112, 1552, "nvfp4", False, "gelu", "f32", False, "f32", 0), (8, 333, 4064, "mxfp4", False, "gelu", "bf16", True, "f32", 5),
    (17, 97, 96, "mxfp4", False, "silu", "bf16", True, "bf16", 7), (40, 4096, 2048, "mxfp4", False, "", "f32", True, "f32", 0),
    (64, 512, 4096, "nvfp4", True, "gelu", "bf16", True, "bf16", 0),
]


@pytest.mark.parametrize("T,N,K,fmt,tile2d,act,bias,res,out,pad", GEMV)
def test_gemv_bias_act(bbs, T, N, K, fmt, tile2d, act, bias, res, out, pad):
    announce(f"linear gemv {T} x {N} x {K} {fmt} {act} bias={bias} residual={res} {out}")
    W = random_mx4(bbs, N, K, 1) if fmt == "mxfp4" else random_nv(bbs, N, K, tile2d, 1)
    w = mx4_64(W) if fmt == "mxfp4" else nv64(W)
    w_std = float(w.std())
    x = normal((T, K), torch.bfloat16, 2, 1 / (w_std * K ** 0.5))
    dtype = DTYPES[out]
    b = normal((N + 3,), DTYPES[bias], 3)[3:] if bias else None         # not aligned to 16 bytes
    r = normal((T, N + pad), dtype, 4)[:, :N] if res else None
    full, y = framed(T, N, dtype, pad)
    kind = int(out == "bf16")
    bbs.nvfp4_gemv_bias_act(2 if fmt == "mxfp4" else 0, x, W, y, kind, bias=b, act=ACTS[act], residual=r)
    z, Ez = with_bias(*product_t(x.double(), w), b)
    within(y, *activated(act, z, Ez, r, False), out == "bf16", "y")
    untouched(full, T, N, "y")
    if res:
        before = y.clone()
        y.copy_(r)
        bbs.nvfp4_gemv_bias_act(2 if fmt == "mxfp4" else 0, x, W, y, kind, bias=b, act=ACTS[act], residual=y)
        assert torch.equal(before, y)


def test_gemv_more_rows_than_a_launch(bbs):
    """More than 2^25 rows go in parts, the bias and the residual with them."""
    announce("linear gemv past 2^25 rows")
    N, K = (1 << 25) + 40, 32
    W = random_mx4(bbs, N, K, 1)
    x, b = normal((1, K), torch.bfloat16, 2), normal((N,), torch.bfloat16, 3)
    r, y = normal((1, N), torch.float32, 4), torch.empty((1, N), device=dev())
    bbs.nvfp4_gemv_bias_act(2, x, W, y, 0, bias=b, act=bbs.ACT_SILU, residual=r)
    for at in (slice(0, 64), slice((1 << 25) - 32, N)):
        w = mx4_64(bbs.MXFP4Tensor(W.codes[at], W.scales[at], 0, K))
        z, Ez = with_bias(*product_t(x.double(), w), b[at])
        within(y[:, at], *activated("silu", z, Ez, r[:, at], False), False, "y")


# ---------------------------------------------------------------------------
# Streams, graphs, calls at once
# ---------------------------------------------------------------------------

def problem(bbs, M, N, K, seed):
    return {"A": random_nv(bbs, M, K, False, seed), "W": random_nv(bbs, N, K, True, seed + 1),
            "x": normal((13, K), torch.bfloat16, seed + 2), "b": normal((N,), torch.bfloat16, seed + 3),
            "r": normal((M, N), torch.bfloat16, seed + 4), "dy": normal((M, N), torch.bfloat16, seed + 5)}


def run_all(bbs, q, stream=None):
    M, N = q["r"].shape
    y, dz = (torch.empty((M, N), dtype=torch.bfloat16, device=dev()) for _ in range(2))
    v, db = torch.empty((13, N), device=dev()), torch.empty((N,), device=dev())
    z8 = bbs.MXFP8Tensor.empty(M, N, device=dev())
    bbs.nvfp4_gemm_bias_act(q["A"], q["W"], y, 1, bias=q["b"], act=bbs.ACT_GELU, residual=q["r"], z_ckpt=z8, stream=stream)
    bbs.mxfp8_bias_act_bwd(q["dy"], z8, bbs.ACT_GELU, dz, db, stream=stream)
    bbs.nvfp4_gemv_bias_act(0, q["x"], q["W"], v, 0, bias=q["b"], act=bbs.ACT_SILU, residual=v.zero_(), stream=stream)
    return y, z8.codes, z8.scales, dz, db, v


def same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


def test_streams_and_graphs(bbs):
    announce("linear operators: stream and graph")
    q = problem(bbs, 272, 544, 256, 1)
    eager = run_all(bbs, q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = run_all(bbs, q)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert same(eager, side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = run_all(bbs, q)
    for i in range(4):
        for k in ("x", "r", "dy"):
            q[k].copy_(torch.roll(q[k], 1, 0))
        q["A"].codes.copy_(torch.roll(q["A"].codes, 3, 0))
        graph.replay()
        eager = run_all(bbs, q)
        torch.cuda.synchronize()
        assert same(eager, cap), i


def test_calls_at_once(bbs):
    announce("linear operators: two streams at once")
    probs = problem(bbs, 528, 1056, 1024, 10), problem(bbs, 528, 1056, 1024, 20)
    alone = [run_all(bbs, q) for q in probs]
    torch.cuda.synchronize()
    both = []
    for s, q in zip((torch.cuda.Stream(), torch.cuda.Stream()), probs):
        with torch.cuda.stream(s):
            for _ in range(6):
                got = run_all(bbs, q)
        both.append(got)
    torch.cuda.synchronize()
    assert same(alone[0], both[0]) and same(alone[1], both[1])


def test_own_workspace_on_another_stream(bbs, monkeypatch):
    """A workspace the call allocates for a given stream is not handed out again while that
    stream has yet to run the call."""
    announce("bias gradient: own workspace, other stream")
    dy, db = normal((2048, 512), torch.bfloat16, 1), torch.empty((512,), device=dev())
    bbs.mxfp8_bias_act_bwd(dy, None, bbs.ACT_NONE, None, db)
    want = db.clone()
    made, keep = [], bbs._used_on
    monkeypatch.setattr(bbs, "_used_on", lambda ws, stream: made.append((ws.data_ptr(), ws.numel())) or keep(ws, stream))
    a, s = torch.ones((4096, 4096), device=dev()), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(40):
            a @ a                                                       # milliseconds
    bbs.mxfp8_bias_act_bwd(dy, None, bbs.ACT_NONE, None, db.zero_(), stream=s)
    other = torch.empty((made[0][1],), device=dev())
    busy = not s.query()
    assert other.data_ptr() != made[0][0]
    torch.cuda.synchronize()
    assert busy and torch.equal(db, want)


def test_bwd_over_a_grid_against_differences(bbs):
    """As test_bwd_is_the_gradient_of_the_forward_pass, at every value of four significant
    bits from 2^-4 to 7.5, which the checkpoint holds exactly beside any other of them."""
    announce("linear bwd against differences, grid")
    e, m = torch.arange(-7, -1, device=dev()), torch.arange(8, 16, device=dev())
    b = torch.ldexp(m[None, :].float(), e[:, None]).flatten()
    b = torch.cat([b, -b])
    M, N, K, h = 16, b.numel(), 16, 2.0 ** -6
    A, W = random_nv(bbs, M, K, False, 1), random_nv(bbs, N, K, False, 2)
    A.codes.zero_()                                                     # z is the bias
    dy = normal((M, N), torch.bfloat16, 3)
    for act in ("silu", "gelu"):
        z8 = bbs.MXFP8Tensor.empty(M, N, device=dev())
        y = [torch.empty((M, N), device=dev()) for _ in range(3)]
        for t, d in zip(y, (-h, h, 0.0)):
            bbs.nvfp4_gemm_bias_act(A, W, t, 0, bias=b + d, act=ACTS[act], z_ckpt=z8)
        assert torch.equal(mx64(z8), b.double().expand(M, N))
        dz, db = torch.empty((M, N), dtype=torch.bfloat16, device=dev()), torch.empty((N,), device=dev())
        bbs.mxfp8_bias_act_bwd(dy, z8, ACTS[act], dz, db)
        diff = (y[1].double() - y[0].double()) / (2 * h) * dy.double()
        # h^2 / 6 of the third derivative (below 8) and the rounding of two values
        off = dy.double().abs() * (8 * h * h / 6 + 32 * ULP * (1 + b.double().abs()) / h)
        assert bool(((dz.double() - diff).abs() <= off + (diff.abs() + off) * 2.0 ** -8).all())
        assert bool(((db.double() - diff.sum(0)).abs() <= off.sum(0) + 64 * ULP * dy.double().abs().sum(0)).all())
