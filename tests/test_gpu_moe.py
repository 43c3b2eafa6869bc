"""The expert layer for a few tokens (nvfp4_moe_gemv) against its definition in 64
bits over the decoded weights.

An up projection is off by the FP32 accumulation bound (K + 32) 2^-24 sum |a b|,
the activation and the product as in gated_ref.py; the hidden value is then held
in 16 significant bits for BF16 outputs (off by 2^-16) and in 24 for FP32 ones
(2^-24, as FP32 itself); the down projection adds the accumulation bound over
its parts, and the sum over the experts, their weights' sums and the residual a
rounding each."""
import pytest

from gated_ref import ULP
from gpu_util import announce, dev
from test_gpu_gated import act_t, nv64, product_t, random_nv, within
from test_gpu_linear import ACTS, DTYPES, framed, mx4_64, normal, random_mx4, same, untouched

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def bbs():
    import bit_block_scaled_amd as b
    return b


def experts(bbs, fmt, E, rows, cols, tile2d, seed):
    """A stack of experts' weights with a decode scale each."""
    if fmt == "mxfp4":
        return random_mx4(bbs, E * rows, cols, seed)
    w = random_nv(bbs, E * rows, cols, tile2d, seed)
    d = (1.0 + torch.arange(E, device=dev()) % 5) * 0.3 / cols ** 0.5
    return bbs.NVFP4Tensor(w.codes, w.scales, d.float(), E * rows, cols, tile2d)


def expert64(bbs, w, E, e):
    rows = w.rows // E
    at = slice(e * rows, (e + 1) * rows)
    if isinstance(w, bbs.MXFP4Tensor):
        return mx4_64(bbs.MXFP4Tensor(w.codes[at], w.scales[at], rows, w.cols))
    srows = rows // 16 if w.tile2d else rows
    return nv64(bbs.NVFP4Tensor(w.codes[at], w.scales[e * srows:(e + 1) * srows], w.s_dec[e:e + 1], rows, w.cols, w.tile2d))


def layer64(bbs, x, ids, weights, E, Wg, Wu, Wd, act, r, bf16):
    """(y, its bound) in 64 bits."""
    T, N = x.shape[0], Wd.rows // E
    y, err = (torch.zeros((T, N), dtype=torch.float64, device=dev()) for _ in range(2))
    size = torch.zeros_like(y)
    for e in sorted(set(ids.flatten().tolist())):
        if not 0 <= e < E:
            continue
        hit = ids == e
        rows = hit.any(1).nonzero()[:, 0]
        w = torch.where(hit, weights.double() if weights is not None else 1.0, 0.0).sum(1)[rows, None]
        u, Eu = product_t(x[rows].double(), expert64(bbs, Wu, E, e))
        if Wg is not None:
            g, Eg = product_t(x[rows].double(), expert64(bbs, Wg, E, e))
            a, _, ea, _ = act_t(act, g)
            h = a * u
            Eh = (u.abs() + Eu) * (1.13 * Eg + ea) + a.abs() * Eu + 2 * ULP * h.abs()
        elif act:
            h, _, ea, _ = act_t(act, u)
            Eh = 1.13 * Eu + ea
        else:
            h, Eh = u, Eu
        Eh = Eh + (h.abs() + Eh) * (2.0 ** -16 if bf16 else 2.0 ** -24)
        d = expert64(bbs, Wd, E, e)
        v, Ev = product_t(h, d)
        Ev = 3 * Ev + Eh @ d.abs().t()                                  # up to three parts a value
        y[rows] += w * v
        size[rows] += w.abs() * (v.abs() + Ev)
        err[rows] += w.abs() * Ev
    k = ids.shape[1]
    err = err + (2 * k + 16) * ULP * size
    if r is not None:
        y, err = y + r.double(), err + 2 * ULP * (r.double().abs() + size)
    return y, err


def routing(T, E, k, kind, seed):
    g = torch.Generator(device=dev()).manual_seed(seed)
    ids = torch.argsort(torch.rand((T, max(E, k)), generator=g, device=dev()), dim=1)[:, :k].to(torch.int32) % E
    if kind == "dropped":
        ids = torch.where(torch.rand((T, k), generator=g, device=dev()) < 0.4, -1, ids).to(torch.int32)
        ids[T // 2] = E                                                 # a token without any
        ids[0, 0] = -2 ** 31
    elif kind == "twice":
        ids = (ids % max(1, E // 2)).to(torch.int32)
    elif kind == "one":
        ids = torch.full_like(ids, E - 1)
    elif kind == "none":
        ids = torch.full_like(ids, -1)
    return ids.contiguous()


# tokens, experts, slots, hidden, features in, out, format, tile, gated, act, weights, residual, output, routing, padding
CASES = [
    (1, 1, 1, 16, 16, 16, "nvfp4", False, True, "silu", True, False, "f32", "", 0),
    (1, 8, 2, 32, 32, 1, "mxfp4", False, False, "", False, True, "bf16", "", 0),
    (1, 64, 8, 208, 512, 272, "nvfp4", True, False, "gelu", True, False, "bf16", "", 8),
    (1, 64, 8, 528, 1040, 144, "nvfp4", False, True, "gelu", True, True, "f32", "", 0),
    (1, 12, 5, 96, 160, 37, "mxfp4", False, True, "silu", True, True, "f32", "dropped", 8),
    (1, 6, 32, 64, 96, 20, "mxfp4", False, False, "silu", True, False, "f32", "twice", 0),
    (1, 3, 2, 2064, 1552, 48, "nvfp4", True, True, "silu", True, True, "bf16", "", 0),
    (2, 64, 8, 272, 528, 160, "nvfp4", False, True, "silu", True, True, "bf16", "", 0),
    (2, 4, 4, 512, 1024, 64, "nvfp4", True, False, "", False, False, "f32", "twice", 8),
    (3, 16, 3, 160, 608, 99, "mxfp4", False, True, "gelu", True, False, "bf16", "dropped", 0),
    (4, 8, 6, 1040, 272, 96, "nvfp4", False, False, "gelu", True, True, "f32", "", 8),
    (4, 5, 5, 144, 80, 32, "nvfp4", True, True, "silu", True, False, "bf16", "one", 0),
    (5, 12, 3, 736, 1568, 1568, "mxfp4", False, True, "gelu", True, True, "f32", "dropped", 0),
    (6, 300, 8, 96, 288, 64, "mxfp4", False, True, "silu", True, True, "bf16", "", 8),
    (7, 40, 1, 112, 144, 112, "nvfp4", True, False, "silu", False, False, "bf16", "", 0),
    (16, 64, 8, 208, 528, 160, "nvfp4", False, True, "silu", True, True, "bf16", "", 0),
    (17, 4, 2, 400, 1040, 48, "nvfp4", True, True, "gelu", True, True, "f32", "", 8),
    (33, 2, 2, 160, 288, 45, "mxfp4", False, False, "", True, False, "f32", "", 0),
    (33, 1000, 4, 32, 64, 33, "mxfp4", False, True, "silu", True, True, "bf16", "dropped", 0),
    (64, 64, 8, 272, 528, 144, "nvfp4", True, True, "silu", True, True, "bf16", "", 0),
    (64, 3, 32, 96, 160, 80, "nvfp4", False, True, "gelu", True, False, "f32", "twice", 8),
    (64, 1024, 32, 32, 32, 16, "mxfp4", False, False, "gelu", True, True, "bf16", "", 0),
    (64, 10, 4, 1024, 640, 32, "nvfp4", False, False, "silu", True, True, "bf16", "one", 0),
    (40, 16, 4, 64, 64, 64, "nvfp4", True, True, "silu", True, True, "f32", "none", 8),
    # a few tokens, hidden rows and experts enough for whole rows a wave
    (1, 12, 6, 4112, 528, 32, "nvfp4", False, True, "silu", True, True, "bf16", "", 0),
    (2, 40, 8, 3200, 272, 48, "nvfp4", True, False, "gelu", True, False, "f32", "dropped", 8),
    (3, 64, 16, 592, 1552, 64, "nvfp4", False, True, "gelu", False, True, "f32", "twice", 0),
    (4, 10, 4, 5216, 784, 80, "nvfp4", True, True, "silu", True, True, "bf16", "", 8),
    # three tokens on (MXFP4; NVFP4: nine), with weights enough for the streaming kernels
    (5, 64, 8, 544, 1568, 1040, "nvfp4", False, False, "silu", True, False, "bf16", "", 0),
    (8, 64, 8, 528, 1552, 1040, "nvfp4", False, True, "gelu", True, True, "f32", "", 8),
    (3, 8, 2, 2080, 2720, 2720, "mxfp4", False, True, "silu", True, True, "bf16", "", 0),
    (4, 16, 3, 2080, 2080, 2080, "mxfp4", False, True, "gelu", True, True, "f32", "dropped", 8),
    (8, 64, 8, 544, 1568, 1040, "mxfp4", False, True, "silu", True, False, "bf16", "", 0),
    (9, 64, 8, 528, 1552, 1040, "nvfp4", False, True, "silu", True, False, "bf16", "twice", 0),
    (9, 100, 12, 544, 608, 1568, "mxfp4", False, True, "gelu", True, True, "f32", "dropped", 8),
    (24, 6, 3, 2064, 4624, 2080, "nvfp4", True, True, "silu", True, True, "f32", "", 0),
    (13, 8, 2, 5136, 1040, 2064, "nvfp4", False, True, "silu", True, False, "bf16", "", 0),
    (64, 6, 2, 4640, 2080, 2085, "mxfp4", False, False, "gelu", True, True, "f32", "", 8),
    (11, 8, 1, 512, 16400, 2064, "nvfp4", False, True, "silu", True, False, "bf16", "", 0),
    (6, 8, 2, 512, 40960, 48, "nvfp4", True, False, "", True, True, "bf16", "", 0),
    (33, 64, 8, 1552, 1552, 160, "nvfp4", True, True, "silu", True, True, "bf16", "", 8),
    (64, 1024, 32, 512, 544, 32, "mxfp4", False, True, "silu", True, False, "bf16", "", 0),
    (40, 48, 32, 1040, 1552, 1040, "nvfp4", False, True, "silu", False, True, "bf16", "twice", 0),
    (64, 16, 4, 2064, 2576, 2064, "nvfp4", False, False, "", True, True, "f32", "one", 0),
    (16, 64, 3, 1056, 1056, 1056, "mxfp4", False, True, "silu", True, True, "f32", "none", 8),
    (17, 64, 8, 1056, 1568, 45, "mxfp4", False, True, "gelu", True, False, "bf16", "", 0),
]


@pytest.mark.parametrize("T,E,k,F,K,N,fmt,tile2d,gated,act,weighted,res,out,kind,pad", CASES)
def test_moe(bbs, T, E, k, F, K, N, fmt, tile2d, gated, act, weighted, res, out, kind, pad):
    announce(f"moe {T} tokens, {k} of {E} experts {kind}, {K} -> {F} -> {N} {fmt} tile2d={tile2d} gated={gated} {act} {out}")
    Wg = experts(bbs, fmt, E, F, K, tile2d, 1) if gated else None
    Wu, Wd = experts(bbs, fmt, E, F, K, tile2d, 2), experts(bbs, fmt, E, N, F, tile2d, 3)
    x = normal((T, K + pad), torch.bfloat16, 4)[:, :K]
    ids = routing(T, E, k, kind, 5)
    weights = torch.softmax(normal((T, k), torch.float32, 6), 1) if weighted else None
    dtype, flag = DTYPES[out], int(out == "bf16")
    r = normal((T, N + pad), dtype, 7)[:, :N] if res else None
    full, y = framed(T, N, dtype, pad)
    f = 2 if fmt == "mxfp4" else 0
    bbs.nvfp4_moe_gemv(f, x, ids, weights, E, Wg, Wu, Wd, y, flag, act=ACTS[act], residual=r)
    ref, err = layer64(bbs, x, ids, weights, E, Wg, Wu, Wd, act, r, bool(flag))
    within(y, ref, err, bool(flag), "y")
    untouched(full, T, N, "y")
    # again, into the residual itself and with a workspace that holds other values: the same bits
    ws = bbs.moe_workspace(T, k, E, F, N, dev()).fill_(0xFF)
    again = r.clone(memory_format=torch.contiguous_format) if res else torch.empty((T, N), dtype=dtype, device=dev())
    bbs.nvfp4_moe_gemv(f, x, ids, weights, E, Wg, Wu, Wd, again, flag, act=ACTS[act], residual=again if res else None, ws=ws)
    assert torch.equal(again, y)
    if kind == "none":
        assert torch.equal(y, r)


def test_tokens_do_not_mix(bbs):
    """NaN and infinite tokens, and NaN weights of experts nobody chose, stay where they are."""
    announce("moe: NaN")
    for T, E, k, fmt, wide in ((4, 16, 3, "nvfp4", 1), (24, 8, 2, "mxfp4", 1), (2, 9, 2, "mxfp4", 1),
                               (24, 8, 2, "mxfp4", 33), (40, 9, 3, "nvfp4", 33)):
        F, K, N = 96 * wide, 160 * wide, 64
        Wg, Wu, Wd = (experts(bbs, fmt, E, r, c, False, i) for i, (r, c) in enumerate(((F, K), (F, K), (N, F))))
        ids = routing(T, E - 1, k, "", 5)                               # the last expert is never chosen
        if fmt == "mxfp4":
            for w in (Wg, Wu, Wd):
                w.scales[(E - 1) * w.rows // E:] = 255
        else:
            for w in (Wg, Wu, Wd):
                w.s_dec[E - 1] = float("nan")
        x, weights = normal((T, K), torch.bfloat16, 4), torch.softmax(normal((T, k), torch.float32, 6), 1)
        call = lambda: (bbs.nvfp4_moe_gemv(2 if fmt == "mxfp4" else 0, x, ids, weights, E, Wg, Wu, Wd, y, 0), y.clone())[1]
        y = torch.empty((T, N), device=dev())
        clean = call()
        x[1, 7], x[T - 1, 9] = float("nan"), float("inf")
        dirty = call()
        assert bool(torch.isfinite(clean).all())
        assert bool(torch.isnan(dirty[1]).all()) and not bool(torch.isfinite(dirty[T - 1]).any())
        keep = [t for t in range(T) if t not in (1, T - 1)]
        assert torch.equal(clean[keep], dirty[keep])


def test_infinite_hidden_value(bbs):
    """A hidden value past BF16's range becomes an infinity, not NaN."""
    announce("moe: hidden value past the range")
    F, K, N = 16, 16, 16
    Wu, Wd = experts(bbs, "nvfp4", 1, F, K, False, 1), experts(bbs, "nvfp4", 1, N, F, False, 2)
    for w in (Wu, Wd):
        w.codes.fill_(0x22), w.scales.fill_(0x38), w.s_dec.fill_(1.0)  # all ones
    x = torch.full((1, K), 2.0 ** 124, dtype=torch.bfloat16, device=dev())
    y = torch.empty((1, N), device=dev())
    ids = torch.zeros((1, 1), dtype=torch.int32, device=dev())
    bbs.nvfp4_moe_gemv(0, x, ids, None, 1, None, Wu, Wd, y, 0, act=bbs.ACT_NONE)
    assert bool(torch.isposinf(y).all())


def test_weights_beyond_32_bits(bbs):
    """More than 2^32 bytes of codes: the last experts."""
    announce("moe past 2^32 bytes of weights")
    E, F, K, N = 600, 512, 32768, 32
    Wu, Wd = experts(bbs, "mxfp4", E, F, K, False, 1), experts(bbs, "mxfp4", E, N, F, False, 2)
    assert Wu.codes.numel() > 1 << 32
    for T in (1, 6):
        x = normal((T, K), torch.bfloat16, 4, 1e-2)
        ids = torch.tensor([[E - 1, 0, E - 2]] * T, dtype=torch.int32, device=dev())
        y = torch.empty((T, N), device=dev())
        bbs.nvfp4_moe_gemv(2, x, ids, None, E, None, Wu, Wd, y, 0, act=bbs.ACT_GELU)
        within(y, *layer64(bbs, x, ids, None, E, None, Wu, Wd, "gelu", None, False), False, "y")


def problem(bbs, T, seed, wide=1):
    E, k, F, K, N = 16, 4, 208 * wide, 272 * wide, 160 * wide
    return {"x": normal((T, K), torch.bfloat16, seed), "ids": routing(T, E, k, "dropped", seed),
            "w": torch.softmax(normal((T, k), torch.float32, seed + 1), 1), "r": normal((T, N), torch.bfloat16, seed + 2),
            "W": [experts(bbs, "nvfp4", E, r, c, True, seed + i) for i, (r, c) in enumerate(((F, K), (F, K), (N, F)))]}


def run(bbs, q, stream=None):
    y, z = torch.empty_like(q["r"]), torch.empty(q["r"].shape, device=dev())
    bbs.nvfp4_moe_gemv(0, q["x"], q["ids"], q["w"], 16, *q["W"], y, 1, act=bbs.ACT_GELU, residual=q["r"], stream=stream)
    bbs.nvfp4_moe_gemv(0, q["x"], q["ids"], q["w"], 16, None, *q["W"][1:], z, 0, stream=stream)
    return y, z


@pytest.mark.parametrize("T,wide", [(1, 1), (3, 1), (3, 10), (20, 1), (20, 10)])
def test_streams_and_graphs(bbs, T, wide):
    """On a side stream, and captured and replayed with new tokens and another
    routing, with eager calls between the replays."""
    announce(f"moe: stream and graph, {T} tokens, {wide}")
    q = problem(bbs, T, 1, wide)
    eager = run(bbs, q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = run(bbs, q)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert same(eager, side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = run(bbs, q)
    for i in range(4):
        q["x"].copy_(torch.roll(q["x"], 1, 1))
        q["ids"].copy_(torch.where(q["ids"] >= 0, (q["ids"] + 3) % 16, q["ids"]))
        graph.replay()
        eager = run(bbs, q)
        torch.cuda.synchronize()
        assert same(eager, cap), i


@pytest.mark.parametrize("wide", [1, 10])
def test_calls_at_once(bbs, wide):
    announce("moe: two streams at once")
    probs = problem(bbs, 20, 10, wide), problem(bbs, 2, 20)
    alone = [run(bbs, q) for q in probs]
    torch.cuda.synchronize()
    both = []
    for s, q in zip((torch.cuda.Stream(), torch.cuda.Stream()), probs):
        with torch.cuda.stream(s):
            for _ in range(8):
                got = run(bbs, q)
        both.append(got)
    torch.cuda.synchronize()
    assert same(alone[0], both[0]) and same(alone[1], both[1])


@pytest.mark.parametrize("T,wide", [(5, 1), (20, 1), (20, 10)])
def test_two_graphs_of_one_workspace(bbs, T, wide):
    """Two captured calls that share a workspace, replayed in turn on one stream."""
    announce("moe: two graphs, one workspace")
    a, b = problem(bbs, T, 1, wide), problem(bbs, T, 30, wide)
    ws = bbs.moe_workspace(T, 4, 16, 208 * wide, 160 * wide, dev())

    def call(q):
        y = torch.empty_like(q["r"])
        bbs.nvfp4_moe_gemv(0, q["x"], q["ids"], q["w"], 16, *q["W"], y, 1, residual=q["r"], ws=ws)
        return y

    want = [call(a), call(b)]
    graphs, got = [], []
    for q in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(call(q))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert same(want, got)
        got[0].zero_(), got[1].zero_()


def test_one_expert_is_the_few_token_block(bbs):
    """One expert chosen by all with weight 1 is the gated block of nvfp4_gated_gemv and
    nvfp4_gemv but for the hidden values' rounding to BF16 there."""
    announce("moe: one expert")
    F, K, N, T = 208, 272, 160, 9
    W = [random_nv(bbs, r, c, True, i) for i, (r, c) in enumerate(((F, K), (F, K), (N, F)))]
    x, ids = normal((T, K), torch.bfloat16, 4), torch.zeros((T, 1), dtype=torch.int32, device=dev())
    h, z = torch.empty((T, F), dtype=torch.bfloat16, device=dev()), torch.empty((T, N), device=dev())
    y = torch.empty((T, N), device=dev())
    bbs.nvfp4_gated_gemv(0, x, W[0], W[1], h, 1)
    bbs.nvfp4_gemv(0, h, W[2], z, 0)
    bbs.nvfp4_moe_gemv(0, x, ids, None, 1, *W, y, 0)
    room = (2.0 ** -8 + 600 * ULP) * (h.double().abs() @ nv64(W[2]).abs().t()) + 2.0 ** -20
    assert bool(((y - z).abs().double() <= room).all())


def test_own_workspace_on_another_stream(bbs, monkeypatch):
    """A workspace the call allocates for a given stream is not handed out again while that
    stream has yet to run the call."""
    announce("moe: own workspace, other stream")
    q = problem(bbs, 20, 1)
    eager = run(bbs, q)
    made = []
    make = bbs.moe_workspace
    monkeypatch.setattr(bbs, "moe_workspace", lambda *a: made.append(make(*a)) or made[-1])
    a, s = torch.ones((4096, 4096), device=dev()), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(40):
            a @ a                                                       # milliseconds
    y = torch.empty_like(q["r"])
    s.wait_stream(torch.cuda.current_stream())
    bbs.nvfp4_moe_gemv(0, q["x"], q["ids"], q["w"], 16, *q["W"], y, 1, act=bbs.ACT_GELU, residual=q["r"], stream=s)
    size, at = made[0].numel(), made.pop().data_ptr()
    other = torch.empty((size,), dtype=torch.uint8, device=dev())
    busy = not s.query()
    assert other.data_ptr() != at
    torch.cuda.synchronize()
    assert busy and torch.equal(y, eager[0])


@pytest.mark.parametrize("op", ["moe", "bias"])
def test_own_workspace_leaves_pending_work_alone(bbs, monkeypatch, op):
    """A workspace the call allocates for a given stream is no block that work on the
    current stream, which the given one does not wait for, still uses."""
    announce(f"{op}: own workspace, other stream, pending work on the current one")
    q = problem(bbs, 20, 1)
    dy, db = normal((2048, 512), torch.bfloat16, 1), torch.empty((512,), device=dev())
    ys = torch.empty_like(q["r"]), torch.empty_like(q["r"])

    def call(i, stream=None):
        if op == "moe":
            bbs.nvfp4_moe_gemv(0, q["x"], q["ids"], q["w"], 16, *q["W"], ys[i], 1, residual=q["r"], stream=stream)
            return ys[i]
        bbs.mxfp8_bias_act_bwd(dy, None, bbs.ACT_NONE, None, db, stream=stream)
        return db

    want = call(0).clone()
    size = bbs.moe_workspace(20, 4, 16, 208, 160).numel() if op == "moe" else bbs.BIAS_PARTS * 512 * 4
    made, keep = [], bbs._used_on
    monkeypatch.setattr(bbs, "_used_on", lambda ws, stream: made.append(ws.data_ptr()) or keep(ws, stream))
    a, s = torch.ones((4096, 4096), device=dev()), torch.cuda.Stream()
    call(1, s)                                                          # the stream's pool has memory
    torch.cuda.synchronize()
    for _ in range(40):
        a @ a                                                           # milliseconds, on the current stream
    used = torch.empty((size,), dtype=torch.uint8, device=dev())
    used.fill_(7)
    sums, at = used.view(-1, 256).sum(1), used.data_ptr()               # read after the call below has run
    del used
    got = call(1, s)
    busy = not torch.cuda.current_stream().query()
    s.synchronize()
    assert made[-1] != at and busy
    assert torch.equal(got, want)
    torch.cuda.synchronize()
    assert bool((sums == 7 * 256).all())


def test_own_workspaces_in_a_capture_of_two_streams(bbs):
    """Calls on a given stream that a capture forks to, each with a workspace of its own, and
    others beside them on the capturing stream: every replay gives the eager bits."""
    announce("own workspaces, captured on a forked stream")
    q = problem(bbs, 20, 1)
    dy, x = normal((512, 256), torch.bfloat16, 1), normal((64, 256), torch.bfloat16, 2)
    s = torch.cuda.Stream()

    def both(stream):
        out = []
        for on in (stream, None):
            y, db = torch.empty_like(q["r"]), torch.empty((256,), device=dev())
            row, col = bbs.NVFP4Tensor.empty(64, 256, device=dev()), bbs.NVFP4Tensor.empty(256, 64, device=dev())
            out += [y, db, row.codes, row.scales, row.s_dec, col.codes, col.scales, col.s_dec]
            if on is not None:
                on.wait_stream(torch.cuda.current_stream())
            bbs.nvfp4_moe_gemv(0, q["x"], q["ids"], q["w"], 16, *q["W"], y, 1, residual=q["r"], stream=on)
            bbs.mxfp8_bias_act_bwd(dy, None, bbs.ACT_NONE, None, db, stream=on)
            bbs.nvfp4_quantize(x, row, col, stream=on)
        torch.cuda.current_stream().wait_stream(s)
        return out

    want = both(None)
    for a, b in zip(want, both(s)):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = both(s)
    for i in range(4):
        q["x"].copy_(torch.roll(q["x"], 1, 1))
        dy.copy_(torch.roll(dy, 1, 0)), x.copy_(torch.roll(x, 1, 1))
        graph.replay()
        eager = both(s)
        torch.cuda.synchronize()
        assert same(eager, cap), i
