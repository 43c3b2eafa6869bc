"""The operators of the gated feed-forward block on 4-bit weights, as cases to be timed and compared.

  gemv         y = x W^T for a few tokens: BF16 activations, NVFP4 or MXFP4 weights
  gated_gemv   h = act(x Wg^T) * (x Wu^T), the same for the block's two up projections
  gated_gemm   the same on NVFP4 activations for many tokens (prompt processing)
  gated_train  the training form: the forward pass keeps the two projections as
               8-bit checkpoints, and the backward pass takes dY back through the
               down projection and the gated activation from them

With `own` false, run() computes the plain form in FP32 torch operations; with
`own` true it calls the library's entry points."""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token through one expert's up projection: latency counts
        {"name": "gemv 1 token, expert", "op": "gemv", "tokens": 1, "n": 1536, "k": 4096, "fmt": "nvfp4",
         "tile": True, "act": "", "out": "bf16"},
        # one token through a dense down projection: a long sum, FP32 out
        {"name": "gemv 1 token, down", "op": "gemv", "tokens": 1, "n": 4096, "k": 14336, "fmt": "nvfp4",
         "tile": False, "act": "", "out": "f32"},
        # a few sequences at sizes that fill no tile
        {"name": "gemv 5 tokens, odd sizes", "op": "gemv", "tokens": 5, "n": 4112, "k": 1552, "fmt": "nvfp4",
         "tile": False, "act": "", "out": "bf16"},
        # a batch of sequences, one token each, through an MXFP4 up projection
        {"name": "gemv 48 tokens, mxfp4", "op": "gemv", "tokens": 48, "n": 14336, "k": 4096, "fmt": "mxfp4",
         "tile": False, "act": "", "out": "bf16"},
        # one token through both up projections of the dense block
        {"name": "gated gemv 1 token", "op": "gated_gemv", "tokens": 1, "n": 14336, "k": 4096, "fmt": "nvfp4",
         "tile": True, "act": "silu", "out": "bf16"},
        # a small batch through one expert's two projections
        {"name": "gated gemv 13 tokens", "op": "gated_gemv", "tokens": 13, "n": 1536, "k": 4096, "fmt": "mxfp4",
         "tile": False, "act": "gelu", "out": "f32"},
        # a prompt at sizes that fill no tile and no slab
        {"name": "gated gemm, odd sizes", "op": "gated_gemm", "tokens": 528, "n": 2736, "k": 1552, "fmt": "nvfp4",
         "tile": False, "act": "silu", "out": "bf16"},
        # one expert's share of a batch of prompts
        {"name": "gated gemm, expert", "op": "gated_gemm", "tokens": 2048, "n": 1536, "k": 4096, "fmt": "nvfp4",
         "tile": True, "act": "gelu", "out": "f32"},
        # long prompts through the dense block
        {"name": "gated gemm, dense", "op": "gated_gemm", "tokens": 8192, "n": 14336, "k": 4096, "fmt": "nvfp4",
         "tile": True, "act": "silu", "out": "bf16"},
        # a training step at sizes that fill no tile and no slab
        {"name": "gated train, odd sizes", "op": "gated_train", "tokens": 272, "n": 1568, "k": 1184,
         "fmt": "nvfp4", "tile": False, "act": "gelu", "out": "bf16"},
        # a training step of a small block
        {"name": "gated train, small", "op": "gated_train", "tokens": 2048, "n": 4096, "k": 1536, "fmt": "nvfp4",
         "tile": True, "act": "silu", "out": "bf16"},
        # a training step of the dense block
        {"name": "gated train, dense", "op": "gated_train", "tokens": 8192, "n": 14336, "k": 4096, "fmt": "nvfp4",
         "tile": True, "act": "silu", "out": "bf16"},
    ]


def draw(rng):
    op = rng.choice(["gemv", "gated_gemv", "gated_gemm", "gated_train"])

    def size(lo, hi, step):
        # spread over the logarithm, a multiple of step
        return max(lo, min(hi, step * round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)))

    few = op in ("gemv", "gated_gemv")
    fmt = rng.choice(["nvfp4", "mxfp4"]) if few else "nvfp4"
    by = 32 if fmt == "mxfp4" or op == "gated_train" else 16
    return {"op": op, "tokens": size(1, 64, 1) if few else size(16, 8192, 16), "n": size(256, 14336, by),
            "k": size(256, 14336 if op == "gemv" else 4096, by), "fmt": fmt,
            "tile": fmt == "nvfp4" and rng.random() < 0.5,
            "act": "" if op == "gemv" else rng.choice(["silu", "gelu"]),
            # gradients taken from 8-bit values are BF16
            "out": "bf16" if op == "gated_train" else rng.choice(["bf16", "f32"])}


# ---------------------------------------------------------------------------
# Inputs: tensors in the library's layouts (codes, scales, decode scale)
# ---------------------------------------------------------------------------

def _nibbles(v):
    """E2M1 codes of values on or between grid points (nearest), packed two a byte, even column low."""
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)
    c = torch.bucketize(v.abs(), mid).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous()


def _to_nvfp4(v, tile):
    """(codes, E4M3 scale bytes, decode scale) of an FP32 matrix, 1x16 blocks or 16x16 tiles."""
    r, c = v.shape
    s_enc = 2688.0 / v.abs().amax()
    a = v.view(r // 16, 16, c // 16, 16).abs().amax(dim=(1, 3)) if tile else v.view(r, c // 16, 16).abs().amax(dim=2)
    sc = (a / 6 * s_enc).clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn)
    full = sc.float().repeat_interleave(16, 0) if tile else sc.float()
    q = v.view(r, c // 16, 16) * (s_enc / full)[:, :, None]
    return _nibbles(q.view(r, c)), sc.view(torch.uint8), (1.0 / s_enc).reshape(1)


def _to_mx(v, top):
    """(values scaled by 2^-k, E8M0 bytes) of an FP32 matrix: 32-blocks, the smallest 2^k with amax <= top 2^k."""
    r, c = v.shape
    m, e = torch.frexp(v.view(r, c // 32, 32).abs().amax(dim=2) / top)
    k = torch.where(m == 0.5, e - 1, e).clamp(-127, 127)
    return torch.ldexp(v.view(r, c // 32, 32), -k[:, :, None]).view(r, c), (k + 127).to(torch.uint8)


def _to_mxfp4(v):
    q, s = _to_mx(v, 6.0)
    return _nibbles(q), s


def _to_mxfp8(v):
    q, s = _to_mx(v, 448.0)
    return q.to(torch.float8_e4m3fn).view(torch.uint8), s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    T, N, K = case["tokens"], case["n"], case["k"]
    few = case["op"] in ("gemv", "gated_gemv")

    def normal(r, c, std):
        return torch.randn((r, c), generator=g, device=dev) * std

    def activation():
        # a few large entries, as the layers' activations have
        x = normal(T, K, 1.0)
        return torch.where(torch.rand((T, K), generator=g, device=dev) < 0.005, x * 20.0, x)

    st = {"case": dict(case)}
    st["x"] = activation().bfloat16() if few else _to_nvfp4(activation(), False)
    for w in ("w",) if case["op"] == "gemv" else ("wg", "wu"):
        v = normal(N, K, K ** -0.5)
        st[w] = _to_nvfp4(v, case["tile"]) if case["fmt"] == "nvfp4" else _to_mxfp4(v)
    kind = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    st["y"] = torch.empty((T, N), dtype=kind, device=dev)
    if case["op"] == "gated_train":
        u = torch.rand((T, K), generator=g, device=dev) - 0.5
        st["dy"] = _to_mxfp8(-7e-4 * u.sign() * torch.log1p(-1.9999998 * u.abs()))     # Laplace, std 1e-3
        st["wt"] = _to_mxfp8(normal(N, K, N ** -0.5))
        st["dgu"] = torch.empty((T, 2 * N), dtype=kind, device=dev)
        st["g8"], st["u8"] = ((torch.empty((T, N), dtype=torch.uint8, device=dev),
                               torch.empty((T, N // 32), dtype=torch.uint8, device=dev)) for _ in range(2))
    return st


# ---------------------------------------------------------------------------
# The plain form: FP32 torch operations
# ---------------------------------------------------------------------------

def _codes_f32(codes):
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    pair = torch.stack((codes & 15, codes >> 4), dim=-1)
    return table[pair.long()].view(codes.shape[0], -1)


def _dequant(case, w):
    """An NVFP4 or MXFP4 matrix in FP32, without NVFP4's decode scale."""
    v = _codes_f32(w[0])
    r, c = v.shape
    if case["fmt"] == "mxfp4":
        return (v.view(r, c // 32, 32) * torch.exp2(w[1].float() - 127)[:, :, None]).view(r, c)
    s = w[1].view(torch.float8_e4m3fn).float()
    s = s.repeat_interleave(16, 0) if s.shape[0] != r else s
    return (v.view(r, c // 16, 16) * s[:, :, None]).view(r, c)


def _product(case, x, w):
    """x w^T in FP32, decode scales applied."""
    few = torch.is_tensor(x)
    a = x.float() if few else _dequant({"fmt": "nvfp4"}, x)
    y = a @ _dequant(case, w).t()
    if case["fmt"] == "nvfp4":
        y = y * (w[2] if few else x[2] * w[2])
    return y


def _sigmoid_arg(case, g):
    """act(g) = g * sigmoid(z): (z, dz/dg)."""
    if case["act"] == "silu":
        return g, torch.ones_like(g)
    c = math.sqrt(2.0 / math.pi)
    return 2 * c * (g + 0.044715 * (g * g * g)), 2 * c * (1 + 3 * 0.044715 * (g * g))


def _act(case, g):
    z, _ = _sigmoid_arg(case, g)
    return g / (1 + torch.exp(-z))


def _act_grad(case, g):
    z, dz = _sigmoid_arg(case, g)
    s = 1 / (1 + torch.exp(-z))
    return s + g * s * (1 - s) * dz


def _mxfp8_f32(codes, scales):
    r, c = codes.shape
    v = codes.view(torch.float8_e4m3fn).float().view(r, c // 32, 32)
    return (v * torch.exp2(scales.float() - 127)[:, :, None]).view(r, c)


def _plain(st):
    case = st["case"]
    kind = st["y"].dtype
    if case["op"] == "gemv":
        return _product(case, st["x"], st["w"]).to(kind)
    g, u = _product(case, st["x"], st["wg"]), _product(case, st["x"], st["wu"])
    h = (_act(case, g) * u).to(kind)
    if case["op"] != "gated_train":
        return h
    # the checkpoints: MXFP8 to nearest, read back
    g, u = _mxfp8_f32(*_to_mxfp8(g)), _mxfp8_f32(*_to_mxfp8(u))
    dh = _mxfp8_f32(*st["dy"]) @ _mxfp8_f32(*st["wt"]).t()
    return {"h": h, "dgate": (dh * u * _act_grad(case, g)).to(kind), "dup": (dh * _act(case, g)).to(kind)}


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------

def _own(st):
    import bit_block_scaled_amd as bbs

    case, y = st["case"], st["y"]
    T, N, K = case["tokens"], case["n"], case["k"]
    kind = bbs.OUT_BF16 if case["out"] == "bf16" else bbs.OUT_F32
    act = bbs.ACT_GELU if case["act"] == "gelu" else bbs.ACT_SILU

    def weight(w):
        if case["fmt"] == "mxfp4":
            return bbs.MXFP4Tensor(w[0], w[1], N, K)
        return bbs.NVFP4Tensor(w[0], w[1], w[2], N, K, case["tile"])

    fmt = bbs.FMT_MXFP4 if case["fmt"] == "mxfp4" else bbs.FMT_NVFP4
    if case["op"] == "gemv":
        bbs.nvfp4_gemv(fmt, st["x"], weight(st["w"]), y, kind)
        return y
    if case["op"] == "gated_gemv":
        bbs.nvfp4_gated_gemv(fmt, st["x"], weight(st["wg"]), weight(st["wu"]), y, kind, act=act)
        return y
    a = bbs.NVFP4Tensor(*st["x"], T, K, False)
    if case["op"] == "gated_gemm":
        bbs.nvfp4_gated_gemm(a, weight(st["wg"]), weight(st["wu"]), y, kind, act=act)
        return y
    g8, u8 = bbs.MXFP8Tensor(*st["g8"], T, N), bbs.MXFP8Tensor(*st["u8"], T, N)
    bbs.nvfp4_gated_gemm(a, weight(st["wg"]), weight(st["wu"]), y, kind, act=act, g_ckpt=g8, u_ckpt=u8)
    dgate, dup = st["dgu"][:, :N], st["dgu"][:, N:]
    bbs.mxfp8_gemm_gated_bwd(bbs.MXFP8Tensor(*st["dy"], T, K), bbs.MXFP8Tensor(*st["wt"], N, K), g8, u8, dgate, dup,
                             kind, act=act)
    return {"h": y, "dgate": dgate, "dup": dup}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    T, N, K = case["tokens"], case["n"], case["k"]
    out = T * N * (2 if case["out"] == "bf16" else 4)
    per = 1 / 2 + (1 / 32 if case["fmt"] == "mxfp4" else 1 / 256 if case["tile"] else 1 / 16)
    mats = 1 if case["op"] == "gemv" else 2
    x = T * K * (2 if case["op"] in ("gemv", "gated_gemv") else 9 / 16)
    b, f = x + mats * N * K * per + out, 2 * mats * T * N * K
    if case["op"] == "gated_train":
        b += (T + N) * K * 33 / 32 + 2 * out
        f += 2 * T * N * K
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def _e4m3_64(b):
    """E4M3 bytes by their fields."""
    b = b.to(torch.int64)
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2((e - 7).double()))
    return torch.where(b >= 128, -mag, mag)


def _e2m1_64(codes):
    """E2M1 nibbles by their fields: even columns low, odd columns high."""
    n = torch.stack((codes & 15, codes >> 4), dim=2).flatten(1)
    e, m = ((n >> 1) & 3).double(), (n & 1).double()
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e - 1))
    return torch.where(n >= 8, -mag, mag)


def _value64(w):
    """The values of an NVFP4 (three parts), MXFP4 (half as many code bytes as values) or MXFP8 matrix."""
    if len(w) == 3:
        v, s = _e2m1_64(w[0]), _e4m3_64(w[1])
        s = s.repeat_interleave(v.shape[0] // s.shape[0], 0).repeat_interleave(16, 1)
        return v.mul_(s).mul_(w[2].double())
    v = _e4m3_64(w[0]) if w[0].shape[1] == 32 * w[1].shape[1] else _e2m1_64(w[0])
    return v.mul_(torch.exp2(w[1].double() - 127).repeat_interleave(32, 1))


def _round8_64(v):
    """v through an 8-bit checkpoint: the smallest 2^k with amax <= 448 2^k, E4M3 to nearest even."""
    b = v.view(v.shape[0], -1, 32)
    a = b.abs().amax(dim=2, keepdim=True)
    k = torch.ceil(torch.log2(a.clamp_min(2.0 ** -140) / 448))
    k = k + (a > 448 * torch.exp2(k)) - (a <= 448 * torch.exp2(k - 1)).double()
    unit = torch.exp2(k.clamp(-127, 127))
    t = b / unit
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(t / step) * step * unit).view(v.shape)


def exact(case, seed):
    st = prepare(case, seed)
    x = st["x"].double() if torch.is_tensor(st["x"]) else _value64(st["x"])
    if case["op"] == "gemv":
        return x @ _value64(st["w"]).t()
    g = x @ _value64(st["wg"]).t()
    u = x @ _value64(st["wu"]).t()

    def act_and_slope(v):
        if case["act"] == "silu":
            s = torch.sigmoid(v)
            return v * s, s * (1 + v * (1 - s))
        r = math.sqrt(2 / math.pi)
        th = torch.tanh(r * (v + 0.044715 * v ** 3))
        return 0.5 * v * (1 + th), 0.5 * (1 + th) + 0.5 * v * (1 - th * th) * r * (1 + 0.134145 * v * v)

    h = act_and_slope(g)[0] * u
    if case["op"] != "gated_train":
        return h
    g, u = _round8_64(g), _round8_64(u)
    a, slope = act_and_slope(g)
    dh = _value64(st["dy"]) @ _value64(st["wt"]).t()
    return {"h": h, "dgate": dh * u * slope, "dup": dh * a}
