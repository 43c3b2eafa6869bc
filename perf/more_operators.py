"""What a layer has around its 4-bit products, as cases to be timed and compared.

  linear        y = act(A W^T + b) + r on NVFP4 operands: the product of a prompt or a training batch
                with bias, activation and residual in its epilogue
  linear_train  its training form: the forward pass keeps z = A W^T + b as an 8-bit checkpoint, and the
                backward pass takes dY through the activation and sums the bias' gradient
  linear_gemv   y = act(x W^T + b) + r for a few tokens: BF16 activations, NVFP4 or MXFP4 weights
  moe           a whole mixture-of-experts layer for a few tokens: every token's chosen experts (gated or
                plain), their weighted sum and a residual

With `own` false, run() computes the plain form in FP32 torch operations; with
`own` true it calls the library's entry points."""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    def linear(name, tokens, n, k, act="", bias="", residual=False, tile=True, out="bf16", op="linear", fmt="nvfp4"):
        return {"name": name, "op": op, "tokens": tokens, "n": n, "k": k, "fmt": fmt, "tile": tile, "act": act,
                "bias": bias, "residual": residual, "out": out}

    def moe(name, tokens, experts, top, hidden, features, act="silu", gated=True, fmt="nvfp4", tile=True,
            residual=False, dropped=False, out="bf16"):
        return {"name": name, "op": "moe", "tokens": tokens, "experts": experts, "top": top, "hidden": hidden,
                "features": features, "act": act, "gated": gated, "fmt": fmt, "tile": tile, "residual": residual,
                "dropped": dropped, "out": out}

    return [
        # a prompt's up projection at sizes that fill no tile and no slab
        linear("linear odd sizes", 528, 2736, 1552, act="gelu", bias="f32", tile=False, out="f32"),
        # a short prompt's down projection back into the residual stream
        linear("linear short prompt", 256, 4096, 1536, bias="bf16", residual=True, out="f32"),
        # long prompts through the dense down projection, into the residual stream
        linear("linear dense down", 8192, 4096, 14336, bias="bf16", residual=True),
        # a training step at sizes that fill no tile and no slab
        linear("linear train odd sizes", 272, 1568, 1184, act="silu", bias="f32", tile=False, op="linear_train"),
        # a training step of the dense up projection
        linear("linear train dense up", 8192, 14336, 4096, act="gelu", bias="bf16", op="linear_train"),
        # one token through a small up projection: latency counts
        linear("linear gemv 1 token", 1, 1536, 4096, act="gelu", bias="bf16", op="linear_gemv"),
        # a batch of sequences, one token each, through the dense down projection
        linear("linear gemv 40 tokens", 40, 4096, 14336, bias="f32", residual=True, tile=False, op="linear_gemv",
               fmt="mxfp4", out="f32"),
        # one token through 8 of 64 plain experts
        moe("moe 1 token 8 of 64", 1, 64, 8, 1536, 4096, act="gelu", gated=False),
        # one token through 2 of 8 experts as wide as the dense block
        moe("moe 1 token 2 of 8", 1, 8, 2, 14336, 4096, residual=True),
        # a few sequences at odd sizes, some slots dropped for lack of room
        moe("moe 5 tokens odd sizes", 5, 12, 3, 736, 1568, act="gelu", fmt="mxfp4", tile=False, residual=True,
            dropped=True, out="f32"),
        # a small batch of sequences, MXFP4 experts
        moe("moe 16 tokens mxfp4", 16, 64, 8, 1536, 4096, fmt="mxfp4", tile=False, residual=True),
        # the largest batch: nearly every expert is read
        moe("moe 64 tokens 8 of 64", 64, 64, 8, 1536, 4096, residual=True),
    ]


def draw(rng):
    op = rng.choice(["linear", "linear_train", "linear_gemv", "moe"])

    def size(lo, hi, step):
        # spread over the logarithm, a multiple of step
        return max(lo, min(hi, step * round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)))

    few = op in ("linear_gemv", "moe")
    fmt = rng.choice(["nvfp4", "mxfp4"]) if few else "nvfp4"
    by = 32 if fmt == "mxfp4" or op == "linear_train" else 16
    tokens = size(1, 64, 1) if few else size(16, 8192, 16)
    tile = fmt == "nvfp4" and rng.random() < 0.5
    # gradients taken from 8-bit values are BF16
    out = "bf16" if op == "linear_train" else rng.choice(["bf16", "f32"])
    if op == "moe":
        experts = size(2, 64, 1)
        features = size(256, 4096, by)
        most = 64 * 1536 * 4096 // (experts * features)          # no more weights than the largest listed case
        return {"op": op, "tokens": tokens, "experts": experts, "top": rng.randint(1, min(8, experts)),
                "hidden": size(256, max(256, min(14336, most // by * by)), by), "features": features,
                "act": rng.choice(["silu", "gelu"]), "gated": rng.random() < 0.7, "fmt": fmt, "tile": tile,
                "residual": rng.random() < 0.5, "dropped": rng.random() < 0.25, "out": out}
    k = size(256, 14336, by)
    n = size(256, 14336 if few else min(14336, 14336 * 4096 // k // by * by), by)
    return {"op": op, "tokens": tokens, "n": n, "k": k, "fmt": fmt, "tile": tile,
            "act": rng.choice(["silu", "gelu"] if op == "linear_train" else ["", "silu", "gelu"]),
            "bias": rng.choice(["bf16", "f32"] if op == "linear_train" else ["", "bf16", "f32"]),
            "residual": op != "linear_train" and rng.random() < 0.5, "out": out}


# ---------------------------------------------------------------------------
# Inputs: tensors in the library's layouts (codes, scales, decode scale)
# ---------------------------------------------------------------------------

def _nibbles(v):
    """E2M1 codes of values on or between grid points (nearest), packed two a byte, even column low."""
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)
    c = torch.bucketize(v.abs(), mid, out_int32=True).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
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


def _kind(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    T = case["tokens"]

    def normal(r, c, std=1.0):
        return torch.randn((r, c), generator=g, device=dev) * std

    def activation(k):
        # a few large entries, as the layers' activations have
        x = normal(T, k)
        return torch.where(torch.rand((T, k), generator=g, device=dev) < 0.005, x * 20.0, x)

    def weight(r, c):
        v = normal(r, c, c ** -0.5)
        return _to_nvfp4(v, case["tile"]) if case["fmt"] == "nvfp4" else _to_mxfp4(v)

    st = {"case": dict(case)}
    if case["op"] == "moe":
        E, F, K, top = case["experts"], case["hidden"], case["features"], case["top"]
        st["x"] = activation(K).bfloat16()
        for name, r, c in (("wg", F, K), ("wu", F, K), ("wd", K, F)):
            if name != "wg" or case["gated"]:
                parts = [weight(r, c) for _ in range(E)]             # an expert's weight is a tensor of its own
                st[name] = tuple(torch.cat(p) for p in zip(*parts))
        # a Zipf law over the experts, as trained routers show
        score = -1.1 * torch.log(torch.randperm(E, generator=g, device=dev) + 1.0)
        score = score - torch.log(-torch.log(torch.rand((T, E), generator=g, device=dev).clamp(1e-9, 1 - 1e-7)))
        st["ids"] = torch.topk(score, top).indices.to(torch.int32)
        if case["dropped"]:
            st["ids"] = torch.where(torch.rand((T, top), generator=g, device=dev) < 0.1, -1, st["ids"]).to(torch.int32)
        st["weights"] = torch.softmax(normal(T, top), dim=1)
        N = K
    else:
        N, K = case["n"], case["k"]
        x = activation(K)
        st["x"] = x.bfloat16() if case["op"] == "linear_gemv" else _to_nvfp4(x, False)
        st["w"] = weight(N, K)
        if case["bias"]:
            st["b"] = normal(1, N, 0.2).reshape(N).to(_kind(case["bias"]))
    kind = _kind(case["out"])
    if case["op"] != "linear_train" and case["residual"]:
        st["r"] = normal(T, N).to(kind)
    st["y"] = torch.empty((T, N), dtype=kind, device=dev)
    if case["op"] == "linear_train":
        u = torch.rand((T, N), generator=g, device=dev) - 0.5
        st["dy"] = (-7e-4 * u.sign() * torch.log1p(-1.9999998 * u.abs())).bfloat16()      # Laplace, std 1e-3
        st["z8"] = (torch.empty((T, N), dtype=torch.uint8, device=dev),
                    torch.empty((T, N // 32), dtype=torch.uint8, device=dev))
        st["dz"] = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
        st["db"] = torch.empty((N,), dtype=torch.bfloat16, device=dev)
    return st


# ---------------------------------------------------------------------------
# The plain form: FP32 torch operations
# ---------------------------------------------------------------------------

def _codes_f32(codes):
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    pair = torch.stack((codes & 15, codes >> 4), dim=-1)
    return table[pair.int()].view(codes.shape[0], -1)


def _dequant(fmt, w):
    """An NVFP4 or MXFP4 matrix in FP32, without NVFP4's decode scale."""
    v = _codes_f32(w[0])
    r, c = v.shape
    if fmt == "mxfp4":
        return (v.view(r, c // 32, 32) * torch.exp2(w[1].float() - 127)[:, :, None]).view(r, c)
    s = w[1].view(torch.float8_e4m3fn).float()
    s = s.repeat_interleave(16, 0) if s.shape[0] != r else s
    return (v.view(r, c // 16, 16) * s[:, :, None]).view(r, c)


def _sigmoid_arg(act, g):
    """act(g) = g * sigmoid(z): (z, dz/dg)."""
    if act == "silu":
        return g, torch.ones_like(g)
    c = math.sqrt(2.0 / math.pi)
    return 2 * c * (g + 0.044715 * (g * g * g)), 2 * c * (1 + 3 * 0.044715 * (g * g))


def _act(act, g):
    if not act:
        return g
    z, _ = _sigmoid_arg(act, g)
    return g / (1 + torch.exp(-z))


def _act_grad(act, g):
    z, dz = _sigmoid_arg(act, g)
    s = 1 / (1 + torch.exp(-z))
    return s + g * s * (1 - s) * dz


def _mxfp8_f32(codes, scales):
    r, c = codes.shape
    v = codes.view(torch.float8_e4m3fn).float().view(r, c // 32, 32)
    return (v * torch.exp2(scales.float() - 127)[:, :, None]).view(r, c)


def _with_residual(st, y):
    y = y + st["r"].float() if "r" in st else y
    return y.to(st["y"].dtype)


def _plain_linear(st):
    case = st["case"]
    a = _dequant("nvfp4", st["x"]) if case["op"] != "linear_gemv" else st["x"].float()
    z = a @ _dequant(case["fmt"], st["w"]).t()
    if case["fmt"] == "nvfp4":
        z = z * (st["w"][2] if case["op"] == "linear_gemv" else st["x"][2] * st["w"][2])
    if "b" in st:
        z = z + st["b"].float()
    y = _with_residual(st, _act(case["act"], z))
    if case["op"] != "linear_train":
        return y
    # the checkpoint: MXFP8 to nearest, read back
    dz = st["dy"].float() * _act_grad(case["act"], _mxfp8_f32(*_to_mxfp8(z)))
    return {"y": y, "dz": dz.to(st["dz"].dtype), "db": dz.sum(dim=0).to(st["db"].dtype)}


def _plain_moe(st):
    case, ids = st["case"], st["ids"].long()
    T, top, E, F, K = case["tokens"], case["top"], case["experts"], case["hidden"], case["features"]
    # the experts of this batch: the chosen ones where they are fewer than all
    if T * top < E:
        chosen = ids.reshape(-1).clamp(min=0)
        again = (chosen[:, None] == chosen[None, :]).tril(-1).any(dim=1)      # an expert that an earlier slot chose
    else:
        chosen = torch.arange(E, device=ids.device)
        again = torch.zeros_like(chosen, dtype=torch.bool)
    A = chosen.numel()

    def experts(w, rows):
        w = [t.view(E, -1, *t.shape[1:])[chosen] for t in w]
        v = _dequant(case["fmt"], [t.flatten(0, 1) for t in w[:2]]).view(A, rows, -1)
        return v * w[2].view(A, 1, 1) if case["fmt"] == "nvfp4" else v

    def project(w):
        return (st["x"].float() @ experts(w, F).view(A * F, K).t()).view(T, A, F)

    u = project(st["wu"])
    h = _act(case["act"], project(st["wg"])) * u if case["gated"] else _act(case["act"], u)
    slot = (ids[:, :, None] == chosen[None, None, :]) & ~again
    share = (st["weights"][:, :, None] * slot).sum(dim=1)                     # [T, A]
    down = experts(st["wd"], K).permute(0, 2, 1).reshape(A * F, K)
    return _with_residual(st, (h * share[:, :, None]).view(T, A * F) @ down)


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------

def _own(st):
    import bit_block_scaled_amd as bbs

    case, y = st["case"], st["y"]
    kind = bbs.OUT_BF16 if case["out"] == "bf16" else bbs.OUT_F32
    act = {"": bbs.ACT_NONE, "silu": bbs.ACT_SILU, "gelu": bbs.ACT_GELU}[case["act"]]
    fmt = bbs.FMT_MXFP4 if case["fmt"] == "mxfp4" else bbs.FMT_NVFP4

    def weight(w, rows, cols):
        if case["fmt"] == "mxfp4":
            return bbs.MXFP4Tensor(w[0], w[1], rows, cols)
        return bbs.NVFP4Tensor(w[0], w[1], w[2], rows, cols, case["tile"])

    if case["op"] == "moe":
        E, F, K = case["experts"], case["hidden"], case["features"]
        wg = weight(st["wg"], E * F, K) if case["gated"] else None
        bbs.nvfp4_moe_gemv(fmt, st["x"], st["ids"], st["weights"], E, wg, weight(st["wu"], E * F, K),
                           weight(st["wd"], E * K, F), y, kind, act=act, residual=st.get("r"))
        return y
    T, N, K = case["tokens"], case["n"], case["k"]
    w = weight(st["w"], N, K)
    if case["op"] == "linear_gemv":
        bbs.nvfp4_gemv_bias_act(fmt, st["x"], w, y, kind, bias=st.get("b"), act=act, residual=st.get("r"))
        return y
    a = bbs.NVFP4Tensor(*st["x"], T, K, False)
    if case["op"] == "linear":
        bbs.nvfp4_gemm_bias_act(a, w, y, kind, bias=st.get("b"), act=act, residual=st.get("r"))
        return y
    z8 = bbs.MXFP8Tensor(*st["z8"], T, N)
    bbs.nvfp4_gemm_bias_act(a, w, y, kind, bias=st["b"], act=act, z_ckpt=z8)
    bbs.mxfp8_bias_act_bwd(st["dy"], z8, act, st["dz"], st["db"])
    return {"y": y, "dz": st["dz"], "db": st["db"]}


def run(state):
    if own:
        return _own(state)
    return _plain_moe(state) if state["case"]["op"] == "moe" else _plain_linear(state)


def work(case):
    T = case["tokens"]
    es = 2 if case["out"] == "bf16" else 4
    per = 1 / 2 + (1 / 32 if case["fmt"] == "mxfp4" else 1 / 256 if case["tile"] else 1 / 16)
    if case["op"] == "moe":
        E, F, K, top = case["experts"], case["hidden"], case["features"], case["top"]
        mats = 3 if case["gated"] else 2
        # the experts that a batch reads: all its slots' while they are few, all there are at the most
        read = min(E, T * top)
        return {"bytes": read * mats * F * K * per + T * K * (2 + es * (2 if case["residual"] else 1)) + 8 * T * top,
                "flops": 2 * mats * T * top * F * K}
    N, K = case["n"], case["k"]
    x = T * K * (2 if case["op"] == "linear_gemv" else 9 / 16)
    b = x + N * K * per + T * N * es * (2 if case["residual"] else 1)
    b += {"": 0, "bf16": 2, "f32": 4}[case["bias"]] * N
    f = 2 * T * N * K
    if case["op"] == "linear_train":
        b += T * N * (33 / 32 + 2 + 2) + 2 * N
        f += 16 * T * N
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
    """The values of an NVFP4 (three parts) or MXFP4 matrix."""
    v = _e2m1_64(w[0])
    if len(w) == 3:
        s = _e4m3_64(w[1])
        s = s.repeat_interleave(v.shape[0] // s.shape[0], 0).repeat_interleave(16, 1)
        return v.mul_(s).mul_(w[2].double())
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


def _act64(act, v):
    """The activation and its slope."""
    if not act:
        return v, torch.ones_like(v)
    if act == "silu":
        s = torch.sigmoid(v)
        return v * s, s * (1 + v * (1 - s))
    r = math.sqrt(2 / math.pi)
    th = torch.tanh(r * (v + 0.044715 * v ** 3))
    return 0.5 * v * (1 + th), 0.5 * (1 + th) + 0.5 * v * (1 - th * th) * r * (1 + 0.134145 * v * v)


def exact(case, seed):
    st = prepare(case, seed)
    r = st["r"].double() if "r" in st else 0.0
    if case["op"] == "moe":
        x, out = st["x"].double(), torch.zeros(st["y"].shape, dtype=torch.float64, device=st["y"].device)
        for e in range(case["experts"]):
            mine = st["ids"] == e
            rows = mine.any(dim=1).nonzero()[:, 0]
            if not rows.numel():
                continue

            def part(name):
                return _value64([t.chunk(case["experts"])[e] for t in st[name]])

            h = x[rows] @ part("wu").t()
            if case["gated"]:
                h = _act64(case["act"], x[rows] @ part("wg").t())[0] * h
            else:
                h = _act64(case["act"], h)[0]
            share = torch.where(mine, st["weights"].double(), 0.0).sum(dim=1)[rows]
            out[rows] += share[:, None] * (h @ part("wd").t())
        return out + r
    x = st["x"].double() if torch.is_tensor(st["x"]) else _value64(st["x"])
    z = x @ _value64(st["w"]).t()
    if "b" in st:
        z = z + st["b"].double()
    y = _act64(case["act"], z)[0] + r
    if case["op"] != "linear_train":
        return y
    dz = st["dy"].double() * _act64(case["act"], _round8_64(z))[1]
    return {"y": y, "dz": dz, "db": dz.sum(dim=0)}
