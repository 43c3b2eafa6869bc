"""NVFP4 quantized layers: torch.autograd.Functions over the C ABI.

QLinear, one linear layer:

The recipe of 4bit.vizuara.ai, sections 8-10 and 13 (Figure 13) and of
Pretraining LLMs with NVFP4 ("Random Hadamard Transforms", "Two-Dimensional
Weight Scaling", "Stochastic Rounding"):

forward   X -> NVFP4 rows (1x16, nearest) for the forward GEMM, and the
          NVFP4 copy of X^T (16-point RHT, stochastic) kept for wgrad;
          W -> NVFP4 with 16x16 tile scales (nearest); Y = X W^T (NVFP4
          GEMM, BF16 out).
backward  dY -> the NVFP4 copy of dY^T (RHT, stochastic) and the MXFP8 rows
          of dY (stochastic); W's NVFP4 copy -> MXFP8 of W^T (stochastic);
          dX = dY W (MXFP8 GEMM, BF16 out); dW = dY^T X (NVFP4 GEMM over the
          two RHT'd copies, FP32 accumulation, written by the kernel in the
          weight's dtype: BF16, nearest even, or FP32).

Every step runs in the library's kernels; this module only allocates the
outputs and passes pointers.  The stochastic roundings of call t draw from
Philox streams 4t .. 4t + 3 under the layer's seed, so a run is reproducible.
Shapes: tokens, in_features and out_features multiples of 32 (the MXFP8
copies block 32 values).
With bias, act or a residual, Y = act(X W^T + b) + R is one kernel that keeps
z = X W^T + b as an 8-bit (MXFP8) checkpoint; the backward pass first takes dY
through the activation and sums the bias' gradient in one pass, and goes on from
dZ as above.  Kept then, in bits a value: 4.5 for X, 8.25 for z with an
activation, and of those only what the wanted gradients read.  Outputs are BF16, and so
is a residual: one of another type is rounded to BF16 first, then added in FP32 and
rounded with the sum.
QLinearInference holds the quantized weight of such a layer, and
QMoEInference a layer of experts; up to GEMV_MAX_TOKENS tokens are answered by the
few-token kernels (activations in BF16).

QGatedMLP, a gated feed-forward block y = (act(x Wg^T) * (x Wu^T)) Wd^T by
the same recipe:

forward   X -> NVFP4 rows and the NVFP4 copy of X^T (RHT, stochastic); the
          stacked [Wg; Wu] and Wd -> NVFP4 with 16x16 tile scales; one kernel
          computes both products, the activation and H, and keeps the two
          products as 8-bit (MXFP8) checkpoints; H -> NVFP4 rows and the
          NVFP4 copy of H^T (RHT, stochastic); Y = H Wd^T.
backward  dY -> the NVFP4 copy of dY^T and MXFP8 rows; Wd's copy -> MXFP8 of
          Wd^T; one kernel computes dH and turns it, with the checkpoints,
          into [dG, dU]; these -> the NVFP4 copy of [dG, dU]^T and MXFP8 rows;
          dWd = dY^T H, d[Wg; Wu] = [dG, dU]^T X (NVFP4), dX = [dG, dU] [Wg; Wu]
          (MXFP8).

Kept for the backward pass, in bits a value: 4.5 for X, 4.5 + 2 * 8.25 for the
hidden values, and of those only what the wanted gradients read (nothing under
torch.no_grad).  Call t draws from Philox streams 8t .. 8t + 7.
QGatedMLPInference holds the quantized weights of such a block and answers
with the matrix-vector kernels (activations in BF16) up to GEMV_MAX_TOKENS
tokens, with the GEMMs beyond.
"""
import torch
from torch.autograd.function import once_differentiable

from . import (ACT_GELU, ACT_NONE, ACT_SILU, FMT_MXFP8, FMT_NVFP4, GEMV_MAX_TOKENS, MOE_MAX_EXPERTS, OUT_BF16,
               OUT_F32, SR, MXFP8Tensor, NVFP4Tensor, amax_workspace, mxfp8_bias_act_bwd, mxfp8_gemm_gated_bwd,
               mxfp8_requantize_t, nvfp4_gated_gemm, nvfp4_gated_gemv, nvfp4_gemm, nvfp4_gemm_bias_act,
               nvfp4_gemv, nvfp4_gemv_bias_act, nvfp4_moe_gemv, nvfp4_quantize, _on_current)


def _bits(t):
    """A BF16 tensor as its 16-bit patterns (no copy when already BF16 and contiguous)."""
    return t.to(torch.bfloat16).contiguous().view(torch.int16)


class QLinearFn(torch.autograd.Function):
    """y = x @ w^T with the NVFP4 recipe; x [..., in], w [out, in] (BF16)."""

    @staticmethod
    def forward(ctx, x, w, seed, step, signs):
        lead = x.shape[:-1]
        K = x.shape[-1]
        N = w.shape[0]
        x2 = _bits(x.reshape(-1, K))
        M = x2.shape[0]
        dev = x.device
        ws = amax_workspace(dev)
        xq = NVFP4Tensor.empty(M, K, device=dev)
        xc = NVFP4Tensor.empty(K, M, device=dev)
        nvfp4_quantize(x2, xq, xc, col_round=SR, col_rng=(seed, 4 * step), col_rht=True,
                       rht_signs=signs, amax_ws=ws)
        wq = NVFP4Tensor.empty(N, K, tile2d=True, device=dev)
        nvfp4_quantize(_bits(w), wq, tile2d=True, amax_ws=ws)
        y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        nvfp4_gemm(FMT_NVFP4, xq, wq, y.view(torch.int16), OUT_BF16)
        ctx.save_for_backward(xc.codes, xc.scales, xc.s_dec, wq.codes, wq.scales, wq.s_dec)
        ctx.dims = (M, K, N, lead, w.dtype)
        ctx.rng = (seed, step, signs)
        return y.reshape(*lead, N)

    @staticmethod
    def backward(ctx, dy):
        M, K, N, lead, wdtype = ctx.dims
        seed, step, signs = ctx.rng
        xcc, xcs, xcd, wqc, wqs, wqd = ctx.saved_tensors
        xc = NVFP4Tensor(xcc, xcs, xcd, K, M, False)
        wq = NVFP4Tensor(wqc, wqs, wqd, N, K, True)
        dev = dy.device
        g = _bits(dy.reshape(M, N))
        gc = NVFP4Tensor.empty(N, M, device=dev)
        gm = MXFP8Tensor.empty(M, N, device=dev)
        nvfp4_quantize(g, None, gc, gm, col_round=SR, col_rng=(seed, 4 * step + 1), col_rht=True,
                       rht_signs=signs, mx8_round=SR, mx8_rng=(seed, 4 * step + 2),
                       amax_ws=amax_workspace(dev))
        wt = MXFP8Tensor.empty(K, N, device=dev)
        mxfp8_requantize_t(wq, wt, SR, (seed, 4 * step + 3))
        dx = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
        nvfp4_gemm(FMT_MXFP8, gm, wt, dx.view(torch.int16), OUT_BF16)
        if wdtype == torch.bfloat16:
            dw = torch.empty((N, K), dtype=torch.bfloat16, device=dev)
            nvfp4_gemm(FMT_NVFP4, gc, xc, dw.view(torch.int16), OUT_BF16)
        else:
            dw = torch.empty((N, K), dtype=torch.float32, device=dev)
            nvfp4_gemm(FMT_NVFP4, gc, xc, dw, OUT_F32)
            dw = dw.to(wdtype)
        return dx.reshape(*lead, K), dw, None, None, None


_ACTS = {"silu": ACT_SILU, "gelu": ACT_GELU}


def _act_code(act):
    return ACT_NONE if act is None else _ACTS[act]


def _aligned(t):
    """A contiguous tensor from a 16-byte aligned address on."""
    return t if t is None or t.data_ptr() % 16 == 0 else t.clone()


def _bias(b):
    """A bias as the kernels read it: adjacent BF16 or FP32 values."""
    return b if b is None else _aligned((b if b.dtype == torch.bfloat16 else b.float()).contiguous())


def _residual(r, rows, features):
    return r if r is None else _aligned(r.reshape(rows, features).to(torch.bfloat16).contiguous())


def _check_residual(r, lead, features):
    if r is not None and r.shape != (*lead, features):
        raise ValueError("residual must have the output's shape")


def _nvfp4_weight(w, ws):
    """The 16x16-tiled NVFP4 copy of a weight."""
    q = NVFP4Tensor.empty(*w.shape, tile2d=True, device=w.device)
    nvfp4_quantize(_bits(w), q, tile2d=True, amax_ws=ws)
    return q


def _halves(q):
    """The upper and lower half of a stacked 16x16-tiled NVFP4 tensor (views)."""
    F = q.rows // 2
    return (NVFP4Tensor(q.codes[:F], q.scales[:F // 16], q.s_dec, F, q.cols, True),
            NVFP4Tensor(q.codes[F:], q.scales[F // 16:], q.s_dec, F, q.cols, True))


def _wgrad(gc, xc, dtype, dev):
    """dW = gc xc^T in the weight's dtype (BF16 and FP32 straight from the kernel)."""
    bf16 = dtype == torch.bfloat16
    dw = torch.empty((gc.rows, xc.rows), dtype=torch.bfloat16 if bf16 else torch.float32, device=dev)
    nvfp4_gemm(FMT_NVFP4, gc, xc, dw, OUT_BF16 if bf16 else OUT_F32)
    return dw.to(dtype)


class QLinearBiasActFn(torch.autograd.Function):
    """y = act(x @ w^T + b) + r; x [..., in], w [out, in], b [out] or None, r [..., out]
    or None.  grad: whether the call is recorded (a Function does not see grad mode
    itself)."""

    @staticmethod
    def forward(ctx, x, w, b, r, act, seed, step, signs, grad=True):
        lead, K, N = x.shape[:-1], x.shape[-1], w.shape[0]
        x2 = _aligned(_bits(x.reshape(-1, K)))
        M, dev = x2.shape[0], x.device
        ws = amax_workspace(dev)
        need_x, need_w, need_b, need_r = (grad and n for n in ctx.needs_input_grad[:4])
        need_z = act != ACT_NONE and (need_x or need_w or need_b)
        xq = NVFP4Tensor.empty(M, K, device=dev)
        xc = NVFP4Tensor.empty(K, M, device=dev) if need_w else None
        nvfp4_quantize(x2, xq, xc, col_round=SR, col_rng=(seed, 4 * step), col_rht=need_w, rht_signs=signs, amax_ws=ws)
        wq = _nvfp4_weight(w, ws)
        z8 = MXFP8Tensor.empty(M, N, device=dev) if need_z else None
        y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        nvfp4_gemm_bias_act(xq, wq, y, OUT_BF16, bias=_bias(b), act=act, z_ckpt=z8,
                            residual=_residual(r, M, N))
        kept4 = (xc, wq if need_x else None)
        ctx.save_for_backward(*(t for q in kept4 for t in ((q.codes, q.scales, q.s_dec) if q else (None,) * 3)),
                              *((z8.codes, z8.scales) if z8 else (None,) * 2))
        ctx.dims = (M, K, N, lead, w.dtype, None if b is None else b.dtype, None if r is None else r.dtype)
        ctx.args = (act, seed, step, signs)
        return y.reshape(*lead, N)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        M, K, N, lead, w_dtype, b_dtype, r_dtype = ctx.dims
        act, seed, step, signs = ctx.args
        t = ctx.saved_tensors
        need_x, need_w, need_b, need_r = ctx.needs_input_grad[:4]
        dev = dy.device
        dx = dw = db = None
        dr = dy.to(r_dtype) if need_r else None
        if need_x or need_w or need_b:
            g = _aligned(_bits(dy.reshape(M, N)))
            z8 = MXFP8Tensor(t[6], t[7], M, N) if act != ACT_NONE else None
            dz = torch.empty_like(g) if z8 and (need_x or need_w) else None
            if need_b:
                db = torch.empty((N,), dtype=b_dtype if b_dtype == torch.bfloat16 else torch.float32, device=dev)
            if dz is not None or db is not None:
                mxfp8_bias_act_bwd(g, z8, act, dz, db)
            if need_b:
                db = db.to(b_dtype)
            g = g if dz is None else dz
        if need_x or need_w:
            gc = NVFP4Tensor.empty(N, M, device=dev) if need_w else None
            gm = MXFP8Tensor.empty(M, N, device=dev) if need_x else None
            nvfp4_quantize(g, None, gc, gm, col_round=SR, col_rng=(seed, 4 * step + 1), col_rht=need_w, rht_signs=signs,
                           mx8_round=SR, mx8_rng=(seed, 4 * step + 2), amax_ws=amax_workspace(dev))
            if need_w:
                dw = _wgrad(gc, NVFP4Tensor(*t[0:3], K, M, False), w_dtype, dev)
            if need_x:
                wt = MXFP8Tensor.empty(K, N, device=dev)
                mxfp8_requantize_t(NVFP4Tensor(*t[3:6], N, K, True), wt, SR, (seed, 4 * step + 3))
                dx = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
                nvfp4_gemm(FMT_MXFP8, gm, wt, dx, OUT_BF16)
                dx = dx.reshape(*lead, K)
        return dx, dw, db, dr, None, None, None, None, None


class QLinear(torch.nn.Module):
    """Linear layer whose forward and backward GEMMs run in NVFP4 / MXFP8 as above.
    weight: [out_features, in_features], BF16; bias: [out_features] or None; act:
    None, "silu" or "gelu", applied to the product and the bias.  The call takes a
    residual [..., out_features] that is added at the end, in FP32 but as its BF16 values
    (an FP32 residual loses what BF16 does not hold)."""

    def __init__(self, in_features, out_features, seed=0, rht_signs=0x5A3C, device="cuda",
                 dtype=torch.bfloat16, bias=False, act=None):
        super().__init__()
        for n in (in_features, out_features):
            if n % 32:
                raise ValueError("in_features and out_features must be multiples of 32")
        if act is not None and act not in _ACTS:
            raise ValueError(f"act must be None or one of {sorted(_ACTS)}")
        self.in_features, self.out_features, self.act = in_features, out_features, act
        self.weight = torch.nn.Parameter(torch.empty((out_features, in_features), device=device,
                                                     dtype=dtype))
        torch.nn.init.normal_(self.weight, std=in_features ** -0.5)
        self.bias = torch.nn.Parameter(torch.zeros((out_features,), device=device, dtype=dtype)) if bias else None
        self.seed, self.rht_signs = seed, rht_signs
        self.step = 0

    def forward(self, x, residual=None):
        if x.shape[-1] != self.in_features:
            raise ValueError("last dimension of x must be in_features")
        if x.numel() // self.in_features % 32:
            raise ValueError("the number of tokens must be a multiple of 32")
        if self.bias is None and self.act is None and residual is None:
            y = QLinearFn.apply(x, self.weight, self.seed, self.step, self.rht_signs)
        else:
            _check_residual(residual, x.shape[:-1], self.out_features)
            if x.numel() == 0:
                raise ValueError("the number of tokens must be a positive multiple of 32")
            _on_current(None, x, self.weight, *(t for t in (self.bias, residual) if t is not None))
            y = QLinearBiasActFn.apply(x, self.weight, self.bias, residual, _act_code(self.act), self.seed, self.step,
                                       self.rht_signs, torch.is_grad_enabled())
        self.step += 1
        return y

    def inference(self):
        """The layer with its weight and bias as they are now, quantized once, for any number of tokens."""
        return QLinearInference(self.weight.detach(), None if self.bias is None else self.bias.detach(), self.act)


class QLinearInference:
    """y = act(x W^T + b) + residual from an NVFP4 weight that is quantized when the
    object is made (a later change of the given tensors does not reach it).  Up to
    GEMV_MAX_TOKENS tokens the activations stay BF16; more tokens are quantized to
    NVFP4 (padded to a multiple of 16 rows) with one decode scale for the call, so
    a token's answer then also depends on the other tokens.  Bias and residual are
    added in FP32; a residual of another type than BF16 is rounded to BF16 first."""

    def __init__(self, weight, bias=None, act=None):
        if act is not None and act not in _ACTS:
            raise ValueError(f"act must be None or one of {sorted(_ACTS)}")
        if weight.dim() != 2 or any(n == 0 or n % 16 for n in weight.shape):
            raise ValueError("weight must be [out, in], both multiples of 16")
        if bias is not None and bias.shape != weight.shape[:1]:
            raise ValueError("bias must be [out]")
        _on_current(None, weight, *(() if bias is None else (bias,)))
        self.act, self.bias = _act_code(act), None if bias is None else _bias(bias).clone()
        self.weight = _nvfp4_weight(weight, amax_workspace(weight.device))

    def __call__(self, x, residual=None):
        K, N = self.weight.cols, self.weight.rows
        if x.shape[-1] != K:
            raise ValueError("last dimension of x does not fit the weight")
        _check_residual(residual, x.shape[:-1], N)
        _on_current(None, x, self.weight.codes, *(() if residual is None else (residual,)))
        lead = x.shape[:-1]
        x2 = _aligned(x.reshape(-1, K).to(torch.bfloat16).contiguous())
        T, dev = x2.shape[0], x.device
        r = _residual(residual, T, N)
        y = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
        if 0 < T <= GEMV_MAX_TOKENS:
            nvfp4_gemv_bias_act(FMT_NVFP4, x2, self.weight, y, OUT_BF16, bias=self.bias, act=self.act, residual=r)
        elif T:
            rows = (T + 15) // 16 * 16
            if rows != T:
                x2 = torch.nn.functional.pad(x2, (0, 0, 0, rows - T))
                r = r if r is None else torch.nn.functional.pad(r, (0, 0, 0, rows - T))
            xq = NVFP4Tensor.empty(rows, K, device=dev)
            nvfp4_quantize(x2, xq, amax_ws=amax_workspace(dev))
            full = y if rows == T else torch.empty((rows, N), dtype=torch.bfloat16, device=dev)
            nvfp4_gemm_bias_act(xq, self.weight, full, OUT_BF16, bias=self.bias, act=self.act, residual=r)
            y = full[:T]
        return y.reshape(*lead, N)


class QGatedMLPFn(torch.autograd.Function):
    """y = (act(x Wg^T) * (x Wu^T)) Wd^T; x [..., K], w_gate_up [2F, K] = [Wg; Wu],
    w_down [N, F]."""

    @staticmethod
    def forward(ctx, x, w_gate_up, w_down, act, seed, step, signs, grad=True):
        """grad: whether the call is recorded (a Function does not see grad mode itself)."""
        lead, K = x.shape[:-1], x.shape[-1]
        F, N = w_gate_up.shape[0] // 2, w_down.shape[0]
        x2 = _bits(x.reshape(-1, K))
        M, dev = x2.shape[0], x.device
        ws = amax_workspace(dev)
        need_x, need_gu, need_d = (grad and n for n in ctx.needs_input_grad[:3])
        need_h = need_x or need_gu           # the backward pass reaches the activation

        def copies(t, rows, cols, stream, keep):
            q = NVFP4Tensor.empty(rows, cols, device=dev)
            c = NVFP4Tensor.empty(cols, rows, device=dev) if keep else None
            nvfp4_quantize(t, q, c, col_round=SR, col_rng=(seed, stream), col_rht=keep, rht_signs=signs,
                           amax_ws=ws)
            return q, c

        xq, xc = copies(x2, M, K, 8 * step, need_gu)
        wq = _nvfp4_weight(w_gate_up, ws)
        h = torch.empty((M, F), dtype=torch.bfloat16, device=dev)
        g8, u8 = (MXFP8Tensor.empty(M, F, device=dev) if need_h else None for _ in range(2))
        nvfp4_gated_gemm(xq, *_halves(wq), h, OUT_BF16, act=act, g_ckpt=g8, u_ckpt=u8)
        hq, hc = copies(h.view(torch.int16), M, F, 8 * step + 1, need_d)
        dq = _nvfp4_weight(w_down, ws)
        y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        nvfp4_gemm(FMT_NVFP4, hq, dq, y, OUT_BF16)
        kept4 = (xc, wq if need_x else None, hc, dq if need_h else None)
        ctx.save_for_backward(*(t for q in kept4 for t in ((q.codes, q.scales, q.s_dec) if q else (None,) * 3)),
                              *(t for q in (g8, u8) for t in ((q.codes, q.scales) if q else (None,) * 2)))
        ctx.dims = (M, K, F, N, lead, w_gate_up.dtype, w_down.dtype)
        ctx.args = (act, seed, step, signs)
        return y.reshape(*lead, N)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        M, K, F, N, lead, gu_dtype, d_dtype = ctx.dims
        act, seed, step, signs = ctx.args
        t = ctx.saved_tensors
        xc = NVFP4Tensor(*t[0:3], K, M, False)
        wq = NVFP4Tensor(*t[3:6], 2 * F, K, True)
        hc = NVFP4Tensor(*t[6:9], F, M, False)
        dq = NVFP4Tensor(*t[9:12], N, F, True)
        g8, u8 = MXFP8Tensor(*t[12:14], M, F), MXFP8Tensor(*t[14:16], M, F)
        dev = dy.device
        ws = amax_workspace(dev)
        need_x, need_gu, need_d = ctx.needs_input_grad[:3]

        def copies(v, cols, col_stream, row_stream):
            c = NVFP4Tensor.empty(cols, M, device=dev)
            r = MXFP8Tensor.empty(M, cols, device=dev)
            nvfp4_quantize(v, None, c, r, col_round=SR, col_rng=(seed, col_stream), col_rht=True,
                           rht_signs=signs, mx8_round=SR, mx8_rng=(seed, row_stream), amax_ws=ws)
            return c, r

        yc, ym = copies(_bits(dy.reshape(M, N)), N, 8 * step + 2, 8 * step + 3)
        dw_down = _wgrad(yc, hc, d_dtype, dev) if need_d else None
        dx = dw_gate_up = None
        if need_x or need_gu:
            wdt = MXFP8Tensor.empty(F, N, device=dev)
            mxfp8_requantize_t(dq, wdt, SR, (seed, 8 * step + 4))
            dgu = torch.empty((M, 2 * F), dtype=torch.bfloat16, device=dev)
            mxfp8_gemm_gated_bwd(ym, wdt, g8, u8, dgu[:, :F], dgu[:, F:], OUT_BF16, act=act)
            gc, gm = copies(dgu.view(torch.int16), 2 * F, 8 * step + 5, 8 * step + 6)
            if need_gu:
                dw_gate_up = _wgrad(gc, xc, gu_dtype, dev)
            if need_x:
                wt = MXFP8Tensor.empty(K, 2 * F, device=dev)
                mxfp8_requantize_t(wq, wt, SR, (seed, 8 * step + 7))
                dx = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
                nvfp4_gemm(FMT_MXFP8, gm, wt, dx, OUT_BF16)
                dx = dx.reshape(*lead, K)
        return dx, dw_gate_up, dw_down, None, None, None, None, None


class QGatedMLP(torch.nn.Module):
    """Gated feed-forward block without biases, act "silu" or "gelu", whose
    GEMMs run as above.  w_gate_up: [2 * hidden, features] (gate rows first),
    w_down: [features, hidden], BF16."""

    def __init__(self, features, hidden, act="silu", seed=0, rht_signs=0x5A3C, device="cuda",
                 dtype=torch.bfloat16):
        super().__init__()
        if act not in _ACTS:
            raise ValueError(f"act must be one of {sorted(_ACTS)}")
        for n in (features, hidden):
            if n <= 0 or n % 32:
                raise ValueError("features and hidden must be positive multiples of 32")
        self.features, self.hidden, self.act = features, hidden, act
        self.w_gate_up = torch.nn.Parameter(torch.empty((2 * hidden, features), device=device, dtype=dtype))
        self.w_down = torch.nn.Parameter(torch.empty((features, hidden), device=device, dtype=dtype))
        torch.nn.init.normal_(self.w_gate_up, std=features ** -0.5)
        torch.nn.init.normal_(self.w_down, std=hidden ** -0.5)
        self.seed, self.rht_signs = seed, rht_signs
        self.step = 0

    def forward(self, x):
        if x.shape[-1] != self.features:
            raise ValueError("last dimension of x must be features")
        _on_current(None, x, self.w_gate_up, self.w_down)
        tokens = x.numel() // self.features
        if tokens == 0 or tokens % 32:
            raise ValueError("the number of tokens must be a positive multiple of 32")
        y = QGatedMLPFn.apply(x, self.w_gate_up, self.w_down, _ACTS[self.act], self.seed, self.step,
                              self.rht_signs, torch.is_grad_enabled())
        self.step += 1
        return y

    def inference(self):
        """The block with its weights as they are now, quantized once, for any number of tokens."""
        return QGatedMLPInference(self.w_gate_up.detach(), self.w_down.detach(), self.act)


class QGatedMLPInference:
    """y = (act(x Wg^T) * (x Wu^T)) Wd^T from NVFP4 weights that are quantized
    when the object is made (later changes of the given weights do not reach
    it).  Up to GEMV_MAX_TOKENS tokens the activations stay BF16; more tokens
    are quantized to NVFP4 (padded to a multiple of 16 rows) for the GEMMs, with
    one decode scale for the call, so a token's answer then also depends on the
    other tokens.  Callers that need BF16 activations give GEMV_MAX_TOKENS
    tokens at a time."""

    def __init__(self, w_gate_up, w_down, act="silu"):
        if act not in _ACTS:
            raise ValueError(f"act must be one of {sorted(_ACTS)}")
        F, K = w_down.shape[1], w_gate_up.shape[1]
        if w_gate_up.shape[0] != 2 * F or any(n == 0 or n % 16 for n in (F, K, w_down.shape[0])):
            raise ValueError("w_gate_up must be [2F, K], w_down [N, F], all multiples of 16")
        _on_current(None, w_gate_up, w_down)
        self.act = _ACTS[act]
        ws = amax_workspace(w_down.device)
        self._stacked = _nvfp4_weight(w_gate_up, ws)
        self.gate, self.up = _halves(self._stacked)
        self.down = _nvfp4_weight(w_down, ws)

    def __call__(self, x):
        K, F, N = self.gate.cols, self.gate.rows, self.down.rows
        if x.shape[-1] != K:
            raise ValueError("last dimension of x does not fit the weights")
        _on_current(None, x, self.down.codes)
        lead = x.shape[:-1]
        x2 = x.reshape(-1, K).to(torch.bfloat16).contiguous()
        T, dev = x2.shape[0], x.device
        y = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
        if 0 < T <= GEMV_MAX_TOKENS:
            h = torch.empty((T, F), dtype=torch.bfloat16, device=dev)
            nvfp4_gated_gemv(FMT_NVFP4, x2, self.gate, self.up, h, OUT_BF16, act=self.act)
            nvfp4_gemv(FMT_NVFP4, h, self.down, y, OUT_BF16)
        elif T:
            rows = (T + 15) // 16 * 16
            if rows != T:
                x2 = torch.nn.functional.pad(x2, (0, 0, 0, rows - T))
            ws = amax_workspace(dev)
            xq = NVFP4Tensor.empty(rows, K, device=dev)
            nvfp4_quantize(x2, xq, amax_ws=ws)
            h = torch.empty((rows, F), dtype=torch.bfloat16, device=dev)
            nvfp4_gated_gemm(xq, self.gate, self.up, h, OUT_BF16, act=self.act)
            hq = NVFP4Tensor.empty(rows, F, device=dev)
            nvfp4_quantize(h, hq, amax_ws=ws)
            full = y if rows == T else torch.empty((rows, N), dtype=torch.bfloat16, device=dev)
            nvfp4_gemm(FMT_NVFP4, hq, self.down, full, OUT_BF16)
            y = full[:T]
        return y.reshape(*lead, N)


_MORE_THAN_32_BITS = (torch.int64, torch.uint32, torch.uint64)


class QMoEInference:
    """A mixture-of-experts layer from NVFP4 weights that are quantized when the
    object is made, each expert's as a tensor of its own: w_up [E, F, K], w_down [E, N,
    F], and w_gate [E, F, K] for gated experts (None: plain ones, act may then be
    None).  The call takes the router's choice: ids [..., k] (integers; outside
    [0, E): no expert) and weights [..., k] (None: 1), and an optional residual
    [..., N], added in FP32 as its BF16 values.  GEMV_MAX_TOKENS tokens go through the kernels at a time (many more
    tokens read the experts' weights again for each group of them)."""

    def __init__(self, w_gate, w_up, w_down, act="silu"):
        if act not in _ACTS and not (act is None and w_gate is None):
            raise ValueError(f"act must be one of {sorted(_ACTS)}, or None without w_gate")
        E, F, K = w_up.shape
        if w_down.dim() != 3 or w_down.shape[0] != E or w_down.shape[2] != F or not 1 <= E <= MOE_MAX_EXPERTS or \
                any(n == 0 or n % 16 for n in (F, K, w_down.shape[1])):
            raise ValueError("w_up must be [E, F, K], w_down [E, N, F], F, K and N multiples of 16")
        if w_gate is not None and w_gate.shape != w_up.shape:
            raise ValueError("w_gate must have w_up's shape")
        _on_current(None, w_up, w_down, *(() if w_gate is None else (w_gate,)))
        self.experts, self.act = E, _act_code(act)
        ws = amax_workspace(w_up.device)
        self.gate, self.up, self.down = (None if w is None else _nvfp4_experts(w, ws) for w in (w_gate, w_up, w_down))

    def __call__(self, x, ids, weights=None, residual=None):
        K, N, lead = self.up.cols, self.down.rows // self.experts, x.shape[:-1]
        if x.shape[-1] != K:
            raise ValueError("last dimension of x does not fit the weights")
        if ids.shape[:-1] != lead or (weights is not None and weights.shape != ids.shape):
            raise ValueError("ids and weights must be [..., k] for x [..., K]")
        if ids.is_floating_point() or ids.dtype == torch.bool:
            raise ValueError("ids must be integers")
        _check_residual(residual, lead, N)
        _on_current(None, x, ids, self.up.codes, *(t for t in (weights, residual) if t is not None))
        x2 = _aligned(x.reshape(-1, K).to(torch.bfloat16).contiguous())
        T, k = x2.shape[0], ids.shape[-1]
        ids = ids.reshape(T, k)
        if ids.dtype in _MORE_THAN_32_BITS:              # what does not fit 32 bits is no expert's number
            ids = ids.to(torch.int64)
            ids = torch.where((ids >= 0) & (ids < self.experts), ids, -1)
        ids = ids.to(torch.int32).contiguous()           # (the kernels drop what is outside [0, E))
        w = None if weights is None else weights.reshape(T, k).float().contiguous()
        r = _residual(residual, T, N)
        y = torch.empty((T, N), dtype=torch.bfloat16, device=x.device)
        for t in range(0, T, GEMV_MAX_TOKENS):
            at = slice(t, t + GEMV_MAX_TOKENS)
            nvfp4_moe_gemv(FMT_NVFP4, x2[at], ids[at], w if w is None else w[at], self.experts, self.gate, self.up,
                           self.down, y[at], OUT_BF16, act=self.act, residual=r if r is None else r[at])
        return y.reshape(*lead, N)


def _nvfp4_experts(w, ws):
    """The 16x16-tiled NVFP4 copies of a stack of weights, one decode scale each, as one tensor."""
    E, rows, cols = w.shape
    q = NVFP4Tensor.empty(E * rows, cols, tile2d=True, n_scales=E, device=w.device)
    for e in range(E):
        at, tiles = slice(e * rows, (e + 1) * rows), slice(e * rows // 16, (e + 1) * rows // 16)
        one = NVFP4Tensor(q.codes[at], q.scales[tiles], q.s_dec[e:e + 1], rows, cols, True)
        nvfp4_quantize(_bits(w[e]), one, tile2d=True, amax_ws=ws)
    return q
