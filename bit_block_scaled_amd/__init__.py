"""Python binding of libbbs.so, the MI355X NVFP4 quantized-linear library.

Argument marshalling, and for the gated and the few-token calls checks of what a
pointer does not tell: every step of the hot path runs in the HIP kernels behind
the C ABI declared in include/bbs.h.  PyTorch is used for device
memory and streams.  The functions have the names of the C entry points and
raise BbsError on a non-zero status.  There is no CPU fallback: importing
this module fails if the library has not been built.
"""
import ctypes as C
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbbs.so")

BBS_OK, BBS_EINVAL, BBS_ENOTSUP, BBS_EHIP = 0, -1, -2, -3
RTN, SR = 0, 1
OUT_F32, OUT_BF16 = 0, 1
FMT_NVFP4, FMT_MXFP8, FMT_MXFP4 = 0, 1, 2
ACT_SILU, ACT_GELU, ACT_NONE = 0, 1, 2
AMAX_WS_FLOATS = 11264
GEMV_MAX_TOKENS = 64
BIAS_PARTS = 64
MOE_MAX_SLOTS, MOE_MAX_EXPERTS = 32, 1024


class Fp4Desc(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("s_dec", C.c_void_p),
                ("rows", C.c_int64), ("cols", C.c_int64), ("tile2d", C.c_int32),
                ("sdec_per_row", C.c_int32)]


class Mx8Desc(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("rows", C.c_int64),
                ("cols", C.c_int64)]


class Mx4Desc(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("rows", C.c_int64),
                ("cols", C.c_int64)]


class S2F6Desc(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("rows", C.c_int64),
                ("cols", C.c_int64)]


class Rng(C.Structure):
    _fields_ = [("seed", C.c_uint64), ("stream", C.c_uint32)]


class QuantArgs(C.Structure):
    _fields_ = [("x", C.c_void_p), ("rows", C.c_int64), ("cols", C.c_int64), ("ld", C.c_int64),
                ("row", C.POINTER(Fp4Desc)), ("row_round", C.c_int32), ("row_rng", Rng),
                ("col", C.POINTER(Fp4Desc)), ("col_round", C.c_int32), ("col_rng", Rng),
                ("col_rht", C.c_int32), ("rht_signs", C.c_uint32),
                ("row_mx8", C.POINTER(Mx8Desc)), ("mx8_round", C.c_int32), ("mx8_rng", Rng),
                ("tile2d", C.c_int32), ("amax_ws", C.c_void_p),
                ("row_per_token", C.c_int32), ("row_four_six", C.c_int32),
                ("gelu", C.c_int32)]


# Fp4Desc, and Mx8Desc or Mx4Desc, as bytes
_FP4_PACK = struct.Struct("@PPPqqii").pack
_MX_PACK = struct.Struct("@PPqq").pack


class BbsError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"bbs status {status}: {msg}")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
    lib = C.CDLL(LIB_PATH)
    vp, i32, i64 = C.c_void_p, C.c_int32, C.c_int64
    lib.nvfp4_quantize.argtypes = [C.POINTER(QuantArgs), vp]
    lib.nvfp4_quantize_noalloc.argtypes = [C.POINTER(QuantArgs), vp]
    lib.mxfp8_requantize_t.argtypes = [C.POINTER(Fp4Desc), C.POINTER(Mx8Desc), i32, Rng, vp]
    lib.nvfp4_gemm.argtypes = [i32, vp, vp, vp, i32, i64, vp]
    lib.grouped_nvfp4_gemm.argtypes = [C.POINTER(Fp4Desc), vp, vp, i32, i64, C.POINTER(Fp4Desc),
                                       i64, vp, i32, i64, vp]
    lib.mxfp4_quantize.argtypes = [vp, i64, i64, i64, C.POINTER(Mx4Desc), i32, Rng, vp]
    lib.nvfp4_gemm_quant.argtypes = [C.POINTER(Fp4Desc), C.POINTER(Fp4Desc), vp, i32,
                                     C.POINTER(Fp4Desc), vp, vp, vp]
    lib.grouped_nvfp4_gemm_quant.argtypes = [C.POINTER(Fp4Desc), vp, vp, i32, i64,
                                             C.POINTER(Fp4Desc), i64, vp, i32, C.POINTER(Fp4Desc),
                                             vp, vp, vp]
    lib.nvfp4_gemm_s2f6.argtypes = [C.POINTER(Fp4Desc), C.POINTER(Fp4Desc), i32, C.c_uint32,
                                    C.POINTER(S2F6Desc), vp]
    lib.grouped_nvfp4_gemm_s2f6.argtypes = [C.POINTER(Fp4Desc), vp, vp, i32, i64,
                                            C.POINTER(Fp4Desc), i64, i32, C.c_uint32,
                                            C.POINTER(S2F6Desc), vp]
    lib.s2f6_quantize.argtypes = [vp, i64, i64, i64, i32, C.c_uint32, C.POINTER(S2F6Desc), vp]
    lib.s2f6_combine.argtypes = [C.POINTER(S2F6Desc), vp, vp, i64, i32, i32, C.c_uint32, vp, i32,
                                 i64, vp]
    lib.nvfp4_gated_gemm.argtypes = [C.POINTER(Fp4Desc), C.POINTER(Fp4Desc), C.POINTER(Fp4Desc), i32,
                                     vp, i32, i64, C.POINTER(Mx8Desc), C.POINTER(Mx8Desc), vp]
    lib.mxfp8_gemm_gated_bwd.argtypes = [C.POINTER(Mx8Desc), C.POINTER(Mx8Desc), C.POINTER(Mx8Desc),
                                         C.POINTER(Mx8Desc), i32, vp, vp, i32, i64, vp]
    lib.nvfp4_gemv.argtypes = [i32, vp, i64, i64, vp, vp, i32, i64, vp]
    lib.nvfp4_gated_gemv.argtypes = [i32, vp, i64, i64, vp, vp, i32, vp, i32, i64, vp]
    lib.nvfp4_gemm_bias_act.argtypes = [vp, vp, vp, i32, i32, vp, i64, vp, vp, i32, i64, vp]
    lib.mxfp8_bias_act_bwd.argtypes = [vp, i64, i64, i64, vp, i32, vp, i64, vp, i32, vp, vp]
    lib.nvfp4_gemv_bias_act.argtypes = [i32, vp, i64, i64, vp, vp, i32, i32, vp, i64, vp, i32, i64, vp]
    lib.nvfp4_moe_gemv.argtypes = [i32, vp, i64, i64, vp, vp, i32, i32, vp, vp, vp, i32, vp, i64, vp, vp, i32, i64, vp]
    lib.nvfp4_moe_ws_bytes.argtypes = [i64, i32, i32, i64, i64]
    lib.nvfp4_moe_ws_bytes.restype = i64
    for f in ("nvfp4_moe_gemv", "nvfp4_gemm_bias_act", "mxfp8_bias_act_bwd", "nvfp4_gemv_bias_act", "nvfp4_gated_gemm", "mxfp8_gemm_gated_bwd", "nvfp4_gemv", "nvfp4_gated_gemv",
              "nvfp4_quantize", "nvfp4_quantize_noalloc", "mxfp8_requantize_t", "nvfp4_gemm", "grouped_nvfp4_gemm",
              "s2f6_quantize", "s2f6_combine", "mxfp4_quantize", "nvfp4_gemm_quant",
              "grouped_nvfp4_gemm_quant", "nvfp4_gemm_s2f6", "grouped_nvfp4_gemm_s2f6"):
        getattr(lib, f).restype = C.c_int
    lib.bbs_strerror.argtypes = [C.c_int]
    lib.bbs_strerror.restype = C.c_char_p
    lib.bbs_last_error.argtypes = []
    lib.bbs_last_error.restype = C.c_char_p
    return lib


lib = _load()


def _check(status):
    if status != BBS_OK:
        raise BbsError(status, lib.bbs_last_error().decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


# of a build of PyTorch without GPUs these are missing, and no call gets here
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream):
    if stream is None:
        # the handle of torch.cuda.current_stream(), without building the Stream object
        return _raw_stream(_device())
    return stream.cuda_stream


# ---------------------------------------------------------------------------
# Tensor containers (device memory comes from PyTorch)
# ---------------------------------------------------------------------------

class NVFP4Tensor:
    """codes [rows, cols/2] u8, scales [rows(/16), cols/16] u8, s_dec [n] f32
    (n = 1, G stacked experts, or rows when sdec_per_row)."""

    def __init__(self, codes, scales, s_dec, rows, cols, tile2d, sdec_per_row=False):
        self.codes, self.scales, self.s_dec = codes, scales, s_dec
        self.rows, self.cols, self.tile2d = rows, cols, int(tile2d)
        self.sdec_per_row = int(sdec_per_row)

    @staticmethod
    def empty(rows, cols, tile2d=False, n_scales=1, device="cuda", sdec_per_row=False):
        srows = rows // 16 if tile2d else rows
        n = rows if sdec_per_row else n_scales
        return NVFP4Tensor(torch.empty((rows, cols // 2), dtype=torch.uint8, device=device),
                           torch.empty((srows, cols // 16), dtype=torch.uint8, device=device),
                           torch.empty((n,), dtype=torch.float32, device=device),
                           rows, cols, tile2d, sdec_per_row)

    def desc(self):
        return Fp4Desc(_ptr(self.codes), _ptr(self.scales), _ptr(self.s_dec), self.rows,
                       self.cols, self.tile2d, self.sdec_per_row)

    def packed(self):
        """The bytes of desc(), 0.4 us cheaper to make."""
        return _FP4_PACK(self.codes.data_ptr(), self.scales.data_ptr(), self.s_dec.data_ptr(), self.rows,
                         self.cols, self.tile2d, self.sdec_per_row)


class MXFP8Tensor:
    """codes [rows, cols] u8 (E4M3), scales [rows, cols/32] u8 (E8M0)."""

    def __init__(self, codes, scales, rows, cols):
        self.codes, self.scales, self.rows, self.cols = codes, scales, rows, cols

    @staticmethod
    def empty(rows, cols, device="cuda"):
        return MXFP8Tensor(torch.empty((rows, cols), dtype=torch.uint8, device=device),
                           torch.empty((rows, cols // 32), dtype=torch.uint8, device=device),
                           rows, cols)

    def desc(self):
        return Mx8Desc(_ptr(self.codes), _ptr(self.scales), self.rows, self.cols)

    def packed(self):
        """As NVFP4Tensor.packed."""
        return _MX_PACK(self.codes.data_ptr(), self.scales.data_ptr(), self.rows, self.cols)


class MXFP4Tensor:
    """codes [rows, cols/2] u8 (E2M1 pairs, even column low), scales [rows, cols/32] u8 (E8M0)."""

    def __init__(self, codes, scales, rows, cols):
        self.codes, self.scales, self.rows, self.cols = codes, scales, rows, cols

    @staticmethod
    def empty(rows, cols, device="cuda"):
        return MXFP4Tensor(torch.empty((rows, cols // 2), dtype=torch.uint8, device=device),
                           torch.empty((rows, cols // 32), dtype=torch.uint8, device=device),
                           rows, cols)

    def desc(self):
        return Mx4Desc(_ptr(self.codes), _ptr(self.scales), self.rows, self.cols)

    def packed(self):
        """As NVFP4Tensor.packed."""
        return _MX_PACK(self.codes.data_ptr(), self.scales.data_ptr(), self.rows, self.cols)


class S2F6Tensor:
    """codes [rows, cols] int8 (value code / 64), scales [rows, cols/32] u8 (E8M0)."""

    def __init__(self, codes, scales, rows, cols):
        self.codes, self.scales, self.rows, self.cols = codes, scales, rows, cols

    @staticmethod
    def empty(rows, cols, device="cuda"):
        return S2F6Tensor(torch.empty((rows, cols), dtype=torch.int8, device=device),
                          torch.empty((rows, cols // 32), dtype=torch.uint8, device=device),
                          rows, cols)

    def desc(self):
        return S2F6Desc(_ptr(self.codes), _ptr(self.scales), self.rows, self.cols)


def amax_workspace(device="cuda"):
    return torch.empty((AMAX_WS_FLOATS,), dtype=torch.float32, device=device)


def _workspace(make, stream):
    """make()'s workspace of this call alone, from the pool of the stream that the call runs
    on (None: the current one).  The allocator orders a block's owners on its own stream only:
    one from another pool may still be in use there by work that `stream` does not wait for."""
    if stream is None:
        return make()
    with torch.cuda.stream(stream):
        return make()


# ---------------------------------------------------------------------------
# Entry points
# ---------------------------------------------------------------------------

def nvfp4_quantize(x, row=None, col=None, row_mx8=None, *, row_round=RTN, row_rng=(0, 0),
                   col_round=RTN, col_rng=(0, 0), col_rht=False, rht_signs=0, mx8_round=RTN,
                   mx8_rng=(0, 0), tile2d=False, amax_ws=None, row_per_token=False,
                   row_four_six=False, gelu=False, stream=None):
    """x: BF16 bit patterns as a [rows, cols] int16/uint16/bfloat16 device tensor
    (row stride x.stride(0)).  row / col: NVFP4Tensor outputs; row_mx8: MXFP8Tensor.
    row_per_token / row_four_six: activation options of the row copy (a
    per-token row copy needs NVFP4Tensor.empty(..., sdec_per_row=True)).
    gelu: the row / row_mx8 copies are of GELU(x) (tanh form, FP32).
    amax_ws: amax_workspace(), allocated on the call's stream if None."""
    rd = row.desc() if row is not None else None
    cd = col.desc() if col is not None else None
    md = row_mx8.desc() if row_mx8 is not None else None
    if amax_ws is None:
        amax_ws = _workspace(lambda: amax_workspace(x.device), stream)
    a = QuantArgs(_ptr(x), x.shape[0], x.shape[1], x.stride(0),
                  C.pointer(rd) if rd else None, row_round, Rng(*row_rng),
                  C.pointer(cd) if cd else None, col_round, Rng(*col_rng),
                  int(col_rht), rht_signs,
                  C.pointer(md) if md else None, mx8_round, Rng(*mx8_rng),
                  int(tile2d), _ptr(amax_ws), int(row_per_token), int(row_four_six),
                  int(gelu))
    _check(lib.nvfp4_quantize(C.byref(a), _stream(stream)))


def nvfp4_quantize_noalloc(x, row=None, col=None, row_mx8=None, *, row_round=RTN, row_rng=(0, 0),
                           col_round=RTN, col_rng=(0, 0), col_rht=False, rht_signs=0,
                           mx8_round=RTN, mx8_rng=(0, 0), tile2d=False, row_per_token=False,
                           row_four_six=False, gelu=False, stream=None):
    """nvfp4_quantize without a workspace argument: the library's own per-GPU
    scratch holds the amax partials (nothing is allocated by the call)."""
    rd = row.desc() if row is not None else None
    cd = col.desc() if col is not None else None
    md = row_mx8.desc() if row_mx8 is not None else None
    a = QuantArgs(_ptr(x), x.shape[0], x.shape[1], x.stride(0),
                  C.pointer(rd) if rd else None, row_round, Rng(*row_rng),
                  C.pointer(cd) if cd else None, col_round, Rng(*col_rng),
                  int(col_rht), rht_signs,
                  C.pointer(md) if md else None, mx8_round, Rng(*mx8_rng),
                  int(tile2d), None, int(row_per_token), int(row_four_six), int(gelu))
    _check(lib.nvfp4_quantize_noalloc(C.byref(a), _stream(stream)))


def mxfp8_requantize_t(src, dst, round=SR, rng=(0, 0), stream=None):
    sd, dd = src.desc(), dst.desc()
    _check(lib.mxfp8_requantize_t(C.byref(sd), C.byref(dd), round, Rng(*rng), _stream(stream)))


def nvfp4_gemm(fmt, A, B, C_out, c_dtype, ldc=None, stream=None):
    ad, bd = A.desc(), B.desc()
    ldc = C_out.stride(0) if ldc is None else ldc
    _check(lib.nvfp4_gemm(fmt, C.byref(ad), C.byref(bd), _ptr(C_out), c_dtype, ldc,
                          _stream(stream)))


def grouped_nvfp4_gemm(A, row_index, group_offsets, G, max_rows, B, N, C_out, c_dtype, ldc=None,
                       stream=None):
    ad, bd = A.desc(), B.desc()
    ldc = C_out.stride(0) if ldc is None else ldc
    _check(lib.grouped_nvfp4_gemm(C.byref(ad), _ptr(row_index), _ptr(group_offsets), G, max_rows,
                                  C.byref(bd), N, _ptr(C_out), c_dtype, ldc, _stream(stream)))


def s2f6_quantize(x, out, rht=True, signs=0, stream=None):
    """Combine wire format encode of x (BF16 patterns [rows, cols]) into the
    S2F6Tensor out, with the 32-point RHT when rht."""
    d = out.desc()
    _check(lib.s2f6_quantize(_ptr(x), x.shape[0], x.shape[1], x.stride(0), int(rht), signs,
                             C.byref(d), _stream(stream)))


def s2f6_combine(inp, src_index, out, weights=None, rht=True, signs=0, out_dtype=OUT_BF16,
                 ldo=None, stream=None):
    """out[t] = inverse RHT of sum_j weights[t, j] * decode(inp row src_index[t, j]);
    src_index: int32 [tokens, k] device tensor, weights: float32 [tokens, k] or None."""
    d = inp.desc()
    T, K = src_index.shape
    ldo = out.stride(0) if ldo is None else ldo
    _check(lib.s2f6_combine(C.byref(d), _ptr(src_index), _ptr(weights), T, K, int(rht), signs,
                            _ptr(out), out_dtype, ldo, _stream(stream)))


def mxfp4_quantize(x, out, round=RTN, rng=(0, 0), stream=None):
    """MXFP4 copy of x (BF16 patterns [rows, cols]) into the MXFP4Tensor out."""
    d = out.desc()
    _check(lib.mxfp4_quantize(_ptr(x), x.shape[0], x.shape[1], x.stride(0), C.byref(d), round,
                              Rng(*rng), _stream(stream)))


def nvfp4_gemm_quant(A, B, s_enc, Y, gelu=False, amax=None, ws=None, stream=None):
    """Y (NVFP4Tensor, 1x16) = NVFP4 copy of (GELU of) the BF16 product A * B^T
    with the encode scale s_enc (a one-element float32 device tensor); amax
    (optional one-element float32 device tensor) receives max |y|."""
    ad, bd, yd = A.desc(), B.desc(), Y.desc()
    if gelu and ws is None:
        ws = _workspace(lambda: amax_workspace(s_enc.device), stream)
    _check(lib.nvfp4_gemm_quant(C.byref(ad), C.byref(bd), _ptr(s_enc), int(gelu), C.byref(yd),
                                _ptr(amax), _ptr(ws), _stream(stream)))


def grouped_nvfp4_gemm_quant(A, row_index, group_offsets, G, max_rows, B, N, s_enc, Y,
                             gelu=False, amax=None, ws=None, stream=None):
    ad, bd, yd = A.desc(), B.desc(), Y.desc()
    if gelu and ws is None:
        ws = _workspace(lambda: amax_workspace(s_enc.device), stream)
    _check(lib.grouped_nvfp4_gemm_quant(C.byref(ad), _ptr(row_index), _ptr(group_offsets), G,
                                        max_rows, C.byref(bd), N, _ptr(s_enc), int(gelu),
                                        C.byref(yd), _ptr(amax), _ptr(ws), _stream(stream)))


def nvfp4_gemm_s2f6(A, B, Y, rht=True, signs=0, stream=None):
    """Y (S2F6Tensor) = combine wire format encode of the BF16 product A * B^T."""
    ad, bd, yd = A.desc(), B.desc(), Y.desc()
    _check(lib.nvfp4_gemm_s2f6(C.byref(ad), C.byref(bd), int(rht), signs, C.byref(yd),
                               _stream(stream)))


def grouped_nvfp4_gemm_s2f6(A, row_index, group_offsets, G, max_rows, B, N, Y, rht=True, signs=0,
                            stream=None):
    """The grouped GEMM with the combine wire format encode of its BF16 output."""
    ad, bd, yd = A.desc(), B.desc(), Y.desc()
    _check(lib.grouped_nvfp4_gemm_s2f6(C.byref(ad), _ptr(row_index), _ptr(group_offsets), G,
                                       max_rows, C.byref(bd), N, int(rht), signs, C.byref(yd),
                                       _stream(stream)))


# The gated and the few-token calls take tensors straight from a model, so what
# the pointers alone do not tell the C ABI is looked at here: type, shape,
# strides, format and device.

_ELEMENTS = {OUT_F32: (torch.float32,), OUT_BF16: (torch.bfloat16, torch.int16, torch.uint16)}
_BF16 = _ELEMENTS[OUT_BF16]
_WEIGHTS = {FMT_NVFP4: NVFP4Tensor, FMT_MXFP4: MXFP4Tensor}


def _output_ld(t, dtype, rows, cols, ld, name):
    """Row stride of an output of rows x cols; with a given one the rows lie ld elements apart from t's first."""
    if ld is None:
        r, c = t.shape
        ld, step = t.stride()
        fits = r >= rows and c >= cols and (step == 1 or cols == 1)
        if rows == 1:
            ld = cols                    # a single row's stride may be anything in PyTorch
    else:
        fits = (rows - 1) * ld + cols <= t.untyped_storage().nbytes() // t.element_size() - t.storage_offset()
    if not fits or t.dtype not in _ELEMENTS.get(dtype, (t.dtype,)):    # an unknown dtype is the C ABI's to refuse
        raise ValueError(f"{name} must hold {rows} x {cols} elements of the output's type, those of a row adjacent")
    return ld


def _on_current(stream, *tensors):
    """The stream's handle; every tensor is on the current GPU, whose stream it is."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError("the tensors must be on one GPU")
    if dev < 0 or dev != _device() or (stream is not None and stream.device_index != dev):
        raise ValueError("the tensors and the stream must be on the current GPU")
    return _raw_stream(dev) if stream is None else stream.cuda_stream


def _used_on(ws, stream):
    """Keeps a workspace from reuse until `stream` is past the call, also if its maker took it
    from another stream's pool (for a block of the stream's own this changes nothing)."""
    if stream is not None:
        ws.record_stream(stream)


def nvfp4_gated_gemm(A, Wg, Wu, H, h_dtype, act=ACT_SILU, g_ckpt=None, u_ckpt=None, ldh=None,
                     stream=None):
    """H = act(A * Wg^T) * (A * Wu^T) in one kernel (NVFP4Tensors A [M, K], Wg and
    Wu [F, K]); g_ckpt and u_ckpt (MXFP8Tensors [M, F], both or neither) receive
    8-bit checkpoints of the two products for mxfp8_gemm_gated_bwd."""
    ldh = _output_ld(H, h_dtype, A.rows, Wg.rows, ldh, "H")
    ckpt = [t for c in (g_ckpt, u_ckpt) if c is not None for t in (c.codes, c.scales)]
    s = _on_current(stream, A.codes, Wg.codes, Wu.codes, H, *ckpt)
    ad, gd, ud = A.desc(), Wg.desc(), Wu.desc()
    g8 = g_ckpt.desc() if g_ckpt is not None else None
    u8 = u_ckpt.desc() if u_ckpt is not None else None
    _check(lib.nvfp4_gated_gemm(C.byref(ad), C.byref(gd), C.byref(ud), act, _ptr(H), h_dtype, ldh,
                                C.byref(g8) if g8 is not None else None,
                                C.byref(u8) if u8 is not None else None, s))


def mxfp8_gemm_gated_bwd(dY, Wt, g_ckpt, u_ckpt, dG, dU, dtype, act=ACT_SILU, ld=None, stream=None):
    """Backward pass of act(g) * u behind a down projection, from the 8-bit
    checkpoints: with dH = dY * Wt^T (MXFP8Tensors [M, K], [F, K]), dG = dH * u *
    act'(g) and dU = dH * act(g), both [M, F] with one row stride (they may be
    the halves of one [M, 2F] tensor)."""
    M, F = dY.rows, Wt.rows
    lds = [_output_ld(t, dtype, M, F, ld, name) for t, name in ((dG, "dG"), (dU, "dU"))]
    if lds[0] != lds[1]:
        raise ValueError("dG and dU must have the same row stride")
    s = _on_current(stream, dY.codes, Wt.codes, g_ckpt.codes, u_ckpt.codes, dG, dU)
    yd, wd, gd, ud = dY.desc(), Wt.desc(), g_ckpt.desc(), u_ckpt.desc()
    _check(lib.mxfp8_gemm_gated_bwd(C.byref(yd), C.byref(wd), C.byref(gd), C.byref(ud), act, _ptr(dG),
                                    _ptr(dU), dtype, lds[0], s))


def _few_tokens(fmt, x, W, Wu, y, y_dtype, ldy, stream):
    """(tokens, row strides of x and y, stream) of a few-token product.  As
    _output_ld and _on_current, in line: the smallest products are bound by the
    host."""
    T, cols = x.shape
    ldx, step = x.stride()
    N, K = W.rows, W.cols
    if cols < K or step != 1 or x.dtype not in _BF16:
        raise ValueError(f"x must hold rows of {K} BF16 patterns, those of a row adjacent")
    kind = _WEIGHTS.get(fmt)
    if kind is None or not isinstance(W, kind) or not isinstance(Wu, kind):
        raise ValueError("fmt must be FMT_NVFP4 or FMT_MXFP4, and the weights in that format")
    if ldy is None:
        r, c = y.shape
        ldy, step = y.stride()
        if r < T or c < N or (step != 1 and N > 1) or y.dtype not in _ELEMENTS.get(y_dtype, (y.dtype,)):
            _output_ld(y, y_dtype, T, N, None, "the output")
    else:
        _output_ld(y, y_dtype, T, N, ldy, "the output")
    if T == 1:
        ldx = K                          # a single row's stride may be anything in PyTorch
        ldy = max(ldy, N)
    dev = x.get_device()
    if dev != y.get_device() or dev != W.codes.get_device() or (Wu is not W and dev != Wu.codes.get_device()) or dev < 0:
        raise ValueError("the tensors must be on one GPU")
    if stream is None and dev == _device():
        return T, ldx, ldy, _raw_stream(dev)
    return T, ldx, ldy, _on_current(stream, x)


def nvfp4_gemv(fmt, x, W, y, y_dtype, ldy=None, stream=None):
    """y = x * W^T for 1 to GEMV_MAX_TOKENS tokens: x BF16 patterns [T, K] (row
    stride x.stride(0)), W an NVFP4Tensor or MXFP4Tensor [N, K] by fmt."""
    T, ldx, ldy, s = _few_tokens(fmt, x, W, W, y, y_dtype, ldy, stream)
    status = lib.nvfp4_gemv(fmt, x.data_ptr(), T, ldx, W.packed(), y.data_ptr(), y_dtype, ldy, s)
    if status:
        _check(status)


def nvfp4_gated_gemv(fmt, x, Wg, Wu, h, h_dtype, act=ACT_SILU, ldh=None, stream=None):
    """h = act(x * Wg^T) * (x * Wu^T) for 1 to GEMV_MAX_TOKENS tokens, operands as
    nvfp4_gemv."""
    T, ldx, ldh, s = _few_tokens(fmt, x, Wg, Wu, h, h_dtype, ldh, stream)
    status = lib.nvfp4_gated_gemv(fmt, x.data_ptr(), T, ldx, Wg.packed(), Wu.packed(), act, h.data_ptr(),
                                  h_dtype, ldh, s)
    if status:
        _check(status)


# A linear layer's bias and residual come as tensors; the type of a bias is its own.

_TYPES = {torch.float32: OUT_F32, torch.bfloat16: OUT_BF16}


def _vector(t, n, name):
    """(pointer, type) of n adjacent float32 or bfloat16 values."""
    if t is None:
        return None, OUT_F32
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1) or t.dtype not in _TYPES:
        raise ValueError(f"{name} must hold {n} adjacent float32 or bfloat16 values")
    return t.data_ptr(), _TYPES[t.dtype]


def _mx8_shape(t, rows, cols, name):
    """An MXFP8Tensor's sizes, and that its tensors hold as much."""
    if not isinstance(t, MXFP8Tensor) or (t.rows, t.cols) != (rows, cols):
        raise ValueError(f"{name} must be an MXFP8Tensor of {rows} x {cols}")
    c, s = t.codes, t.scales
    if c.itemsize != 1 or s.itemsize != 1 or c.numel() < rows * cols or s.numel() < rows * (cols // 32) or \
            not (c.is_contiguous() and s.is_contiguous()):
        raise ValueError(f"{name} must hold {rows} x {cols} adjacent codes and their scales")


def nvfp4_gemm_bias_act(A, B, out, out_dtype, bias=None, act=ACT_NONE, residual=None, z_ckpt=None, ldo=None,
                        ldr=None, stream=None):
    """out = act(A * B^T + bias) + residual in one kernel (NVFP4Tensors A [M, K], B
    [N, K]; bias [N] float32 or bfloat16; residual [M, N] of out's type, out itself
    allowed); z_ckpt (MXFP8Tensor [M, N]) receives the 8-bit checkpoint of A * B^T
    + bias for mxfp8_bias_act_bwd."""
    M, N = A.rows, B.rows
    ldo = _output_ld(out, out_dtype, M, N, ldo, "out")
    if residual is not None:
        ldr = _output_ld(residual, out_dtype, M, N, ldr, "residual")
    b, b_dtype = _vector(bias, N, "bias")
    tensors, zd = [out, A.codes, A.scales, A.s_dec, B.codes, B.scales, B.s_dec], None
    if bias is not None:
        tensors.append(bias)
    if residual is not None:
        tensors.append(residual)
    if z_ckpt is not None:
        _mx8_shape(z_ckpt, M, N, "z_ckpt")
        tensors += (z_ckpt.codes, z_ckpt.scales)
        zd = z_ckpt.packed()
    s = _on_current(stream, *tensors)
    _check(lib.nvfp4_gemm_bias_act(A.packed(), B.packed(), b, b_dtype, act, _ptr(residual), ldr or 0, zd, _ptr(out),
                                   out_dtype, ldo, s))


def mxfp8_bias_act_bwd(dY, z_ckpt, act, dZ=None, dbias=None, ws=None, stream=None):
    """Backward pass of act(z) + residual, z = product + bias, from the 8-bit
    checkpoint of z: dZ = dY * act'(z) and dbias = its sum over the rows.  dY and dZ:
    BF16 patterns [M, N] (dZ may be dY); dbias: [N] float32 or bfloat16; z_ckpt is
    not read, and may be None, with ACT_NONE.  ws: BIAS_PARTS * N float32 of
    workspace for dbias (allocated on the call's stream if None)."""
    M, N = dY.shape
    ldy = _output_ld(dY, OUT_BF16, M, N, None, "dY")
    ldz = _output_ld(dZ, OUT_BF16, M, N, None, "dZ") if dZ is not None else 0
    if z_ckpt is not None:
        _mx8_shape(z_ckpt, M, N, "z_ckpt")
    elif act != ACT_NONE:
        raise ValueError("an activation's backward pass needs z_ckpt")
    b, b_dtype = _vector(dbias, N, "dbias")
    own = dbias is not None and ws is None
    if dbias is not None:
        if own:
            ws = _workspace(lambda: torch.empty((BIAS_PARTS * N,), dtype=torch.float32, device=dY.device), stream)
        elif ws.dtype != torch.float32 or not ws.is_contiguous() or ws.numel() < BIAS_PARTS * N:
            raise ValueError(f"ws must hold {BIAS_PARTS * N} adjacent float32 values")
    tensors, zd = [dY], None
    if z_ckpt is not None:
        tensors += (z_ckpt.codes, z_ckpt.scales)
        zd = z_ckpt.packed()
    if dZ is not None:
        tensors.append(dZ)
    if dbias is not None:
        tensors += (dbias, ws)
    s = _on_current(stream, *tensors)
    _check(lib.mxfp8_bias_act_bwd(_ptr(dY), M, N, ldy, zd, act, _ptr(dZ), ldz, b, b_dtype, _ptr(ws), s))
    if own:
        _used_on(ws, stream)


def nvfp4_gemv_bias_act(fmt, x, W, y, y_dtype, bias=None, act=ACT_NONE, residual=None, ldy=None, ldr=None,
                        stream=None):
    """y = act(x * W^T + bias) + residual for 1 to GEMV_MAX_TOKENS tokens, x, W and y
    as nvfp4_gemv; bias [N] float32 or bfloat16, residual [T, N] of y's type (y
    itself allowed)."""
    T, ldx, ldy, s = _few_tokens(fmt, x, W, W, y, y_dtype, ldy, stream)
    b, b_dtype = _vector(bias, W.rows, "bias")
    if residual is not None:
        ldr = _output_ld(residual, y_dtype, T, W.rows, ldr, "residual")
    dev = x.get_device()
    if (bias is not None and bias.get_device() != dev) or (residual is not None and residual.get_device() != dev) or \
            W.scales.get_device() != dev or (fmt == FMT_NVFP4 and W.s_dec.get_device() != dev):
        raise ValueError("the tensors must be on one GPU")
    status = lib.nvfp4_gemv_bias_act(fmt, x.data_ptr(), T, ldx, W.packed(), b, b_dtype, act, _ptr(residual), ldr or 0,
                                     y.data_ptr(), y_dtype, ldy, s)
    if status:
        _check(status)


def moe_workspace(tokens, k, experts, hidden, features, device="cuda"):
    """Workspace of an nvfp4_moe_gemv call of these sizes."""
    n = lib.nvfp4_moe_ws_bytes(tokens, k, experts, hidden, features)
    if n < 0:
        _check(n)
    return torch.empty((n,), dtype=torch.uint8, device=device)


def nvfp4_moe_gemv(fmt, x, ids, weights, experts, Wg, Wu, Wd, y, y_dtype, act=ACT_SILU, residual=None, ws=None,
                   ldy=None, ldr=None, stream=None):
    """A whole mixture-of-experts layer for 1 to GEMV_MAX_TOKENS tokens: y[t] =
    residual[t] + sum over j of weights[t, j] * expert ids[t, j] of x[t], the experts
    gated (Wg, Wu: stacked [experts * F, K], Wd: [experts * N, F]) or plain (Wg None).
    x BF16 patterns [T, K]; ids int32 [T, k] (entries outside [0, experts) add
    nothing), weights float32 [T, k] or None (1); weights in the format fmt (NVFP4
    with one decode scale an expert); residual [T, N] of y's type, y itself allowed;
    ws: moe_workspace(...), allocated on the call's stream if None."""
    if not 1 <= experts <= MOE_MAX_EXPERTS:
        raise ValueError(f"experts must be in [1, {MOE_MAX_EXPERTS}]")
    T, cols = x.shape
    ldx, step = x.stride()
    K, F, N = Wu.cols, Wd.cols, Wd.rows // experts
    if cols != K or step != 1 or x.dtype not in _BF16:
        raise ValueError(f"x must hold rows of {K} BF16 patterns, those of a row adjacent")
    kind, tensors = _WEIGHTS.get(fmt), [x, ids, y]
    for w in (Wu, Wd) if Wg is None else (Wu, Wd, Wg):
        if kind is None or not isinstance(w, kind):
            raise ValueError("fmt must be FMT_NVFP4 or FMT_MXFP4, and the weights in that format")
        if kind is NVFP4Tensor:
            d = w.s_dec
            if d.numel() != experts or d.dtype is not torch.float32 or not d.is_contiguous():
                raise ValueError("NVFP4 weights need one float32 decode scale an expert, adjacent")
            tensors += (w.codes, w.scales, d)
        else:
            tensors += (w.codes, w.scales)
    if ids.dim() != 2 or ids.shape[0] != T or ids.dtype != torch.int32 or not ids.is_contiguous():
        raise ValueError(f"ids must be a contiguous int32 tensor of {T} rows")
    k = ids.shape[1]
    if weights is not None:
        if weights.shape != ids.shape or weights.dtype != torch.float32 or not weights.is_contiguous():
            raise ValueError("weights must be a contiguous float32 tensor of ids' shape")
        tensors.append(weights)
    ldy = _output_ld(y, y_dtype, T, N, ldy, "y")
    if residual is not None:
        ldr = _output_ld(residual, y_dtype, T, N, ldr, "residual")
        tensors.append(residual)
    if T == 1:
        ldx = K                          # a single row's stride may be anything in PyTorch
    own = ws is None
    if own:
        ws = _workspace(lambda: moe_workspace(T, k, experts, F, N, x.device), stream)
    elif ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.numel() < lib.nvfp4_moe_ws_bytes(T, k, experts, F, N):
        raise ValueError("ws must be a moe_workspace of the call's sizes")
    s = _on_current(stream, ws, *tensors)
    _check(lib.nvfp4_moe_gemv(fmt, x.data_ptr(), T, ldx, ids.data_ptr(), _ptr(weights), k, experts,
                              None if Wg is None else Wg.packed(), Wu.packed(), Wd.packed(), act, _ptr(residual),
                              ldr or 0, ws.data_ptr(), y.data_ptr(), y_dtype, ldy, s))
    if own:
        _used_on(ws, stream)
