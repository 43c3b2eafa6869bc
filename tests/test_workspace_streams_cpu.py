"""On which stream a call makes the workspace that it allocates itself.  The
allocator hands a block out again as soon as it is freed, ordered with the stream
whose pool it is from and with no other: a workspace from another stream's pool can
be one that work there still reads and writes.  The library and the streams are
replaced by recorders, so nothing runs on a GPU."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

import bit_block_scaled_amd as bbs                                          # noqa: E402
from test_gated_bindings_cpu import bf  # noqa: E402

E, T, K, F, N = 4, 3, 64, 32, 48


@pytest.fixture
def made(monkeypatch):
    """[(entry point, the stream that was current when its workspace was made)] of the calls"""
    on, blocks, seen = [None], {}, []
    empty = torch.empty

    @contextlib.contextmanager
    def stream(s):
        on.append(s)
        yield
        on.pop()

    def recorded(*a, **kw):
        t = empty(*a, **kw)
        blocks[t.data_ptr()] = on[-1]
        keep.append(t)
        return t

    def entry(name, at):
        def call(*a):
            ws = a[0]._obj.amax_ws if name == "nvfp4_quantize" else a[at]
            seen.append((name, blocks.get(getattr(ws, "value", ws), "not made by the call")))
            return 0
        return call

    keep = []
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty", recorded)
    for name, at in (("mxfp8_bias_act_bwd", 10), ("nvfp4_moe_gemv", 14), ("nvfp4_quantize", 0), ("nvfp4_gemm_quant", 6),
                     ("grouped_nvfp4_gemm_quant", 11)):
        monkeypatch.setattr(bbs.lib, name, entry(name, at))
    monkeypatch.setattr(bbs, "_on_current", lambda stream, *t: 0)
    monkeypatch.setattr(bbs, "_stream", lambda stream: 0)
    monkeypatch.setattr(bbs, "_used_on", lambda ws, stream: None)
    return seen


def bwd(stream=None, ws=None):
    bbs.mxfp8_bias_act_bwd(bf(T, N), None, bbs.ACT_NONE, None, torch.zeros(N), ws=ws, stream=stream)


def moe(stream=None, ws=None):
    stack = lambda r, c: bbs.NVFP4Tensor.empty(E * r, c, device="cpu", n_scales=E)      # noqa: E731
    bbs.nvfp4_moe_gemv(0, bf(T, K), torch.zeros((T, 2), dtype=torch.int32), None, E, stack(F, K), stack(F, K), stack(N, F),
                       bf(T, N), 1, ws=ws, stream=stream)


def nv(rows, cols):
    return bbs.NVFP4Tensor.empty(rows, cols, device="cpu")


def quantize(stream=None, ws=None):
    bbs.nvfp4_quantize(bf(32, K), nv(32, K), amax_ws=ws, stream=stream)


def gemm_quant(stream=None, ws=None):
    bbs.nvfp4_gemm_quant(nv(32, K), nv(N, K), torch.ones(1), nv(32, N), gelu=True, ws=ws, stream=stream)


def grouped_quant(stream=None, ws=None):
    bbs.grouped_nvfp4_gemm_quant(nv(32, K), None, torch.zeros(2, dtype=torch.int32), 1, 32, nv(N, K), N, torch.ones(1),
                                 nv(32, N), gelu=True, ws=ws, stream=stream)


CALLS = {"mxfp8_bias_act_bwd": bwd, "nvfp4_moe_gemv": moe, "nvfp4_quantize": quantize, "nvfp4_gemm_quant": gemm_quant,
         "grouped_nvfp4_gemm_quant": grouped_quant}


@pytest.mark.parametrize("name", CALLS)
def test_own_workspace_is_made_on_the_calls_stream(made, name):
    CALLS[name](stream="given")
    CALLS[name]()
    assert made == [(name, "given"), (name, None)]


@pytest.mark.parametrize("name", CALLS)
def test_given_workspace_is_used(made, name):
    kind = torch.uint8 if name == "nvfp4_moe_gemv" else torch.float32
    CALLS[name](stream="given", ws=torch.zeros(1 << 16, dtype=kind))
    assert made == [(name, "not made by the call")]
