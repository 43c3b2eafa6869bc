"""The bindings' given row strides and streams, and outputs larger than the
result: what the plain calls give, and nothing written beside it."""
import pytest

import test_gpu_gated as G
from gpu_util import announce, dev

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def bbs():
    import bit_block_scaled_amd as b
    return b


def test_given_strides_and_streams(bbs):
    announce("gated bindings: given strides and streams")
    T, M, F, K, P = 5, 48, 96, 160, 8
    A, Wg, Wu = G.random_nv(bbs, M, K, False, 1), G.random_nv(bbs, F, K, True, 2), G.random_nv(bbs, F, K, True, 3)
    dY, Wt = G.random_mx(bbs, M, K, 4), G.random_mx(bbs, F, K, 5)
    c = G.random_mx(bbs, M, F, 6), G.random_mx(bbs, M, F, 7)
    x = torch.randn((T, K), device=dev()).bfloat16()
    bf = lambda r, k: torch.full((r, k), 7.0, dtype=torch.bfloat16, device=dev())           # noqa: E731
    side = torch.cuda.Stream()

    def run(place, kw):
        """place(rows): an output of that many rows and F columns, with the arguments that describe it."""
        y, v, h, d = place(T), place(T), place(M), place(M)
        e = place(M)
        bbs.nvfp4_gemv(0, x, Wg, y, 1, **kw("ldy"))
        bbs.nvfp4_gated_gemv(0, x, Wg, Wu, v, 1, **kw("ldh"))
        bbs.nvfp4_gated_gemm(A, Wg, Wu, h, 1, **kw("ldh"))
        bbs.mxfp8_gemm_gated_bwd(dY, Wt, *c, d, e, 1, **kw("ld"))
        return y, v, h, d, e

    plain = run(lambda r: bf(r, F), lambda name: {})
    torch.cuda.synchronize()
    wide = run(lambda r: bf(r + 1, F + P)[:, :F], lambda name: {})                          # more rows, wider rows
    flat = run(lambda r: bf(1, (r + 1) * (F + P)).view(-1), lambda name: {name: F + P})     # rows of a flat buffer
    side.wait_stream(torch.cuda.current_stream())
    other = run(lambda r: bf(r, F), lambda name: {"stream": side})
    torch.cuda.synchronize()
    for p, w, f, o in zip(plain, wide, flat, other):
        r = len(p)
        f = f.view(r + 1, F + P)
        assert torch.equal(p, w[:r]) and torch.equal(p, f[:r, :F]) and torch.equal(p, o)
        assert bool((w[r] == 7).all()) and bool((f[:, F:] == 7).all()) and bool((f[r] == 7).all())
        assert bool((w.as_strided((r + 1, P), (F + P, 1), w.storage_offset() + F) == 7).all())
    with pytest.raises(ValueError):
        bbs.nvfp4_gemv(0, x.cpu(), Wg, bf(T, F), 1)
    with pytest.raises(ValueError):
        bbs.nvfp4_gated_gemm(A, Wg, Wu, bf(M, F).cpu(), 1)
