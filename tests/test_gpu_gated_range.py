"""The gated backward pass over every checkpoint value an MXFP8 block can hold:
every code at every block scale whose value is finite in FP32.  With dH = 1 and
u = 1 the outputs are the slope act'(g) and act(g) themselves."""
import numpy as np
import pytest

from gated_ref import ULP, act64, act_slope64, sigma64, _z
from gpu_util import announce, dev, host, to_dev

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def bbs():
    import bit_block_scaled_amd as b
    return b


def e4m3(codes):
    c = codes.astype(np.int64)
    e, m = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * np.exp2(e - 7.0))
    return np.where(c >= 128, -v, v)


def every_value():
    """255 x 256 codes and 255 x 8 scale bytes: row b holds every code at scale 2^(b - 127);
    NaN codes and codes whose value reaches 2^128 stand as +-1 times the scale."""
    codes = np.tile(np.arange(256, dtype=np.uint8), (255, 1))
    scales = np.repeat(np.arange(255, dtype=np.uint8)[:, None], 8, axis=1)
    unit = np.exp2(np.arange(255) - 127.0)[:, None]
    bad = ((codes & 0x7F) == 0x7F) | (np.abs(e4m3(codes)) * unit >= 2.0 ** 128)
    codes = np.where(bad, (codes & 0x80) | 0x38, codes).astype(np.uint8)
    return codes, scales, e4m3(codes) * unit


def one_hot(bbs, rows, K, code=0x38, byte=127):
    """Rows whose first value is code * 2^(byte - 127) and the rest zeros."""
    c = torch.zeros((rows, K), dtype=torch.uint8, device=dev())
    c[:, 0] = code
    s = torch.full((rows, K // 32), byte, dtype=torch.uint8, device=dev())
    return bbs.MXFP8Tensor(c, s, rows, K)


def tiled(bbs, codes, scales, M, F):
    """The pattern repeated over an M x F checkpoint (F a multiple of 32)."""
    r = -(-M // codes.shape[0]), -(-F // codes.shape[1])
    return bbs.MXFP8Tensor(to_dev(np.ascontiguousarray(np.tile(codes, r)[:M, :F])),
                           to_dev(np.ascontiguousarray(np.tile(scales, r)[:M, :F // 32])), M, F)


def full(bbs, M, F, code, byte):
    return bbs.MXFP8Tensor(torch.full((M, F), code, dtype=torch.uint8, device=dev()),
                           torch.full((M, F // 32), byte, dtype=torch.uint8, device=dev()), M, F)


# Rounding as in gated_ref.py, but with a bound below the reciprocal's range that
# does not grow with g.  Where e^-z passes 2^126 (z < -87.3) the reciprocal may flush,
# and past 2^128 s is 0.  There |g| sigma(z) <= 89 e^-87.3 < 89 2^-125 (SiLU; it falls
# as |g| grows, and GELU has |g| about 10), and the slope's second term is the same
# times dz/dg <= 24 (GELU, |g| about 10): both below 2^-117.
TINY = 2.0 ** -117


def bounds(act, g):
    with np.errstate(over="ignore"):
        z, dz = _z(act, np.clip(g, -64, 64))       # beyond, s is 0 or 1 and s q is 0
    s, q = sigma64(z), sigma64(-z)
    ag = np.minimum(np.abs(g), 64)
    ea = 16 * ULP * np.abs(g) * s + 6 * ULP * ag * s * q * np.abs(z) + TINY
    es = 24 * ULP * (s + ag * s * q * dz) + 6 * ULP * np.abs(z) * s * q * (1 + ag * dz) + TINY
    return ea, es


def exact(act, g):
    """act(g) and its slope; at |g| > 1000 both are those of the sign alone."""
    far = np.abs(g) > 1000
    near = np.where(far, 0.0, g)
    a = np.where(far, np.maximum(g, 0.0), act64(act, near))
    return a, np.where(far, (g > 0) * 1.0, act_slope64(act, near))


def check(got, ref, E, bf16, g, what):
    tol = E + (np.abs(ref) + E) * 2.0 ** -8 if bf16 else E
    bad = ~(np.abs(got - ref) <= tol)
    at = np.argwhere(bad)
    assert len(at) == 0, (what, len(at), *(v[tuple(at[0])] for v in (g, got, ref, tol)))


# the small tiles, the 128-row tiles, and the large tiles with whole and partial slabs
@pytest.mark.parametrize("M,F,K", [(255, 256, 32), (2500, 3360, 128), (2500, 3360, 2048), (2500, 3360, 2080)])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_slope_over_every_checkpoint_value(bbs, M, F, K, bf16, act):
    announce(f"gated bwd range {M} x {F} x {K} bf16={bf16} {act}")
    codes, scales, g = every_value()
    d = torch.full((2, M, F), 7.0, dtype=torch.bfloat16 if bf16 else torch.float32, device=dev())
    bbs.mxfp8_gemm_gated_bwd(one_hot(bbs, M, K), one_hot(bbs, F, K), tiled(bbs, codes, scales, M, F),
                             full(bbs, M, F, 0x38, 127), d[0], d[1], int(bf16), act=int(act == "gelu"))
    torch.cuda.synchronize()
    got = host(d.float()).astype(np.float64)
    g = np.tile(g, (-(-M // 255), -(-F // 256)))[:M, :F]
    a, sl = exact(act, g)
    ea, es = bounds(act, g)
    check(got[0], sl, es, bf16, g, "slope")
    check(got[1], a, ea, bf16, g, "act")


@pytest.mark.parametrize("T,N,gated", [(1, (1 << 30) + 4096, False), (2, (1 << 29) + 4112, True)])
def test_rows_beyond_a_launch(bbs, T, N, gated):
    """More rows than one launch has threads for: every output is written.  K = 16, weights 1
    and 2 by parts of 2^20 rows, so y = 16 or 32 times the token's value."""
    announce(f"gemv {T} x {N} rows, gated={gated}")
    K = 16
    part = (torch.arange(N, device=dev()) >> 20) % 2
    codes = torch.where(part.bool(), 0x44, 0x22).to(torch.uint8)[:, None].repeat(1, K // 2)
    W = bbs.NVFP4Tensor(codes, torch.full((N, 1), 0x38, dtype=torch.uint8, device=dev()),
                        torch.ones(1, device=dev()), N, K, False)
    x = torch.arange(1, T + 1, device=dev()).bfloat16()[:, None].repeat(1, K)
    y = torch.full((T, N), 7.0, dtype=torch.bfloat16, device=dev())
    if gated:
        bbs.nvfp4_gated_gemv(0, x, W, W, y, 1)
    else:
        bbs.nvfp4_gemv(0, x, W, y, 1)
    for t in range(T):
        ref = 16.0 * (t + 1) * (1 + part.float())
        if gated:
            ref = ref * ref                        # SiLU of 16 and more is g (1 - 2^-23 at most)
        assert torch.equal(y[t].float(), ref.bfloat16().float()), t


@pytest.mark.parametrize("T", [1, 3, 7, 64])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_longest_rows_of_the_few_token_products(bbs, T, fmt):
    """K = 2^26, the most the calls take, and 80 rows: a weight of 2 in the last place of row n,
    one of 1 at n 2^19 and zeros elsewhere, x counting in powers of two."""
    announce(f"gemv {T} x 80 x 2^26 {fmt}")
    N, K = 80, 1 << 26
    codes = torch.zeros((N, K // 2), dtype=torch.uint8, device=dev())
    at = torch.arange(N, device=dev()) << 19
    codes[torch.arange(N, device=dev()), at // 2] = 2                     # 1 in the even column
    codes[:, -1] = 4 << 4                                                 # 2 in the last column
    x = torch.zeros((T, K), dtype=torch.bfloat16, device=dev())
    x[:, at] = torch.exp2((torch.arange(N, device=dev()) % 7).double()).bfloat16()
    x[:, -1] = torch.arange(1, T + 1, device=dev()).bfloat16()
    if fmt == "nvfp4":
        W = bbs.NVFP4Tensor(codes, torch.full((N, K // 16), 0x38, dtype=torch.uint8, device=dev()),
                            torch.ones(1, device=dev()), N, K, False)
    else:
        W = bbs.MXFP4Tensor(codes, torch.full((N, K // 32), 127, dtype=torch.uint8, device=dev()), N, K)
    y, h = (torch.full((T, N), 7.0, dtype=torch.float32, device=dev()) for _ in range(2))
    bbs.nvfp4_gemv(0 if fmt == "nvfp4" else 2, x, W, y, 0)
    bbs.nvfp4_gated_gemv(0 if fmt == "nvfp4" else 2, x, W, W, h, 0)
    t, n = np.arange(1, T + 1)[:, None], np.arange(N)[None]
    ref = np.exp2(n % 7) + 2.0 * t
    assert np.array_equal(host(y).astype(np.float64), ref)
    sq, E = ref * act64("silu", ref), 32 * ULP * ref * ref                # 16 roundings, and 6 of z
    assert np.all(np.abs(host(h) - sq) <= E)
