"""The statistical limit of FP32 sums, and what it tells apart.

A sum of K products of independent signs walks as sqrt(j) s after j of them (s
their RMS), and each addition rounds by at most 2^-24 of the sum, RMS 2^-24 /
sqrt(3) of it: 2^-24 s K / sqrt(6) in all for one long chain, that is 2^-24
sqrt(K / 6) of the result's RMS; every other order adds fewer or smaller
roundings.  The limit is twice that, rounded up, with eight roundings more for
the block scales, the joining of split sums and the output's scale."""
import numpy as np
import pytest


def sum_limit(K):
    return 2.0 ** -24 * (K ** 0.5 + 8)


def rounded(v, bits):
    """v to `bits` significant bits, nearest."""
    m, e = np.frexp(v)
    return np.ldexp(np.round(m * 2 ** bits), e - bits)


@pytest.mark.parametrize("K", [512, 4096, 14336])
def test_limit_tells_short_sums_apart(K):
    rng = np.random.default_rng(1)
    p = (rng.standard_normal((512, K)) * rng.standard_normal((512, K))).astype(np.float32).astype(np.float64)
    ref = p.sum(1)
    rel = lambda y: np.sqrt(np.mean((y - ref) ** 2) / np.mean(ref ** 2))    # noqa: E731
    # one chain in FP32
    acc = np.zeros(512, np.float32)
    for k in range(K):
        acc = acc + p[:, k].astype(np.float32)
    assert rel(acc.astype(np.float64)) <= sum_limit(K)
    # eight partial sums, each rounded once: FP32, FP16 (11 bits), BF16 (8 bits)
    parts = p.reshape(512, 8, -1).sum(2)
    assert rel(rounded(parts, 24).sum(1)) <= sum_limit(K)
    assert rel(rounded(parts, 11).sum(1)) > 8 * sum_limit(K)
    assert rel(rounded(parts, 8).sum(1)) > 64 * sum_limit(K)
