"""The expert numbers that QMoEInference hands to the expert layer, by the integer type
they come in.  The kernels are replaced by recorders, so nothing runs on a GPU."""
import pytest

torch = pytest.importorskip("torch")

from bit_block_scaled_amd import layer as L                                 # noqa: E402

K, F, N = 32, 16, 16


@pytest.fixture
def seen(monkeypatch):
    ids = []
    for name, f in (("nvfp4_quantize", lambda *a, **kw: None), ("_on_current", lambda *a: 0),
                    ("nvfp4_moe_gemv", lambda fmt, x, i, *a, **kw: ids.append(i))):
        monkeypatch.setattr(L, name, f)
    return ids


def layer(E):
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)                    # noqa: E731
    return L.QMoEInference(bf(E, F, K), bf(E, F, K), bf(E, N, F))


KINDS = (torch.int8, torch.uint8, torch.int16, torch.uint16, torch.int32, torch.uint32, torch.int64, torch.uint64)


@pytest.mark.parametrize("E", [9, 130, 200, 255, 256, 1000])
@pytest.mark.parametrize("kind", KINDS)
def test_ids_of_every_type(seen, kind, E):
    """What is in [0, E) arrives as it is, everything else as no expert's number."""
    info = torch.iinfo(kind)
    # the type's ends, around E and its image in eight bits, and numbers whose lower bits are an expert's
    want = [info.min, info.max, info.max - 1, 0, 1, 5, 100, 127, E - 1, E, E + 1, -1, -E, (1 << 32) + 2, (1 << 40), (1 << 63) + 1]
    want = [v for v in want if info.min <= v <= info.max]
    # (torch builds unsigned 64-bit values past 2^63 from their signed image)
    ids = torch.tensor([v - (1 << 64) if v >= 1 << 63 else v for v in want], dtype=torch.int64)
    ids = (ids.view(torch.uint64) if kind == torch.uint64 else ids.to(kind)).reshape(1, -1)
    assert info.bits == 64 or ids.to(torch.int64).flatten().tolist() == want
    layer(E)(torch.zeros((1, K)), ids)
    got, = seen
    assert got.dtype == torch.int32 and got.shape == ids.shape and got.is_contiguous()
    for v, g in zip(want, got.flatten().tolist()):
        assert g == v if 0 <= v < E else not 0 <= g < E, (v, g)


def test_strided_ids(seen):
    ids = torch.arange(24, dtype=torch.int32).reshape(4, 6)[:, ::2]
    layer(9)(torch.zeros((4, K)), ids)
    assert seen[0].is_contiguous() and [v for v in seen[0].flatten().tolist() if 0 <= v < 9] == [0, 2, 4, 6, 8]
