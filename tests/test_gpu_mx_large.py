"""The microscaled operators on tensors of more than 2^31 values, against the same calls on runs of their rows."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available() or torch.cuda.get_device_properties(0).total_memory < 64 << 30,
                                 reason="needs a CUDA device with 64 GB")]

import audio_driven_talking_b200 as fh  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
ROWS, COLS = 140001, 16384


def runs(rows, n):
    return [(i, min(rows, i + n)) for i in range(0, rows, n)]


@pytest.fixture(autouse=True)
def give_memory_back():
    yield
    torch.cuda.empty_cache()


def values(seed, *shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(seed))


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_quantize_and_back(fmt):
    x = values(1, ROWS, COLS)
    q = fh.quantize(x, fmt)
    back = fh.dequantize(q, BF)
    for i, j in runs(ROWS, 20000):
        part = fh.quantize(x[i:j], fmt)
        assert torch.equal(q.data[i:j], part.data) and torch.equal(back[i:j], fh.dequantize(part, BF))


def test_add_rms_norm():
    x, res, a = values(1, ROWS, COLS), values(2, ROWS, COLS), values(3, COLS, dtype=F32)
    total, y = fh.add_rms_norm(x, res, a, out="mxfp8")
    for i, j in runs(ROWS, 20000):
        t, p = fh.add_rms_norm(x[i:j], res[i:j], a, out="mxfp8")
        assert torch.equal(total[i:j], t) and torch.equal(y.data[i:j], p.data)


def test_rows_far_apart():
    x = torch.empty((5, 1 << 29), dtype=BF, device="cuda")
    v = x[:, :4096].normal_()
    a, b = fh.quantize(v), fh.quantize(v.contiguous())
    assert torch.equal(a.data, b.data) and torch.equal(a.scales, b.scales)


@pytest.mark.parametrize("N", [40032, 40001])     # results that leave by TMA, and rows off 16-byte boundaries
def test_linear_mx(N):
    M, K = 60001, 64
    A, W = fh.quantize(values(1, M, K), "mxfp4"), fh.quantize(values(2, N, K), "mxfp4")
    y = fh.linear_mx(A, W)
    for i in range(0, M, 128 * 100):               # whole scale tiles
        j = min(M, i + 128 * 100)
        part = fh.MXTensor(A.data[i:j], A.scales[i // 128 * 512:(j + 127) // 128 * 512], (j - i, K), A.fmt)
        assert torch.equal(y[i:j], fh.linear_mx(part, W))
