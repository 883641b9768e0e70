"""add_rms_norm on rows whose squares leave float32's range: their norm is as finite as any other's.

The bound is that of the other rows, 64 u of |n| (1 + |a|) + |c| with u = 2^-24: the row is scaled by a power
of two, exactly, but for values 2^-126 of its largest and smaller, which the inputs do not have."""
import numpy as np
import pytest

import mx_reference as mx

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

import audio_driven_talking_b200 as fh  # noqa: E402

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
SIZES = [1e15, 1e18, 3e18, 1e19, 1e25, 1e30, 3e37, 1e-10, 1e-15, 1e-18, 1e-22, 1e-28, 1e-34]


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def check(got, y, tol):
    if isinstance(got, fh.MXTensor):
        mx.check_result(got, y, tol)
        return
    half = 0.0 if got.dtype == F32 else 2.0 ** -8
    d = np.abs(f64(got) - y) - (half * np.abs(y) + (1 + half) * tol)
    assert np.isfinite(f64(got)).all() and (d <= 0).all(), float(d.max())


@pytest.mark.parametrize("out", [F32, BF, "mxfp8", "mxfp4"])
@pytest.mark.parametrize("D", [32, 256, 1536, 2400, 6144, 16384])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_rows_of_every_size(D, eps, out):
    rng = np.random.default_rng(D)
    for M, xt, rt in ((len(SIZES), F32, BF), (300, BF, F32)):
        size = np.resize(np.array(SIZES), M)[:, None]
        x, res = (torch.from_numpy((rng.uniform(0.5, 2, (M, D)) * rng.choice([-1, 1], (M, D)) * size).astype(np.float32)).cuda().to(t)
                  for t in (xt, rt))
        a, c = (torch.from_numpy(rng.standard_normal(D).astype(np.float32)).cuda() for _ in range(2))
        total, y = fh.add_rms_norm(x, res, a, c, out=out, eps=eps)
        assert torch.equal(total, (x.float() + res.float()).to(xt))
        t, e = f64(total), float(np.float32(eps))
        n = t / np.sqrt((t ** 2).mean(1, keepdims=True) + e)
        g, h = f64(a), f64(c)
        check(y, n * (1 + g) + h, 64 * U * (np.abs(n) * (1 + np.abs(g)) + np.abs(h)))


def test_the_largest_rows_and_the_others_beside_them():
    """Rows of float32's largest number; their neighbours' results are those without them."""
    D = 512
    x = torch.randn(9, D, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    zero, g = torch.zeros(9, D, device="cuda"), torch.ones(D, device="cuda")
    want = fh.add_rms_norm(x, zero, g, out=F32)[1]
    x[2], x[5], x[7] = torch.finfo(F32).max, -torch.finfo(F32).max, 0.0
    got = fh.add_rms_norm(x, zero, g, out=F32)[1]
    assert (got[2] - 1).abs().max() <= 64 * U and (got[5] + 1).abs().max() <= 64 * U and not got[7].any()
    keep = [0, 1, 3, 4, 6, 8]
    assert torch.equal(got[keep], want[keep])


def test_rows_with_an_infinity_or_a_nan_among_large_values():
    x = torch.full((3, 256), 1e25, device="cuda")
    x[0, 3], x[1, 100] = float("inf"), float("nan")
    y = fh.add_rms_norm(x, torch.zeros_like(x), torch.ones(256, device="cuda"), out=F32)[1]
    assert y[0, 3].isnan() and not y[0, 4:].any()             # inf / inf, and 1e25 / inf
    assert y[1].isnan().all()
    assert ((y[2] - 1).abs() <= 64 * U).all()
