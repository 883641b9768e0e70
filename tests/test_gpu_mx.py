"""The microscaled operators on the GPU against 64-bit references: quantisation bit for bit, the
norm and the block-scaled product within bounds counted from their roundings, and runs of them
together - in a graph, on other streams, in place.

Bounds. u = 2^-24 is half a step of float32. The norm's result is a chain of at most 64 + 5 + 32
additions of squares (relative error 101 u, halved by the square root) and a dozen further
roundings: 64 u of |n| (1 + |a|) + |c|. A product of length K is accumulated in float32 with at
most a whole step 2 u per addition: 2 u (K + 8) of sum |A| |W| + |bias|, times 1.13, the largest
slope of GELU, plus 16 u of the result for the activation itself. Results in bf16 add half a step,
2^-8 of their value; microscaled ones what mx_reference.check_result states."""
import numpy as np
import pytest

import mx_reference as mx

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

import audio_driven_talking_b200 as fh  # noqa: E402

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
FMTS = ["mxfp8", "mxfp4"]


def dev(a, dtype=F32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(dtype)


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def randn(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def check_values(got, y, tol):
    """A float32 or bf16 result against 64 bits."""
    half = 0.0 if got.dtype == F32 else 2.0 ** -8
    d = np.abs(f64(got) - y) - (half * np.abs(y) + (1 + half) * tol)
    assert np.isfinite(f64(got)).all() and (d <= 0).all(), float(d.max())


def check_any(got, y, tol):
    if isinstance(got, fh.MXTensor):
        mx.check_result(got, y, tol)
    else:
        check_values(got, y, tol)


# ------------------------------------------------------------------------------ quantise
def edge_rows(K, fmt):
    """Blocks at the format's edges: ties, the largest element and its neighbours, zeros, the ends of float32."""
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] if fmt == "mxfp4"
                    else [448.0, 432.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 0.0, 1.0])
    top, f32 = mx.TOP[fmt], np.float32
    rows = []
    for s in (1.0, 2.0 ** -20, 2.0 ** 90):
        rows.append(np.resize(np.concatenate([ties, -ties]) * s, K))
    for m in (top, np.nextafter(f32(top), f32(1e9)), np.nextafter(f32(top), f32(0)), 2.0 ** 127 * 1.75, 2.0 ** -126,
              2.0 ** -149, 3 * 2.0 ** -140, top * 2.0 ** -127, np.finfo(f32).max):
        rows.append(np.resize(np.array([m, -m / 2, 0.0, m / 3], dtype=f32), K))
    rows.append(np.zeros(K))
    return np.array(rows, dtype=f32)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("M,K", [(1, 32), (1, 1536), (3, 64), (31, 96), (127, 128), (128, 128), (129, 160), (300, 1568),
                                 (257, 4128), (1280, 1536)])
def test_quantize_and_back(M, K, dtype, fmt):
    x = randn(M + K, M, K) * np.exp(2 * randn(M * K + 1, K))
    edges = edge_rows(K, fmt)
    x[:min(M, len(edges))] = edges[:min(M, len(edges))]
    x = dev(x, dtype)
    q = fh.quantize(x, fmt)
    el, byte = mx.quantize(f64(x), fmt)
    gel, gbyte, flat = mx.read(q)
    assert np.array_equal(gbyte, byte)
    assert np.array_equal(gel, el)
    assert not mx.padding(flat, M, K).any()
    # float32's largest number, (2 - 2^-23) 2^127, is 255.99... 2^120 in e4m3, whose step there is 16:
    # the element is 256, and 256 * 2^120 = 2^128 reads back as infinite in float32; all else is exact.
    # (In bf16 the same number is an infinity to begin with, and its block NaN.)
    with np.errstate(over="ignore"):
        want = mx.values(el, byte).astype(np.float32)
    np.testing.assert_array_equal(fh.dequantize(q).cpu().numpy(), want)
    np.testing.assert_array_equal(f64(fh.dequantize(q, BF)), f64(torch.from_numpy(want).to(BF)))


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_blocks_that_are_not_finite(fmt):
    x = randn(5, 140, 128)
    x[0, 3], x[1, 40], x[2, 127], x[139, 64] = np.nan, np.inf, -np.inf, np.nan
    for dtype in (F32, BF):
        t = dev(x, dtype)
        back = f64(fh.dequantize(fh.quantize(t, fmt)))
        nan = np.zeros((140, 4), dtype=bool)
        nan[0, 0] = nan[1, 1] = nan[2, 3] = nan[139, 2] = True
        nan = np.repeat(nan, 32, axis=1)
        assert np.isnan(back[nan]).all()
        el, byte = mx.quantize(np.where(nan, 0.0, f64(t)), fmt)
        assert np.array_equal(back[~nan], mx.values(el, byte)[~nan])


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_rows_apart(fmt):
    for dtype, gap in ((F32, 4), (BF, 8), (BF, 1000)):
        big = dev(randn(6, 133, 160 + gap), dtype)
        a, b = fh.quantize(big[:, :160], fmt), fh.quantize(big[:, :160].contiguous(), fmt)
        assert torch.equal(a.data, b.data) and torch.equal(a.scales, b.scales)
    with pytest.raises(fh.FHError, match="stride"):
        fh.quantize(dev(randn(6, 133, 162))[:, :160], fmt)
    with pytest.raises(fh.FHError, match="unaligned"):
        fh.quantize(dev(randn(6, 4, 164))[:, 1:161], fmt)
    with pytest.raises(ValueError, match="contiguous rows"):
        fh.quantize(dev(randn(6, 160, 160)).t(), fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_dequantize_every_code_and_scale(fmt):
    """Any bytes at all: every code under every scale, e4m3's NaN and the NaN scale among them."""
    M, K = 257, 32 * (8 if fmt == "mxfp8" else 1)
    q = fh.MXTensor.empty(M, K, fmt, "cuda")
    codes = np.arange(256, dtype=np.uint8) if fmt == "mxfp8" else np.resize(np.arange(256, dtype=np.uint8), 16)
    data = np.tile(codes, (M, 1)) if fmt == "mxfp8" else (np.arange(M)[:, None] * 16 + codes).astype(np.uint8)
    byte = np.repeat((np.arange(M) % 256).astype(np.uint8)[:, None], K // 32, axis=1)
    q.data.copy_(torch.from_numpy(data))
    q.scales.copy_(torch.from_numpy(mx.tile(byte, K)))
    want = mx.values(mx.unpack(data, fmt), byte)
    with np.errstate(over="ignore"):
        w32 = torch.from_numpy(want.astype(np.float32))
    assert torch.equal(fh.dequantize(q).cpu().nan_to_num(7.5), w32.nan_to_num(7.5))
    assert torch.equal(fh.dequantize(q, BF).cpu().nan_to_num(7.5), w32.to(BF).nan_to_num(7.5))


# ------------------------------------------------------------------------------ residual + norm
def norm_reference(total, a, c, streams, eps):
    M, D = total.shape
    n = total / np.sqrt((total ** 2).mean(1, keepdims=True) + eps)
    r = np.arange(M) // (M // streams)
    a = np.broadcast_to(a, (streams, D))[r]
    if c is None:
        return n * a, 64 * U * np.abs(n) * np.abs(a)
    c = np.broadcast_to(c, (streams, D))[r]
    return n * (1 + a) + c, 64 * U * (np.abs(n) * (1 + np.abs(a)) + np.abs(c))


@pytest.mark.parametrize("out", [F32, BF, "mxfp8", "mxfp4"])
@pytest.mark.parametrize("M,D,streams,mod,xt,rt", [
    (1, 32, 1, False, F32, BF), (1, 1536, 1, True, F32, BF), (5, 96, 5, True, BF, BF), (130, 160, 2, True, BF, F32),
    (777, 1568, 1, False, BF, BF), (256, 512, 2, False, F32, F32), (99, 1024, 3, True, F32, BF), (7, 2048, 7, True, F32, F32),
    (129, 2080, 1, False, F32, BF), (33, 4096, 3, True, BF, F32), (20, 6144, 2, True, F32, BF), (6, 8224, 2, True, F32, F32),
    (4, 16384, 1, False, BF, BF), (1280, 1536, 1, True, F32, BF)])
def test_add_rms_norm(M, D, streams, mod, xt, rt, out):
    x, res = dev(4 * randn(M + D, M, D), xt), dev(randn(M + D + 1, M, D), rt)
    a = dev(0.3 * randn(D, streams, D)) if mod else dev(1 + 0.1 * randn(D, streams, D))
    c = dev(0.3 * randn(D + 1, streams, D)) if mod else None
    if streams == 1:
        a, c = a[0], None if c is None else c[0]
    total, y = fh.add_rms_norm(x, res, a, c, out=out, eps=1e-6)
    assert torch.equal(total, (x.float() + res.float()).to(xt))
    want, tol = norm_reference(f64(total), f64(a), None if c is None else f64(c), streams, 1e-6)
    check_any(y, want, tol)
    again = fh.add_rms_norm(x, res, a, c, out=out, eps=1e-6)[1]
    if isinstance(y, fh.MXTensor):
        assert torch.equal(y.data, again.data) and torch.equal(y.scales, again.scales)
    else:
        assert torch.equal(y, again)


@pytest.mark.parametrize("M", [3, 256, 259])
@pytest.mark.parametrize("D", [64, 256, 480, 512, 640, 1024, 1280, 1792, 2048, 2240, 2400, 2720, 3616, 4096, 4640, 5344, 6144, 8192, 12320])
def test_add_rms_norm_widths(D, M):
    """Row widths at and between the shapes that share a row, for few rows and many."""
    for xt, rt, mod, out in ((F32, BF, True, "mxfp8"), (BF, BF, False, "mxfp4"), (BF, F32, True, BF), (F32, F32, False, F32)):
        x, res = dev(4 * randn(M + D, M, D), xt), dev(randn(M + D + 1, M, D), rt)
        a, c = dev(1 + 0.1 * randn(D, D)), dev(0.3 * randn(D + 1, D)) if mod else None
        total, y = fh.add_rms_norm(x, res, a, c, out=out)
        assert torch.equal(total, (x.float() + res.float()).to(xt))
        check_any(y, *norm_reference(f64(total), f64(a), None if c is None else f64(c), 1, 1e-6))


def test_add_rms_norm_in_place_and_zero_rows():
    x, res = dev(randn(1, 50, 1536)), dev(randn(2, 50, 1536))
    x[7] = 0
    res[7] = 0
    g = dev(1 + 0.1 * randn(3, 1536))
    want, y = fh.add_rms_norm(x, res, g, out="mxfp8")
    assert not y.data[7].any()                            # 0 / sqrt(0 + eps)
    for target in (x.clone(), res.clone()):
        args = (target, res) if torch.equal(target, x) else (x, target)
        total, y2 = fh.add_rms_norm(*args, g, out="mxfp8", sum_out=target)
        assert total is target and torch.equal(target, want)
        assert torch.equal(y2.data, y.data) and torch.equal(y2.scales, y.scales)
    with pytest.raises(fh.FHError, match="overlaps"):     # shifted by one row
        big = dev(randn(4, 51, 1536))
        fh.add_rms_norm(big[:50], res, g, sum_out=big[1:])


@pytest.mark.parametrize("D", [64, 1536, 3104, 8224])
def test_add_rms_norm_on_16_byte_boundaries(D):
    """Inputs, sum and vectors that lie on 16 bytes but not on 32."""
    M = 37

    def off(a, dtype=F32):
        t = dev(a, dtype)
        skip = 16 // t.element_size()
        buf = torch.empty(t.numel() + skip, dtype=dtype, device="cuda")
        buf[skip:] = t.reshape(-1)
        v = buf[skip:].view(t.shape)
        assert v.data_ptr() % 32 == 16
        return v

    for xt, rt in ((F32, BF), (BF, F32), (F32, F32)):
        x, res, a, c = randn(D, M, D), randn(D + 1, M, D), 0.3 * randn(D + 2, D), randn(D + 3, D)
        want = fh.add_rms_norm(dev(x, xt), dev(res, rt), dev(a), dev(c), out="mxfp8")
        total = off(np.zeros((M, D)), xt)
        got = fh.add_rms_norm(off(x, xt), off(res, rt), off(a), off(c), out="mxfp8", sum_out=total)
        assert torch.equal(got[0], want[0])
        assert torch.equal(got[1].data, want[1].data) and torch.equal(got[1].scales, want[1].scales)
    q = fh.quantize(off(randn(D, M, D)), "mxfp4")
    p = fh.quantize(dev(randn(D, M, D)), "mxfp4")
    assert torch.equal(q.data, p.data) and torch.equal(q.scales, p.scales)


def test_add_rms_norm_rows_that_are_not_finite():
    x, res = dev(randn(1, 9, 256)), dev(randn(2, 9, 256), BF)
    x[2, 5], res[6, 200] = float("inf"), float("nan")
    g = dev(np.ones(256))
    clean = fh.add_rms_norm(dev(randn(1, 9, 256)), dev(randn(2, 9, 256), BF), g, out="mxfp8")[1]
    q = fh.add_rms_norm(x, res, g, out="mxfp8")[1]
    back = f64(fh.dequantize(q))
    assert np.isnan(back[6]).all() and np.isnan(back[2]).any()
    keep = [0, 1, 3, 4, 5, 7, 8]
    assert torch.equal(q.data[keep], clean.data[keep])


def test_add_rms_norm_refuses():
    x, g = dev(randn(1, 6, 64)), dev(np.ones(64))
    for bad in (lambda: fh.add_rms_norm(x, x[:5], g), lambda: fh.add_rms_norm(x, x, g[:32]),
                lambda: fh.add_rms_norm(x, x, g.expand(4, 64).contiguous()), lambda: fh.add_rms_norm(x, x, g, g.expand(2, 64)),
                lambda: fh.add_rms_norm(x, x, g.to(BF)), lambda: fh.add_rms_norm(x[:, ::2], x[:, ::2], g[:32]),
                lambda: fh.add_rms_norm(x, x, g, sum_out=x.to(BF)), lambda: fh.add_rms_norm(x, x, g.cpu())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        fh.add_rms_norm(x.half(), x, g)
    with pytest.raises(fh.FHError, match="multiple of 32"):
        fh.add_rms_norm(x[:, :48].contiguous(), x[:, :48].contiguous(), g[:48], out=BF)


# ------------------------------------------------------------------------------ product
def operands(seed, M, N, K, fmt):
    A = fh.quantize(dev(randn(seed, M, K) * np.exp(0.5 * randn(seed + 1, K))), fmt)
    W = fh.quantize(dev(randn(seed + 2, N, K) / np.sqrt(K)), fmt)
    return A, W, dev(0.5 * randn(seed + 3, N))


def gelu64(y):
    return 0.5 * y * (1 + np.tanh(np.sqrt(2 / np.pi) * (y + 0.044715 * y ** 3)))


def linear_reference(A, W, bias, act):
    """Values and bound; on the GPU in 64 bits for the products of many terms."""
    a, w = fh.dequantize(A).double(), fh.dequantize(W).double()
    b = torch.zeros(w.shape[0], dtype=torch.float64, device="cuda") if bias is None else bias.double()
    y, mag = f64(a @ w.t() + b), f64(a.abs() @ w.abs().t() + b.abs())
    tol = 2 * U * (A.shape[1] + 8) * mag
    return (gelu64(y), 1.13 * tol + 16 * U * np.abs(gelu64(y))) if act else (y, tol)


SHAPES = [(1, 1, 32), (1, 128, 32), (1, 9216, 1536), (2, 33, 64), (7, 32, 96), (31, 96, 128), (128, 128, 128), (128, 256, 256),
          (129, 130, 160), (130, 160, 288), (437, 1001, 1568), (256, 512, 512), (257, 288, 544), (300, 1536, 1024),
          (640, 896, 2080), (1280, 1536, 1536), (1000, 8960, 320), (64, 4608, 8960), (2000, 2048, 96), (4100, 1056, 1536)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_mx(M, N, K, fmt):
    A, W, bias = operands(M + N + K, M, N, K, fmt)
    y, tol = linear_reference(A, W, bias, None)
    first = fh.linear_mx(A, W, bias, out=F32)
    check_values(first, y, tol)
    assert torch.equal(first, fh.linear_mx(A, W, bias, out=F32))
    check_values(fh.linear_mx(A, W, bias), y, tol)
    g, gtol = linear_reference(A, W, bias, "gelu")
    check_values(fh.linear_mx(A, W, bias, act="gelu", out=F32), g, gtol)
    if N % 32 == 0:
        for kind in FMTS:
            mx.check_result(fh.linear_mx(A, W, bias, act="gelu", out=kind), g, gtol)
    else:
        with pytest.raises(ValueError, match="multiple of 32"):
            fh.linear_mx(A, W, bias, out="mxfp8")
    y0, tol0 = linear_reference(A, W, None, None)
    check_values(fh.linear_mx(A, W), y0, tol0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(1, 1, 8960), (1, 64, 8960), (1, 1536, 8960), (3, 200, 4096), (33, 96, 8960), (128, 160, 8960),
                                   (129, 129, 8960), (200, 512, 8960), (300, 1000, 8960), (64, 4608, 8960), (17, 1056, 3008),
                                   (250, 32, 16384), (1, 32, 1 << 18)])
def test_linear_mx_few_rows_and_a_long_inner_dimension(M, N, K, fmt):
    """Products whose few tiles are shared by clusters of two, four and eight CTAs."""
    test_linear_mx(M, N, K, fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("N", [1, 2, 4, 7, 8, 12, 16, 24, 31, 40, 63, 65, 72, 100, 120, 127, 136])
def test_linear_mx_narrow_results(N, fmt):
    """Rows of results shorter than a box, on and off 16-byte boundaries, in both float types."""
    for M, K in ((3, 64), (130, 1024), (5, 8960)):
        A, W, bias = operands(N + K, M, N, K, fmt)
        y, tol = linear_reference(A, W, bias, "gelu")
        for out in (BF, F32):
            check_values(fh.linear_mx(A, W, bias, act="gelu", out=out), y, tol)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(4096, 4096, 1536), (4097, 4224, 2080), (2500, 8961, 1536), (3900, 8960, 1568), (8640, 1536, 4096),
                                   (1280, 4608, 1536), (1300, 4641, 1568), (100, 12320, 544), (1, 16384, 1536), (64, 18000, 96)])
def test_linear_mx_wide_tiles(M, N, K, fmt):
    """Several rounds of 256-column tiles, the last one of halves, on ragged edges; tiles of 192 columns;
    and few rows against many columns."""
    A, W, bias = operands(M + N + K, M, N, K, fmt)
    y, tol = linear_reference(A, W, bias, "gelu")
    for out in (BF, F32, "mxfp8", "mxfp4") if N % 32 == 0 else (BF, F32):
        check_any(fh.linear_mx(A, W, bias, act="gelu", out=out), y, tol)


@pytest.mark.parametrize("fmt", FMTS)
def test_linear_mx_scales_reach_the_right_blocks(fmt):
    """Operands of ones under scales that are different everywhere: sums of powers of two, exact."""
    M, N, K = 300, 270, 640
    rng = np.random.default_rng(3)
    sides = []
    for rows in (M, N):
        q = fh.quantize(torch.ones(rows, K, device="cuda"), fmt)
        el, byte, flat = mx.read(q)
        byte = (byte.astype(int) + rng.integers(-2, 3, byte.shape)).astype(np.uint8)
        q.scales.copy_(torch.from_numpy(mx.tile(byte, K)))
        sides.append((q, mx.values(el, byte)))
    want = sides[0][1] @ sides[1][1].T
    assert np.array_equal(f64(fh.linear_mx(sides[0][0], sides[1][0], out=F32)), want)


@pytest.mark.parametrize("fmt", FMTS)
def test_linear_mx_nan_blocks_stay_in_their_rows(fmt):
    M, N, K = 200, 160, 256
    x, w = randn(1, M, K), randn(2, N, K)
    x[150, 200] = np.nan
    w[33, 7] = np.inf
    y = f64(fh.linear_mx(fh.quantize(dev(x), fmt), fh.quantize(dev(w), fmt), out=F32))
    nan = np.zeros((M, N), dtype=bool)
    nan[150], nan[:, 33] = True, True
    assert np.array_equal(np.isnan(y), nan)
    g = f64(fh.linear_mx(fh.quantize(dev(x), fmt), fh.quantize(dev(w), fmt), act="gelu", out=F32))
    assert np.array_equal(np.isnan(g), nan)
    q = fh.linear_mx(fh.quantize(dev(x), fmt), fh.quantize(dev(w), fmt), out="mxfp8")
    back = f64(fh.dequantize(q))
    assert np.isnan(back[150]).all() and np.isnan(back[:, 32:64]).all()
    assert np.isfinite(np.delete(np.delete(back, 150, 0), np.s_[32:64], 1)).all()


def test_linear_mx_gelu_tails():
    """Results from far below zero to far above, without overflow: -0 or tiny values, and x itself."""
    A = fh.quantize(torch.ones(1, 32, device="cuda"), "mxfp8")
    W = fh.quantize(torch.zeros(2048, 32, device="cuda"), "mxfp8")
    bias = torch.cat([torch.linspace(-12, 12, 2040, device="cuda"),
                      torch.tensor([-3e38, -1e20, -1e5, -50.0, 50.0, 1e5, 1e20, 3e38], device="cuda")])
    inf = bias.clone()
    inf[100], inf[201] = float("inf"), -float("inf")
    far = f64(fh.linear_mx(A, W, inf, act="gelu", out=F32))[0]
    assert far[100] == np.inf and abs(far[201]) < 2.0 ** -28
    got = f64(fh.linear_mx(A, W, bias, act="gelu", out=F32))[0]
    want = gelu64(f64(bias))
    # relative to x: the tanh form's own cancellation at the far negative end is not the kernel's
    assert np.isfinite(got).all()
    # four neighbours share a reciprocal: what the infinities change in the others are its roundings, the
    # three products into it, itself (2 u) and the three out of it, 8 u each way at most
    rest = np.delete(np.arange(2048), [100, 201])
    assert (np.abs(far - got)[rest] <= 16 * U * np.abs(got[rest])).all()
    assert (np.abs(got - want) <= 64 * U * np.abs(want) + 2 * U * np.abs(np.clip(f64(bias), -12, 12)) + U * np.abs(f64(bias)) * (f64(bias) > 0)).all()


def test_linear_mx_refuses():
    A, W, b = operands(1, 8, 64, 64, "mxfp8")
    A4, _, _ = operands(1, 8, 64, 64, "mxfp4")
    A32, _, _ = operands(1, 8, 64, 32, "mxfp8")
    for bad in (lambda: fh.linear_mx(A4, W, b), lambda: fh.linear_mx(A32, W, b), lambda: fh.linear_mx(A, W, b[:32]),
                lambda: fh.linear_mx(A, W, b.to(BF)), lambda: fh.linear_mx(A, W, b.cpu()), lambda: fh.linear_mx(A, W, b, out=torch.half),
                lambda: fh.linear_mx(fh.MXTensor(A.data, A.scales[:256], A.shape, A.fmt), W, b),
                lambda: fh.linear_mx(fh.MXTensor(A.data.view(torch.int8), A.scales, A.shape, A.fmt), W, b),
                lambda: fh.linear_mx(A, fh.MXTensor(W.data.cpu(), W.scales, W.shape, W.fmt), b)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(fh.FHError, match="unaligned"):
        fh.linear_mx(A, W, torch.zeros(65, device="cuda")[1:])


# ------------------------------------------------------------------------------ memory, streams, runs of them
def raw(lib, name, *args):
    fh._check(getattr(lib, name)(*args, torch.cuda.current_stream().cuda_stream))


@pytest.mark.parametrize("M,N,K", [(1, 32, 32), (130, 288, 160), (300, 1056, 544), (1281, 1568, 1536)])
def test_nothing_is_written_past_the_results(M, N, K):
    lib, guard = fh.load_library(), 4096
    A, W, bias = operands(9, M, N, K, "mxfp8")
    x, res = dev(randn(1, M, K)), dev(randn(2, M, K), BF)
    g = dev(np.ones(K))

    def buf(n):
        return torch.full((n + guard,), 0xA5, dtype=torch.uint8, device="cuda")

    for kind, size in ((fh.FH_F32, 32), (fh.FH_BF16, 16), (fh.FH_MXFP8, 8), (fh.FH_MXFP4, 4)):
        nb, kb = M * N * size // 8, M * K * size // 8
        is_mx = kind >= fh.FH_MXFP8
        for n, cols, op in ((nb, N, "linear"), (kb, K, "norm"), (kb, K, "quantize")):
            ns = mx.scale_count(M, cols) if is_mx else 0
            data, scales = buf(n), buf(ns)
            sp = scales.data_ptr() if is_mx else None
            if op == "linear":
                raw(lib, "fh_op_linear_mx", A.data.data_ptr(), A.scales.data_ptr(), W.data.data_ptr(), W.scales.data_ptr(),
                    bias.data_ptr(), M, N, K, fh.FH_MXFP8, 0, kind, data.data_ptr(), sp)
            elif op == "norm":
                total = buf(M * K * 4)
                raw(lib, "fh_op_add_rms_norm", x.data_ptr(), 0, res.data_ptr(), 1, total.data_ptr(), g.data_ptr(), None, 0, M, M,
                    K, 1e-6, kind, data.data_ptr(), sp)
                assert (total[M * K * 4:] == 0xA5).all()
            elif is_mx:
                raw(lib, "fh_op_quantize", x.data_ptr(), K, M, K, 0, kind, data.data_ptr(), sp)
            torch.cuda.synchronize()
            assert (data[n:] == 0xA5).all() and (scales[ns:] == 0xA5).all()


def feed_forward(x, res, gain, w1, b1, w2, b2, gain2, mid, out):
    """The block's run of them: norm, FFN1 with its GELU, FFN2, and the next norm."""
    s, h = fh.add_rms_norm(x, res, gain, out=mid)
    u = fh.linear_mx(h, w1, b1, act="gelu", out=mid)
    f = fh.linear_mx(u, w2, b2)
    return s, h, u, f, *fh.add_rms_norm(s, f, gain2, out=out)


def ff_inputs(seed, M, D, H, fmt):
    return [dev(randn(seed, M, D)), dev(randn(seed + 1, M, D), BF), dev(1 + 0.1 * randn(seed + 2, D)),
            fh.quantize(dev(randn(seed + 3, H, D) / np.sqrt(D)), fmt), dev(0.1 * randn(seed + 4, H)),
            fh.quantize(dev(randn(seed + 5, D, H) / np.sqrt(H)), fmt), dev(0.1 * randn(seed + 6, D)), dev(1 + 0.1 * randn(seed + 7, D))]


def flat(results):
    for t in results:
        if isinstance(t, fh.MXTensor):
            yield t.data
            yield t.scales
        else:
            yield t


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,D,H", [(1, 1536, 8960), (200, 384, 1024), (333, 416, 992), (1280, 1536, 8960)])
def test_feed_forward(M, D, H, fmt):
    """Each step of the run against 64 bits on what the step before it gave."""
    x, res, g, w1, b1, w2, b2, g2 = args = ff_inputs(11, M, D, H, fmt)
    s, h, u, f, s2, y = feed_forward(*args, fmt, BF)
    assert torch.equal(s, x + res.float())
    check_any(h, *norm_reference(f64(s), f64(g), None, 1, 1e-6))
    check_any(u, *linear_reference(h, w1, b1, "gelu"))
    check_any(f, *linear_reference(u, w2, b2, None))
    assert torch.equal(s2, s + f.float())
    check_any(y, *norm_reference(f64(s2), f64(g2), None, 1, 1e-6))


@pytest.mark.parametrize("fmt", FMTS)
def test_feed_forward_captured_and_replayed(fmt):
    """One graph of the run, replayed on inputs refilled in place, bit for bit the eager run; two
    graphs replayed side by side on two streams keep their own results."""
    M, D, H = 300, 384, 1024
    ins = [ff_inputs(s, M, D, H, fmt) for s in (21, 22)]
    eager = [[t.clone() for t in flat(feed_forward(*i, fmt, "mxfp8"))] for i in ins]
    graphs = []
    for i in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = feed_forward(*i, fmt, "mxfp8")
        graphs.append((g, list(flat(out))))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(5):
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (_, out), want in zip(graphs, eager):
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    ins[0][0].copy_(ins[1][0])
    ins[0][1].copy_(ins[1][1])
    graphs[0][0].replay()
    again = [t.clone() for t in graphs[0][1]]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, flat(feed_forward(*ins[0], fmt, "mxfp8"))))


def test_other_streams():
    """Two runs in flight at once on streams of their own, given by argument as torch streams and as
    handles; memory of inputs that are dropped meanwhile is not reused before the work is done."""
    fmt = "mxfp8"
    ins = [ff_inputs(s, 500, 384, 1024, fmt) for s in (31, 32)]
    want = [[t.clone() for t in flat(feed_forward(*i, fmt, BF))] for i in ins]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for k, st in enumerate(streams):
            x, res, g, w1, b1, w2, b2, g2 = ins[k]
            arg = st if k == 0 else st.cuda_stream
            s, h = fh.add_rms_norm(x, res, g, out=fmt, stream=arg)
            u = fh.linear_mx(h, w1, b1, act="gelu", out=fmt, stream=arg)
            f = fh.linear_mx(u, w2, b2, stream=arg)
            s2, y = fh.add_rms_norm(s, f, g2, out=BF, stream=arg)
            got[k] = [s, h, u, f, s2, y]
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(a, b) for a, b in zip(flat(got[k]), want[k]))
    x = dev(randn(1, 64, 64))
    torch.cuda.synchronize()
    q = fh.quantize(x, "mxfp4", stream=0)                  # the legacy default stream
    back = fh.dequantize(q, stream=torch.cuda.default_stream())
    torch.cuda.synchronize()
    assert torch.equal(back, fh.dequantize(fh.quantize(x, "mxfp4")))


def test_a_wait_that_ran_out_is_reported():
    """A bounded wait of a kernel with no arriving party runs out (about a second): the next product
    raises it once and launches nothing, as does sync_operators; the calls after them work."""
    A, W, bias = operands(1, 40, 64, 64, "mxfp8")
    want = fh.linear_mx(A, W, bias)
    fh.sync_operators()
    for report in (lambda: fh.linear_mx(A, W, bias), fh.sync_operators):
        fh._check(fh.load_library().fh_op_probe_wait_timeout(torch.cuda.current_stream().cuda_stream))
        torch.cuda.synchronize()
        with pytest.raises(fh.FHError, match="ran out") as e:
            report()
        assert e.value.code == fh.FH_ERR_TIMEOUT
        assert torch.equal(fh.linear_mx(A, W, bias), want)
        fh.sync_operators()


def test_calls_from_several_threads():
    """Threads with streams of their own, at once: checks, allocations and launches share nothing."""
    import threading
    ins = [ff_inputs(s, 200, 384, 1024, "mxfp8") for s in range(41, 45)]
    want = [[t.clone() for t in flat(feed_forward(*i, "mxfp8", BF))] for i in ins]
    torch.cuda.synchronize()
    good = [False] * len(ins)

    def work(k):
        with torch.cuda.stream(torch.cuda.Stream()):
            good[k] = all(torch.equal(a, b) for _ in range(10)
                          for a, b in zip(flat(feed_forward(*ins[k], "mxfp8", BF)), want[k]))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(ins))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(good)


def test_first_call_inside_a_capture():
    """Nothing that the first calls set up is forbidden while a stream captures: a fresh process, whose
    first calls are recorded and replayed."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = (
        "import torch, audio_driven_talking_b200 as fh\n"
        "x = torch.randn(64, 256, device='cuda'); g = torch.ones(256, device='cuda'); torch.cuda.synchronize()\n"
        "def run():\n"
        "    s, h = fh.add_rms_norm(x, x, g)\n"
        "    y = fh.linear_mx(h, h, out='mxfp4')\n"
        "    return [s, h.data, y.data, fh.dequantize(y), fh.quantize(x).data]\n"
        "graph = torch.cuda.CUDAGraph()\n"
        "with torch.cuda.graph(graph): got = run()\n"
        "graph.replay(); torch.cuda.synchronize()\n"
        "assert all(torch.equal(a, b) for a, b in zip(got, run()))\n"
        "print('equal')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "equal" in r.stdout, r.stderr[-2000:]


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two devices")
def test_tensors_of_another_device():
    x = torch.randn(64, 128, device="cuda:1")
    q = fh.quantize(x)
    y = fh.linear_mx(q, q)
    assert q.device.index == 1 and y.get_device() == 1 and torch.cuda.current_device() == 0
    with pytest.raises(ValueError, match="cuda:1"):
        fh.linear_mx(fh.quantize(x.to("cuda:0")), q)
