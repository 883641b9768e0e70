"""linear_mx on sums that float32 holds exactly, and by its norm-wise error, in every tile form.

Exact: elements are the integers -4 .. 4 and scales 1/2, 1, 2, different everywhere, so products are
multiples of 1/4 and at most 64. A sum of them, in any order and with any of its additions cut off instead
of rounded, is exact while sum |A| |W| + |bias| < 2^24 / 4, which each case checks. So a float32 result has
to be the sum bit for bit, and a bf16 or microscaled one its rounding.

Norm-wise: the tensor core adds K / 32 blocks of 32 products (mxfp4: K / 64 of 64) to the running sum; an
addition that cuts off loses less than a step 2u of it, u = 2^-24, and the running sums' norm over all results
does not pass that of the final ones, whose terms are independent. Inside a block at most 64 more steps of
values that are smaller still. So ||error|| <= 2u (K / 32 + 64) ||y||, which at K = 8960 is 4e-5 of the norm,
where a block of 32 left out would be 6e-2."""
import numpy as np
import pytest

import mx_reference as mx
from mx_shapes import SHAPES

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

import audio_driven_talking_b200 as fh  # noqa: E402

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
FMTS = ["mxfp8", "mxfp4"]


def generator(seed):
    return torch.Generator("cuda").manual_seed(seed)


def operand(seed, rows, K, fmt):
    """(MXTensor, its values in 64 bits) of integers -4 .. 4 under scales 1/2, 1, 2."""
    g = generator(seed)
    v = torch.randint(-4, 5, (rows, K), device="cuda", generator=g)
    if fmt == "mxfp8":
        data = v.to(F32).to(torch.float8_e4m3fn).view(torch.uint8)
    else:                                           # 0, 1, 2, 3, 4 are the e2m1 codes 0, 2, 4, 5, 6
        code = torch.tensor([0, 2, 4, 5, 6], device="cuda")[v.abs()] + 8 * (v < 0)
        data = (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8)
    byte = torch.randint(126, 129, (rows, K // 32), device="cuda", generator=g)
    flat = torch.from_numpy(mx.tile(byte.cpu().numpy().astype(np.uint8), K)).cuda()
    values = v.double().view(rows, K // 32, 32) * torch.exp2(byte.double() - 127)[..., None]
    return fh.MXTensor(data, flat, (rows, K), fmt), values.view(rows, K)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_exact_sums(M, N, K, fmt):
    A, a = operand(M + K, M, K, fmt)
    W, w = operand(N + K + 1, N, K, fmt)
    bias = torch.randint(-100, 101, (N,), device="cuda", generator=generator(N)).to(F32)
    y = a @ w.t() + bias.double()
    assert float((a.abs() @ w.abs().t()).max()) + 100 < 2.0 ** 22
    assert torch.equal(fh.linear_mx(A, W, bias, out=F32).double(), y)
    assert torch.equal(fh.linear_mx(A, W, bias), y.to(F32).to(BF))
    assert torch.equal(fh.linear_mx(A, W, out=F32).double(), y - bias.double())
    if N % 32 == 0 and M * N <= 1 << 21:
        for out in FMTS:
            el, byte, flat = mx.read(fh.linear_mx(A, W, bias, out=out))
            want = mx.quantize(y.cpu().numpy(), out)
            assert np.array_equal(el, want[0]) and np.array_equal(byte, want[1]) and not mx.padding(flat, M, N).any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_norm_wise_error(M, N, K, fmt):
    g = generator(M + N + K)
    A = fh.quantize(torch.randn(M, K, device="cuda", generator=g) * torch.exp(0.5 * torch.randn(K, device="cuda", generator=g)), fmt)
    W = fh.quantize(torch.randn(N, K, device="cuda", generator=g) / K ** 0.5, fmt)
    y = fh.dequantize(A).double() @ fh.dequantize(W).double().t()
    error = fh.linear_mx(A, W, out=F32).double() - y
    assert float(error.norm() / y.norm()) <= 2 * U * (K / 32 + 64)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(2148, 2289, 64), (2148, 2304, 64), (1078, 4872, 768), (5643, 8610, 96), (2304, 2304, 96)])
def test_tiles_of_192_columns_with_gelu(M, N, K, fmt):
    """Bias, GELU and every result type, on ragged edges; the bounds are those of the other forms: 2u (K + 8) of
    sum |A| |W| + |bias| for the sum, times 1.13 and 16 u more for GELU."""
    g = generator(M + N + K)
    A = fh.quantize(torch.randn(M, K, device="cuda", generator=g), fmt)
    W = fh.quantize(torch.randn(N, K, device="cuda", generator=g) / K ** 0.5, fmt)
    bias = 0.5 * torch.randn(N, device="cuda", generator=g)
    a, w = fh.dequantize(A).double(), fh.dequantize(W).double()
    y = a @ w.t() + bias.double()
    tol = 2 * U * (K + 8) * (a.abs() @ w.abs().t() + bias.double().abs())
    z = 0.5 * y * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (y + 0.044715 * y ** 3)))
    ztol = 1.13 * tol + 16 * U * z.abs()
    for out, half in ((F32, 0.0), (BF, 2.0 ** -8)):
        got = fh.linear_mx(A, W, bias, act="gelu", out=out).double()
        assert (got - z).abs().le(half * z.abs() + (1 + half) * ztol).all()
    if N % 32 == 0:
        for out in FMTS:
            mx.check_result(fh.linear_mx(A, W, bias, act="gelu", out=out), z.cpu().numpy(), ztol.cpu().numpy())
