"""Refused calls of the microscaled operators, on the CPU: the C entry points check their
arguments before any device work, the binding before it calls them. And the oracle's own
number format against its definition, element by element."""
import ctypes

import numpy as np
import pytest

import audio_driven_talking_b200 as fh
import mx_reference as mx
from audio_driven_talking_b200 import build as fhbuild

torch = pytest.importorskip("torch")

P = 1 << 20      # an aligned address that is never read
FAR = 1 << 40


@pytest.fixture(scope="module")
def lib():
    fhbuild.build()
    return fh.load_library()


@pytest.mark.parametrize("M,K", [(1, 32), (128, 128), (129, 160), (777, 1568)])
def test_sizes(lib, M, K):
    assert lib.fh_mx_data_bytes(M, K, fh.FH_MXFP8) == M * K
    assert lib.fh_mx_data_bytes(M, K, fh.FH_MXFP4) == M * K // 2
    assert lib.fh_mx_scale_bytes(M, K) == mx.scale_count(M, K) == fh.MXTensor.scale_bytes(M, K)
    off = mx.offsets(M, K)
    assert len(np.unique(off)) == off.size and off.max() < mx.scale_count(M, K)


def test_sizes_that_do_not_exist(lib):
    assert lib.fh_mx_data_bytes(4, 33, fh.FH_MXFP8) == 0
    assert lib.fh_mx_data_bytes(4, 32, fh.FH_BF16) == 0
    assert lib.fh_mx_scale_bytes(0, 32) == 0
    assert lib.fh_mx_scale_bytes(1, (1 << 20) + 32) == 0


QUANT = dict(x=P, ldx=64, M=2, K=64, dtype=fh.FH_F32, mxtype=fh.FH_MXFP8, data=P, scales=P, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(x=None), fh.FH_ERR_ARG), (dict(x=P + 4), fh.FH_ERR_ARG), (dict(data=P + 8), fh.FH_ERR_ARG),
    (dict(scales=None), fh.FH_ERR_ARG), (dict(dtype=fh.FH_MXFP8), fh.FH_ERR_ARG), (dict(mxtype=fh.FH_BF16), fh.FH_ERR_ARG),
    (dict(M=0), fh.FH_ERR_SHAPE), (dict(K=48), fh.FH_ERR_SHAPE), (dict(K=0), fh.FH_ERR_SHAPE), (dict(ldx=32), fh.FH_ERR_SHAPE),
    (dict(ldx=66), fh.FH_ERR_SHAPE), (dict(ldx=68, dtype=fh.FH_BF16), fh.FH_ERR_SHAPE)])
def test_quantize_refuses(lib, change, code):
    assert lib.fh_op_quantize(*{**QUANT, **change}.values()) == code


DEQUANT = dict(data=P, scales=P, M=2, K=64, mxtype=fh.FH_MXFP4, out=P, dtype=fh.FH_F32, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(data=None), fh.FH_ERR_ARG), (dict(out=P + 2), fh.FH_ERR_ARG), (dict(mxtype=0), fh.FH_ERR_ARG),
    (dict(dtype=3), fh.FH_ERR_ARG), (dict(K=31), fh.FH_ERR_SHAPE), (dict(M=-1), fh.FH_ERR_SHAPE)])
def test_dequantize_refuses(lib, change, code):
    assert lib.fh_op_dequantize(*{**DEQUANT, **change}.values()) == code


NORM = dict(x=P, x_dtype=0, res=FAR, res_dtype=1, sum=P, a=P, c=P, bstride=0, rows=4, M=4, D=64, eps=1e-6, out_type=2, out=P,
            scales=P, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(x=None), fh.FH_ERR_ARG), (dict(a=None), fh.FH_ERR_ARG), (dict(c=P + 4), fh.FH_ERR_ARG), (dict(x_dtype=2), fh.FH_ERR_ARG),
    (dict(out_type=4), fh.FH_ERR_ARG), (dict(scales=None), fh.FH_ERR_ARG), (dict(out_type=0), fh.FH_ERR_ARG),
    (dict(eps=-1.0), fh.FH_ERR_ARG), (dict(eps=float("nan")), fh.FH_ERR_ARG), (dict(D=80), fh.FH_ERR_SHAPE),
    (dict(D=16384 + 32), fh.FH_ERR_SHAPE), (dict(M=0), fh.FH_ERR_SHAPE), (dict(rows=0), fh.FH_ERR_SHAPE),
    (dict(bstride=-4), fh.FH_ERR_SHAPE), (dict(bstride=2), fh.FH_ERR_SHAPE),
    (dict(sum=P + 16), fh.FH_ERR_ARG),                      # partly over x
    (dict(sum=FAR), fh.FH_ERR_ARG),                         # over res, which has another type
    (dict(sum=FAR + 64, res_dtype=0), fh.FH_ERR_ARG)])      # partly over res
def test_add_rms_norm_refuses(lib, change, code):
    assert lib.fh_op_add_rms_norm(*{**NORM, **change}.values()) == code


LINEAR = dict(A=P, sA=P, W=P, sW=P, bias=P, M=4, N=64, K=64, mxtype=2, act=0, out_type=1, out=P, scales=None, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(A=None), fh.FH_ERR_ARG), (dict(sW=P + 8), fh.FH_ERR_ARG), (dict(bias=P + 4), fh.FH_ERR_ARG),
    (dict(mxtype=1), fh.FH_ERR_ARG), (dict(act=2), fh.FH_ERR_ARG), (dict(out_type=-1), fh.FH_ERR_ARG),
    (dict(scales=P), fh.FH_ERR_ARG), (dict(out_type=3), fh.FH_ERR_ARG), (dict(out=None), fh.FH_ERR_ARG),
    (dict(K=40), fh.FH_ERR_SHAPE), (dict(N=0), fh.FH_ERR_SHAPE), (dict(M=0), fh.FH_ERR_SHAPE),
    (dict(N=(1 << 20) + 1), fh.FH_ERR_SHAPE), (dict(N=40, out_type=2, scales=P), fh.FH_ERR_SHAPE)])
def test_linear_mx_refuses(lib, change, code):
    assert lib.fh_op_linear_mx(*{**LINEAR, **change}.values()) == code


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(4, 64)
    q = fh.MXTensor.empty(4, 64, "mxfp8", "cpu")
    assert q.data.shape == (4, 64) and q.scales.numel() == 512 and "mxfp8" in repr(q)
    with pytest.raises(ValueError, match="CUDA"):
        fh.quantize(x)
    with pytest.raises(ValueError, match="format"):
        fh.quantize(x, "fp8")
    with pytest.raises(TypeError):
        fh.quantize(x.numpy())
    with pytest.raises(ValueError, match="CUDA"):
        fh.dequantize(q)
    with pytest.raises(TypeError):
        fh.dequantize(x)
    with pytest.raises(ValueError, match="CUDA"):
        fh.add_rms_norm(x, x, torch.ones(64))
    with pytest.raises(ValueError, match="out="):
        fh.add_rms_norm(x, x, torch.ones(64), out="fp8")
    with pytest.raises(ValueError, match="out="):
        fh.add_rms_norm(x, x, torch.ones(64), out=torch.float16)
    with pytest.raises(TypeError):
        fh.linear_mx(x, q)
    with pytest.raises(ValueError, match="act="):
        fh.linear_mx(q, q, act="relu")
    with pytest.raises(ValueError, match="microscaled shape"):
        fh.dequantize(fh.MXTensor(q.data, q.scales, (4, 48), "mxfp8"))


def test_reference_elements():
    """The 64-bit reference's tables: largest values, neighbours, ties to the even code."""
    assert np.nanmax(mx.element_table("mxfp8")) == 448.0 and mx.element_table("mxfp8")[1] == 2.0 ** -9
    assert mx.round_element(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0, 6.0]), "mxfp4").tolist() == [
        0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, -4.0, 6.0]
    assert mx.round_element(np.array([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 432.0]), "mxfp8").tolist() == [
        16.0, 20.0, 0.0, 2.0 ** -8, 448.0]
    assert mx.scale_exponent(np.array([448.0, np.nextafter(448.0, 500), 0.0, 2.0 ** -140]), "mxfp8").tolist() == [0, 1, -127, -127]
    assert mx.scale_exponent(np.array([6.0, 6.1, 3.0, 1.5]), "mxfp4").tolist() == [0, 1, -1, -2]
