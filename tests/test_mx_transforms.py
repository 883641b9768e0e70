"""The microscaled operators under torch's transforms: a tensor that wraps another one has no memory
of its own and is refused with an ordinary error, for each operand and in each transform."""
import pytest

torch = pytest.importorskip("torch")

import audio_driven_talking_b200 as fh  # noqa: E402
from audio_driven_talking_b200 import build as fhbuild  # noqa: E402

M, K = 4, 64


def operands(device):
    """x, gain, and an MXTensor, of one shape each."""
    q = fh.MXTensor(torch.zeros(M, K, dtype=torch.uint8, device=device), torch.zeros(512, dtype=torch.uint8, device=device),
                    (M, K), "mxfp8")
    return torch.zeros(M, K, device=device), torch.ones(K, device=device), q


def calls(device):
    """name: (the tensor that gets wrapped, the call on what wraps it)."""
    x, g, q = operands(device)
    codes = lambda t: fh.MXTensor(t, q.scales, q.shape, q.fmt)  # noqa: E731
    scales = lambda t: fh.MXTensor(q.data, t, q.shape, q.fmt)  # noqa: E731
    return {
        "quantize": (x, lambda t: fh.quantize(t)),
        "dequantize": (q.data, lambda t: fh.dequantize(codes(t))),
        "dequantize scales": (q.scales, lambda t: fh.dequantize(scales(t))),
        "norm x": (x, lambda t: fh.add_rms_norm(t, x, g)),
        "norm res": (x, lambda t: fh.add_rms_norm(x, t, g)),
        "norm a": (g, lambda t: fh.add_rms_norm(x, x, t)),
        "norm c": (g, lambda t: fh.add_rms_norm(x, x, g, t)),
        "norm sum_out": (x, lambda t: fh.add_rms_norm(x, x, g, sum_out=t)),
        "linear A": (q.data, lambda t: fh.linear_mx(codes(t), q)),
        "linear W scales": (q.scales, lambda t: fh.linear_mx(q, scales(t))),
        "linear bias": (g[:M], lambda t: fh.linear_mx(q, q, t)),
    }


NAMES = ["quantize", "dequantize", "dequantize scales", "norm x", "norm res", "norm a", "norm c", "norm sum_out", "linear A",
         "linear W scales", "linear bias"]


def under_vmap(call, t):
    torch.vmap(lambda r: (call(r), r)[1])(t.unsqueeze(0))


def under_grad(call, t):
    torch.func.grad(lambda r: (call(r), r.sum())[1])(t)


def under_jvp(call, t):
    torch.func.jvp(lambda r: (call(r), r)[1], (t,), (t.clone(),))


def check(name, device):
    t, call = calls(device)[name]
    transforms = [under_vmap] + ([under_grad, under_jvp] if t.is_floating_point() else [])
    for transform in transforms:
        with pytest.raises(ValueError, match="no storage"):
            transform(call, t)


@pytest.mark.parametrize("name", NAMES)
def test_wrapped_tensors_are_refused(name):
    """On the CPU, with tensors that only claim to be on a device: nothing of the call gets that far."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    fhbuild.build()
    with FakeTensorMode():
        check(name, "cuda:0")


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")
@pytest.mark.parametrize("name", NAMES)
def test_wrapped_tensors_are_refused_on_the_gpu(name):
    check(name, "cuda:0")
    x, _, _ = operands("cuda:0")
    assert not fh.dequantize(fh.quantize(x)).any()         # the calls after it work
