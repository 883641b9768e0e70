"""The microscaled operators give no gradients: a call whose result autograd would take for a constant
without a word is refused, and passes where gradients are off or the tensor is detached."""
import pytest

torch = pytest.importorskip("torch")

import audio_driven_talking_b200 as fh  # noqa: E402
from audio_driven_talking_b200 import build as fhbuild  # noqa: E402

M, K = 4, 64


def calls(device):
    """name: (a tensor of the call, the call)."""
    x, g = torch.ones(M, K, device=device), torch.ones(K, device=device)
    q = fh.MXTensor(torch.zeros(M, K, dtype=torch.uint8, device=device), torch.zeros(512, dtype=torch.uint8, device=device),
                    (M, K), "mxfp8")
    return {"quantize": (x, lambda t: fh.quantize(t)),
            "norm x": (x, lambda t: fh.add_rms_norm(t, x, g)),
            "norm res": (x, lambda t: fh.add_rms_norm(x, t, g)),
            "norm a": (g, lambda t: fh.add_rms_norm(x, x, t)),
            "norm c": (g, lambda t: fh.add_rms_norm(x, x, g, t)),
            "norm sum_out": (x, lambda t: fh.add_rms_norm(x, x, g, sum_out=t)),
            "linear bias": (g[:M], lambda t: fh.linear_mx(q, q, t))}


NAMES = ["quantize", "norm x", "norm res", "norm a", "norm c", "norm sum_out", "linear bias"]


def check_refusals(name, device):
    t, call = calls(device)[name]
    leaf = t.clone().requires_grad_()
    for bad in (leaf, leaf * 2):
        with pytest.raises(ValueError, match="gradient"):
            call(bad)
    with torch.autograd.forward_ad.dual_level():
        with pytest.raises(ValueError, match="gradient"):
            call(torch.autograd.forward_ad.make_dual(t.clone(), t.clone()))


@pytest.mark.parametrize("name", NAMES)
def test_refused(name):
    """On the CPU, with tensors that only claim to be on a device."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    fhbuild.build()
    with FakeTensorMode():
        check_refusals(name, "cuda:0")


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")
@pytest.mark.parametrize("name", NAMES)
def test_taken_without_gradients(name):
    check_refusals(name, "cuda:0")
    t, call = calls("cuda:0")[name]
    leaf = t.clone().requires_grad_()
    flat = lambda r: [p for v in (r if isinstance(r, tuple) else (r,))  # noqa: E731
                      for p in ((v.data, v.scales) if isinstance(v, fh.MXTensor) else (v,))]
    want = flat(call(t.clone()))
    with torch.no_grad():
        off = flat(call(leaf.clone().requires_grad_()))
    for got in (off, flat(call(leaf.detach()))):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
