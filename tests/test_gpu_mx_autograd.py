"""The microscaled operators beside autograd: they give no gradients, and must not corrupt others'."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

import audio_driven_talking_b200 as fh  # noqa: E402


def rows(seed, *shape):
    return torch.randn(shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))


@pytest.mark.parametrize("target", ["x", "res", "view"])
def test_sum_out_over_a_saved_tensor_is_seen_by_its_backward(target):
    """w * t saves t for w's gradient; a sum written into t makes that gradient wrong, so it has to raise."""
    x, res, g = rows(1, 6, 64), rows(2, 6, 64), rows(3, 64)
    t = res if target == "res" else x
    w = torch.ones(6, 64, device="cuda", requires_grad=True)
    y = (w * t).sum()
    before = t._version
    fh.add_rms_norm(x, res, g, sum_out=x.view(6, 64) if target == "view" else t)
    assert t._version == before + 1
    with pytest.raises(RuntimeError, match="inplace operation"):
        y.backward()


def test_a_sum_of_its_own_leaves_the_inputs_as_they_were():
    x, res, g = rows(1, 6, 64), rows(2, 6, 64), rows(3, 64)
    w = torch.ones(6, 64, device="cuda", requires_grad=True)
    y = (w * x).sum()
    fh.add_rms_norm(x, res, g, sum_out=torch.empty_like(x))
    fh.add_rms_norm(x, res, g)
    y.backward()
    assert torch.equal(w.grad, x)


def test_inference_tensors():
    """Read anywhere, written in inference mode only, as torch has it."""
    with torch.inference_mode():
        x, res, g = rows(1, 6, 64), rows(2, 6, 64), rows(3, 64)
        want = x + res
        total, _ = fh.add_rms_norm(x, res, g, sum_out=x)
        assert total is x and torch.equal(x, want)
        plain = rows(1, 6, 64)
    with pytest.raises(ValueError, match="inference"):
        fh.add_rms_norm(plain, res, g, sum_out=plain)
    assert torch.equal(fh.add_rms_norm(plain, res, g)[0], want)
