"""Operators whose tensor maps need a context bound to the calling thread, as the first CUDA call of a
thread: launches bind the device's context, but the maps are encoded before the launch."""
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

import audio_driven_talking_b200 as fh  # noqa: E402

BF = torch.bfloat16


def rows(seed, *shape, dtype=torch.float32):
    return torch.randn(shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).to(dtype)


def linear_mx():
    q = fh.quantize(rows(1, 200, 256))
    return lambda: fh.linear_mx(q, q)


def linear():
    A, W, b = rows(1, 256, 256, dtype=BF), rows(2, 256, 256, dtype=BF), rows(3, 256)
    return lambda: fh.linear(A, W, b)


def attention():
    q, k = (rows(s, 1, 2, 128, 128, dtype=BF) for s in (1, 2))
    v, ssq = rows(3, 1, 2, 128, 128, dtype=torch.float16), torch.ones(128, 4, device="cuda") * 128
    return lambda: fh.attention(q, k, v, ssq)


@pytest.mark.parametrize("operator", [linear_mx, linear, attention])
def test_first_cuda_call_of_a_thread(operator):
    call = operator()
    want = call()                 # torch keeps the result's memory, so that the thread's call allocates none
    again = [call() for _ in range(2)]
    del again
    torch.cuda.synchronize()
    got = []

    def work():
        try:
            got.append(call())
        except fh.FHError as e:
            got.append(e)

    for _ in range(2):
        t = threading.Thread(target=work)
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert not [e for e in got if isinstance(e, fh.FHError)]
    assert len(got) == 2 and all(torch.equal(r, want) for r in got)
