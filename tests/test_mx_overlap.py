"""add_rms_norm's sum over the vectors a and c: other rows' CTAs write it while a row reads them, so the
call is refused, at the first and the last byte that they could share."""
import pytest

import audio_driven_talking_b200 as fh
from audio_driven_talking_b200 import build as fhbuild

torch = pytest.importorskip("torch")

MB = 1 << 20
M, D, STREAMS = 8, 64, 4
SUM = M * D * 4                   # bytes of the float32 sum
VEC = STREAMS * D * 4             # and of the streams' vectors
NORM = dict(x=1 * MB, x_dtype=0, res=2 * MB, res_dtype=1, sum=3 * MB, a=4 * MB, c=5 * MB, bstride=D, rows=M // STREAMS, M=M, D=D,
            eps=1e-6, out_type=2, out=6 * MB, scales=7 * MB, stream=None)


@pytest.mark.parametrize("vector", ["a", "c"])
@pytest.mark.parametrize("at", [0, SUM - 16, 16 - VEC])
def test_sum_over_a_vector_is_refused(vector, at):
    fhbuild.build()
    lib = fh.load_library()
    assert lib.fh_op_add_rms_norm(*{**NORM, vector: NORM["sum"] + at}.values()) == fh.FH_ERR_ARG
    assert "a or c" in lib.fh_last_error().decode()


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")
def test_sum_beside_the_vectors():
    """A sum that ends where the vectors begin is taken, one that holds them is not."""
    room = torch.randn(2 * M, D, device="cuda")
    x, a = room[:M], room[M:M + STREAMS]
    res = torch.randn(M, D, device="cuda")
    want = fh.add_rms_norm(x.clone(), res, a.clone(), out=torch.float32)
    for bad in (lambda: fh.add_rms_norm(x, res, x[0], sum_out=x), lambda: fh.add_rms_norm(x, res, a, x[:STREAMS], sum_out=x),
                lambda: fh.add_rms_norm(res, res, a, sum_out=room[STREAMS:STREAMS + M])):
        with pytest.raises(fh.FHError, match="a or c"):
            bad()
    total, y = fh.add_rms_norm(x, res, a, out=torch.float32, sum_out=x)
    assert total is x and torch.equal(total, want[0]) and torch.equal(y, want[1])
