"""The rule that picks linear_mx's tile form, on the CPU: the shapes of the GPU's tests reach every form,
in both formats."""
import ctypes

import pytest

import audio_driven_talking_b200 as fh
from audio_driven_talking_b200 import build as fhbuild
from mx_shapes import BY_FORM

SMS = 148


class Tile(ctypes.Structure):
    _fields_ = [("bn", ctypes.c_int), ("pair", ctypes.c_bool), ("split", ctypes.c_int)]


@pytest.fixture(scope="module")
def rule():
    fhbuild.build()
    fn = getattr(fh.load_library(), "_ZN2fh12gemm_mx_tileEiiiii")  # fh::gemm_mx_tile(M, N, K, fmt, sms)
    fn.restype, fn.argtypes = Tile, [ctypes.c_int] * 5
    return lambda M, N, K, fmt: (lambda t: (t.bn, t.pair, t.split))(fn(M, N, K, fmt, SMS))


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("form", BY_FORM)
def test_shapes_reach_their_form(rule, form, fmt):
    for shape in BY_FORM[form]:
        assert rule(*shape, fmt) == form, shape


@pytest.mark.parametrize("fmt", [0, 1])
def test_forms_that_need_two_row_tiles_or_several_stages_have_them(rule, fmt):
    import random
    rng = random.Random(7)
    for _ in range(5000):
        M, N, K = (int(2 ** rng.uniform(0, top)) for top in (15, 14, 9))
        bn, pair, split = rule(M, N, 32 * K, fmt)
        assert (bn, pair, split) in BY_FORM
        assert not pair or M > 128
        assert split <= -(-32 * K // (256 if fmt else 128))
