"""The operator benchmark's microscaled entries, on the CPU: parsing and the byte counts."""
import pytest

import audio_driven_talking_b200.opbench as ob


@pytest.mark.parametrize("op", ["quantize", "add_rms_norm", "linear_mx"])
def test_microscaled_operators_are_accepted(op):
    a = ob.parser().parse_args([op, "--format", "mxfp4", "--out", "mxfp8"])
    assert (a.op, a.format, a.out, a.act) == (op, "mxfp4", "mxfp8", None)
    assert ob.parser().parse_args([op, "--act", "gelu"]).act == "gelu"
    with pytest.raises(SystemExit):
        ob.parser().parse_args([op, "--format", "fp8"])


def test_bytes_of_each_kind():
    assert [ob._mx_bytes(4, 64, k) for k in ("f32", "bf16", "mxfp8", "mxfp4")] == [1024, 512, 264, 136]
