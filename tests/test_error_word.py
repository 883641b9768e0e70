"""The operators' error word when several threads ask for it: what was latched once is reported once."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "audio_driven_talking_b200", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_one_of_several_threads_is_told(tmp_path):
    exe = str(tmp_path / "race")
    subprocess.run(["g++", "-O2", "-std=c++20", "-pthread", "-I", CSRC, os.path.join(HERE, "error_word_race.cpp"), "-o", exe],
                   check=True, capture_output=True, timeout=120)
    r = subprocess.run([exe, "50000", "4"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == ["50000", "0", "0"]


@pytest.mark.gpu
def test_one_of_several_threads_is_told_of_a_wait_that_ran_out():
    """A bounded wait with no arriving party runs out (about a second); four threads ask at once, and one
    call after another works again."""
    import threading

    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import audio_driven_talking_b200 as fh

    q = fh.quantize(torch.randn(40, 64, device="cuda"))
    want = fh.linear_mx(q, q)
    fh._check(fh.load_library().fh_op_probe_wait_timeout(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    told, start = [], threading.Barrier(4)

    def ask():
        start.wait()
        try:
            fh.linear_mx(q, q)
        except fh.FHError as e:
            told.append(e.code)

    threads = [threading.Thread(target=ask) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert told == [fh.FH_ERR_TIMEOUT]
    assert torch.equal(fh.linear_mx(q, q), want)
