"""The host code of the log probabilities and of the gradients' norm and clipping under
AddressSanitizer (CPU only): tests/c/host_check_answers.cpp drives their argument checks, the overlaps
of up to 64 ranks' arrays and of thousands of tensors, and their workspace sizes."""

from tests.test_host_asan_rows import run


def test_host_code_is_clean_under_asan():
    res = run("host_check_answers")
    assert res.returncode == 0, res.stdout[-4000:] + res.stderr[-4000:]
    assert "PASSED" in res.stdout
