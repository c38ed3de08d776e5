"""Workspaces are cleared in the order of the stream that uses them (CPU only):
tests/c/host_check_streams.cpp puts its own account of streams, allocations and launches in the
place of the HIP runtime's calls and runs the all-reduce calls that allocate, grow, renew and reset
workspaces; build() compiles it, with AddressSanitizer on the library's host code."""

from tests.test_host_asan_rows import run


def test_workspaces_are_cleared_in_stream_order():
    res = run("host_check_streams")
    assert res.returncode == 0, res.stdout[-4000:] + res.stderr[-4000:]
    assert "PASSED" in res.stdout
