"""The row operators' host code under AddressSanitizer (CPU only).

tests/c/host_check_rows.cpp drives their argument checks, the overlaps of up to 196
arrays in a call, and their workspace sizes, against a copy of ra_rows_api.cpp built
with the sanitizer (build() compiles it).  Any heap or stack misuse aborts it."""

import os
import subprocess

from ring_all_reduce_schedule_amd import build
from tests.conftest import ROOT


def run(name):
    path = os.path.join(ROOT, "tests", "c", name)
    assert os.path.exists(path), f"tests/c/{name} is missing: run build() first"
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1")
    return subprocess.run([path], capture_output=True, text=True, timeout=300, env=env)


def test_row_operators_host_code_is_clean_under_asan():
    res = run("host_check_rows")
    assert res.returncode == 0, res.stdout[-4000:] + res.stderr[-4000:]
    assert "PASSED" in res.stdout


def test_every_host_source_is_built_with_the_sanitizer():
    """Each .cpp of the library is compiled with it, and its plain object is not linked."""
    objs = [os.path.join(build.BUILD, os.path.splitext(s)[0] + ".o") for s in build.SOURCES]
    commands = build.host_check_commands(objs)
    host = [s for s in build.SOURCES if s.endswith(".cpp")]
    assert len(host) >= 2
    for src in host:
        made = [c for c in commands if "-fsanitize=address" in c and any(a.endswith(os.sep + src) for a in c)]
        assert len(made) == 1, src
        plain = os.path.join(build.BUILD, os.path.splitext(src)[0] + ".o")
        links = [c for c in commands if "-lamdhip64" in c]
        assert len(links) == 2
        for link in links:
            assert plain not in link and made[0][made[0].index("-o") + 1] in link, src
