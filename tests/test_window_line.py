"""The division of windowed attention's work, compiled for the host (tests/window_line.cu) and run on random
batches: one sequence to forty, contexts of one key to 2^31 - 4096, one worker to 1300, groups above a tile, windows
and sinks of any size, lengths that break a constraint."""
import os
import re
import subprocess

import pytest

from paged_kv_cache_206_gb300 import build_lib

SOURCE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "window_line.cu")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("line") / "window_line")
    r = subprocess.run([build_lib.nvcc(), "-std=c++17", "-O1", *build_lib.ARCH, "--expt-relaxed-constexpr",
                        f"-I{build_lib.INCLUDE}", f"-I{build_lib.CSRC}", SOURCE, "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    return exe


@pytest.mark.parametrize("seed", range(4))
def test_every_unit_is_some_workers_once(program, seed):
    r = subprocess.run([program, str(seed), "120"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    batches, tiles, divided = map(int, re.findall(r"\d+", r.stdout))
    assert batches == 840 and tiles > 10000 and divided > 1000
