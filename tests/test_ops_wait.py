"""The limit of the product's waits: two seconds in which the warp ran, however
long the process was suspended in between."""
import subprocess
from pathlib import Path

import pytest

from gpu_util import dev  # noqa: F401
from weight_communication_gb300 import build

HERE = Path(__file__).resolve().parent


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = tmp_path_factory.mktemp("wait") / "wait_limit"
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-O2", str(HERE / "wait_limit.cu"), "-o", str(exe)],
                   check=True, capture_output=True)
    return exe


def results(exe, what):
    run = subprocess.run([str(exe), what], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, (run.returncode, run.stdout, run.stderr)
    return {k: int(v) for k, v in (line.split() for line in run.stdout.splitlines())}


def test_limit_counts_the_time_that_ran(program):
    """Looks 1 us apart: two seconds of them with or without the clock's wrap;
    a suspension counts for no more than 10 ms."""
    got = results(program, "host")
    assert got["steady"] == got["wrapping"] == 2_000_000_000
    for name in ("suspended_1h", "suspended_2s"):
        assert 1_990_000_000 <= got[name] <= 2_000_000_000, name


@pytest.mark.gpu
def test_a_wait_that_nothing_answers_ends(dev, program):  # noqa: F811
    got = results(program, "gpu")
    assert got["answered"] == 1 and got["lost"] == 1 and got["count"] == 1
    # no try between two looks may be cut off by the 10 ms that a gap counts for
    assert 1_990_000_000 <= got["ns"] <= 3_000_000_000
