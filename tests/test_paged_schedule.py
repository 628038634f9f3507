"""The integer arithmetic behind the attention over a paged cache
(csrc/paged_schedule.h) against plain loops over every key, on the host: the
clamping of lengths, the blocks and rows that copies touch, the masks, and
the dealing out of blocks and whole tiles to workers (mbarrier_model/paged_model.cpp).  A
planted mistake in the model must make it fail."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "mbarrier_model", "paged_model.cpp")
CSRC = os.path.join(os.path.dirname(HERE), "async_barrier_pipelined_gb300", "csrc")


def run(tmp_path, text):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    src, exe = tmp_path / "model.cpp", tmp_path / "model"
    src.write_text(text)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined",
                    "-fno-sanitize-recover=undefined", "-I", CSRC, str(src), "-o", str(exe)],
                   check=True)
    return subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)


def test_schedule_holds(tmp_path):
    r = run(tmp_path, open(SRC).read())
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout + r.stderr


@pytest.mark.parametrize("right,wrong", [
    ("any |= sees(r.len - r.n + t, k, m);\n    CHECK", "any |= sees(r.len - r.n + t + 1, k, m);\n    CHECK"),
    ("CHECK(done == nb);", "CHECK(done == nb + 1);"),
    ("load[c] + share <= std::max(hi, most + 1)", "load[c] + share < std::min(hi, most + 1)"),
    ("if (shares(mid) < rest) lo", "if (shares(mid) < rest - workers - 9) lo"),
    ("v = sees(r.len - r.n + t, k, m);\n            any", "v = sees(r.len - r.n + t - 1, k, m);\n            any"),
])
def test_a_planted_mistake_is_found(tmp_path, right, wrong):
    text = open(SRC).read()
    assert right in text
    r = run(tmp_path, text.replace(right, wrong))
    assert r.returncode != 0 and not r.stdout.startswith("ok ")
