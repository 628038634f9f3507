"""The host models of csrc/paged_schedule.h find mistakes planted in a copy of
that header (each of which still compiles)."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "async_barrier_pipelined_gb300", "csrc")
MODELS = os.path.join(HERE, "mbarrier_model")
HEADER = open(os.path.join(CSRC, "paged_schedule.h")).read()


def run(tmp_path, model, header):
    """The model's run on a header of this text."""
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    (tmp_path / "paged_schedule.h").write_text(header)
    exe = tmp_path / "model"
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", str(tmp_path), "-I", CSRC,
                    os.path.join(MODELS, model), "-o", str(exe)], check=True)
    return subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)


@pytest.mark.parametrize("model", ["paged_model.cpp", "paged_deal_model.cpp"])
def test_models_hold(tmp_path, model):
    r = run(tmp_path, model, HEADER)
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout + r.stderr


@pytest.mark.parametrize("right,wrong", [
    # lengths
    ("s1 > total_q ||", "s1 > total_q + 1 ||"),
    ("r.len = (int)lmin(lmax(len, 0), room);", "r.len = (int)lmax(len, 0);"),
    # blocks of a tile
    ("s.end = imax(p1 + 1, 0);", "s.end = imax(p1, 0);"),
    ("(int)lmax(0, (int64_t)p0 - m.window + 1)", "(int)lmax(0, (int64_t)p0 - m.window + 2)"),
    ("(m.sinks - 1) / BLOCK_KEYS + 1, s.fb)", "(m.sinks - 1) / BLOCK_KEYS, s.fb)"),
    ("j < s.sblk ? j : s.fb + (j - s.sblk)", "j <= s.sblk ? j : s.fb + (j - s.sblk)"),
    # what is copied, and from where
    ("k0 + rows > s.first || k0 < m.sinks", "k0 + rows > s.first + 1 || k0 < m.sinks"),
    ("k0 + rows > s.first || k0 < m.sinks", "k0 + rows > s.first"),
    ("g.shift = left > 0 && left < rows ? rows - left : 0;", "g.shift = 0;"),
    ("g.shift = left > 0 && left < rows ? rows - left : 0;",
     "g.shift = left > 0 && left < rows ? rows - left - 1 : 0;"),
    # masks
    ("(int64_t)k > (int64_t)p - m.window ||", "(int64_t)k >= (int64_t)p - m.window ||"),
    ("lmax((int64_t)k - pos0, 0) * group", "lmax((int64_t)k - pos0 + 1, 0) * group"),
    ("lmax((int64_t)k - pos0 + m.window, 0) * group", "lmax((int64_t)k - pos0 + m.window - 1, 0) * group"),
    ("imin(imax(p - k0 + 1, 0), BLOCK_KEYS)", "imin(imax(p - k0, 0), BLOCK_KEYS)"),
    ("lmax((int64_t)p - k0 + 1 - m.window, 0)", "lmax((int64_t)p - k0 - m.window, 0)"),
    ("sk = imin(imax(m.sinks - k0, 0), hi);", "sk = 0;"),
    ("const int shift = rows - over;", "const int shift = rows - over - 1;"),
    ("return k1 <= p0 &&", "return k0 <= p0 &&"),
    # shares
    ("(blocks + workers - 1) / workers);\n}\n\n// Where", "blocks / workers);\n}\n\n// Where"),
    ("return 2 * w + ((int64_t)w * per < L ? 1 : 0);", "return 2 * w;"),
    ("(tiles / workers - 1) * workers", "(tiles / workers) * workers"),
    ("return imax(1, level - load);", "return imax(0, level - load);"),
    ("return most_load + (rest + workers - 1) / workers;", "return most_load;"),
    ("imin(before, rest - (workers - c))", "imin(before, rest - (workers - c) + 1)"),
])
def test_a_mistake_in_the_header_is_found(tmp_path, right, wrong):
    assert HEADER.count(right) == 1
    r = run(tmp_path, "paged_model.cpp", HEADER.replace(right, wrong))
    assert r.returncode != 0 and not r.stdout.startswith("ok ")


@pytest.mark.parametrize("right,wrong", [
    ("if (shares(mid) < rest) lo", "if (shares(mid) <= rest) lo"),
    ("if (shares(mid) < rest) lo", "if (shares(mid) < rest - 1) lo"),
    ("while (hi - lo > 1) {", "while (hi - lo > 2) {"),
    ("return hi;\n}\nGF16_HD int deal_start", "return lo;\n}\nGF16_HD int deal_start"),
])
def test_a_mistake_in_the_level_is_found(tmp_path, right, wrong):
    assert HEADER.count(right) == 1
    r = run(tmp_path, "paged_deal_model.cpp", HEADER.replace(right, wrong))
    assert r.returncode != 0 and not r.stdout.startswith("ok ")
