"""The serving example (examples/paged_serving.py) against the same layers in
FP32 without a cache."""
from __future__ import annotations

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "paged_serving.py")


def test_serving_example_matches_the_plain_form():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from async_barrier_pipelined_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("paged_serving", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    # Two layers of about ten binary16 roundings each on the way of a number,
    # each at most 2^-11 of it; independent, so their root-sum-square with a
    # factor of 2 for the residual's growth: 2 * sqrt(20) * 2^-11 = 4.4e-3.
    assert m.main(["--steps", "24"]) < 4.4e-3
