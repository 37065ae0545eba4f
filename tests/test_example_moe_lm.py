"""The example runs the quantizers, grouped GEMMs, activation checkpoints, the loss
and the few-token layer together: it learns, and generation agrees with the
training pass."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_example_trains_and_generates():
    print("case: example moe_lm", flush=True)
    spec = importlib.util.spec_from_file_location("moe_lm", os.path.join(ROOT, "examples", "moe_lm.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    first, last, off, _ = m.main(steps=20)
    assert last < 0.7 * first, (first, last)
    # the training pass quantizes its activations to 4 bits (E1M2: up to half a
    # step of 1/7 of a block's largest, some 10 % of a typical element, twice
    # in a row), generation does not
    assert off < 0.35, off
