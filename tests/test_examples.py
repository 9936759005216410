"""The examples run, and what they compute is right."""

import importlib.util
import os

import pytest

from quantized_weight_linear_amd import nq

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("fmt", [nq.NQ_KV_BF16, nq.NQ_KV_E4M3])
def test_speculative_steps(fmt):
    spec = importlib.util.spec_from_file_location("speculative_steps", os.path.join(ROOT, "examples", "speculative_steps.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    worst, used, left = example.main(fmt)
    # BF16 outputs: half a unit in the last place of 8 bits, at most 2^-9, for the output and again for the weights
    # that the values are multiplied with, and as much again for all else.
    assert worst <= 3 * 2.0 ** -9
    # 303, 50, 302 and 307 tokens in pages of 64: the first's 4 whole pages are the third's and fourth's too, each of
    # the three has a fifth page of its own, and the second has one page.
    assert (used, left) == (4 + 3 + 1, 0)
