"""The example runs, keeps drafted tokens, and its cache equals a single pass's.

The two passes' activations differ by float32 rounding in the linears (at most 1e-3, the linears'
bound; the batch sizes differ) and in attention, which moves a code only where a value lies next to
the border of two codes: a share of at most 1e-3 * 15 / 1 of the values by one step of 1/15 of a
block's range, about 4 standard deviations.  In the 2-norm that is sqrt(0.015) * 4/15 + 1e-3 < 0.04."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_speculative_decoding_example():
    spec = importlib.util.spec_from_file_location("speculative_decode", os.path.join(ROOT, "examples", "speculative_decode.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    said = []
    kept, worst = mod.main(steps=5, say=said.append)
    assert kept > 0 and worst < 0.04 and len(said) == 2
