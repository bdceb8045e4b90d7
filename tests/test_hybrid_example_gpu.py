"""The hybrid decode step of the example: every operator in one path.

A sequence decoded in a batch over shared prompt pages and decoded alone over
its own pages differ in the order of the attention's sums only: a bf16
rounding or so of the attention's output (2^-8 of it), which the two blocks
after it pass on.  Without the same keys, positions or states the outputs
differ by their own size."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,prompt,tokens", [(6, 200, 5), (1, 8, 2), (70, 33, 2)])
def test_a_sequence_in_the_batch_is_the_sequence_alone(batch, prompt, tokens):
    import hybrid_decode
    assert hybrid_decode.main(batch, prompt, tokens, verbose=False) <= 2.0 ** -5
