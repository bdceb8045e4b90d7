"""The page pool, the 4-bit cache and the attention over it as they are used together.

A continuation in a forked, trimmed and compacted pool and the same sequence alone hold
the same codes in other pages: their outputs differ in the order of the attention's sums,
a bf16 rounding or so (2^-8) of the attention's output, which the layer after it passes
on.  A code may then move by one too (a sixteenth of its group's range, in one of the two
layers' caches).  With other tokens' rows or another length they differ by their own size."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prompt,tokens,children", [(77, 6, 3), (16, 3, 1), (5, 2, 12), (301, 4, 7)])
def test_continuations_are_the_sequences_alone(prompt, tokens, children):
    import paged_decode
    assert paged_decode.main(prompt, tokens, children, verbose=False) <= 2.0 ** -5
