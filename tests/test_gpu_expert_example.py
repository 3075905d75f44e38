"""The expert-layer example runs, and its two ways to the experts' part agree."""
import os
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,experts", [(300, 16), (5, 8), (1500, 64)])
def test_example(tokens, experts):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import expert_layer
    # The way over all experts rounds its sum to bf16, half a step 2^-8 of each value.  The
    # products add the same blocks in the same order, but the few-row kernel (a few tokens of the
    # dense way) adds them in another: a sum next to a rounding border can then round to the other
    # side, and with it one of the 768 gated values' codes, a step of 2^-3 of one term: 2^-3 /
    # sqrt(768) of a token's norm.  Two of those in a single token, and the rounding, stay below
    # 2^-6.
    assert expert_layer.main(["--tokens", str(tokens), "--experts", str(experts)]) <= 2.0 ** -6
