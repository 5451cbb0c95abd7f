"""The example that runs the full-attention operators together (examples/hybrid_block.py): the same
tokens as whole prompts, as prompts in two parts, and as steps.

The ways differ in roundings: attention's p to bf16 (2^-8 of each term), the cache's values to bf16
where they are read back (2^-8; the steps take them as they are), the delta rule's prompt path
(held elsewhere to 5e-3 of its outputs), and what an 8-bit rounding behind them may turn into a
step of e4m3 (2^-4) where a value lies near the middle between two: the outputs of one layer are
held to 3e-2 as a whole, as those of recurrent_block.py.

Through both layers the steps' keys and values differ from the prompts' by what the recurrent layer
does, d of their size, before they are quantised.  Of 32 normal values the largest is 2.1 sigma on
average, so a step of the 4-bit codes is s = 2.1 sigma / 7 = 0.3 sigma; two values |x - y| apart
get codes that differ with probability |x - y| / s, and then by s: a mean square of |x - y| s, on
average 0.8 d sigma 0.3 sigma.  Relative to sigma that is a root of 0.24 d: 4.9e-2 for d = 1e-2,
which is what is left of the 3e-2 above after a third of the way (recurrence, norm and projection).
With the 3e-2 of the attention layer's own: sqrt(4.9e-2^2 + 3e-2^2) = 5.8e-2."""
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.gpu
@pytest.mark.parametrize("lens,new", [((70, 1, 130), 8), ((300,), 3), ((5,) * 20, 4)])
def test_steps_and_parts_agree_with_whole_prompts(lens, new):
    import hybrid_block
    in_parts, alone, steps = hybrid_block.compare(lens, new)
    assert in_parts <= 3e-2 and alone <= 3e-2 and steps <= 5.8e-2
