"""The example that runs the operators together (examples/recurrent_block.py): the same tokens
as steps and as part of a prompt.

The two ways differ in the recurrences' rounding (the delta-rule prompt path works in chunks on
the tensor cores, held elsewhere to 5e-3 of its outputs), which an 8-bit rounding behind it may
turn into a step of e4m3 (2^-4) where a value lies near the middle between two: the outputs are
held to 3e-2 as a whole."""
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.gpu
@pytest.mark.parametrize("lens,new", [((70, 1, 130), 8), ((300,), 3), ((5,) * 20, 4)])
def test_steps_agree_with_the_prompt(lens, new):
    import recurrent_block
    rel, _ = recurrent_block.compare(lens, new)
    assert rel <= 3e-2
