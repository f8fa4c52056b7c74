"""The decode loop of examples/decode_step.py runs all operators together."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_decode_loop():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import decode_step
    lines = []
    said = decode_step.run(steps=40, batch=3, say=lines.append)
    assert len(lines) == 40 and all(0 <= t < decode_step.VOCAB for words in said for t in words)
    assert all(len(words) > 41 for words in said)           # some drafts stood
    cached = eval(lines[-1].split("cached ")[1])            # every request came over its budget and was cut to it
    assert cached == [decode_step.BUDGET] * 3
    # the same seeds say the same words
    assert said == decode_step.run(steps=40, batch=3, say=lambda s: None)
