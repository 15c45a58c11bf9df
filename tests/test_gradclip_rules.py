"""Rules of the gradient-clipping code that show without a GPU."""
import os
import re

import pytest

from newton_schulz_norm_b200 import build


def _code(name):
    with open(os.path.join(build.CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


@pytest.mark.parametrize("load", [r"__ldg\b", r"\.nc\b", r"__restrict__"])
def test_gradients_that_a_launch_may_write_are_read_coherently(load):
    """The non-coherent path asks for memory that nothing writes while the
    kernel runs; the one-cluster clip writes in place what it has read."""
    assert not re.search(load, _code("gradclip.cu"))
