"""Rules that the kernels' sources keep and that no run can show: what they
guard against holds or fails by the compiler's or the scheduler's choice."""
from __future__ import annotations

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "activation_sparse_gated_relu_b200", "csrc")


def code(name: str) -> str:
    """A source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_no_warp_mask_from_the_lanes_that_happen_to_be_there():
    # the lanes that reach a point together after a branch are the compiler's choice: a shuffle whose mask asks for them
    # may leave a lane's partner out
    for name in sorted(os.listdir(CSRC)):
        assert "__activemask" not in code(name), name
