"""Lane masks of warp-wide operations in the CUDA sources.

What __activemask() returns says which lanes run together at that moment, not which will be at the
next instruction, so it must not be the member mask of a vote, match or shuffle: lanes named in it
that come later leave the others waiting. A mask comes from a vote that whole warps take part in."""

import glob
import os
import re

import pytest

from conftest import ROOT

FILES = sorted(glob.glob(os.path.join(ROOT, "descriptor_build_gb300", "csrc", "*.cu*")))


@pytest.mark.parametrize("path", FILES, ids=[os.path.basename(f) for f in FILES])
def test_no_mask_is_taken_from_the_lanes_that_happen_to_be_active(path):
    code = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)
    assert "__activemask" not in code and "activemask.b32" not in code
