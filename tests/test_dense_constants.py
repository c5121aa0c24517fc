"""The host tests play the kernels' rules in Python; the constants they use are the kernels'."""
import os
import re

import pytest

from tests import test_dense_host as H

CSRC = os.path.join(os.path.dirname(__file__), "..", "sparse_attention_decode_03_b200", "csrc")


def constant(file, name):
    with open(os.path.join(CSRC, file)) as f:
        found = re.findall(rf"\bconstexpr (?:int|float) (?:[^;]*, )?{name} = (\d+)\b", f.read())
    assert len(found) == 1, f"{name} in {file}: {found}"
    return int(found[0])


@pytest.mark.parametrize("file,name,value", [
    ("dense_decode.cu", "kPieceCost", H.PIECE_COST), ("dense_decode.cu", "kMinPlaces", H.MIN_PLACES),
    ("dense_decode.cu", "kTile", 16), ("dense_decode.cu", "kMaxCtas", 256),
    ("evict.cu", "kUnitBlocks", H.UNIT), ("evict.cu", "kSmallUnit", 4), ("evict.cu", "kLook", 128 // 32)])
def test_constants_that_host_tests_restate(file, name, value):
    assert constant(file, name) == value
