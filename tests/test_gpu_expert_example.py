"""The example from training to 4-bit serving runs, learns, and its quantised layer stays near the bf16 one."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_expert_ffn_example():
    import expert_ffn
    got = expert_ffn.main(12)
    assert got["losses"][-1] < got["losses"][0]
    assert got["prompt"] < 0.4 and got["token"] < 0.4
