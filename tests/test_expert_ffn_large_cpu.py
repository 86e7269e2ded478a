"""Every variant of the whole layer for few tokens that reads its weights as data not used again is run by some GPU test, in each form of
the weights (the rules, compiled for the host)."""
import pytest

from test_fp8_tiles_cpu import DOWN, UP, VALUES, down_of, up_of, variants  # noqa: F401
from test_gpu_expert_ffn import STREAMED
from test_gpu_expert_ffn_large import LARGE


@pytest.mark.parametrize("form", list(VALUES))
def test_every_streamed_variant_runs_on_the_gpu(variants, form):  # noqa: F811
    got = variants("l", [(VALUES[form], *c) for f, *c in STREAMED + LARGE if f == form])
    assert up_of(got) >= {v for v in UP if v[2]} and down_of(got) >= {v for v in DOWN if v[3]}
