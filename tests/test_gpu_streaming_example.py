"""The example that runs quantizer, windowed attention, its gradient and the paged cache together."""

import os
import sys

import pytest
import torch

from gpu_util import announce, needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_example(dtype):
    import streaming_attention as example
    announce("example", dtype=dtype)
    losses, worst, missing, live = example.main(dtype=dtype, steps=5, quiet=True)
    assert losses[-1] < losses[0]
    # each side rounds its weights and its result once (u of the largest value at most each), and sums in float32
    assert worst <= 4 * torch.finfo(dtype).eps / 2 + 400 * 2.0 ** -24
    # listeners keep the window's pages, the sinks' one and the one being written
    assert missing == 0 and 0 < live <= 3 * (-(-example.WINDOW // example.PAGE) + 2)
