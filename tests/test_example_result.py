"""What the expert-layer example prints is the layer: its difference to float32 is e4m3's.

A code is off by at most half a step of 2^-3 in [1, 2): 2^-3 / sqrt(12) = 3.6 % rms of a factor at
most.  Gate and up have two factors each (5.1 %), which silu passes on at most 1.5 times for
gates around 1 (7.6 %); the down product has two more: sqrt(7.6^2 + 5.1^2 + 2 * 3.6^2) = 10.5 %,
and below 12 % with the bfloat16 roundings.  A row of the wrong expert, token or weight would be off
by the size of the result."""

import pytest

from gpu_util import require_gpu
from test_example_expert_layer import _example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,experts,top_k,dim,ffn", [(1, 16, 4, 1024, 1536), (50, 5, 5, 300, 700), (900, 64, 8, 512, 260)])
def test_difference_to_float32(tokens, experts, top_k, dim, ffn):
    require_gpu()
    names = ("--tokens", "--experts", "--top-k", "--dim", "--ffn")
    args = [str(a) for pair in zip(names, (tokens, experts, top_k, dim, ffn)) for a in pair]
    assert _example().main(args) < 0.12
