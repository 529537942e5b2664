"""GPU group norm beyond the sizes that one launch takes, in the shapes that the
smaller tests cover below them."""

import pytest
import torch

from tests.rowops_cases import DTYPES, ragged
from tests.test_gpu_norm import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", ["none", "relu", "silu"])
@pytest.mark.parametrize("C,G", [(64, 8), (48, 3), (80, 10)])
def test_norm_large_activations_and_dropout(dtype, name, C, G):
    run(9001, C, G, ragged(C, 9001, 5), dtype, name, drop=(77 + C, 1 << 33, 5, 0.2), seed=C)


@pytest.mark.parametrize("C,G", [(16, 16), (16, 1), (48, 16), (48, 48), (112, 7), (128, 1), (272, 17), (272, 16), (528, 33)])
def test_norm_large_channels_and_groups(C, G):
    run(5000, C, G, [2500, 0, 1, 2499], torch.float32, "silu", seed=C)
    run(5000, C, G, [5000], torch.bfloat16, "none", seed=C + 1)


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_large_many_samples(dtype):
    # more samples than a wave has lanes, several in a tile and several tiles to one, empty ones among them
    run(12000, 32, 4, [1, 0, 2, 3, 114] * 100, dtype, "silu", seed=4)
    run(20000, 64, 4, ragged(6, 20000, 90), dtype, "none", seed=5)


@pytest.mark.parametrize("n", [511, 512, 513, 1023, 1025, 4095, 4096, 4097])
def test_norm_around_the_one_launch_limits(n):
    run(n, 32, 2, [n], torch.float32, "silu", seed=n)
    run(n, 32, 1, ragged(n, n, 4), torch.bfloat16, "silu", drop=(5, n, 1, 0.1), seed=n)
