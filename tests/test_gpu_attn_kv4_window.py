"""Windows near the largest whole number hide nothing."""
import numpy as np
import pytest

from test_gpu_attn_kv4 import _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 4, 2 ** 31 - 250])
@pytest.mark.parametrize("lengths,new", [([3, 0], [6, 40]), ([70, 3, 0, 500], [300, 6, 200, 400])])
def test_rows_before_their_sequence(window, lengths, new):
    _check(np.random.default_rng(new[0]), lengths, new, 8, 2, 128, window=window)
