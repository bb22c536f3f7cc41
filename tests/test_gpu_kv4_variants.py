"""The kernels' variants for many rows, long items and many sequences."""
import numpy as np
import pytest
import torch

import test_gpu_qk_rope as rope
from test_gpu_attn_kv4 import _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_q,n_kv,D", [(8, 1, 128), (14, 2, 64), (4, 4, 128)])
@pytest.mark.parametrize("window", [0, 1500])
@pytest.mark.parametrize("lengths,new", [([2600], [100]), ([4000, 1501, 64], [290, 130, 40])])
def test_prompt_items_cut_across_ctas(n_q, n_kv, D, window, lengths, new):
    """More than 16 pages an item: pieces, tickets and joins; the second call finds the counters that the first left."""
    _check(np.random.default_rng(sum(lengths) + D), lengths, new, n_q, n_kv, D, window=window, pad=8, repeat=2)


@pytest.mark.parametrize("n_q,n_kv,D", [(8, 1, 128), (8, 2, 64)])
def test_three_hundred_sequences(n_q, n_kv, D):
    """More sequences than a CTA's threads (streaming), and than are added up at once (prompts)."""
    rng = np.random.default_rng(D)
    lengths = [int(x) for x in rng.integers(0, 200, 300)]
    _check(rng, lengths, [1] * 300, n_q, n_kv, D, repeat=2)
    new = [int(x) for x in rng.integers(0, 45, 300)]
    _check(rng, [x + y for x, y in zip(lengths, new)], new, n_q, n_kv, D, repeat=2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n_kv,D", [(4, 128), (3, 64)])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("lengths,new", [([1003, 1401], [900, 1400]), ([2500, 3, 1700], [2399, 2, 1700])])
def test_append_and_read_of_many(dtype, n_kv, D, pairs, lengths, new):
    """A warp a token, four tokens a CTA of the read; first places odd and even."""
    rope.test_append_and_read(dtype, n_kv, D, pairs, lengths, new)
