"""Keys that are all zero in the 8-bit cache, with softmax scales down to where their score
factor underflows."""
import numpy as np
import pytest
import torch

from tests.test_gpu_decode_q8 import check, decode, make

pytestmark = pytest.mark.gpu

# query tokens of 8 heads over one KV head: 8, 16, 24, 40 and 128 rows
TOKENS = [1, 2, 3, 5, 16]


@pytest.mark.parametrize("scale", [None, 1e-7, 1e-12, 1e-30])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lq", TOKENS)
def test_keys_that_are_all_zero(Lq, d, scale):
    """Scale byte 1 throughout: the factor of the scores is subnormal or underflows, and every
    key that is there counts the same."""
    q, k, v, lens = make(107, 3, 8, 1, Lq, 300, d, [300, 131, 0])
    k = (np.zeros_like(k[0]), np.ones_like(k[1]), torch.zeros_like(k[2]))
    o, lse = decode(q, k, v, lens, scale=scale)
    check(o, lse, q, k, v, lens, scale=scale)
