"""NaN codes in the 8-bit cache below its length, through the decode with few query rows per
KV head and with many."""
import math

import pytest
import torch

from tests.q8_helpers import quantise
from tests.test_gpu_decode_q8 import decode, make

pytestmark = pytest.mark.gpu

# query tokens of 8 heads over one KV head: 8, 16, 24, 40 and 128 rows
TOKENS = [1, 2, 3, 5, 16]


def same_bits_but(got, want, nan):
    got, want = got.cpu(), want.cpu()
    assert torch.equal(got.isnan(), nan)
    assert torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("page,ctas", [(0, 0), (16, 0), (0, 1), (64, 3)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lq", TOKENS)
def test_nan_codes_give_nan(Lq, d, page, ctas):
    """A NaN code of a key: its rows' O and LSE; of a value: its column of O.  Whatever the
    row's scale is beside the others'."""
    B, Hq, Hkv, Lk = 2, 16, 2, 700
    q, k, v, lens = make(101, B, Hq, Hkv, Lq, Lk, d, [700, 333])
    for byte in (127, 1):  # 1: the value's scale vanishes beside its tile's
        for code in (0x7F, 0xFF):
            for x in (k, v):
                x[1][0, 1, 515] = x[1][1, 0, 332] = byte
            want, want_lse = decode(q, k, v, lens, page, ctas)
            kn, vn = (k[0].copy(),) + k[1:], (v[0].copy(),) + v[1:]
            kn[0][0, 1, 515, d - 1] = code
            nan = torch.zeros(B, Hq, Lq, dtype=torch.bool)
            nan[0, 8:] = True
            o, lse = decode(q, kn, v, lens, page, ctas)
            same_bits_but(o, want, nan[..., None].expand(o.shape))
            same_bits_but(lse, want_lse, nan)
            vn[0][1, 0, 332, 17] = code
            column = torch.zeros(B, Hq, Lq, d, dtype=torch.bool)
            column[1, :8, :, 17] = True
            o, lse = decode(q, k, vn, lens, page, ctas)
            same_bits_but(o, want, column)
            assert torch.equal(lse, want_lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lq", TOKENS)
def test_a_nan_value_counts_where_its_weight_underflows(Lq, d):
    """Keys 300 below the others in their score, as the second piece of a unit that two CTAs
    share: the weight of the whole piece is 0 in fp32, and 0 times NaN is NaN."""
    q, k, v, lens = make(102, 1, 8, 1, Lq, 1024, d, [1024])
    q[..., 0] = 8
    x = k[2].clone()
    x[..., 0] = 0
    x[:, :, 512:] = 0
    x[:, :, 512:, 0] = -300 / 8 * math.sqrt(d)
    code, e, val = quantise(x)
    k = (code, e, torch.from_numpy(val).to(torch.bfloat16))
    want, want_lse = decode(q, k, v, lens, 0, 2)
    v[0][0, 0, 1000, 17] = 0x7F
    column = torch.zeros(1, 8, Lq, d, dtype=torch.bool)
    column[..., 17] = True
    for ctas in (2, 1, 0):
        o, lse = decode(q, k, v, lens, 0, ctas)
        assert torch.equal(o.isnan().cpu(), column)
    o, lse = decode(q, k, v, lens, 0, 2)
    same_bits_but(o, want, column)
    assert torch.equal(lse, want_lse)
