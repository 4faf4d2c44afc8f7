"""NaN through the split-KV and the shared-prefix decode, at every number of query rows
per KV head: in a query, in a key or a value that a row sees, in the prefix.  A NaN score
makes its row's sums NaN, so O and LSE of the row are NaN; a NaN value makes its column of
O NaN and leaves LSE.  All other outputs keep their bits."""
import math

import numpy as np
import pytest
import torch

import sm_attn_fwd_b200 as ab
from tests.test_gpu_prefix import make, run

pytestmark = pytest.mark.gpu

B, HKV, LP, LK = 3, 2, 700, 300
LENS = [300, 131, 0]
# query heads and tokens over two KV heads: 4, 40, 128 and 136 rows per KV head
ROWS = [(8, 1), (16, 5), (16, 16), (16, 17)]


def same_bits_but(got, want, nan):
    """NaN where `nan` says so, the bits of `want` elsewhere."""
    got, want = got.cpu(), want.cpu()
    assert torch.equal(got.isnan(), nan)
    assert torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Lq", ROWS)
def test_shared_prefix(Hq, Lq, d, page):
    data = make(71, B, Hq, HKV, Lq, LP, LK, d, LENS)
    want, want_lse = run(*data, page=page)
    group = Hq // HKV
    rows = torch.zeros(B, Hq, Lq, dtype=torch.bool)

    def check(nan_o, nan_lse, **at):
        q, kp, vp, k, v, lens = (x.clone() if isinstance(x, torch.Tensor) else x for x in data)
        for name, index in at.items():
            {"q": q, "kp": kp, "vp": vp, "k": k, "v": v}[name][index] = math.nan
        o, lse = run(q, kp, vp, k, v, lens, page=page)
        same_bits_but(o, want, nan_o.expand(o.shape))
        same_bits_but(lse, want_lse, nan_lse)

    one = rows.clone()
    one[:, 3, Lq - 1] = True
    check(one[..., None], one, q=(slice(None), 3, Lq - 1, 5))
    # a key, and a value, of sequence 1's own cache
    mine = rows.clone()
    mine[1, :group] = True
    check(mine[..., None], mine, k=(1, 0, 70, 3))
    column = torch.zeros(B, Hq, Lq, d, dtype=torch.bool)
    column[1, group:, :, 9] = True
    check(column, rows, v=(1, 1, 130, 9))
    # a key, and a value, of the prefix: every sequence's
    head = rows.clone()
    head[:, group:] = True
    check(head[..., None], head, kp=(1, 699, 0))
    column = torch.zeros(B, Hq, Lq, d, dtype=torch.bool)
    column[:, :group, :, d - 1] = True
    check(column, rows, vp=(0, 400, d - 1))


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Lq", ROWS)
def test_split_kv(Hq, Lq, d, splits):
    q, _, _, k, v, _ = make(72, 2, Hq, HKV, Lq, 1, 600, d, [600, 200])
    kv = torch.tensor([600, 200], dtype=torch.int32, device="cuda")

    def decode():
        out = ab.attn_decode_splitkv(q.cuda(), k.cuda(), v.cuda(), kv, num_splits=splits)
        torch.cuda.synchronize()
        return out

    want, want_lse = decode()
    group = Hq // HKV
    nan = torch.zeros(2, Hq, Lq, dtype=torch.bool)
    nan[:, 3, 0] = True          # a query of both sequences
    nan[0, group:] = True        # a key of sequence 0, KV head 1
    q[:, 3, 0, 1] = math.nan
    k[0, 1, 450, 2] = math.nan
    k[1, :, 200:] = math.nan     # past the end: not seen
    v[1, :, 200:] = math.nan
    o, lse = decode()
    same_bits_but(o, want, nan[..., None].expand(o.shape))
    same_bits_but(lse, want_lse, nan)
    assert ab.attn_get_device_error() == (ab.ATTN_OK, 0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Lq", ROWS)
def test_a_nan_value_counts_where_its_weight_underflows(Hq, Lq, d):
    """Keys 300 below the others in their score, in a split or in a cache of their own: the
    weight of the whole partial result is 0 in fp32, and 0 times NaN is NaN."""
    q, kp, vp, k, v, _ = make(73, 1, Hq, HKV, Lq, 256, 256, d, [256])
    q[..., 0], kp[..., 0], k[..., 0] = 8, 0, -300 / 8 * math.sqrt(d)
    want, want_lse = run(q, kp, vp, k, v, np.asarray([256], np.int32))
    v[0, 1, 200, 9] = math.nan
    column = torch.zeros(want.shape, dtype=torch.bool)
    column[:, Hq // HKV:, :, 9] = True
    o, lse = run(q, kp, vp, k, v, np.asarray([256], np.int32))
    same_bits_but(o, want, column)
    assert torch.equal(lse, want_lse)
    kk, vv = torch.cat([kp[None], k], 2).cuda(), torch.cat([vp[None], v], 2).cuda()
    kv = torch.tensor([512], dtype=torch.int32, device="cuda")
    o, _ = ab.attn_decode_splitkv(q.cuda(), kk, vv, kv, num_splits=2)
    assert torch.equal(o.isnan().cpu(), column)
    assert ab.attn_get_device_error() == (ab.ATTN_OK, 0)
