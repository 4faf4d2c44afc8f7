"""How the 8-bit decode rounds its weights: few query rows per KV head (up to 16 at
d = 128, 32 at d = 64) hold P times the value scale in f16, more of them P in bf16.

f16: relative to the largest P 2^ve of the row it is 2^7 or more, so a weight carries
2^-11 of itself, or half of f16's smallest step, 2^-25, which is 2^-32 of that largest
one:
  |dO| <= 2^-8 |O| + (2^-11 + 2^-12) sum_j p_j |v_j| + n 2^-32 max_j(p_j 2^ve_j) max|code|,
the last 2^-12 for fp32 scores, exponentials and sums.  A running fp32 sum of N positive
terms is off by at most N 2^-24 of itself; a thread adds at most n / 64 of a row's n keys
(a CTA has 8 warps or more, and each thread one of eight keys), so LSE is off by at most
n / 64 * 2^-24 + 1e-5 + 1e-6 max|s|.
"""
import math

import numpy as np
import pytest
import torch

import sm_attn_fwd_b200 as ab
from tests.q8_helpers import as_codes
from tests.test_gpu_decode_q8 import decode, make

pytestmark = pytest.mark.gpu


def few_rows(d, rows):
    return rows <= (32 if d == 64 else 16)


@pytest.mark.parametrize("drop", [19.25, 22.25, 25.5, 27.75])
@pytest.mark.parametrize("d,group", [(128, 8), (128, 16), (64, 8), (64, 16), (64, 32), (128, 32)])
def test_a_long_flat_tail_below_a_dominant_key(d, group, drop):
    """Every warp of the one CTA sees a key with all the weight in its first 32 and then a long
    tail of weights 2^-drop.  Half of the columns are 0 in the dominant keys, so that they
    show the tail alone."""
    n, sinks = 1 << 18, np.arange(0, 512, 32)
    scale = drop * math.log(2) / 16
    q = torch.zeros(1, group, 1, d, dtype=torch.bfloat16)
    q[..., 0] = 1
    kc = np.zeros((1, 1, n, d), np.uint8)
    kc[0, 0, sinks, 0] = 0x58            # 16: the score 16 * scale = drop * ln 2
    vc = np.full((1, 1, n, d), 0x38, np.uint8)  # 1
    vc[0, 0, sinks, d // 2:] = 0
    e = torch.full((1, 1, n), 127, dtype=torch.uint8, device="cuda")
    o, lse = ab.attn_decode_splitkv_q8(
        q.cuda(), as_codes(kc).cuda(), as_codes(vc).cuda(), e, e,
        torch.tensor([n], dtype=torch.int32, device="cuda"), scale=scale, num_ctas=1)
    assert ab.attn_get_device_error() == (ab.ATTN_OK, 0)
    s = float(np.float32(scale)) * 16    # the call takes fp32
    tail = (n - len(sinks)) * math.exp(-s)
    total = len(sinks) + tail
    want = np.where(np.arange(d) < d // 2, 1.0, tail / total)
    tol = 2.0 ** -8 * want + (2.0 ** -11 + 2.0 ** -12) * want + n * 2.0 ** -32 / total
    if not few_rows(d, group):           # bf16: relative at every size
        tol = (2.0 ** -8 + 2.0 ** -8 + 2.0 ** -12) * want
    err = np.abs(o.float().cpu().double().numpy() - want)
    assert (err <= tol).all(), (err.max(-1).max(), want[-1])
    lse_err = np.abs(lse.cpu().double().numpy() - (math.log(total) + s)).max()
    assert lse_err <= n / 64 * 2.0 ** -24 + 1e-5 + 1e-6 * s


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 8, 16, 17, 24, 32, 33, 128])
@pytest.mark.parametrize("n", [2, 3, 5, 40, 300])
def test_rounding_of_the_weights(d, group, n):
    """Few keys with values that nearly cancel show the rounding of P itself."""
    q, k, v, lens = make(200 + n, 1, group, 1, 1, n, d, [n])
    # v_j = +-(1 + 2^-3 random): the alternating sum of weights near 1 / n
    q = (q.float() * 0.05).to(torch.bfloat16)
    g = torch.Generator().manual_seed(n)
    x = 1 + torch.randint(0, 3, (1, 1, n, d), generator=g) / 8
    x = x * torch.where(torch.arange(n) % 2 == 0, 1.0, -1.0)[:, None]
    code = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert torch.equal(torch.from_numpy(code).view(torch.float8_e4m3fn).float(), x)
    v = (code, np.full((1, 1, n), 127, np.uint8), x.to(torch.bfloat16))
    o, lse = decode(q, k, v, lens)
    s = q[0, :, 0].double() @ k[2][0, 0].double().T / math.sqrt(d)
    p = torch.softmax(s, -1)
    ro = (p @ x[0, 0].double()).numpy()
    ra = (p @ x[0, 0].double().abs()).numpy()
    top = p.max(-1, keepdim=True).values.numpy()
    if few_rows(d, group):
        tol = (2.0 ** -11 + 2.0 ** -12) * ra + n * 2.0 ** -32 * 1.25 * top
    else:
        tol = (2.0 ** -8 + 2.0 ** -12) * ra
    err = np.abs(o[0, :, 0].float().cpu().double().numpy() - ro)
    assert (err <= 2.0 ** -8 * np.abs(ro) + tol).all(), err.max()


@pytest.mark.parametrize("d,group", [(128, 8), (128, 16), (64, 8), (64, 16), (64, 32), (128, 32)])
@pytest.mark.parametrize("c", [0.5, 1, 2, 4, 5, 7, 8, 9, 15, 16, 17, 32, 64, 1024])
def test_large_scores_that_grow_by_little(c, d, group):
    """Base-2 scores of about 2^23 c, where fp32's steps are as large as the differences, and
    c more in later keys: no weight may overflow.  All values are 1, so O is 1 up to P's
    rounding and O's own."""
    n = 2048
    q = torch.zeros(1, group, 1, d, dtype=torch.bfloat16)
    q[..., 0], q[..., 1] = 2.0 ** 15, 1
    kc = np.zeros((1, 1, n, d), np.uint8)
    kc[..., 0] = 0x78                    # 256: a score of 2^23
    kc[0, 0, n // 2:, 1] = 0x38          # and 1 more
    vc = np.full((1, 1, n, d), 0x38, np.uint8)
    e = torch.full((1, 1, n), 127, dtype=torch.uint8, device="cuda")
    for ctas in (1, 0):
        o, lse = ab.attn_decode_splitkv_q8(
            q.cuda(), as_codes(kc).cuda(), as_codes(vc).cuda(), e, e,
            torch.tensor([n], dtype=torch.int32, device="cuda"), scale=c * math.log(2),
            num_ctas=ctas)
        p_round = 2.0 ** -11 if few_rows(d, group) else 2.0 ** -8
        assert float((o.float() - 1).abs().max()) <= 2.0 ** -8 + p_round + 2.0 ** -12
        assert bool(lse.isfinite().all())
