"""Scale bytes of the 8-bit cache at both ends of their range, through read-back and the
decode with few query rows per KV head and with many."""
import numpy as np
import pytest
import torch

import oracle
import sm_attn_fwd_b200 as ab
from tests.q8_helpers import as_codes
from tests.test_gpu_decode_q8 import decode

pytestmark = pytest.mark.gpu

# query tokens of 8 heads over one KV head: 8 and 16 rows
TOKENS = [1, 2]


def codes_of(values, shape, seed):
    """Random codes with magnitudes among `values` (exact e4m3 numbers), and their numbers."""
    g = torch.Generator().manual_seed(seed)
    x = torch.tensor(values)[torch.randint(0, len(values), shape, generator=g)]
    x = x * (torch.randint(0, 2, shape, generator=g) * 2 - 1)
    return x.to(torch.float8_e4m3fn).view(torch.uint8).numpy(), x


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lq", TOKENS)
def test_scale_byte_0_is_2_to_the_minus_127(Lq, d):
    """Values of about 2^-124, and keys of that size under queries of about 2^100 (an 8-bit
    score is q times code in fp32 before its scale).  P in bf16 or better, O in bf16, fp32
    between."""
    B, Hq, Hkv, Lk = 1, 8, 1, 300
    lens = np.asarray([Lk], np.int32)
    planes = []
    for seed in (1, 2):
        code, x = codes_of([4.0, 5.0, 7.0, 10.0, 52.0], (B, Hkv, Lk, d), seed)
        exact = (x.double() * 2.0 ** -127).to(torch.bfloat16)
        assert torch.equal(exact.double(), x.double() * 2.0 ** -127)
        planes.append((code, np.zeros((B, Hkv, Lk), np.uint8), exact))
    k, v = planes
    q = torch.randn(B, Hq, Lq, d, generator=torch.Generator().manual_seed(3))
    q = (q * 2.0 ** 100).to(torch.bfloat16)
    o, lse = decode(q, k, v, lens)
    kv = torch.from_numpy(lens)
    ro, rl = oracle.attn_fwd(q, k[2], v[2], kv_lens=kv)
    ra, _ = oracle.attn_fwd(q, k[2], v[2].abs(), kv_lens=kv)
    err = np.abs(o.float().cpu().double().numpy() - ro)
    # 2^-134: half of bf16's smallest step
    assert (err <= 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2.0 ** -12) * ra + 2.0 ** -134).all()
    assert np.abs(lse.cpu().double().numpy() - rl).max() <= 1e-4
    kr, vr = ab.attn_cache_read_q8(*(as_codes(x[0]).cuda() for x in (k, v)),
                                   *(torch.from_numpy(x[1]).cuda() for x in (k, v)), kv.cuda())
    assert torch.equal(kr.cpu(), k[2]) and torch.equal(vr.cpu(), v[2])
