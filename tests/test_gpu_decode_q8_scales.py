"""Scale bytes of the 8-bit cache at both ends of their range, through read-back and the
decode with few query rows per KV head and with many."""
import numpy as np
import pytest
import torch

import oracle
import sm_attn_fwd_b200 as ab
from tests.q8_helpers import as_codes
from tests.test_gpu_decode_q8 import check, decode, make

pytestmark = pytest.mark.gpu

# query tokens of 8 heads over one KV head: 8, 16, 24, 40 and 128 rows
TOKENS = [1, 2, 3, 5, 16]


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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lq", TOKENS)
def test_scale_bytes_above_247_count_as_247(Lq, d):
    """No bf16 row needs a byte above 247; larger ones count as 247 everywhere, and reach no
    other key."""
    B, Hq, Hkv, Lk = 1, 8, 1, 300
    q, k, v, lens = make(105, B, Hq, Hkv, Lq, Lk, d, [Lk])
    at = [3, 64, 130, 299]
    for x in (k, v):
        x[0][0, 0, at] = 0x01            # 2^-9: values of 2^111
        x[0][0, 0, at, ::2] = 0x81
    got = []
    for bytes_ in ([247] * 4, [248, 250, 254, 255]):
        vv = (v[0], v[1].copy())
        vv[1][0, 0, at] = bytes_
        kk = (k[0], k[1].copy())
        kk[1][0, 0, at[0]] = bytes_[0]
        both = [as_codes(k[0]).cuda(), as_codes(v[0]).cuda(), torch.from_numpy(kk[1]).cuda(),
                torch.from_numpy(vv[1]).cuda(), torch.tensor([Lk], dtype=torch.int32).cuda()]
        got.append(list(decode(q, k, vv, lens)) + list(decode(q, kk, v, lens)) +
                   list(ab.attn_cache_read_q8(*both)))
    for a, b in zip(*got):
        assert torch.equal(a.cpu().view(torch.int16), b.cpu().view(torch.int16))
    assert bool(got[0][0].isfinite().all())
    assert float(got[0][5][0, 0, 3, 1]) == 2.0 ** 111


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lq", [5, 16])
def test_a_zero_row_with_any_scale_byte_is_zero(Lq, d):
    """Many query rows: a value row whose codes are all 0 adds nothing whatever its byte is,
    and its neighbours keep their values."""
    q, k, v, lens = make(106, 1, 8, 1, Lq, 300, d, [300])
    at = [0, 62, 63, 128, 298]
    v[0][0, 0, at] = 0
    v[2][0, 0, at] = 0
    for byte in (0, 1, 246, 247, 248, 251, 252, 255):
        v[1][0, 0, at] = byte
        o, lse = decode(q, k, v, lens)
        check(o, lse, q, k, v, lens)
