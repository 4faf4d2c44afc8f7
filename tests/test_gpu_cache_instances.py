"""Sizes and layouts that take kernel instances of their own: long appends and read-backs
(several rows per lane group), 17 to 32 query rows per KV head at d = 64 over the 8-bit
cache, paged shared prefixes with many query rows; and every scale byte a row can get."""
import numpy as np
import pytest
import torch

import sm_attn_fwd_b200 as ab
import tests.test_gpu_cache_q8 as cache
import tests.test_gpu_decode_q8 as dec
import tests.test_gpu_prefix as prefix
from tests.q8_helpers import as_codes, quantise

pytestmark = pytest.mark.gpu

# rows * d / 8 lanes above 148 * 2048
LONG = [
    # seed, B, Hkv, Ln, Lk_max, d, page, kind
    (31, 3, 5, 2600, 2700, 128, 0, "spread"),
    (32, 3, 5, 5200, 5201, 64, 0, "normal"),
    (33, 3, 5, 2600, 2816, 128, 64, "edges"),
    (34, 3, 5, 5200, 5248, 64, 16, "spread"),
]


def many(rows, d):
    return rows * (d // 8) > 2 * 148 * 2048


@pytest.mark.parametrize("case", LONG, ids=lambda c: f"ln{c[3]}_d{c[5]}_p{c[6]}_{c[7]}")
@pytest.mark.parametrize("ragged", [False, True])
def test_long_append_is_the_definition_bit_for_bit(case, ragged):
    assert many(case[1] * case[2] * case[3], case[5])
    cache.run_append(case, ragged)


@pytest.mark.parametrize("case", LONG, ids=lambda c: f"ln{c[3]}_d{c[5]}_p{c[6]}_{c[7]}")
def test_long_read_back_is_exact_and_leaves_the_rest(case):
    assert many(case[1] * case[2] * case[4], case[5])
    cache.test_read_back_is_exact_and_leaves_the_rest(case)


@pytest.mark.parametrize("d", [64, 128])
def test_long_append_and_read_back_of_nan_and_infinity(d):
    B, Hkv, Ln = 3, 5, 2600 * 128 // d
    k = cache.rows(35, (B, Hkv, Ln, d))
    at = torch.randperm(B * Hkv * Ln, generator=torch.Generator().manual_seed(36))[:300]
    flat = k.view(-1, d)
    flat[at[:100], 5] = float("nan")
    flat[at[100:200], d - 1] = float("inf")
    flat[at[200:], 8] = -float("inf")
    args = [torch.zeros(B, Hkv, Ln, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
            for _ in "kv"]
    args += [torch.zeros(B, Hkv, Ln, dtype=torch.uint8, device="cuda") for _ in "kv"]
    kv = torch.full((B,), Ln, dtype=torch.int32, device="cuda")
    ab.attn_cache_append_q8(k.cuda(), k.cuda(), *args, kv)
    kr, vr = ab.attn_cache_read_q8(*args, kv)
    cache.dev_ok()
    finite = torch.where(k.isfinite(), k, torch.zeros_like(k))
    _, e, val = quantise(finite)
    assert np.array_equal(args[2].cpu().numpy(), e) and torch.equal(args[2], args[3])
    want = torch.from_numpy(val)
    limit = (448.0 * torch.exp2(torch.from_numpy(e).double() - 127))[..., None].expand(k.shape)
    want = torch.where(k.isinf(), limit * k.float().sign(), want)
    nan = k.isnan()
    assert torch.equal(kr.cpu().isnan(), nan) and torch.equal(vr.cpu().isnan(), nan)
    assert torch.equal(kr.cpu().double()[~nan], want[~nan])


@pytest.mark.parametrize("d", [64, 128])
def test_every_scale_byte(d):
    """Rows whose largest element is the largest with its scale byte, or the smallest."""
    tops, want = [], []
    for e in range(1, 248):
        lo, hi = 1.7578125 * 2.0 ** (e - 120), 1.75 * 2.0 ** (e - 119)
        if e == 1:
            lo = 0.0
        if e == 247:
            hi = float(torch.finfo(torch.bfloat16).max)
        tops += [lo, hi]
        want += [e, e]
    n = len(tops)
    g = torch.Generator().manual_seed(37)
    top = torch.tensor(tops, dtype=torch.float64)[:, None]
    x = (torch.rand(n, d, generator=g, dtype=torch.float64) * 2 - 1) * top * 0.99
    x[torch.arange(n), torch.randint(0, d, (n,), generator=g)] = top[:, 0]
    k = x.to(torch.bfloat16).view(1, 1, n, d)
    code, e, val = quantise(k)
    assert e[0, 0].tolist() == want
    args = [torch.zeros(1, 1, n, d, dtype=torch.uint8, device="cuda") for _ in "kv"]
    exps = [torch.zeros(1, 1, n, dtype=torch.uint8, device="cuda") for _ in "kv"]
    codes = [a.view(torch.float8_e4m3fn) for a in args]
    kv = torch.tensor([n], dtype=torch.int32, device="cuda")
    ab.attn_cache_append_q8(k.cuda(), (-k).cuda(), *codes, *exps, kv)
    kr, vr = ab.attn_cache_read_q8(*codes, *exps, kv)
    cache.dev_ok()
    assert np.array_equal(exps[0].cpu().numpy(), e) and torch.equal(exps[0], exps[1])
    assert np.array_equal(args[0].cpu().numpy(), code)
    back = torch.from_numpy(val).to(torch.bfloat16)
    assert torch.equal(kr.cpu().view(torch.int16), back.view(torch.int16))
    assert torch.equal(vr.cpu(), -back)


ROWS_32 = [
    # B, Hq, Hkv, Lq, Lk_max, (lo, hi), page, num_ctas
    (2, 17, 1, 1, 700, (1, 700), 0, 0),
    (3, 32, 2, 2, 1000, (0, 1000), 0, 3),
    (2, 8, 1, 3, 500, (1, 500), 16, 0),
    (2, 40, 2, 1, 900, (1, 900), 64, 1),
    (1, 32, 1, 1, 20000, (20000, 20000), 256, 0),
    (70, 20, 1, 1, 300, (0, 300), 0, 9),
    (3, 31, 1, 1, 129, (127, 129), 32, 0),
]


@pytest.mark.parametrize("case", ROWS_32, ids=lambda c: f"b{c[0]}_r{c[1] // c[2] * c[3]}_lk{c[4]}_p{c[6]}")
def test_17_to_32_query_rows_at_d64(case):
    B, Hq, Hkv, Lq, Lk, (lo, hi), page, ctas = case
    assert 17 <= Hq // Hkv * Lq <= 32
    lens = np.random.default_rng(B + Hq).integers(lo, hi + 1, B)
    q, k, v, lens = dec.make(40 + B, B, Hq, Hkv, Lq, Lk, 64, lens)
    o, lse = dec.decode(q, k, v, lens, page, ctas)
    dec.check(o, lse, q, k, v, lens)


@pytest.mark.parametrize("n", [0, 1, 31, 32, 33, 255, 256, 257, 300])
def test_17_to_32_query_rows_at_every_tail_length(n):
    for page in (0, 16):
        q, k, v, lens = dec.make(50 + n, 2, 24, 1, 1, 300, 64, [n, 300 - n])
        o, lse = dec.decode(q, k, v, lens, page, 1)
        dec.check(o, lse, q, k, v, lens)


MANY_ROWS = [
    # B, Hq, Hkv, Lq, Lp, Lk_max, d, (lo, hi), page, num_splits
    (3, 34, 2, 1, 300, 40, 128, (0, 40), 16, 0),       # 17 rows
    (5, 16, 2, 5, 777, 300, 128, (1, 300), 64, 0),     # 40 rows
    (3, 16, 2, 16, 513, 200, 128, (0, 200), 256, 2),   # 128 rows
    (2, 16, 2, 17, 400, 70, 128, (1, 70), 32, 0),      # 136 rows
    (4, 24, 1, 1, 500, 90, 64, (0, 90), 16, 0),        # 24 rows
    (3, 33, 1, 1, 700, 130, 64, (0, 130), 16, 3),
    (2, 32, 2, 16, 129, 500, 64, (1, 500), 128, 0),    # 256 rows
]


@pytest.mark.parametrize("case", MANY_ROWS, ids=lambda c: f"r{c[1] // c[2] * c[3]}_d{c[6]}_p{c[8]}")
def test_paged_prefix_with_many_query_rows(case):
    B, Hq, Hkv, Lq, Lp, Lk, d, (lo, hi), page, ns = case
    lens = np.random.default_rng(Lp).integers(lo, hi + 1, B)
    data = prefix.make(60 + B, B, Hq, Hkv, Lq, Lp, Lk, d, lens)
    o, lse = prefix.run(*data, page=page, num_splits=ns)
    prefix.check(o, lse, *data)
