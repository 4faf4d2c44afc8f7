"""Decode over the 8-bit cache against the double-precision oracle on the values the
cache stands for (exact in bf16, which the oracle takes).

Tolerance.  The codes, scales and Q enter exactly; scores and sums are fp32.  P is
rounded to f16 (2^-11 relative) for the second product and O to bf16 (2^-8) at the
end, so |dO| <= 2^-8 |O| + 2^-11 sum_j P_ij |v_j| + the fp32 part; with max|v| as
the bound of the weighted mean, 2^-8 |O| + 2^-10 max|v| holds with a factor of two to
spare for the fp32 sums.  With more than 32 query rows per KV head P is rounded to
bf16 (2^-8) instead: 2^-8 |O| + (2^-8 + 2^-12) sum_j P_ij |v_j|, the sum being the
oracle's output for |V| and 2^-12 the fp32 part.  LSE: fp32 scores of magnitude s carry 2^-22 s, the base-2
exponential and logarithm 2^-21 each: 1e-5 + 1e-6 max|s|.
"""
import math

import numpy as np
import pytest
import torch

import oracle
import sm_attn_fwd_b200 as ab
from tests.q8_helpers import as_codes, quantise, random_table, to_pages

pytestmark = pytest.mark.gpu


def make(seed, B, Hq, Hkv, Lq, Lk, d, lens, k_gain=None, v_gain=None, q_gain=1.0):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(B, Hq, Lq, d, generator=g) * q_gain).to(torch.bfloat16)
    out = [q]
    for gain in (k_gain, v_gain):
        x = torch.randn(B, Hkv, Lk, d, generator=g)
        if gain is not None:
            x = x * gain
        code, e, val = quantise(x.to(torch.bfloat16))
        exact = torch.from_numpy(val).to(torch.bfloat16)
        assert torch.equal(exact.double(), torch.from_numpy(val))  # the oracle's input is the cache
        out.append((code, e, exact))
    return out[0], out[1], out[2], np.asarray(lens, np.int32)


def poison(x, lens):
    code, e = x[0].copy(), x[1].copy()
    for b, n in enumerate(lens):
        code[b, :, n:], e[b, :, n:] = 0x7F, 255  # NaN codes, infinite scales
    return code, e


def decode(q, k, v, lens, page=0, num_ctas=0, scale=None, **kw):
    """num_ctas = 0: one per SM; 1: no unit is cut; few: pieces, their merge, whole units
    in between."""
    (kc, ke), (vc, ve) = poison(k, lens), poison(v, lens)
    kv = torch.from_numpy(lens).cuda()
    if page:
        B, _, Lk = kc.shape[:3]
        per_seq = -(-Lk // page)
        num_pages = B * per_seq + 3
        table = random_table(5, B, per_seq, num_pages)
        kc, vc = (to_pages(x, table, num_pages, page, 0x7F) for x in (kc, vc))
        ke, ve = (to_pages(x, table, num_pages, page, 255) for x in (ke, ve))
        for b, n in enumerate(lens):   # entries past the last page are never read
            table[b, -(-n // page):] = 1 << 30
        args = (as_codes(kc).cuda(), as_codes(vc).cuda(), torch.from_numpy(ke).cuda(),
                torch.from_numpy(ve).cuda(), torch.from_numpy(table).cuda(), kv)
        o, lse = ab.attn_decode_paged_q8(q.cuda(), *args, num_ctas=num_ctas, scale=scale, **kw)
    else:
        args = (as_codes(kc).cuda(), as_codes(vc).cuda(), torch.from_numpy(ke).cuda(),
                torch.from_numpy(ve).cuda(), kv)
        o, lse = ab.attn_decode_splitkv_q8(q.cuda(), *args, num_ctas=num_ctas, scale=scale,
                                           **kw)
    torch.cuda.synchronize()
    st, bits = ab.attn_get_device_error()
    assert st == ab.ATTN_OK, (st, bits)
    return o, lse


def check(o, lse, q, k, v, lens, scale=None):
    kv = torch.from_numpy(lens)
    scale = 1.0 / math.sqrt(q.shape[-1]) if scale is None else scale
    ro, rl = oracle.attn_fwd(q, k[2], v[2], kv_lens=kv, scale=scale)
    o = o.float().cpu().double().numpy()
    lse = lse.cpu().double().numpy()
    B, Hq, Lq, d = q.shape
    wide = Hq // k[2].shape[1] * Lq > 32
    ra = oracle.attn_fwd(q, k[2], v[2].abs(), kv_lens=kv, scale=scale)[0] if wide else None
    for b in range(B):
        if lens[b] == 0:
            assert np.all(o[b] == 0) and np.all(np.isneginf(lse[b]))
            continue
        vmax = v[2][b, :, :lens[b]].float().abs().amax().item()
        kmax = k[2][b, :, :lens[b]].float().norm(dim=-1).max()  # rows past the end may hold anything
        smax = float(q[b].float().norm(dim=-1).max() * kmax) * scale
        err = np.abs(o[b] - ro[b])
        assert np.isfinite(o[b]).all()
        p_err = (2.0 ** -8 + 2.0 ** -12) * ra[b] if wide else 2.0 ** -10 * vmax
        assert (err <= 2.0 ** -8 * np.abs(ro[b]) + p_err).all(), (b, err.max(), vmax)
        assert np.abs(lse[b] - rl[b]).max() <= 1e-5 + 1e-6 * smax, b


SHAPES = [
    # seed, B, Hq, Hkv, Lq, Lk_max, d, (lo, hi), page, num_ctas
    (1, 2, 8, 1, 1, 300, 128, (1, 300), 0, 0),
    (2, 3, 16, 2, 1, 1000, 128, (1, 1000), 0, 3),
    (3, 3, 16, 2, 1, 1000, 64, (1, 1000), 0, 1),
    (4, 2, 5, 5, 1, 129, 64, (1, 129), 0, 0),
    (5, 1, 1, 1, 1, 1, 128, (1, 1), 0, 0),
    (6, 1, 1, 1, 1, 1, 64, (1, 1), 0, 1),
    (7, 4, 10, 2, 3, 513, 64, (1, 513), 0, 5),       # 15 rows: a padded 16-row tile
    (8, 2, 16, 2, 2, 700, 128, (1, 700), 0, 2),      # 16 rows
    (9, 2, 16, 2, 4, 700, 128, (1, 700), 0, 1),      # 32 rows
    (10, 2, 40, 4, 5, 400, 128, (1, 400), 0, 2),     # 50 rows: two row tiles
    (11, 2, 32, 2, 16, 640, 128, (1, 640), 0, 2),    # 256 rows
    (12, 2, 32, 2, 16, 640, 64, (600, 640), 0, 0),
    (13, 3, 16, 2, 1, 500, 128, (1, 500), 16, 0),
    (14, 3, 16, 2, 1, 500, 64, (1, 500), 16, 2),
    (15, 2, 8, 2, 2, 700, 128, (1, 700), 32, 0),
    (16, 2, 8, 2, 2, 700, 64, (1, 700), 64, 1),
    (17, 2, 16, 2, 16, 900, 128, (1, 900), 128, 3),
    (18, 2, 16, 2, 1, 900, 128, (1, 900), 256, 0),
    (19, 2, 64, 8, 1, 4100, 128, (4000, 4100), 0, 0),
    (20, 1, 8, 1, 1, 65536, 64, (65536, 65536), 0, 0),
    (21, 3, 16, 2, 16, 1500, 128, (1, 1500), 16, 0),  # 128 rows, pages inside a tile
    (22, 3, 16, 2, 16, 1500, 64, (1, 1500), 32, 2),
    (23, 2, 33, 1, 1, 777, 128, (300, 777), 0, 1),    # 33 rows
    (24, 2, 130, 2, 2, 777, 64, (1, 777), 64, 1),     # 130 rows: a full tile and 2 rows
    (25, 1, 64, 1, 2, 16384, 128, (16384, 16384), 256, 0),
    (26, 2, 34, 2, 3, 5000, 64, (1, 5000), 0, 4),     # 51 rows
    (27, 70, 8, 1, 1, 600, 128, (0, 600), 0, 0),      # more sequences than a warp has lanes
    (28, 70, 16, 2, 1, 300, 64, (0, 300), 16, 9),
    (29, 40, 16, 1, 3, 400, 128, (0, 400), 32, 13),   # 48 rows
    (30, 1, 2, 2, 1, 40000, 128, (40000, 40000), 0, 0),  # a unit over many CTAs
    (31, 1, 64, 1, 1, 40000, 128, (40000, 40000), 64, 0),
    (32, 3, 8, 1, 1, 4000, 128, (0, 4000), 0, 1000),  # more CTAs than tiles
]


@pytest.mark.parametrize("case", SHAPES,
                         ids=lambda c: f"s{c[0]}_r{c[2] // c[3] * c[4]}_lk{c[5]}_d{c[6]}_p{c[8]}_n{c[9]}")
def test_matches_the_oracle_with_poison_past_the_end(case):
    seed, B, Hq, Hkv, Lq, Lk, d, (lo, hi), page, ns = case
    lens = np.random.default_rng(seed).integers(lo, hi + 1, B)
    q, k, v, lens = make(seed, B, Hq, Hkv, Lq, Lk, d, lens)
    o, lse = decode(q, k, v, lens, page, ns)
    check(o, lse, q, k, v, lens)


@pytest.mark.parametrize("ns", [1, 3])
@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 256, 257, 300])
def test_every_tail_length(n, ns):
    """Lengths around a 16-key block, a warp's unit, a page, a split; and an empty sequence."""
    for page, d, Lq in ((0, 128, 1), (0, 64, 1), (16, 128, 1), (0, 128, 5), (16, 64, 5),
                        (32, 128, 5)):
        q, k, v, lens = make(40 + n, 2, 8, 1, Lq, 300, d, [n, 300 - n])
        o, lse = decode(q, k, v, lens, page, ns)
        check(o, lse, q, k, v, lens)


@pytest.mark.parametrize("Lq", [1, 6])
@pytest.mark.parametrize("d", [64, 128])
def test_one_key_of_huge_scale_and_no_weight(d, Lq):
    """A value row 2^40 larger than the rest with a softmax weight of about 2^-90 must not
    cost the other rows their precision (nor the other way round)."""
    B, Hq, Hkv, Lk = 1, 8, 1, 200
    q, k, v, lens = make(61, B, Hq, Hkv, Lq, Lk, d, [Lk], q_gain=0.25)
    g = torch.Generator().manual_seed(62)
    x = torch.randn(B, Hkv, Lk, d, generator=g)
    x[:, :, 77] *= 2.0 ** 40
    vv = quantise(x.to(torch.bfloat16))
    v = (vv[0], vv[1], torch.from_numpy(vv[2]).to(torch.bfloat16))
    # key 77 points away from every query: its score is far below the others
    qq = torch.ones(B, Hq, Lq, d)
    q = qq.to(torch.bfloat16)
    kk = torch.randn(B, Hkv, Lk, d, generator=g) * 0.1
    kk[:, :, 77] = -64.0 / math.sqrt(d)
    kq = quantise(kk.to(torch.bfloat16))
    k = (kq[0], kq[1], torch.from_numpy(kq[2]).to(torch.bfloat16))
    o, lse = decode(q, k, v, lens)
    ro, rl = oracle.attn_fwd(q, k[2], v[2], kv_lens=torch.from_numpy(lens))
    small = np.abs(x.numpy()).reshape(-1, d)[np.arange(Lk) != 77].max()
    w77 = 2.0 ** 40 * 4 * math.exp(-64.0 + 8.0)   # the huge row's whole part of O, at most
    assert w77 < 2.0 ** -10 * small
    err = np.abs(o.float().cpu().double().numpy() - ro)
    p_round = 2.0 ** -10 if Lq == 1 else 2.0 ** -8   # of |v|'s maximum: P in f16, in bf16
    assert (err <= 2.0 ** -8 * np.abs(ro) + p_round * small).all(), err.max()
    assert np.abs(lse.cpu().double().numpy() - rl).max() <= 1e-4


@pytest.mark.parametrize("Lq", [1, 9])
def test_scales_over_many_binades(Lq):
    """K and V rows whose scales span 2^+-20, Q tiny and huge per head."""
    g = torch.Generator().manual_seed(71)
    B, Hq, Hkv, Lk, d = 2, 8, 2, 400, 128
    vg = torch.exp2(torch.randint(-20, 21, (B, Hkv, Lk, 1), generator=g).float())
    q, k, v, lens = make(72, B, Hq, Hkv, Lq, Lk, d, [400, 333], v_gain=vg)
    hg = torch.exp2(torch.arange(Hq).float() * 4 - 16).view(1, Hq, 1, 1)
    q = (q.float() * hg).to(torch.bfloat16)
    o, lse = decode(q, k, v, lens)
    ro, rl = oracle.attn_fwd(q, k[2], v[2], kv_lens=torch.from_numpy(lens))
    o = o.float().cpu().double().numpy()
    # the weighted mean of |v| bounds the f16 rounding of P row by row
    ra, _ = oracle.attn_fwd(q, k[2], v[2].abs(), kv_lens=torch.from_numpy(lens))
    smax = np.abs(rl).max() + 10
    err = np.abs(o - ro)
    # scores of magnitude s carry 2^-22 s in fp32, so P carries that much relative error
    p_round = 2.0 ** -10 if Lq == 1 else 2.0 ** -8 + 2.0 ** -12
    assert (err <= 2.0 ** -8 * np.abs(ro) + (p_round + 2.0 ** -20 * smax) * ra).all(), err.max()
    assert np.abs(lse.cpu().double().numpy() - rl).max() <= 1e-5 + 1e-6 * smax


@pytest.mark.parametrize("Lq", [1, 9])
def test_all_zero_values_and_zero_queries(Lq):
    B, Hq, Hkv, Lk, d = 1, 8, 2, 100, 64
    q, k, v, lens = make(81, B, Hq, Hkv, Lq, Lk, d, [100], v_gain=0.0)
    o, lse = decode(q, k, v, lens)
    assert bool((o == 0).all())
    rl = oracle.attn_fwd(q, k[2], v[2], kv_lens=torch.from_numpy(lens))[1]
    assert np.abs(lse.cpu().double().numpy() - rl).max() <= 1e-4
    q0 = torch.zeros_like(q)
    q, k, v, lens = make(82, B, Hq, Hkv, Lq, Lk, d, [100])
    o, lse = decode(q0, k, v, lens)
    check(o, lse, q0, k, v, lens)
    assert np.abs(lse.cpu().numpy() - math.log(100)).max() < 1e-6


def test_empty_sequences_everywhere():
    """Empty sequences first, last, between and alone."""
    for lens in ([0, 0, 5, 0, 300, 0], [0] * 6, [129, 0, 0, 0, 0, 1]):
        for Lq in (1, 20):
            q, k, v, lens_ = make(33, 6, 4, 1, Lq, 300, 128, lens)
            for ctas in (0, 1, 2):
                o, lse = decode(q, k, v, lens_, num_ctas=ctas)
                check(o, lse, q, k, v, lens_)


@pytest.mark.parametrize("Lq", [1, 2, 16])
def test_workspace_is_the_documented_size_and_starts_with_anything(Lq):
    q, k, v, lens = make(34, 5, 16, 2, Lq, 900, 128, [900, 1, 450, 0, 129])
    for ctas in (0, 3, 11):
        need = ab.attn_decode_q8_workspace_size(16, 2, Lq, 128, ctas)
        ws = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN
        o, lse = decode(q, k, v, lens, num_ctas=ctas, workspace=ws)
        check(o, lse, q, k, v, lens)
        assert bool((ws[need:] == 0xFF).all())


def test_append_then_decode_as_a_serving_loop():
    """Prompt in, then tokens one by one: cache written by append, decoded each step,
    captured once in a graph and replayed; each step equals the oracle on the
    read-back values."""
    B, Hq, Hkv, Lk, d, page = 3, 8, 2, 96, 128, 16
    per_seq = Lk // page
    num_pages = B * per_seq
    table = torch.from_numpy(random_table(9, B, per_seq, num_pages)).cuda()
    kp, vp = (torch.full((num_pages, Hkv, page, d), 0x7F, dtype=torch.uint8,
                         device="cuda").view(torch.float8_e4m3fn) for _ in "kv")
    ke, ve = (torch.full((num_pages, Hkv, page), 255, dtype=torch.uint8, device="cuda")
              for _ in "kv")
    g = torch.Generator().manual_seed(91)
    prompt = torch.tensor([40, 1, 33], dtype=torch.int32)
    k0, v0 = (torch.randn(B, Hkv, 40, d, generator=g).to(torch.bfloat16) for _ in "kv")
    kv = prompt.cuda()
    ab.attn_cache_append_paged_q8(k0.cuda(), v0.cuda(), kp, vp, ke, ve, table, kv, new_lens=kv)
    q = torch.zeros(B, Hq, 1, d, dtype=torch.bfloat16, device="cuda")
    k1, v1 = (torch.zeros(B, Hkv, 1, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")

    def step():
        kv.add_(1)
        ab.attn_cache_append_paged_q8(k1, v1, kp, vp, ke, ve, table, kv)
        return ab.attn_decode_paged_q8(q, kp, vp, ke, ve, table, kv)

    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    before = kv.clone()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    kv.copy_(before)
    with torch.cuda.graph(graph):
        o, lse = step()
    kv.copy_(before)
    for i in range(6):
        for t in (q, k1, v1):
            t.copy_(torch.randn(t.shape, generator=g).to(torch.bfloat16))
        graph.replay()
        kr, vr = ab.attn_cache_read_paged_q8(kp, vp, ke, ve, table, kv)
        torch.cuda.synchronize()
        lens = kv.cpu().numpy()
        assert np.array_equal(lens, prompt.numpy() + i + 1)
        # the rows just written are the definition's
        _, _, val = quantise(k1.cpu())
        for b in range(B):
            assert np.array_equal(kr[b, :, lens[b] - 1].cpu().double().numpy(), val[b, :, 0])
        check(o, lse, q.cpu(), (None, None, kr.cpu()), (None, None, vr.cpu()), lens)
    st, bits = ab.attn_get_device_error()
    assert st == ab.ATTN_OK, (st, bits)


@pytest.mark.parametrize("Lq", [1, 16])
def test_two_calls_at_once_on_two_streams_and_repeated_calls_are_bit_equal(Lq):
    q, k, v, lens = make(95, 4, 16, 2, Lq, 2000, 128, [2000, 1, 777, 1500])
    o0, l0 = decode(q, k, v, lens)
    (kc, ke), (vc, ve) = poison(k, lens), poison(v, lens)
    args = (q.cuda(), as_codes(kc).cuda(), as_codes(vc).cuda(), torch.from_numpy(ke).cuda(),
            torch.from_numpy(ve).cuda(), torch.from_numpy(lens).cuda())
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(ab.attn_decode_splitkv_q8(*args))
    torch.cuda.synchronize()
    for o, lse in got:
        assert torch.equal(o, o0) and torch.equal(lse, l0)


def test_bad_lengths_and_pages_are_flagged():
    q, k, v, lens = make(97, 2, 8, 2, 1, 64, 64, [64, 64])
    (kc, ke), (vc, ve) = poison(k, lens), poison(v, lens)
    args = [as_codes(kc).cuda(), as_codes(vc).cuda(), torch.from_numpy(ke).cuda(),
            torch.from_numpy(ve).cuda()]
    for bad in ([65, 3], [-1, 64]):
        ab.attn_decode_splitkv_q8(q.cuda(), *args, torch.tensor(bad, dtype=torch.int32).cuda())
        torch.cuda.synchronize()
        st, _ = ab.attn_get_device_error()
        assert st == ab.ATTN_ERR_INVALID_ARG
    pool = [x.view(torch.uint8).view(8, 2, 16, -1).view(torch.float8_e4m3fn) for x in args[:2]]
    pool += [x.view(8, 2, 16) for x in args[2:]]
    for bad in (8, -1):
        table = torch.tensor([[0, 1, 2, bad], [4, 5, 6, 7]], dtype=torch.int32).cuda()
        ab.attn_decode_paged_q8(q.cuda(), *pool, table, torch.from_numpy(lens).cuda())
        torch.cuda.synchronize()
        st, _ = ab.attn_get_device_error()
        assert st == ab.ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lq", [1, 4, 16])
def test_scores_that_overflow_to_minus_infinity_have_no_weight(Lq, d):
    """The first 200 keys score below fp32's range (2^20 * -2^115 in one column, which the
    other keys have 0 in), whole blocks, warps and tiles of them; Q's other columns lie
    2^20 below its largest, well inside what the scaled Q keeps."""
    B, Hq, Hkv, Lk = 2, 8, 2, 500
    q, k, v, lens = make(83, B, Hq, Hkv, Lq, Lk, d, [500, 333])
    q[..., 0] = 2.0 ** 20
    x = k[2].clone()
    x[..., 0] = 0
    x[:, :, :200, 0] = -2.0 ** 115
    code, e, val = quantise(x)
    exact = torch.from_numpy(val).to(torch.bfloat16)
    o, lse = decode(q, (code, e, exact), v, lens)
    kv = torch.from_numpy(lens - 200).to(torch.int32)
    kk, vv = exact[:, :, 200:].contiguous(), v[2][:, :, 200:].contiguous()
    ro, rl = oracle.attn_fwd(q, kk, vv, kv_lens=kv)
    ra, _ = oracle.attn_fwd(q, kk, vv.abs(), kv_lens=kv)
    o = o.float().cpu().double().numpy()
    assert np.isfinite(o).all()
    assert (np.abs(o - ro) <= 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2.0 ** -12) * ra).all()
    assert np.abs(lse.cpu().double().numpy() - rl).max() <= 2e-5


@pytest.mark.parametrize("Lq", [1, 4, 16])
def test_a_nan_query_gives_nan_in_its_row_only(Lq):
    B, Hq, Hkv, Lk, d = 2, 8, 2, 700, 128
    q, k, v, lens = make(84, B, Hq, Hkv, Lq, Lk, d, [700, 1])
    want, want_lse = decode(q, k, v, lens)
    q[:, 3, Lq - 1, 5] = math.nan
    o, lse = decode(q, k, v, lens)
    assert bool(o[:, 3, Lq - 1].isnan().all()) and bool(lse[:, 3, Lq - 1].isnan().all())
    rest = torch.ones(Hq, Lq, dtype=torch.bool)
    rest[3, Lq - 1] = False
    assert torch.equal(o[:, rest], want[:, rest]) and torch.equal(lse[:, rest], want_lse[:, rest])
