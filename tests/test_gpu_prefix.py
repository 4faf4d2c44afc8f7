"""Shared-prefix decode against the double-precision oracle on the concatenation of the
prefix and each sequence's own keys.

Tolerance: P is rounded to bf16 (2^-8 relative) for the second product and O to bf16 at
the end; sums are fp32.  |dO| <= 2^-8 |O| + (2^-8 + 2^-12) sum_j P_ij |v_j|, the last
factor's 2^-12 for the fp32 scores, exponentials and sums; the sum is the oracle's output
for |V|.  LSE: 1e-5 + 1e-6 times the largest |score| the norms allow.
"""
import math

import numpy as np
import pytest
import torch

import oracle
import sm_attn_fwd_b200 as ab
from tests.q8_helpers import random_table, to_pages

pytestmark = pytest.mark.gpu


def bf(x):
    return x.to(torch.bfloat16)


def make(seed, B, Hq, Hkv, Lq, Lp, Lk, d, lens):
    g = torch.Generator().manual_seed(seed)
    q = bf(torch.randn(B, Hq, Lq, d, generator=g))
    kp, vp = (bf(torch.randn(Hkv, Lp, d, generator=g)) for _ in "kv")
    k, v = (bf(torch.randn(B, Hkv, Lk, d, generator=g)) for _ in "kv")
    return q, kp, vp, k, v, np.asarray(lens, np.int32)


def poison(x, lens):
    x = x.clone()
    for b, n in enumerate(lens):
        x[b, :, n:] = float("nan")
    return x


def page_args(kp, vp, k, v, lens, page, seed=3):
    """The pool, the prefix's table and the block table of the same data."""
    B, Hkv, Lk, d = k.shape
    Lp = kp.shape[1]
    per_seq, n_prefix = -(-Lk // page), -(-Lp // page)
    num_pages = B * per_seq + n_prefix + 2
    ids = np.random.default_rng(seed).permutation(num_pages).astype(np.int32)
    pt, bt = ids[:n_prefix], ids[n_prefix:n_prefix + B * per_seq].reshape(B, per_seq)
    pools = []
    for xp, x in ((kp, k), (vp, v)):
        pool = torch.full((num_pages, Hkv, page, d), float("nan"), dtype=torch.bfloat16)
        for i in range(n_prefix):
            part = xp[:, i * page:(i + 1) * page]
            pool[pt[i], :, :part.shape[1]] = part
        for b in range(B):
            for i in range(per_seq):
                part = x[b, :, i * page:(i + 1) * page]
                pool[bt[b, i], :, :part.shape[1]] = part
        pools.append(pool.cuda())
    return pools + [torch.from_numpy(pt.copy()).cuda(), Lp, torch.from_numpy(bt.copy()).cuda()]


def run(q, kp, vp, k, v, lens, page=0, **kw):
    k, v = poison(k, lens), poison(v, lens)
    kv = torch.from_numpy(lens).cuda()
    if page:
        o, lse = ab.attn_decode_shared_prefix_paged(q.cuda(), *page_args(kp, vp, k, v, lens, page),
                                                    kv, **kw)
    else:
        o, lse = ab.attn_decode_shared_prefix(q.cuda(), kp.cuda(), vp.cuda(), k.cuda(), v.cuda(),
                                              kv, **kw)
    torch.cuda.synchronize()
    st, bits = ab.attn_get_device_error()
    assert st == ab.ATTN_OK, (st, bits)
    return o, lse


def check(o, lse, q, kp, vp, k, v, lens, scale=None):
    B, Hq, Lq, d = q.shape
    Lp, Lk = kp.shape[1], k.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    kk = torch.cat([kp.expand(B, *kp.shape), k], 2).contiguous()
    vv = torch.cat([vp.expand(B, *vp.shape), v], 2).contiguous()
    for b, n in enumerate(lens):
        kk[b, :, Lp + n:], vv[b, :, Lp + n:] = 0, 0
    kv = torch.from_numpy(lens + Lp).to(torch.int32)
    ro, rl = oracle.attn_fwd(q, kk, vv, kv_lens=kv, scale=scale)
    ra, _ = oracle.attn_fwd(q, kk, vv.abs(), kv_lens=kv, scale=scale)
    o = o.float().cpu().double().numpy()
    assert np.isfinite(o).all()
    err = np.abs(o - ro)
    tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2.0 ** -12) * ra
    assert (err <= tol).all(), float((err - tol).max())
    smax = float(q.float().norm(dim=-1).max() * kk.float().norm(dim=-1).max()) * scale
    assert np.abs(lse.cpu().double().numpy() - rl).max() <= 1e-5 + 1e-6 * smax


SHAPES = [
    # seed, B, Hq, Hkv, Lq, Lp, Lk_max, d, (lo, hi), page, num_splits
    (1, 1, 1, 1, 1, 1, 1, 128, (0, 1), 0, 0),
    (2, 1, 1, 1, 1, 1, 1, 64, (1, 1), 0, 0),
    (3, 4, 32, 8, 1, 2064, 129, 128, (1, 129), 0, 0),     # 16 rows of one tile
    (4, 33, 8, 2, 1, 300, 40, 128, (0, 40), 0, 0),        # 132 rows: a full tile and 4 rows
    (5, 65, 8, 2, 1, 500, 30, 64, (0, 30), 0, 3),         # 260 rows: two tiles and 4 rows
    (6, 26, 10, 2, 2, 257, 33, 128, (0, 33), 0, 2),       # 10 rows a sequence: 12 fit in a tile
    (7, 9, 6, 2, 7, 129, 20, 64, (1, 20), 0, 1),          # 21 rows a sequence: 6 fit
    (8, 3, 16, 2, 16, 400, 70, 128, (1, 70), 0, 0),       # 128 rows: a sequence a tile
    (9, 3, 16, 2, 17, 400, 70, 64, (1, 70), 0, 2),        # 136 rows: two tiles a sequence
    (10, 2, 24, 2, 23, 130, 12, 128, (0, 12), 0, 0),      # 276 rows: three tiles a sequence
    (11, 8, 16, 2, 1, 1000, 100, 128, (0, 100), 16, 0),
    (12, 8, 16, 2, 1, 1000, 100, 64, (0, 100), 16, 3),
    (13, 40, 16, 4, 1, 777, 60, 128, (1, 60), 32, 2),
    (14, 5, 8, 2, 4, 513, 200, 64, (1, 200), 64, 0),
    (15, 5, 8, 2, 4, 640, 200, 128, (1, 200), 128, 5),
    (16, 40, 8, 1, 2, 700, 300, 128, (1, 300), 256, 0),
    (17, 64, 64, 8, 1, 4096, 64, 128, (1, 64), 0, 0),
    (18, 2, 2, 2, 1, 20000, 8, 64, (0, 8), 0, 0),
]


@pytest.mark.parametrize("case", SHAPES, ids=lambda c: (
    f"s{c[0]}_b{c[1]}_g{c[2] // c[3] * c[4]}_lp{c[5]}_d{c[7]}_p{c[9]}_n{c[10]}"))
def test_matches_the_oracle_on_the_concatenation(case):
    seed, B, Hq, Hkv, Lq, Lp, Lk, d, (lo, hi), page, ns = case
    lens = np.random.default_rng(seed).integers(lo, hi + 1, B)
    data = make(seed, B, Hq, Hkv, Lq, Lp, Lk, d, lens)
    o, lse = run(*data, page=page, num_splits=ns)
    check(o, lse, *data)


@pytest.mark.parametrize("Lp", [1, 2, 63, 127, 128, 129, 255, 256, 257, 384])
def test_every_prefix_tail(Lp):
    for page, d, B in ((0, 128, 2), (0, 64, 40), (16, 128, 40), (64, 64, 2)):
        data = make(100 + Lp, B, 8, 1, 1, Lp, 20, d, np.arange(B) % 21)
        for ns in (1, 2):
            o, lse = run(*data, page=page, num_splits=ns)
            check(o, lse, *data)


def test_prefix_alone_is_every_sequences_attention_over_it():
    data = make(7, 6, 8, 2, 1, 600, 5, 128, [0] * 6)
    o, lse = run(*data)
    check(o, lse, *data)


def test_large_scores_and_one_dominant_key():
    """A key in the prefix, or in a sequence's own cache, that takes all the weight."""
    q, kp, vp, k, v, lens = make(8, 4, 8, 2, 1, 300, 50, 64, [50, 50, 10, 0])
    q = bf(q.float() * 4)
    kp[:, 123] = bf(q[0, :2, 0].float() * 2)
    k[1, :, 7] = bf(q[1, :2, 0].float() * 3)
    data = (q, kp, vp, k, v, lens)
    o, lse = run(*data)
    check(o, lse, *data)


def test_equals_the_decode_on_the_copied_prefix():
    """The same numbers as attn_decode_splitkv on a cache that holds the prefix's copy,
    within both results' own tolerances."""
    data = make(9, 6, 16, 2, 2, 512, 128, 128, [128, 1, 64, 100, 3, 77])
    q, kp, vp, k, v, lens = data
    o, lse = run(*data)
    kk = torch.cat([kp.expand(6, *kp.shape), k], 2).contiguous().cuda()
    vv = torch.cat([vp.expand(6, *vp.shape), v], 2).contiguous().cuda()
    o2, l2 = ab.attn_decode_splitkv(q.cuda(), kk, vv, torch.from_numpy(lens + 512).cuda())
    check(o2, l2, *data)
    assert (o.float() - o2.float()).abs().max() <= 2 * (2 ** -8 + 2 ** -8 + 2 ** -12) * 4.5
    assert (lse - l2).abs().max() <= 1e-4


def test_captured_graph_workspace_reuse_and_two_streams():
    """One workspace reused by calls of other shapes, a captured call replayed with new
    queries and lengths, and two streams with a workspace each: always the same bits."""
    data = make(10, 33, 16, 2, 1, 1030, 90, 128, np.arange(33) * 2)
    q, kp, vp, k, v, lens = data
    o0, l0 = run(*data)
    dev = [x.cuda() for x in (q, kp, vp, k, v)] + [torch.from_numpy(lens).cuda()]
    need = ab.attn_decode_shared_prefix_workspace_size(33, 16, 2, 1, 1030, 90, 128)
    ws = [torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    small = make(11, 3, 4, 2, 1, 200, 30, 64, [1, 2, 30])
    so, sl = run(*small, workspace=ws[0])
    check(so, sl, *small)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s, w in zip(streams, ws):
            with torch.cuda.stream(s):
                got.append(ab.attn_decode_shared_prefix(*dev, workspace=w))
    torch.cuda.synchronize()
    for o, lse in got:
        assert torch.equal(o, o0) and torch.equal(lse, l0)
    assert bool((ws[0][need:] == 0xFF).all()) and bool((ws[1][need:] == 0xFF).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = ab.attn_decode_shared_prefix(*dev, workspace=ws[0])
    q2 = bf(torch.randn(q.shape, generator=torch.Generator().manual_seed(12)))
    lens2 = lens[::-1].copy()
    dev[0].copy_(q2)
    dev[5].copy_(torch.from_numpy(lens2))
    # rows that come into play were poisoned nowhere: the cache on the device is whole
    graph.replay()
    torch.cuda.synchronize()
    check(o, lse, q2, kp, vp, k, v, lens2)
    assert ab.attn_get_device_error()[0] == ab.ATTN_OK


def test_bad_lengths_and_pages_are_flagged():
    data = make(13, 3, 8, 2, 1, 100, 40, 64, [40, 3, 0])
    q, kp, vp, k, v, lens = data
    dev = [x.cuda() for x in (q, kp, vp, k, v)]
    for bad in ([41, 3, 0], [40, -1, 0]):
        ab.attn_decode_shared_prefix(*dev, torch.tensor(bad, dtype=torch.int32).cuda())
        torch.cuda.synchronize()
        assert ab.attn_get_device_error()[0] == ab.ATTN_ERR_INVALID_ARG
    args = page_args(kp, vp, k, v, lens, 16)
    for bad in (-1, 1 << 20):
        table = args[2].clone()
        table[2] = bad
        ab.attn_decode_shared_prefix_paged(q.cuda(), args[0], args[1], table, *args[3:],
                                           torch.from_numpy(lens).cuda())
        torch.cuda.synchronize()
        assert ab.attn_get_device_error()[0] == ab.ATTN_ERR_INVALID_ARG


def test_binding_rejects_wrong_shapes_and_types():
    q, kp, vp, k, v, lens = make(14, 2, 8, 2, 1, 40, 20, 64, [20, 3])
    q, kp, vp, k, v = (x.cuda() for x in (q, kp, vp, k, v))
    kv = torch.from_numpy(lens).cuda()
    pool = torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    pt = torch.zeros(3, dtype=torch.int32, device="cuda")
    bt = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    bad = [
        lambda: ab.attn_decode_shared_prefix(q, kp[:1], vp, k, v, kv),
        lambda: ab.attn_decode_shared_prefix(q, kp[None], vp[None], k, v, kv),
        lambda: ab.attn_decode_shared_prefix(q, kp, vp[:, :30], k, v, kv),
        lambda: ab.attn_decode_shared_prefix(q, kp.half(), vp, k, v, kv),
        lambda: ab.attn_decode_shared_prefix(q[:1], kp, vp, k, v, kv),
        lambda: ab.attn_decode_shared_prefix(q, kp, vp, k, v, kv[:1]),
        lambda: ab.attn_decode_shared_prefix(q, kp, vp, k, v, kv, o=q.float()),
        lambda: ab.attn_decode_shared_prefix(q, kp, vp, k, v, kv, lse=q),
        lambda: ab.attn_decode_shared_prefix_paged(q, pool, pool, pt, 49, bt, kv),
        lambda: ab.attn_decode_shared_prefix_paged(q, pool, pool, pt, 32, bt, kv),
        lambda: ab.attn_decode_shared_prefix_paged(q, pool, pool, pt.long(), 40, bt, kv),
        lambda: ab.attn_decode_shared_prefix_paged(q, pool, pool, pt, 40, None, kv),
        lambda: ab.attn_decode_shared_prefix_paged(q, pool, pool, pt, 40, bt[:1], kv),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"case {i} was accepted")
    with pytest.raises(ab.AttnError):
        ab.attn_decode_shared_prefix(q, kp, vp, k, v, kv,
                                     workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert ab.attn_get_device_error()[0] == ab.ATTN_OK


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq", [4, 12, 80])
def test_scores_that_overflow_to_minus_infinity_have_no_weight(Hq, d):
    """The first 70 keys of every own cache score below fp32's range (2^83 * -2^83 in one
    column, which the other keys have 0 in), whole blocks and warps of them."""
    B, Hkv, Lq, Lp, Lk = 3, 2, 1, 200, 300
    lens = [300, 70, 131]
    q, kp, vp, k, v, lens = make(61, B, Hq, Hkv, Lq, Lp, Lk, d, lens)
    q[..., 0] = 2.0 ** 83
    kp[..., 0] = 0
    k[..., 0] = 0
    k[:, :, :70, 0] = -2.0 ** 83
    o, lse = run(q, kp, vp, k, v, lens)
    # the same without those keys
    k2, v2 = k[:, :, 70:].contiguous(), v[:, :, 70:].contiguous()
    kk = torch.cat([kp.expand(B, *kp.shape), k2], 2).contiguous()
    vv = torch.cat([vp.expand(B, *vp.shape), v2], 2).contiguous()
    kv = torch.from_numpy(np.maximum(lens - 70, 0) + Lp).to(torch.int32)
    ro, rl = oracle.attn_fwd(q, kk, vv, kv_lens=kv)
    ra, _ = oracle.attn_fwd(q, kk, vv.abs(), kv_lens=kv)
    o = o.float().cpu().double().numpy()
    assert np.isfinite(o).all()
    assert (np.abs(o - ro) <= 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2.0 ** -12) * ra).all()
    # scores of the other keys: at most 10 in magnitude, so 1e-5 + 1e-6 * 10
    assert np.abs(lse.cpu().double().numpy() - rl).max() <= 2e-5


def test_a_nan_query_gives_nan_in_its_row_only():
    B, Hq, Hkv, Lq, Lp, Lk, d = 3, 8, 2, 1, 700, 300, 128
    q, kp, vp, k, v, lens = make(62, B, Hq, Hkv, Lq, Lp, Lk, d, [300, 0, 131])
    want, want_lse = run(q, kp, vp, k, v, lens)
    q[:, 3, 0, 5] = math.nan
    o, lse = run(q, kp, vp, k, v, lens)
    assert bool(o[:, 3].isnan().all()) and bool(lse[:, 3].isnan().all())
    rest = [h for h in range(Hq) if h != 3]
    assert torch.equal(o[:, rest], want[:, rest]) and torch.equal(lse[:, rest], want_lse[:, rest])
