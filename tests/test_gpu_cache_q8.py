"""The 8-bit cache on the GPU: append and read-back against the format's definition
(tests/q8_helpers.py), bit for bit, and what they must not touch."""
import math

import numpy as np
import pytest
import torch

import sm_attn_fwd_b200 as ab
from tests.q8_helpers import as_codes, quantise, random_table, to_pages

pytestmark = pytest.mark.gpu

GUARD = 0xA5  # what the cache holds where nothing may be written


def rows(seed, shape, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if kind == "spread":      # row norms over many binades, so every scale byte region occurs
        x *= torch.exp2(torch.randint(-60, 60, shape[:-1] + (1,), generator=g).float())
    elif kind == "tiny":      # down to bf16's subnormals
        x *= torch.exp2(torch.randint(-140, -120, shape[:-1] + (1,), generator=g).float())
    elif kind == "ties":      # multiples of half a code step: every rounding is a tie or exact
        x = torch.randint(-64, 65, shape, generator=g).float()
    elif kind == "edges":     # the largest element at, just below and just above a scale border
        top = torch.tensor([448.0, 447.0, 450.0, 224.0, 225.0, 1.75, 1.7578125, 0.0])
        pick = torch.randint(0, 8, shape[:-1], generator=g)
        x = x.clamp(-1, 1) * 0.5
        x[..., 3] = -top[pick]
        x[pick == 7] = 0.0
    return x.to(torch.bfloat16)


def dev_ok():
    torch.cuda.synchronize()
    st, bits = ab.attn_get_device_error()
    assert st == ab.ATTN_OK, (st, bits)


CASES = [
    # seed, B, Hkv, Ln, Lk_max, d, page, kind
    (1, 3, 2, 1, 40, 128, 0, "normal"),
    (2, 64, 8, 1, 33, 128, 0, "spread"),
    (3, 1, 1, 1, 1, 64, 0, "normal"),
    (4, 2, 3, 70, 131, 64, 0, "ties"),
    (5, 2, 3, 70, 131, 128, 0, "edges"),
    (6, 2, 1, 50, 64, 128, 16, "tiny"),
    (7, 3, 2, 33, 96, 64, 32, "spread"),
    (8, 2, 2, 129, 256, 128, 128, "normal"),
    (9, 5, 4, 1, 48, 64, 16, "edges"),
]


def run_append(case, ragged):
    seed, B, Hkv, Ln, Lk, d, page, kind = case
    g = np.random.default_rng(seed)
    k, v = rows(seed, (B, Hkv, Ln, d), kind), rows(seed + 100, (B, Hkv, Ln, d), kind)
    lens = g.integers(Ln, Lk + 1, B).astype(np.int32)
    new = g.integers(0, Ln + 1, B).astype(np.int32) if ragged else np.full(B, Ln, np.int32)
    want = {}
    for name, x in (("k", k), ("v", v)):
        code, e, _ = quantise(x)
        c = np.full((B, Hkv, Lk, d), GUARD, np.uint8)
        s = np.full((B, Hkv, Lk), GUARD, np.uint8)
        for b in range(B):
            at = slice(lens[b] - new[b], lens[b])
            c[b, :, at], s[b, :, at] = code[b, :, :new[b]], e[b, :, :new[b]]
        want[name] = (c, s)
    table = None
    if page:
        per_seq = -(-Lk // page)
        num_pages = B * per_seq + 2
        table = random_table(seed, B, per_seq, num_pages)
        want = {n: (to_pages(c, table, num_pages, page, GUARD),
                    to_pages(s, table, num_pages, page, GUARD)) for n, (c, s) in want.items()}
    bufs = []
    for n in ("k", "v"):
        bufs.append(torch.full(want[n][0].shape, GUARD, dtype=torch.uint8, device="cuda"))
    exps = [torch.full(want[n][1].shape, GUARD, dtype=torch.uint8, device="cuda") for n in "kv"]
    codes = [x.view(torch.float8_e4m3fn) for x in bufs]
    kv = torch.from_numpy(lens).cuda()
    nl = torch.from_numpy(new).cuda() if ragged else None
    if page:
        ab.attn_cache_append_paged_q8(k.cuda(), v.cuda(), *codes, *exps,
                                      torch.from_numpy(table).cuda(), kv, new_lens=nl)
    else:
        ab.attn_cache_append_q8(k.cuda(), v.cuda(), *codes, *exps, kv, new_lens=nl)
    dev_ok()
    for i, n in enumerate("kv"):
        assert np.array_equal(exps[i].cpu().numpy(), want[n][1]), n
        assert np.array_equal(bufs[i].cpu().numpy(), want[n][0]), n


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"s{c[0]}_ln{c[3]}_d{c[5]}_p{c[6]}_{c[7]}")
@pytest.mark.parametrize("ragged", [False, True])
def test_append_is_the_definition_bit_for_bit(case, ragged):
    run_append(case, ragged)


def test_append_infinities_and_nan():
    """An infinity saturates at the scale its row's finite values give, NaN stays NaN."""
    k = rows(11, (1, 1, 3, 128))
    k[0, 0, 0, 5] = math.inf
    k[0, 0, 0, 6] = -math.inf
    k[0, 0, 1, 7] = math.nan
    codes = [torch.zeros(1, 1, 3, 128, dtype=torch.uint8, device="cuda") for _ in range(2)]
    exps = [torch.zeros(1, 1, 3, dtype=torch.uint8, device="cuda") for _ in range(2)]
    ab.attn_cache_append_q8(k.cuda(), k.cuda(), *[c.view(torch.float8_e4m3fn) for c in codes],
                            *exps, torch.tensor([3], dtype=torch.int32, device="cuda"))
    dev_ok()
    finite = k.clone()
    finite[0, 0, 0, 5] = finite[0, 0, 0, 6] = finite[0, 0, 1, 7] = 0.0
    want, e, _ = quantise(finite)
    want[0, 0, 0, 5], want[0, 0, 0, 6], want[0, 0, 1, 7] = 0x7E, 0xFE, 0x7F
    for i in range(2):
        assert np.array_equal(exps[i].cpu().numpy(), e)
        got = codes[i].cpu().numpy()
        got[0, 0, 1, 7] &= 0x7F  # NaN's sign is free
        assert np.array_equal(got, want)


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"s{c[0]}_ln{c[3]}_d{c[5]}_p{c[6]}_{c[7]}")
def test_read_back_is_exact_and_leaves_the_rest(case):
    seed, B, Hkv, _, Lk, d, page, kind = case
    g = np.random.default_rng(seed + 50)
    lens = g.integers(0, Lk + 1, B).astype(np.int32)
    Lout = -(-Lk // page) * page if page else Lk
    if page:
        per_seq = Lout // page
        num_pages = B * per_seq + 1
        table = random_table(seed, B, per_seq, num_pages)
    want, args = [], []
    for x in (rows(seed, (B, Hkv, Lk, d), kind), rows(seed + 1, (B, Hkv, Lk, d), kind)):
        code, e, val = quantise(x)
        w = torch.full((B, Hkv, Lout, d), 7.0, dtype=torch.bfloat16)
        for b in range(B):
            # exact in bf16 down to its subnormals, where torch rounds as the kernel must
            w[b, :, :lens[b]] = torch.from_numpy(val[b, :, :lens[b]]).to(torch.bfloat16)
            code[b, :, lens[b]:], e[b, :, lens[b]:] = 0x7F, 255  # NaN past the end
        want.append(w)
        if page:
            code = to_pages(code, table, num_pages, page)
            e = to_pages(e, table, num_pages, page)
        args.append((as_codes(code).cuda(), torch.from_numpy(e).cuda()))
    out = [torch.full((B, Hkv, Lout, d), 7.0, dtype=torch.bfloat16, device="cuda")
           for _ in range(2)]
    flat = (args[0][0], args[1][0], args[0][1], args[1][1])
    kv = torch.from_numpy(lens).cuda()
    if page:
        ab.attn_cache_read_paged_q8(*flat, torch.from_numpy(table).cuda(), kv, k=out[0], v=out[1])
    else:
        ab.attn_cache_read_q8(*flat, kv, k=out[0], v=out[1])
    dev_ok()
    for got, w in zip(out, want):
        assert torch.equal(got.cpu().view(torch.int16), w.view(torch.int16))


@pytest.mark.parametrize("d", [64, 128])
def test_nan_codes_read_back_as_nan(d):
    code, e, val = quantise(rows(13, (1, 1, 5, d)))
    code[0, 0, 2, 7], code[0, 0, 2, d - 1], code[0, 0, 4, 0] = 0x7F, 0xFF, 0x7F
    want = torch.from_numpy(val).to(torch.bfloat16)
    want[0, 0, 2, 7] = want[0, 0, 2, d - 1] = want[0, 0, 4, 0] = math.nan
    c, x = as_codes(code).cuda(), torch.from_numpy(e).cuda()
    k, v = ab.attn_cache_read_q8(c, c, x, x, torch.tensor([5], dtype=torch.int32, device="cuda"))
    dev_ok()
    for got in (k, v):
        assert torch.equal(got.cpu().isnan(), want.isnan())
        assert torch.equal(got.cpu().nan_to_num(0.0), want.nan_to_num(0.0))


def test_more_pairs_than_a_grid_dimension_holds():
    """70,000 (sequence, head) pairs of one key each: written, and read back."""
    B, d = 70000, 64
    k = rows(14, (B, 1, 1, d))
    code, e, val = quantise(k)
    cv = [torch.zeros(B, 1, 1, d, dtype=torch.uint8, device="cuda") for _ in "kv"]
    ex = [torch.zeros(B, 1, 1, dtype=torch.uint8, device="cuda") for _ in "kv"]
    kv = torch.ones(B, dtype=torch.int32, device="cuda")
    args = [c.view(torch.float8_e4m3fn) for c in cv] + ex
    ab.attn_cache_append_q8(k.cuda(), k.cuda(), *args, kv)
    kr, vr = ab.attn_cache_read_q8(*args, kv)
    dev_ok()
    assert np.array_equal(cv[0].cpu().numpy(), code) and np.array_equal(ex[1].cpu().numpy(), e)
    assert np.array_equal(kr.cpu().double().numpy(), val) and torch.equal(kr, vr)


def test_out_of_range_lengths_and_pages_are_skipped_and_flagged():
    B, Hkv, Ln, Lk, d = 4, 2, 3, 16, 64
    k = rows(21, (B, Hkv, Ln, d)).cuda()
    cases = [([16, 17, 2, 8], None), ([16, -1, 5, 8], None), ([16, 8, 8, 8], [3, 4, -1, 3])]
    for lens, new in cases:
        codes = [torch.full((B, Hkv, Lk, d), GUARD, dtype=torch.uint8, device="cuda")
                 for _ in range(2)]
        exps = [torch.full((B, Hkv, Lk), GUARD, dtype=torch.uint8, device="cuda")
                for _ in range(2)]
        nl = None if new is None else torch.tensor(new, dtype=torch.int32, device="cuda")
        ab.attn_cache_append_q8(k, k, *[c.view(torch.float8_e4m3fn) for c in codes], *exps,
                                torch.tensor(lens, dtype=torch.int32, device="cuda"), new_lens=nl)
        torch.cuda.synchronize()
        st, _ = ab.attn_get_device_error()
        assert st == ab.ATTN_ERR_INVALID_ARG
        for b in range(B):
            n = Ln if new is None else new[b]
            bad = not (0 <= n <= Ln and n <= lens[b] <= Lk)
            assert bool((exps[0][b] == GUARD).all()) == bad, (lens, new, b)
    # a page id outside the pool: its rows are not written (append) or read as zeros (read)
    pages = [torch.full((2, Hkv, 16, d), GUARD, dtype=torch.uint8, device="cuda") for _ in "kv"]
    exps = [torch.full((2, Hkv, 16), GUARD, dtype=torch.uint8, device="cuda") for _ in "kv"]
    table = torch.tensor([[0, 2], [-1, 1]], dtype=torch.int32, device="cuda")
    kv = torch.tensor([18, 17], dtype=torch.int32, device="cuda")
    cv = [c.view(torch.float8_e4m3fn) for c in pages]
    ab.attn_cache_append_paged_q8(k[:2].contiguous(), k[:2].contiguous(), *cv, *exps, table, kv)
    torch.cuda.synchronize()
    st, _ = ab.attn_get_device_error()
    assert st == ab.ATTN_ERR_INVALID_ARG
    written = (exps[0] != GUARD).cpu().numpy()
    want = np.zeros((2, Hkv, 16), bool)
    want[0, :, 15] = True   # sequence 0: position 15 in page 0; 16 and 17 are in page 2 (bad)
    want[1, :, 0] = True    # sequence 1: 14 and 15 in page -1 (bad); 16 in page 1
    assert np.array_equal(written, want)
    kr, _ = ab.attn_cache_read_paged_q8(*cv, *exps, table, kv)
    torch.cuda.synchronize()
    st, _ = ab.attn_get_device_error()
    assert st == ab.ATTN_ERR_INVALID_ARG
    assert bool((kr[0, :, 16:18] == 0).all()) and bool((kr[1, :, :16] == 0).all())


def test_append_and_read_in_a_captured_graph_on_a_side_stream():
    """Captured once and replayed with new contents: the replay sees the new rows and lengths."""
    B, Hkv, Lk, d = 3, 2, 64, 128
    codes = [torch.zeros(B, Hkv, Lk, d, dtype=torch.uint8, device="cuda") for _ in "kv"]
    cv = [c.view(torch.float8_e4m3fn) for c in codes]
    exps = [torch.ones(B, Hkv, Lk, dtype=torch.uint8, device="cuda") for _ in "kv"]
    k = torch.zeros(B, Hkv, 1, d, dtype=torch.bfloat16, device="cuda")
    kv = torch.ones(B, dtype=torch.int32, device="cuda")
    out = [torch.zeros(B, Hkv, Lk, d, dtype=torch.bfloat16, device="cuda") for _ in "kv"]

    def step():
        ab.attn_cache_append_q8(k, k, *cv, *exps, kv)
        ab.attn_cache_read_q8(*cv, *exps, kv, k=out[0], v=out[1])

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    want = torch.zeros(B, Hkv, Lk, d, dtype=torch.float64)
    for pos in range(5):
        x = rows(30 + pos, (B, Hkv, 1, d))
        k.copy_(x)
        kv.fill_(pos + 1)
        graph.replay()
        want[:, :, pos] = torch.from_numpy(quantise(x)[2])[:, :, 0]
    dev_ok()
    assert torch.equal(out[0][:, :, :5].cpu().double(), want[:, :, :5])
    assert torch.equal(out[0], out[1])
