"""The 8-bit cache's entry points without a GPU: host-side rejection in the C ABI and
in the Python binding, and the format's reference (tests/q8_helpers.py) itself."""
import ctypes

import numpy as np
import pytest
import torch

import sm_attn_fwd_b200 as ab
from tests.q8_helpers import VALUES, quantise, round_e4m3

A = ctypes.c_void_p(0x10000)   # fake, aligned: rejected calls never touch it
M = ctypes.c_void_p(0x10008)   # not 16-byte aligned


def test_the_references_codes_are_torchs():
    """Every value table entry and every rounding of the numpy reference equals torch's
    float8_e4m3fn, on all e4m3 values, all midpoints between them and random values."""
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert np.array_equal(codes.double().numpy(), VALUES)
    y = np.concatenate([VALUES, (VALUES[1:] + VALUES[:-1]) / 2,
                        np.random.default_rng(0).uniform(0, 448, 5000)])
    y = np.concatenate([y, -y])
    _, c = round_e4m3(y)
    t = torch.from_numpy(y).to(torch.float32).to(torch.float64).numpy()
    keep = t == y  # torch rounds from fp32
    want = torch.from_numpy(y).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert keep.sum() > 500 and np.array_equal(c[keep], want[keep])


def test_scale_bytes_of_known_rows():
    x = torch.tensor([[448.0, 0], [450.0, 0], [1.75, 0], [1.7578125, 1], [0, 0], [2.0 ** -133, 0]])
    _, e, val = quantise(x.to(torch.bfloat16))
    assert e.tolist() == [127, 128, 119, 120, 1, 1]
    assert val[0, 0] == 448.0 and val[2, 0] == 1.75 and val[5, 0] == 2.0 ** -133


def _append(paged=False, **kw):
    a = dict(k=A, v=A, kc=A, vc=A, ke=A, ve=A, table=A, kv=A, new=None, B=2, Hkv=2, Ln=3, Lk=64,
             page=16, per=4, n=8, d=128)
    a.update(kw)
    lib = ab.load_library()
    head = (a["k"], a["v"], a["kc"], a["vc"], a["ke"], a["ve"])
    if paged:
        return lib.attn_cache_append_paged_q8(*head, a["table"], a["kv"], a["new"], a["B"],
                                              a["Hkv"], a["Ln"], a["page"], a["per"], a["n"],
                                              a["d"], None)
    return lib.attn_cache_append_q8(*head, a["kv"], a["new"], a["B"], a["Hkv"], a["Ln"], a["Lk"],
                                    a["d"], None)


def _read(paged=False, **kw):
    a = dict(k=A, v=A, kc=A, vc=A, ke=A, ve=A, table=A, kv=A, B=2, Hkv=2, Lk=64, page=16, per=4,
             n=8, d=128)
    a.update(kw)
    lib = ab.load_library()
    head = (a["kc"], a["vc"], a["ke"], a["ve"])
    if paged:
        return lib.attn_cache_read_paged_q8(*head, a["table"], a["kv"], a["k"], a["v"], a["B"],
                                            a["Hkv"], a["page"], a["per"], a["n"], a["d"], None)
    return lib.attn_cache_read_q8(*head, a["kv"], a["k"], a["v"], a["B"], a["Hkv"], a["Lk"],
                                  a["d"], None)


def _decode(paged=False, **kw):
    a = dict(q=A, kc=A, vc=A, ke=A, ve=A, table=A, o=A, lse=A, kv=A, B=2, Hq=16, Hkv=2, Lq=1,
             Lk=1024, page=16, per=64, n=128, d=128, scale=0.1, ns=0, ws=ctypes.c_void_p(0x100000),
             wsb=1 << 30)
    a.update(kw)
    lib = ab.load_library()
    head = (a["q"], a["kc"], a["vc"], a["ke"], a["ve"])
    tail = (a["d"], a["scale"], a["ns"], a["ws"], a["wsb"], None)
    if paged:
        return lib.attn_decode_paged_q8(*head, a["table"], a["o"], a["lse"], a["kv"], a["B"],
                                        a["Hq"], a["Hkv"], a["Lq"], a["page"], a["per"], a["n"],
                                        *tail)
    return lib.attn_decode_splitkv_q8(*head, a["o"], a["lse"], a["kv"], a["B"], a["Hq"], a["Hkv"],
                                      a["Lq"], a["Lk"], *tail)


INV, UNS, WSP = ab.ATTN_ERR_INVALID_ARG, ab.ATTN_ERR_UNSUPPORTED, ab.ATTN_ERR_WORKSPACE
BAD_PAGES = [(dict(table=None), INV), (dict(table=ctypes.c_void_p(0x10002)), INV),
             (dict(page=24), INV), (dict(page=8), INV), (dict(page=1 << 17), INV),
             (dict(per=0), INV), (dict(n=0), INV), (dict(page=65536, per=32768), UNS),
             (dict(n=1 << 30, Hkv=4, Hq=16), UNS)]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INV), (dict(v=None), INV), (dict(kc=None), INV), (dict(ve=None), INV),
    (dict(kv=None), INV), (dict(k=M), INV), (dict(vc=M), INV), (dict(kv=ctypes.c_void_p(0x10002)), INV),
    (dict(new=ctypes.c_void_p(0x10002)), INV), (dict(B=0), INV), (dict(Hkv=0), INV),
    (dict(Ln=0), INV), (dict(d=96), UNS), (dict(d=256), UNS),
    (dict(B=1 << 15, Hkv=1 << 8, Ln=1 << 8, n=8), UNS)])
def test_append_rejects_on_host(paged, kw, status):
    assert _append(paged, **kw) == status


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INV), (dict(kc=None), INV), (dict(ke=None), INV), (dict(v=M), INV),
    (dict(B=-1), INV), (dict(d=80), UNS), (dict(B=1 << 16, Hkv=1 << 10, n=8), UNS)])
def test_read_rejects_on_host(paged, kw, status):
    assert _read(paged, **kw) == status


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INV), (dict(o=M), INV), (dict(ke=None), INV), (dict(lse=None), INV),
    (dict(Hq=15), INV), (dict(Lq=0), INV), (dict(B=0), INV), (dict(scale=0.0), INV),
    (dict(scale=float("inf")), INV), (dict(ns=-1), INV), (dict(ns=4097), INV), (dict(d=96), UNS), (dict(ws=None), WSP),
    (dict(wsb=64), WSP), (dict(ws=ctypes.c_void_p(0x100010)), WSP)])
def test_decode_rejects_on_host(paged, kw, status):
    assert _decode(paged, **kw) == status


@pytest.mark.parametrize("call", [_append, _read, _decode])
@pytest.mark.parametrize("kw,status", BAD_PAGES)
def test_bad_pages_are_rejected_on_host(call, kw, status):
    assert call(True, **kw) == status


def test_lengths_of_a_contiguous_cache():
    assert _append(Lk=0) == INV and _read(Lk=0) == INV and _decode(Lk=0) == INV
    assert _decode(Lk=0x7fffffff) == UNS
    assert _append(B=1, Hkv=1, Ln=0x7fffffff) == UNS and _read(B=1, Hkv=1, Lk=0x7ffffff0) == UNS
    # more (sequence, head) pairs times key tiles than the 32-bit line of work holds
    assert _decode(B=1 << 20, Hq=16, Hkv=16, Lk=1 << 30) == UNS


def test_decode_workspace_holds_two_partials_per_cta():
    for d, rows, tile in ((128, 8, 8), (128, 9, 16), (128, 17, 128), (64, 17, 32), (64, 33, 128),
                          (128, 300, 128), (64, 1, 8)):
        for ctas in (1, 7, 148):
            part = 2 * ctas * tile
            want = (part * d * 4 + 255) // 256 * 256 + part * 4
            assert ab.attn_decode_q8_workspace_size(rows, 1, 1, d, ctas) == want
    assert ab.load_library().attn_decode_q8_workspace_size(8, 3, 1, 128, 0) == 0
    with pytest.raises(ab.AttnError):
        ab.attn_decode_q8_workspace_size(8, 1, 1, 128, -1)
    need = ab.attn_decode_q8_workspace_size(16, 2, 1, 128, 5)
    assert _decode(ns=5, wsb=need - 1) == WSP


def test_binding_rejects_host_tensors_and_missing_tables():
    k = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    c = torch.zeros(1, 2, 8, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    e = torch.zeros(1, 2, 8, dtype=torch.uint8)
    kv = torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ab.attn_cache_append_q8(k, k, c, c, e, e, kv)
    with pytest.raises(ValueError, match="CUDA"):
        ab.attn_cache_read_q8(c, c, e, e, kv)
    with pytest.raises(ValueError, match="CUDA"):
        ab.attn_decode_splitkv_q8(k, c, c, e, e, kv)
    for call in (lambda t: ab.attn_cache_append_paged_q8(k, k, c, c, e, e, t, kv),
                 lambda t: ab.attn_cache_read_paged_q8(c, c, e, e, t, kv),
                 lambda t: ab.attn_decode_paged_q8(k, c, c, e, e, t, kv)):
        with pytest.raises(ValueError, match="block_table"):
            call(None)


@pytest.mark.gpu
def test_binding_rejects_wrong_shapes_types_and_strides():
    dev = "cuda"
    k = torch.zeros(2, 2, 1, 64, dtype=torch.bfloat16, device=dev)
    q = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device=dev)
    c = torch.zeros(2, 2, 16, 64, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
    e = torch.zeros(2, 2, 16, dtype=torch.uint8, device=dev)
    kv = torch.ones(2, dtype=torch.int32, device=dev)
    wide = torch.zeros(2, 2, 16, 128, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
    table = torch.zeros(2, 1, dtype=torch.int32, device=dev)
    bad = [
        lambda: ab.attn_cache_append_q8(k, k, c, c, e, e, kv[:1]),
        lambda: ab.attn_cache_append_q8(k, k, c, c, e, e, kv.long()),
        lambda: ab.attn_cache_append_q8(k, k, c, c, e, e[:, :, :8], kv),
        lambda: ab.attn_cache_append_q8(k, k, c, wide[..., :64], e, e, kv),
        lambda: ab.attn_cache_append_q8(k.half(), k, c, c, e, e, kv),
        lambda: ab.attn_cache_append_q8(k[:1], k, c, c, e, e, kv),
        lambda: ab.attn_cache_append_q8(k, k, c.view(torch.uint8), c, e, e, kv),
        lambda: ab.attn_cache_append_q8(k, k, c, c, e, e, kv, new_lens=kv[:1]),
        lambda: ab.attn_cache_append_paged_q8(k, k, c, c, e, e, table.long(), kv),
        lambda: ab.attn_cache_append_paged_q8(k, k, c, c, e, e, table[:1], kv),
        lambda: ab.attn_cache_read_q8(c, c, e, e, kv, k=k, v=k),
        lambda: ab.attn_cache_read_q8(c, c, e.int(), e, kv),
        lambda: ab.attn_decode_splitkv_q8(q[:1], c, c, e, e, kv),
        lambda: ab.attn_decode_splitkv_q8(q, wide, wide, e, e, kv),
        lambda: ab.attn_decode_splitkv_q8(q, c, c, e, e, kv, o=q.float()),
        lambda: ab.attn_decode_splitkv_q8(q, c, c, e, e, kv, lse=kv.float()),
        lambda: ab.attn_decode_paged_q8(q, c, c, e, e, kv, kv),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"case {i} was accepted")
    with pytest.raises(ab.AttnError):   # 3 query heads over 2 KV heads
        ab.attn_decode_splitkv_q8(q[:, :3].contiguous(), c, c, e, e, kv)
    torch.cuda.synchronize()
    assert ab.attn_get_device_error()[0] == ab.ATTN_OK
