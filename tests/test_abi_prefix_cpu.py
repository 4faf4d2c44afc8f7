"""The shared-prefix decode's entry points without a GPU: the plan, the workspace's
arithmetic and host-side rejection."""
import ctypes

import pytest

import sm_attn_fwd_b200 as ab

A = ctypes.c_void_p(0x10000)
M = ctypes.c_void_p(0x10008)
INV, UNS, WSP = ab.ATTN_ERR_INVALID_ARG, ab.ATTN_ERR_UNSUPPORTED, ab.ATTN_ERR_WORKSPACE


def call(paged=False, **kw):
    a = dict(q=A, kp=A, vp=A, pt=A, k=A, v=A, bt=A, o=A, lse=A, kv=A, B=4, Hq=16, Hkv=2, Lq=1,
             Lp=1000, Lk=64, page=16, per=4, n=64, d=128, scale=0.1, ns=0,
             ws=ctypes.c_void_p(0x100000), wsb=1 << 30)
    a.update(kw)
    lib = ab.load_library()
    tail = (a["d"], a["scale"], a["ns"], a["ws"], a["wsb"], None)
    if paged:
        return lib.attn_decode_shared_prefix_paged(
            a["q"], a["k"], a["v"], a["pt"], a["bt"], a["o"], a["lse"], a["kv"], a["B"], a["Hq"],
            a["Hkv"], a["Lq"], a["Lp"], a["page"], a["per"], a["n"], *tail)
    return lib.attn_decode_shared_prefix(a["q"], a["kp"], a["vp"], a["k"], a["v"], a["o"], a["lse"],
                                         a["kv"], a["B"], a["Hq"], a["Hkv"], a["Lq"], a["Lp"],
                                         a["Lk"], *tail)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=M), INV), (dict(o=None), INV),
    (dict(lse=ctypes.c_void_p(0x10002)), INV), (dict(kv=None), INV), (dict(B=0), INV),
    (dict(Hq=15), INV), (dict(Lq=0), INV), (dict(Lp=0), INV), (dict(ns=-1), INV),
    (dict(scale=0.0), INV), (dict(scale=float("nan")), INV), (dict(d=96), UNS), (dict(ws=None), WSP),
    (dict(ws=ctypes.c_void_p(0x100010)), WSP), (dict(wsb=1000), WSP)])
def test_rejects_on_host(paged, kw, status):
    assert call(paged, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(pt=None), INV), (dict(pt=ctypes.c_void_p(0x10002)), INV), (dict(bt=None), INV),
    (dict(page=24), INV), (dict(per=0), INV), (dict(n=0), INV), (dict(page=65536, per=32768), UNS)])
def test_paged_rejects_on_host(kw, status):
    assert call(True, **kw) == status


def test_contiguous_rejects_on_host():
    assert call(kp=None) == INV and call(vp=M) == INV and call(Lk=0) == INV
    assert call(Lp=0x7fffffff) == UNS and call(Lk=0x7fffffff) == UNS


def plan(*args):
    chunk = ctypes.c_int(0)
    n = ab.load_library().attn_decode_shared_prefix_num_splits(*args, ctypes.byref(chunk))
    return n, chunk.value


def test_split_plan_covers_the_prefix():
    for B, Hq, Hkv, Lq in ((1, 1, 1, 1), (4, 32, 8, 1), (64, 64, 8, 1), (64, 64, 8, 16),
                           (3, 6, 2, 50)):
        for Lp in (1, 127, 128, 129, 2064, 32768, 100001):
            for ns in (0, 1, 3, 1 << 20):
                for Lk, d in ((1, 128), (1000, 64), (1 << 20, 128)):
                    n, chunk = plan(B, Hq, Hkv, Lq, Lp, Lk, d, ns)
                    assert chunk % 128 == 0 and n * chunk >= Lp and (n - 1) * chunk < Lp
                    if ns:
                        assert n <= ns
    assert plan(4, 16, 2, 1, 1000, 100, 128, 3) == (3, 384)
    assert plan(4, 16, 2, 1, 1000, 100, 128, 100) == (8, 128)
    assert plan(0, 16, 2, 1, 1000, 9, 64, 0)[0] == -1
    assert plan(4, 15, 2, 1, 1000, 9, 64, 0)[0] == -1
    assert plan(4, 16, 2, 1, 0, 9, 64, 0)[0] == -1
    assert plan(4, 16, 2, 1, 10, 0, 64, 0)[0] == -1
    assert plan(4, 16, 2, 1, 10, 9, 64, -1)[0] == -1


def test_split_plan_leaves_sms_to_the_caches_where_that_is_planned():
    """A short prefix and short caches with few query rows: prefix CTAs on part of the
    SMs.  However long the caches may get, a prefix CTA's key tiles stay within 1.4 times
    the fewest (counted with 9 for what they do not change).  Many query rows: the caches
    go through another kernel, and the plan does not depend on them."""
    sms = 148
    if ab.torch.cuda.is_available():
        sms = ab.torch.cuda.get_device_properties(0).multi_processor_count
    n, chunk = plan(4, 32, 8, 1, 2064, 129, 128, 0)
    assert 8 * n <= sms * 2 // 3 and chunk >= 256
    fewest = plan(4, 32, 8, 1, 2064, 1, 128, 0)[1] // 128
    for Lk in (1, 129, 5000, 1 << 20):
        assert plan(4, 32, 8, 1, 2064, Lk, 128, 0)[1] // 128 + 9 <= 1.4 * (max(fewest, 1) + 9)
    assert plan(8, 64, 2, 4, 9000, 1, 128, 0) == plan(8, 64, 2, 4, 9000, 1 << 20, 128, 0)
    assert plan(2, 2147483646, 1073741823, 1, 100, 100, 128, 0)[0] >= -1  # no overflow


def test_workspace_holds_both_parts():
    """Few query rows per KV head: the prefix's splits, a row per output row and two
    partials per CTA; many: the prefix's splits and the decode's."""
    B, Hkv, Lp, Lk = 4, 2, 3000, 700
    for d, Hq, Lq, tile in ((64, 16, 2, 16), (128, 16, 1, 8), (64, 16, 4, 32), (128, 16, 4, 0),
                            (64, 32, 4, 0)):
        np_, _ = plan(B, Hq, Hkv, Lq, Lp, Lk, d, 5)
        ns, _ = ab.attn_decode_num_splits(B, Hq, Hkv, Lq, Lk, d)
        rows = B * Hq * Lq
        sms = 148  # without a device
        if ab.torch.cuda.is_available():
            sms = ab.torch.cuda.get_device_properties(0).multi_processor_count
        part = (np_ + 1) * rows + 2 * sms * tile if tile else (np_ + ns) * rows
        want = (part * d * 4 + 255) // 256 * 256 + part * 4
        assert ab.attn_decode_shared_prefix_workspace_size(B, Hq, Hkv, Lq, Lp, Lk, d, 5) == want
    with pytest.raises(ab.AttnError):
        ab.attn_decode_shared_prefix_workspace_size(B, 16, 3, 1, Lp, Lk, 64)


def test_binding_rejects_host_tensors():
    import torch
    q = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    p = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    k = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    kv = torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ab.attn_decode_shared_prefix(q, p, p, k, k, kv)
    with pytest.raises(ValueError, match="CUDA"):
        ab.attn_decode_shared_prefix_paged(q, k, k, kv, 8, kv.view(1, 1), kv)
