"""The native part of the Python binding: memory it allocates for a call on another
stream than the current one, tensors and numbers it refuses, calls from two threads."""
import threading

import numpy as np
import pytest
import torch

import sm_attn_fwd_b200 as ab
from tests.q8_helpers import quantise

pytestmark = pytest.mark.gpu


def case(seed=5, B=3, Hq=4, Hkv=2, Lq=1, Lk=200, d=128):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(B, Hq, Lq, d, generator=g).to(torch.bfloat16).cuda()
    planes = []
    for _ in range(2):
        code, e, _ = quantise(torch.randn(B, Hkv, Lk, d, generator=g).to(torch.bfloat16))
        planes.append((torch.from_numpy(code).cuda().view(torch.float8_e4m3fn),
                       torch.from_numpy(e).cuda()))
    lens = torch.tensor([Lk, 7, 0], dtype=torch.int32, device="cuda")
    return q, planes[0][0], planes[1][0], planes[0][1], planes[1][1], lens


def test_memory_of_a_call_on_another_stream_is_not_handed_out_before_it_is_done():
    a = case()
    q = a[0]
    o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    need = ab.attn_decode_q8_workspace_size(4, 2, 1, 128)
    want, want_lse = ab.attn_decode_splitkv_q8(*a)
    torch.cuda.synchronize()

    def block():
        t = torch.empty(need, dtype=torch.uint8, device="cuda")
        return t.data_ptr()

    first = block()
    ab.attn_decode_splitkv_q8(*a, o=o, lse=lse)
    assert block() == first  # the workspace came from and went back to this block
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # about 0.1 s
    ab.attn_decode_splitkv_q8(*a, o=o, lse=lse, stream=side)
    assert not side.query()
    assert block() != first  # still in use by the sleeping stream
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, want_lse)


def test_a_call_on_another_stream_gives_the_same_bits():
    a = case()
    want = ab.attn_decode_splitkv_q8(*a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ab.attn_decode_splitkv_q8(*a, stream=side)
    k, v = ab.attn_cache_read_q8(*a[1:], stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    k2, v2 = ab.attn_cache_read_q8(*a[1:])
    torch.cuda.synchronize()
    for b, n in enumerate(a[5].tolist()):
        assert torch.equal(k[b, :, :n], k2[b, :, :n]) and torch.equal(v[b, :, :n], v2[b, :, :n])


def test_calls_from_two_threads_give_the_same_bits():
    a = case()
    want = ab.attn_decode_splitkv_q8(*a)
    torch.cuda.synchronize()
    bad = []

    def loop():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(50):
                o, lse = ab.attn_decode_splitkv_q8(*a)
                s.synchronize()
                if not (torch.equal(o, want[0]) and torch.equal(lse, want[1])):
                    bad.append(1)

    threads = [threading.Thread(target=loop) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_numbers_and_tensors_that_do_not_fit_are_refused():
    a = case()
    q, lens = a[0], a[5]
    dec = ab.attn_decode_splitkv_q8
    for kw in ({"num_ctas": 1 << 40}, {"num_ctas": "x"}, {"scale": "x"}, {"o": q[:, :, :, ::2]},
               {"o": q.float()}, {"lse": torch.empty(3, device="cuda")},
               {"workspace": torch.empty(1 << 20, dtype=torch.uint8)}, {"workspace": 7}):
        with pytest.raises(ValueError):
            dec(*a, **kw)
    for i, bad in ((0, q[:2]), (0, q[..., :64]), (0, None), (1, a[1].view(torch.uint8)),
                   (2, a[2][:, :, :100]), (3, a[3][:, :, :100]), (5, lens.long()),
                   (5, lens[:2]), (5, lens.cpu())):
        b = list(a)
        b[i] = bad
        with pytest.raises(ValueError):
            dec(*b)
    with pytest.raises(ab.AttnError):
        dec(*a, num_ctas=-1)
    with pytest.raises(ab.AttnError):
        dec(*a, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert ab.attn_get_device_error() == (ab.ATTN_OK, 0)
