"""The 8-bit cache format in plain numpy float64, for the tests.

A row's scale byte e is the smallest integer >= 1 with max|x| <= 448 * 2^(e - 127);
its codes are the e4m3 values nearest to x * 2^(127 - e), ties to even.  Written
from the definition: e4m3 values as numbers, no bit tricks.
"""
import numpy as np
import torch


def e4m3_values():
    """Every non-negative finite e4m3 value in ascending order (code i is entry i)."""
    v = [m * 2.0 ** -9 for m in range(8)]
    v += [(1 + m / 8.0) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return np.array(v[:-1])  # the last is NaN's code


VALUES = e4m3_values()


def round_e4m3(y):
    """(signed e4m3 values, codes) nearest to y (|y| <= 448), ties to the even code."""
    a = np.abs(y)
    hi = np.searchsorted(VALUES, a)                 # first value >= a
    hi = np.minimum(hi, len(VALUES) - 1)
    lo = np.maximum(hi - 1, 0)
    d_hi, d_lo = VALUES[hi] - a, a - VALUES[lo]
    pick = np.where(d_hi < d_lo, hi, np.where(d_lo < d_hi, lo, np.where(hi % 2 == 0, hi, lo)))
    pick = np.where(VALUES[hi] == a, hi, pick)
    sign = np.signbit(y)
    return np.where(sign, -VALUES[pick], VALUES[pick]), (pick | (sign << 7)).astype(np.uint8)


def quantise(x):
    """bf16 tensor [..., d] -> (codes uint8, scale bytes uint8, values float64)."""
    x = x.float().cpu().double().numpy()
    top = np.abs(x).max(-1)
    e = np.ones(top.shape, dtype=np.int64)
    for byte in range(2, 255):                      # smallest byte that holds the row
        e = np.where(top > 448.0 * 2.0 ** (byte - 1 - 127), byte, e)
    s = 2.0 ** (e - 127.0)
    val, code = round_e4m3(x / s[..., None])
    return code, e.astype(np.uint8), val * s[..., None]


def as_codes(code):
    return torch.from_numpy(code).view(torch.float8_e4m3fn)


def to_pages(x, table, num_pages, page, fill=0):
    """A cache [B, Hkv, L, ...] (numpy) laid out in pages [num_pages, Hkv, page, ...]."""
    B, H, L = x.shape[:3]
    pool = np.full((num_pages, H, page) + x.shape[3:], fill, dtype=x.dtype)
    for b in range(B):
        for j in range(L):
            pool[table[b, j // page], :, j % page] = x[b, :, j]
    return pool


def random_table(seed, B, pages_per_seq, num_pages):
    rng = np.random.default_rng(seed)
    return rng.permutation(num_pages)[:B * pages_per_seq].reshape(B, pages_per_seq).astype(np.int32)
