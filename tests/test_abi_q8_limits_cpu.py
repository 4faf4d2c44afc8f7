"""Sizes of append and read-back at the limit of their 32-bit counters, refused on the host.

The grid holds (sequence, head) pairs as y * z with y = min(pairs, 65535), so the last
block's number is up to ceil(pairs / 65535) * 65535 - 1, which must fit as well."""
import pytest

import sm_attn_fwd_b200 as ab
from tests.test_abi_q8_cpu import _append, _read

UNS = ab.ATTN_ERR_UNSUPPORTED
LIMIT = 2 ** 31 - 1 - 65535


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("rows", [LIMIT + 1, 32768 * 65535 + 1, 2 ** 31 - 4097, 2 ** 31 - 1])
def test_too_many_pairs(paged, rows):
    assert _append(paged, B=rows, Hkv=1, Ln=1) == UNS
    if not paged:
        assert _read(B=rows, Hkv=1, Lk=1) == UNS


def test_the_limit_keeps_every_block_number_in_32_bits():
    for pairs in (1, 65535, 65536, LIMIT - 65535, LIMIT):
        y = min(pairs, 65535)
        assert -(-pairs // y) * y - 1 <= 2 ** 31 - 1 and -(-pairs // y) <= 65535
