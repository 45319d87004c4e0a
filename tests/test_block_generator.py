"""The dropout reference's generator against the known answers that the authors of Philox4x32-10
publish with it (Salmon, Moraes, Dror, Shaw, SC 2011), for counters and keys that are not zero."""
import pytest

import block_reference as ref

ONES = 0xFFFFFFFF


def _block(counter, key):
    """Ten rounds on four counter words with two key words."""
    c, k = list(counter), list(key)
    for _ in range(10):
        p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(q >> 32) ^ c[1] ^ k[0], q & ONES, (p >> 32) ^ c[3] ^ k[1], p & ONES]
        k = [(k[0] + 0x9E3779B9) & ONES, (k[1] + 0xBB67AE85) & ONES]
    return c


@pytest.mark.parametrize("counter,key,words", [
    ((0,) * 4, (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((ONES,) * 4, (ONES, ONES), (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_known_answers(counter, key, words):
    assert tuple(_block(counter, key)) == words


@pytest.mark.parametrize("seed,offset", [(0, 0), (0xDEADBEEF12345678, (1 << 40) + 17),
                                         ((1 << 64) - 1, (1 << 64) - 1), (1 << 32, 1 << 33)])
def test_words_are_those_of_consecutive_counters(seed, offset):
    want = []
    for i in range(9):
        want += _block((i, 0, offset & ONES, offset >> 32), (seed & ONES, seed >> 32))
    assert ref.philox_words(35, seed, offset) == want[:35]
