"""The Philox4x32-10 that the dropout tests take as their reference, against the
generator's published vectors (Salmon et al., 2011, known-answer file)."""
import random

import numpy as np
import pytest

VECTORS = [
    ((0,) * 4, (0,) * 2, (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
]


def _block(counter, key):
    """One block in Python integers, round by round."""
    c, k = list(counter), list(key)
    for _ in range(10):
        p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(q >> 32) ^ c[1] ^ k[0], q & 0xFFFFFFFF, (p >> 32) ^ c[3] ^ k[1], p & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return tuple(c)


@pytest.mark.parametrize("counter,key,words", VECTORS)
def test_published_vectors(counter, key, words):
    assert _block(counter, key) == words


def test_the_dropout_reference_is_that_generator():
    from .test_head_gpu import _philox
    rng = random.Random(1)
    for seed, offset, stream in ((2 ** 64 - 1, 2 ** 63 - 1, 1), (0, 0, 0),
                                 *((rng.getrandbits(64), rng.getrandbits(63), s) for s in (0, 1))):
        got = _philox(seed, offset, 5, stream)
        for i in range(5):
            want = _block((i, 0, offset & 0xFFFFFFFF, offset >> 32 | stream << 31), (seed & 0xFFFFFFFF, seed >> 32))
            assert tuple(int(v) for v in got[i].astype(np.uint64)) == want
