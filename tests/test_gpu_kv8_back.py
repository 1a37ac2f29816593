"""Rows of the 8-bit cache that go back and continue, as rv.h allows it: to any
multiple of `block`, and elsewhere to at most `block` positions below the
highest end that the row has reached since the first token of that block was
last written."""
import random

import pytest
import torch

from test_gpu_kv8 import Cache, check_cache, data

pytestmark = pytest.mark.gpu


def legal(block, length, ends, p):
    """ends[q]: the highest end reached since position q was last written."""
    return p <= length and (p % block == 0 or p >= ends[p // block * block] - block)


@pytest.mark.parametrize("block,hd,fmt,act", [(16, 64, 0, 1), (32, 128, 1, 0), (64, 64, 0, 0)])
def test_rows_go_back_as_far_as_they_may(block, hd, fmt, act):
    rng = random.Random(block)
    Hkv, N, pool = 2, 6 * block, 40 * block
    k, v = data(61, 1, pool, Hkv, hd, act), data(62, 1, pool, Hkv, hd, act)
    c = Cache(1, Hkv, hd, N, block, fmt, act)
    row, ends, back = [], {}, 0
    for step in range(60):
        p = len(row)
        if row and rng.random() < 0.6:  # the farthest legal place, or any other
            ok = [x for x in range(len(row)) if legal(block, len(row), ends, x)]
            odd = [x for x in ok if x % block]
            p = rng.choice([ok[0], odd[0] if odd else ok[0], rng.choice(ok)])
            back += 1
        n = min(rng.choice([1, 1, 3, block - 1, block + 2, 3 * block]), N - p)
        if n < 1:
            p, n = 0, 5
        at = rng.randrange(pool - n)
        c.append(k[:, at:at + n].contiguous(), v[:, at:at + n].contiguous(), [p])
        row = row[:p] + list(range(at, at + n))
        for q in range(p, p + n):
            ends[q] = 0
        for q in ends:
            ends[q] = max(ends[q], p + n)
        check_cache(c, k[:, row], v[:, row], [len(row)])
    assert back > 20 and int(c.err) == 0
