"""Rows of the 8-bit cache copied to rows: every byte, and no other."""
import numpy as np
import pytest
import torch

import token_level_early_gb300 as rv
from answers_util import copy_rows
from test_gpu_kv8 import Cache, check_cache, data

pytestmark = pytest.mark.gpu


def bits(t):
    return t.view(torch.uint8 if t.dtype == torch.uint8 else torch.int16 if t.element_size() == 2 else torch.int32).cpu().numpy()


def random_cache(seed, rows, Hkv, hd, max_seq, block, fmt=0, act=1):
    c = Cache(rows, Hkv, hd, max_seq, block, fmt, act)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for t in c.codes + c.scale + c.tail:
        t.view(torch.uint8).random_(0, 256, generator=g)
    return c


def run(src, dst, pairs, length=True, stream=None):
    f, t, n = (torch.tensor([p[i] for p in pairs], dtype=torch.int32).cuda() for i in range(3))
    torch.cuda.synchronize()
    rv.kv8_copy(src.c, dst.c, len(pairs), f.data_ptr(), t.data_ptr(), n.data_ptr() if length else None, dst.err.data_ptr(), stream)
    torch.cuda.synchronize()


def check(src, dst, pairs, length=True):
    """Runs the copy and compares the whole destination."""
    most = min(src.T, dst.T)
    use = [(a, b, min(max(m, 0), most) if length else most) for a, b, m in pairs]
    ref = [copy_rows(bits(x), bits(y), use, per) for kind, per in (("codes", 1), ("scale", dst.block), ("tail", None))
           for x, y in zip(getattr(src, kind), getattr(dst, kind))]
    run(src, dst, pairs, length)
    for r, t in zip(ref, dst.codes + dst.scale + dst.tail):
        assert np.array_equal(r, bits(t))


@pytest.mark.parametrize("hd,block,Hkv", [(64, 16, 1), (128, 64, 2), (64, 128, 3), (128, 32, 1)])
@pytest.mark.parametrize("rows,pairs", [
    (2, [(0, 1, 1)]), (2, [(1, 0, 130)]), (4, [(0, 1, 300), (0, 2, 300), (0, 3, 299)]), (4, [(0, 1, 70), (1, 0, 64), (3, 2, 0), (2, 3, 65)]),
    (5, [(0, 1, 9), (1, 2, 200), (2, 3, 17), (3, 4, 300), (4, 0, 299)]), (3, [(0, 0, 20), (1, 1, 300)]),
    (4, [(0, 1, 300), (2, 1, 20), (3, 1, 128)]), (4, [(-1, 2, 50), (1, -2, 50), (0, 3, 63)])])
def test_copy_in_place(rows, pairs, hd, block, Hkv):
    """Forks, exchanges, cycles, rows onto themselves, one destination several
    times (the last counts), unused pairs."""
    c = random_cache(1, rows, Hkv, hd, 300, block)
    check(c, c, pairs)
    assert int(c.err) == 0


@pytest.mark.parametrize("fmt,act", [(0, 0), (1, 1)])
def test_copy_between_caches_of_different_lengths(fmt, act):
    src, dst = random_cache(2, 3, 2, 64, 200, 32, fmt, act), random_cache(3, 5, 2, 64, 777, 32, fmt, act)
    check(src, dst, [(2, 0, 200), (0, 4, 1), (2, 2, 33)])
    check(dst, src, [(4, 1, 200), (3, 0, 160)])
    check(src, dst, [(0, 1, 0), (1, 3, 0)], length=False)  # as many as both hold
    assert int(src.err) == 0 and int(dst.err) == 0


def test_copy_reports_rows_and_lengths_that_are_too_large():
    c = random_cache(4, 3, 1, 64, 100, 16)
    for pairs in ([(3, 0, 10), (1, 2, 10)], [(0, 7, 10), (1, 2, 10)], [(0, 1, 101)], [(0, 2, 2 ** 31 - 1)]):
        check(c, c, pairs)
        assert int(c.err) == 64
        c.err.zero_()
    check(c, c, [(0, 1, -5)])
    assert int(c.err) == 0


@pytest.mark.parametrize("n", [63, 64, 200, 1024])
def test_copy_many_pairs(n):
    """A random map of rows onto rows in place, some sources many times."""
    c = random_cache(n, n, 1, 64, 40, 16)
    rng = np.random.default_rng(n)
    to = rng.permutation(n)
    pairs = [(int(rng.integers(0, n if i % 3 else 5)), int(b), int(rng.integers(0, 41))) for i, b in enumerate(to)]
    check(c, c, pairs)


def test_copy_many_duplicates():
    c = random_cache(5, 40, 2, 64, 70, 16)
    rng = np.random.default_rng(5)
    check(c, c, [(int(rng.integers(-2, 40)), int(rng.integers(-2, 40)), int(rng.integers(0, 71))) for _ in range(300)])


def test_copy_long_rows():
    """Many items a block: codes whose byte offsets go far, and all heads."""
    c = random_cache(6, 3, 4, 128, 20011, 64)
    check(c, c, [(0, 2, 20011), (2, 0, 19999)])


@pytest.mark.parametrize("n", [1, 3, 5, 48])
def test_copy_rows_with_many_scales(n):
    """Several items of scales a head, the last of them short, rows that change places."""
    c = random_cache(8, n + 1, 1, 64, 20011 if n < 48 else 3011, 16)
    rng = np.random.default_rng(n)
    to = rng.permutation(n + 1)
    check(c, c, [(i, int(to[i]), int(rng.integers(c.T // 2, c.T + 1))) for i in range(n)])


def test_a_fork_is_continued_as_the_source_could_be():
    """Fork inside a block, append different tokens to each: both hold what they
    were given, the open block quantised anew from the tail."""
    B, Hkv, hd, block, act, n = 3, 2, 64, 16, 1, 37
    k, v = data(1, 1, n, Hkv, hd, act), data(2, 1, n, Hkv, hd, act)
    more_k, more_v = data(3, B, 21, Hkv, hd, act), data(4, B, 21, Hkv, hd, act)
    c = Cache(B, Hkv, hd, 64, block, 0, act)
    c.append(k, v, [0])
    back = n - 3  # forked three tokens before the source's end
    run(c, c, [(0, 1, n), (0, 2, back)])
    c.append(more_k, more_v, [n, n, back])
    kk, vv = (torch.zeros(B, 64, Hkv, hd, dtype=torch.bfloat16).cuda() for _ in range(2))
    for b, m in enumerate((n, n, back)):
        for full, old, new in ((kk, k, more_k), (vv, v, more_v)):
            full[b, :m], full[b, m:m + 21] = old[0, :m], new[b]
    check_cache(c, kk, vv, [n + 21, n + 21, back + 21])


def test_copy_captured_and_replayed():
    """A graph of two copies, with other rows and lengths at its replay."""
    c = random_cache(7, 6, 2, 128, 500, 32)
    f, t, n = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([0, 1], [2, 3], [500, 500]))
    start = [x.clone() for x in c.codes + c.scale + c.tail]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        for _ in range(2):
            rv.kv8_copy(c.c, c.c, 2, f.data_ptr(), t.data_ptr(), n.data_ptr(), c.err.data_ptr(), torch.cuda.current_stream().cuda_stream)
    for a, b, m in (([0, 1], [1, 0], [300, 301]), ([5, 4], [4, 2], [17, 480])):
        for x, y in zip(c.codes + c.scale + c.tail, start):
            x.copy_(y)
        for x, v in ((f, a), (t, b), (n, m)):
            x.copy_(torch.tensor(v, dtype=torch.int32))
        ref = [bits(x) for x in c.codes + c.scale + c.tail]
        pairs = list(zip(a, b, m))
        for _ in range(2):
            ref = [copy_rows(r, r, pairs, per) for r, per in zip(ref, (1, 1, 32, 32, None, None))]
        graph.replay()
        torch.cuda.synchronize()
        for r, x in zip(ref, c.codes + c.scale + c.tail):
            assert np.array_equal(r, bits(x))
