"""Row copies between caches that have a part of their memory in common are
refused, before any GPU work.  The pointers are numbers that no call may
dereference."""
import pytest

import token_level_early_gb300 as rv
from test_ops_cpu import cache

NAMES = ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail")
B, HKV, HD, SEQ, BLOCK = 4, 8, 128, 1000, 64
N = -(-SEQ // BLOCK) * BLOCK
SIZE = dict(zip(NAMES, (B * HKV * N * HD,) * 2 + (B * HKV * (N // BLOCK) * 4,) * 2 + (B * HKV * 2 * BLOCK * HD * 2,) * 2))


def laid_out(start, **kw):
    """A cache whose six arrays lie one behind the other from `start` on, and where they end."""
    at, p = start, {}
    for name in NAMES:
        p[name] = at
        at += SIZE[name]
    return dict(p, **kw), at


def message(src, dst):
    with pytest.raises(rv.RVError) as e:  # (pointers that are no memory are refused later, with other words)
        rv.kv8_copy(cache(**src), cache(**dst), 1, 0x10000, 0x10000, None, None)
    return e.value.code, str(e.value)


def overlap(src, dst):
    code, text = message(src, dst)
    return code == rv.RV_EINVAL and "share" in text


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("row", [-3, -1, 1, 3])
def test_a_range_of_rows_inside_the_others_arrays(name, row):
    """One array of the source begins some rows behind (or before) the destination's."""
    dst, end = laid_out(1 << 30)
    src, _ = laid_out(end + (1 << 20))
    src[name] = dst[name] + row * (SIZE[name] // B)
    assert overlap(src, dst) and overlap(dst, src)


@pytest.mark.parametrize("one,two", [("k_codes", "v_codes"), ("v_tail", "k_scale"), ("k_scale", "v_codes")])
def test_different_arrays_over_each_other(one, two):
    dst, end = laid_out(1 << 30)
    src, _ = laid_out(end)
    src[one] = dst[two] + SIZE[two] - 16
    assert overlap(src, dst) and overlap(dst, src)


def test_all_arrays_a_row_on():
    """The descriptor of rows 1.. of a cache, against the cache."""
    dst, _ = laid_out(1 << 30)
    src = {n: p + SIZE[n] // B for n, p in dst.items()}
    assert overlap(dict(src, max_batch=B - 1), dst) and overlap(dst, dict(src, max_batch=B - 1))


def test_memory_side_by_side_and_one_cache_are_not_refused():
    """End to end, and two ranges of rows of the same arrays that do not meet."""
    dst, end = laid_out(1 << 30)
    src, _ = laid_out(end)
    assert not overlap(src, dst) and not overlap(dst, src) and not overlap(dst, dst)
    low, high = dict(dst, max_batch=1), {n: p + SIZE[n] // B for n, p in dst.items()}
    assert not overlap(low, dict(high, max_batch=B - 1)) and not overlap(dict(high, max_batch=B - 1), low)


def test_sizes_beyond_the_address_space():
    """A descriptor whose arrays would end behind the last address: counted without a wrap."""
    big, _ = laid_out(1 << 20, max_batch=65535, n_kv_heads=1024, max_seq=2 ** 31 - 257)
    small, _ = laid_out(1 << 40, n_kv_heads=1024)
    assert overlap(big, small) and overlap(small, big)
