"""Row copies between two descriptors of one cache's arrays."""
import numpy as np
import pytest
import torch

import token_level_early_gb300 as rv
from answers_util import copy_rows
from test_gpu_kv8_copy import bits, random_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("up", [True, False])
def test_ranges_of_rows_that_do_not_meet(up):
    """Rows 0..1 and 2..4 of one cache as caches of their own, copied either way."""
    whole = random_cache(3, 5, 2, 64, 130, 32)
    arrays = whole.codes + whole.scale + whole.tail

    def part(first, rows):
        return rv.KV8(rows, 2, 64, 130, 32, 0, 1, *(t[first].data_ptr() for t in arrays))

    low, high, pairs = part(0, 2), part(2, 3), [(0, 1, 130), (1, 0, 77)]
    src, dst = (low, high) if up else (high, low)
    cut = (slice(0, 2), slice(2, 5)) if up else (slice(2, 5), slice(0, 2))
    want = []
    for i, t in enumerate(arrays):
        y = bits(t).copy()
        y[cut[1]] = copy_rows(y[cut[0]], y[cut[1]], pairs, (1, 1, 32, 32, None, None)[i])
        want.append(y)
    f, t, n = (torch.tensor([p[i] for p in pairs], dtype=torch.int32).cuda() for i in range(3))
    torch.cuda.synchronize()
    rv.kv8_copy(src, dst, 2, f.data_ptr(), t.data_ptr(), n.data_ptr(), whole.err.data_ptr())
    torch.cuda.synchronize()
    assert int(whole.err) == 0
    for y, x in zip(want, arrays):
        assert np.array_equal(y, bits(x))


def test_a_row_inside_the_destination_is_refused():
    """The same arrays a row on: nothing is copied."""
    whole = random_cache(4, 4, 1, 64, 64, 16)
    arrays = whole.codes + whole.scale + whole.tail
    before = [x.clone() for x in arrays]
    src = rv.KV8(3, 1, 64, 64, 16, 0, 1, *(t[1].data_ptr() for t in arrays))
    zero = torch.zeros(1, dtype=torch.int32).cuda()
    with pytest.raises(rv.RVError):
        rv.kv8_copy(src, whole.c, 1, zero.data_ptr(), zero.data_ptr(), None, None)
    torch.cuda.synchronize()
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(arrays, before))
