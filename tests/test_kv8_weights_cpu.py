"""The bound that the GPU tests of the attention's two-term weights use holds for
two terms and fails without the second, or with its sign turned."""
import numpy as np
import pytest

from kv8_util import quantise
from kv8_weights_util import bound, case, product


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("n", [2, 3, 7, 33])
def test_bound_tells_one_term_from_two(n, fmt):
    q, k, v = case(n, 24, n, 64)
    k, v = quantise(k, fmt, 32)[0], quantise(v, fmt, 32)[0]
    worst = {1: 0.0, 2: 0.0, -2: 0.0}
    for row in q:
        ref, tol = bound(row, k, v, 32)
        for terms in worst:
            worst[terms] = max(worst[terms], float((np.abs(product(row, k, v, terms) - ref) / tol).max()))
    assert worst[2] < 0.5 and worst[1] > 1.2 and worst[-2] > 1.2, worst
