"""min-p compares logits, not the whole-number weights that the draw sums up:
tokens whose weights are rounded to the largest one's are below a min-p of 1 all
the same."""
import math

import pytest
import torch

from test_gpu_sample import call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("x,t", [([0.0, -1e-20, -1e-13, 0.0], 1.0), ([1.0, 1.0 - 2.0 ** -8, 1.0 - 2.0 ** -8, 1.0], 1e11)])
@pytest.mark.parametrize("k", [0, 3])
def test_a_min_p_of_one_keeps_the_equals_of_the_largest(x, t, k, dtype):
    """All four have the weight 2^40 (the smallest ratio, 1 - 10^-13, is 0.11 below it); two are the largest.  k = 3 drops
    the last of the order.  Logs are below 2: half a step of fp32 is 2^-24."""
    rows = torch.tensor([x] * 4, dtype=dtype).cuda()
    u, B = [0.0, 0.49, 0.51, 0.99], 4
    ids, lp = call(rows, t=[t] * B, k=[k] * B, m=[1.0] * B, u=u)
    assert ids == [0, 0, 3, 3] and all(abs(v - math.log(0.5)) < 2.0 ** -23 for v in lp)
    ids, lp = call(rows, t=[t] * B, k=[k] * B, m=[0.999] * B, u=u)  # every one of them
    assert ids == ([0, 1, 2, 3] if k == 0 else [0, 1, 1, 3])
    assert all(abs(v + math.log(4 if k == 0 else 3)) < 2.0 ** -23 for v in lp)
