"""Draws from the largest vocabularies: a block's share of a row is beyond what leaves
room for two blocks in a multiprocessor (fp32 from 132,000 on), up to the documented
limit.  Definition and tolerances: test_gpu_sample."""
import math

import pytest
import torch

from test_gpu_sample import check, logits, spaced, uniform

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [200003, 262144])
def test_settings(V, dtype):
    """Each setting, each for a row of its own (the rows' kept tokens differ widely)."""
    x = logits(V, 5, V, dtype)
    check(x, t=[1.0, 0.8, 1.3, 0.9, 0.0], k=[0, 50, 0, V - 1, 0], p=[1.0, 1.0, 0.95, 0.999, 1.0], m=[0.0, 0.0, 0.0, 0.01, 0.0], u=uniform(V, 5))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("off,V", [(1, 200003), (3, 262144), (7, 262141)])
def test_rows_that_begin_anywhere(off, V, dtype):
    """The first element off a 16-byte boundary, the neighbours larger than any logit."""
    flat = torch.full((off + V + 9,), 60000.0, dtype=dtype).cuda()
    x = flat[off:off + V].view(1, V)
    x.copy_(logits(off, 1, V, dtype))
    check(x, t=[0.7], p=[0.9], u=[0.6])


@pytest.mark.parametrize("dtype", TYPES)
def test_the_last_token(dtype):
    """Nearly all the weight on the last element, and the number just below one."""
    V = 262144
    x = torch.zeros(1, V, dtype=dtype).cuda()
    x[0, V - 1] = 30.0
    check(x, u=[0.5])
    check(x, t=[5.0], u=[1.0 - 2.0 ** -24])


@pytest.mark.parametrize("dtype", TYPES)
def test_equal_logits(dtype):
    """Far more elements at the border than are listed: the border is found among all, ties go by index."""
    V = 262144
    x = torch.full((4, V), 1.25).to(dtype).cuda()
    x[3, ::3] = 1.25 - 2.0
    check(x, k=[100003, 0, 200000, 0], p=[1.0, 0.5, 0.75, 0.9], u=[0.999, 0.999, 0.999, 0.9])


@pytest.mark.parametrize("dtype", TYPES)
def test_flat_rows(dtype):
    """Logits of few values close together, borders far down the order."""
    x = spaced(5, 3, 262144, 0.0, 0.5).to(dtype)
    check(x, t=[1.0, 0.5, 2.0], k=[0, 130000, 200000], p=[0.9, 1.0, 0.6], u=uniform(7, 3))


def test_absent_tokens():
    """Most tokens banned, one row all of them."""
    V = 262144
    x = logits(2, 2, V)
    x[0, 5:] = -math.inf
    x[1] = -math.inf
    check(x, p=[0.9, 0.9], u=[0.7, 0.7])
