"""Rows that hold copies of a prompt and go on from it by themselves: the cache
attention on them against the definition of what each row stands for, prompt and
new tokens quantised together (an open block is quantised anew from originals,
however its tokens came in).  Bounds: kv8_util.attention."""
import numpy as np
import pytest
import torch

from kv8_util import attention, lse_tolerance, quantise
from test_gpu_answers import ACT, copy
from test_gpu_kv8 import Cache, data, f64

pytestmark = pytest.mark.gpu


def outputs(q, k, v, scale, fmt, block, Hkv):
    """One row: q [H][hd], originals k, v [n][Hkv][hd] -> (out, lse, D, bound of an output type) of each head."""
    kk, vv = (np.stack([quantise(x[:, j], fmt, block)[0] for j in range(Hkv)], 1) for x in (k, v))
    grp = q.shape[0] // Hkv
    return [attention(q[h], kk[:, h // grp], vv[:, h // grp], scale, k.shape[0], block) for h in range(q.shape[0])]


@pytest.mark.parametrize("act,fmt,hd,block", [(1, 0, 128, 32), (0, 1, 64, 32), (1, 1, 64, 16), (0, 0, 128, 64)])
def test_copies_of_a_prompt_and_what_follows(act, fmt, hd, block):
    """Six copies, a token each a step, a new order of the rows behind every step.  What a lost
    token, rows exchanged or nothing at all would give lies outside the bounds."""
    n, rows, Hkv, H, steps = 93, 6, 2, 4, 4
    name = {0: "float16", 1: "bfloat16"}[act]
    pk, pv = data(1, 1, n, Hkv, hd, act, spread=False), data(2, 1, n, Hkv, hd, act, spread=False)
    pre, whole = Cache(1, Hkv, hd, n, block, fmt, act), Cache(rows, Hkv, hd, n + 32, block, fmt, act)
    pre.append(pk, pv, [0])
    copy(pre, whole, [(0, b, n) for b in range(rows)])
    hold = [[f64(x)[0]] * rows for x in (pk, pv)]  # each row's originals
    rng, scale = np.random.default_rng(5), hd ** -0.5
    for step in range(steps):
        g = torch.Generator().manual_seed(50 + step)
        v, q = (torch.randn(rows, 1, heads, hd, generator=g).to(ACT[act]) for heads in (Hkv, H))
        k = (0.5 * q.float().view(rows, 1, Hkv, H // Hkv, hd).sum(3)).to(ACT[act])  # the queries lean towards their token
        k, v, q = k.cuda(), v.cuda(), q.cuda()
        whole.append(k, v, [n + step] * rows)
        hold = [[np.concatenate([old[b], f64(x)[b]]) for b in range(rows)] for old, x in zip(hold, (k, v))]
        out, lse = whole.attention(q, scale, [n + step] * rows)
        ref = [outputs(f64(q)[b, 0], hold[0][b], hold[1][b], scale, fmt, block, Hkv) for b in range(rows)]
        for b in range(rows):
            lost = outputs(f64(q)[b, 0], hold[0][b][:-1], hold[1][b][:-1], scale, fmt, block, Hkv)
            other = outputs(f64(q)[b, 0], hold[0][(b + 1) % rows], hold[1][(b + 1) % rows], scale, fmt, block, Hkv)
            for h, (o, l, D, bound) in enumerate(ref[b]):
                tol = bound(name)
                assert (np.abs(f64(out)[b, 0, h] - o) <= tol).all(), (step, b, h)
                assert abs(float(lse[b, 0, h]) - l) <= lse_tolerance(l, D), (step, b, h)
                for wrong in (lost[h][0], other[h][0], np.zeros(hd)):
                    assert (np.abs(wrong - o) > 4.0 * tol).any(), (step, b, h)
        order = [int(x) for x in (rng.integers(0, rows, rows) if step % 2 else rng.permutation(rows))]
        copy(whole, whole, [(a, b, n + step + 1) for b, a in enumerate(order)])
        hold = [[old[a] for a in order] for old in hold]
    assert int(whole.err) == 0
