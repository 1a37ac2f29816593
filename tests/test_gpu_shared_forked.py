"""The two ways to attend over a prompt that rows share, on the same originals: the
prefix read once beside each row's own cache, and the prompt copied into each row.
Each against the definition of what it quantises; the new tokens take a real
share of the weight."""
import numpy as np
import pytest
import torch

import token_level_early_gb300 as rv
from answers_util import attention_parts
from kv8_util import attention, lse_tolerance, quantise
from test_gpu_kv8 import Cache, data, f64
from test_gpu_kv8_shared import call, queries

pytestmark = pytest.mark.gpu


def values(x, fmt, block):
    """What a cache of tokens x [n][Hkv][hd] stands for."""
    return np.stack([quantise(x[:, j], fmt, block)[0] for j in range(x.shape[1])], 1)


@pytest.mark.parametrize("n,fmt,act,hd,block", [(331, 0, 1, 128, 32), (150, 1, 0, 64, 64), (64, 0, 0, 64, 16), (1, 1, 1, 128, 16)])
def test_shared_and_forked_rows_against_their_definitions(n, fmt, act, hd, block):
    B, Hkv, H, new = 5, 2, 8, 3
    grp, scale, name = H // Hkv, hd ** -0.5, {0: "float16", 1: "bfloat16"}[act]
    pk, pv = data(1, 1, n, Hkv, hd, act, spread=False), data(2, 1, n, Hkv, hd, act, spread=False)
    nk, nv = data(7, B, new, Hkv, hd, act, spread=False), data(8, B, new, Hkv, hd, act, spread=False)
    q = queries(9, B, 1, H, hd, act)
    nk[:, -1] = 0.5 * q.float().view(B, Hkv, grp, hd).sum(2)  # the queries lean towards the last token
    pre, own, whole = Cache(1, Hkv, hd, n, block, fmt, act), Cache(B, Hkv, hd, 16, block, fmt, act), Cache(B, Hkv, hd, n + 16, block, fmt, act)
    pre.append(pk, pv, [0])
    own.append(nk, nv, [0] * B)
    f, t, m = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([0] * B, list(range(B)), [n] * B))
    torch.cuda.synchronize()
    rv.kv8_copy(pre.c, whole.c, B, f.data_ptr(), t.data_ptr(), m.data_ptr(), whole.err.data_ptr())
    whole.append(nk, nv, [n] * B)
    one, l1 = call(pre, own, q, B, scale, [n], [new - 1] * B)
    two, l2 = whole.attention(q, scale, [n + new - 1] * B)
    assert int(whole.err) == 0
    pre_k, pre_v = (values(f64(x)[0], fmt, block) for x in (pk, pv))
    for b in range(B):
        own_k, own_v = (values(f64(x)[b], fmt, block) for x in (nk, nv))
        all_k, all_v = (values(np.concatenate([f64(p)[0], f64(x)[b]]), fmt, block) for p, x in ((pk, nk), (pv, nv)))
        for h in range(H):
            j, qq = h // grp, f64(q)[b, 0, h]
            a, la, da, ba = attention_parts(qq, [(pre_k[:, j], pre_v[:, j], block), (own_k[:, j], own_v[:, j], block)], scale, act == 0)
            c, lc, dc, bc = attention(qq, all_k[:, j], all_v[:, j], scale, n + new, block)
            for got, l, ref, lr, d, tol in ((one, l1, a, la, da, ba(name)), (two, l2, c, lc, dc, bc(name))):
                assert (np.abs(f64(got)[b, 0, h] - ref) <= tol).all(), (b, h)
                assert abs(float(l[b, 0, h]) - lr) <= lse_tolerance(lr, d), (b, h)
                without = attention(qq, pre_k[:, j], pre_v[:, j], scale, n, block)[0]  # no new token
                assert (np.abs(without - ref) > 4.0 * tol).any(), (b, h)
