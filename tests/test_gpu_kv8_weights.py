"""The attention's weights as two fp16 terms: fp16 caches, and fp32 outputs of
bf16 caches (bound and its CPU check in kv8_weights_util)."""
import numpy as np
import pytest
import torch

from kv8_weights_util import bound, case
from test_gpu_kv8 import ACT, Cache, expect, f64, room  # noqa: F401 (room is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [2, 3, 7, 33])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("hd,block,H", [(64, 16, 4), (64, 32, 12), (64, 64, 24), (128, 16, 24), (128, 32, 4), (128, 64, 12)])
def test_attention_weights_of_two_terms(hd, block, H, fmt, act, n, room):
    q, k, v = case(n, H, n, hd)
    q, k, v = (torch.from_numpy(x).to(ACT[act]).cuda() for x in (q[None, None], k[None, :, None], v[None, :, None]))
    c = Cache(1, 1, hd, max(n, room), block, fmt, act)
    c.append(k, v, [0])
    kk, vv = expect(c, f64(k)[0], n)[0][:, 0], expect(c, f64(v)[0], n)[0][:, 0]
    out, _ = c.attention(q, 1.0, [n - 1], out=torch.full(q.shape, 7.0, dtype=torch.float32).cuda())
    got, qq = f64(out)[0, 0], f64(q)[0, 0]
    for h in range(H):
        ref, tol = bound(qq[h], kk, vv, block)
        err = np.abs(got[h] - ref)
        assert (err <= tol).all(), (h, float((err / tol).max()))


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("hd,H", [(64, 1), (64, 24), (128, 16)])
def test_attention_small_values_beside_large_ones(hd, H, fmt, act, room):
    """Columns of V whose codes are +-1 in blocks whose scale another column
    sets, a first position of most of the weight: the error of a column goes by
    its own values, not by the block's largest."""
    n, block = 40, 32
    g = np.random.default_rng(3)
    q, k, _ = case(4, H, n, hd)
    k[0, 0] = 12.0
    k[1:, 0] = g.uniform(0.0, 4.0, n - 1)
    v = g.choice([-1.0, 1.0], (n, hd)) * 2.0 ** -7
    v[:, 5] = g.uniform(-0.8, 0.8, n)
    v[::block, 5] = 127.0 / 128.0 if fmt == 0 else 448.0 / 512.0   # scales of 2^-7 and 2^-9: all the small values are codes
    q, k, v = (torch.from_numpy(x).to(ACT[act]).cuda() for x in (q[None, None], k[None, :, None], v[None, :, None]))
    c = Cache(1, 1, hd, max(n, room), block, fmt, act)
    c.append(k, v, [0])
    kk, vv = expect(c, f64(k)[0], n)[0][:, 0], expect(c, f64(v)[0], n)[0][:, 0]
    small = np.delete(np.arange(hd), 5)
    assert (np.abs(vv[:, small]) == 2.0 ** -7).all()
    out, _ = c.attention(q, 1.0, [n - 1], out=torch.full(q.shape, 7.0, dtype=torch.float32).cuda())
    got, qq = f64(out)[0, 0], f64(q)[0, 0]
    for h in range(H):
        ref, tol = bound(qq[h], kk, vv, block)
        err = np.abs(got[h] - ref)
        assert (err <= tol).all(), (h, float((err / tol).max()))
