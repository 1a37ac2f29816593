"""The cache attention at the ends of its types' ranges: large scores, queries,
keys and values that are finite, weights far below the largest.

With one position's score far above all others the definition's result is that
position's value, however large the scores: its weight is the only one above
zero, so the output may be off by the weight's rounding to fp16 (2^-11), the
fp32 steps (2^-12) and its own half step."""
import math

import numpy as np
import pytest
import torch

import token_level_early_gb300 as rv
from kv8_util import U, attention
from test_gpu_kv8 import ACT, Cache, check_attention, data, expect, f64, room  # noqa: F401 (room is a fixture)

pytestmark = pytest.mark.gpu


def one_hot(seed, n, hd, act, fmt, block, qmag, kmag, room, vmag=1.0, win=None, dtype=None):
    """Two KV heads with a query head each: (cache, q, k values, v values, the winning position of each head)."""
    g = torch.Generator().manual_seed(seed)
    Hkv = 2
    q = torch.sign(torch.randn(1, 1, Hkv, hd, generator=g)) * (1 + 0.9 * torch.rand(1, 1, Hkv, hd, generator=g)) * qmag
    k = torch.randn(1, n, Hkv, hd, generator=g).clamp(-1, 1) * 0.25 * kmag
    v = torch.randn(1, n, Hkv, hd, generator=g).clamp(-1, 1) * vmag
    win = [n // 3, n - 1] if win is None else win
    for h in range(Hkv):
        k[0, win[h], h] = torch.sign(q[0, 0, h]) * kmag
    q, k, v = (x.to(ACT[act]).cuda() for x in (q, k, v))
    c = Cache(1, Hkv, hd, max(n, room), block, fmt, act)
    c.append(k, v, [0])
    return c, q, expect(c, f64(k)[0], n)[0], expect(c, f64(v)[0], n)[0], win


def check_one_hot(c, q, kk, vv, win, out, lse, scale=1.0):
    name = str(out.dtype).split(".")[1]
    for h, p in enumerate(win):
        z = scale * (kk[:, h] @ f64(q)[0, 0, h])
        d = abs(scale) * 2.0 * np.abs(kk[:, h]).max() * np.abs(f64(q)[0, 0, h]).sum()
        rest = np.delete(z, p).max()
        assert z[p] - rest > 0.2 * d > 1000.0          # 2^-19 d is what a score may be off by
        tol = (2.0 ** -11 + 2.0 ** -12 + U[name]) * np.abs(vv[p, h])
        err = np.abs(f64(out)[0, 0, h] - vv[p, h])
        assert (err <= tol).all(), (h, float((err / np.maximum(tol, 1e-300)).max()))
        assert abs(float(lse[0, 0, h]) - z[p]) <= 2.0 ** -19 * d


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("act,qmag,kmag", [(0, 2.0 ** 10, 2.0 ** 10), (0, 30000.0, 30000.0), (1, 2.0 ** 11, 2.0 ** 11), (1, 2.0 ** 15, 2.0 ** 12),
                                           (1, 2.0 ** 15, 2.0 ** 15), (1, 2.0 ** 40, 2.0 ** 15), (1, 2.0 ** 20, 2.0 ** 60)])
def test_attention_large_scores(act, qmag, kmag, hd, fmt, room):
    """Scores from 2^26 to 2^86: their fp32 steps are larger than the softmax's whole range."""
    c, q, kk, vv, win = one_hot(1, 300, hd, act, fmt, 32, qmag, kmag, room)
    out, lse = c.attention(q, 1.0, [299])
    check_one_hot(c, q, kk, vv, win, out, lse)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("qmag,kmag,scale", [(2.0 ** 105, 2.0 ** -92, 1.0), (2.0 ** 126, 2.0 ** -93, 1.0), (2.0 ** 126, 2.0 ** -20, 1.0), (2.0 ** -13, 2.0 ** 126, 1.0),
                                             (2.0 ** 60, 2.0 ** 50, 1.0), (2.0 ** 110, 1.0, 128 ** -0.5), (2.0 ** -110, 2.0 ** 126, 1.0), (2.0 ** 126, 2.0 ** -93, 4.0),
                                             (2.0 ** -120, 0.125, 3.0 * 2.0 ** 126), (2.0 ** 20, 2.0 ** 100, 2.0 ** -100)])
def test_attention_queries_and_keys_over_the_whole_range(qmag, kmag, scale, fmt, room):
    """bf16 queries and keys anywhere in the type's range, as long as scale x |q| x |k| stays below 2^119."""
    c, q, kk, vv, win = one_hot(2, 200, 128, 1, fmt, 64, qmag, kmag, room)
    out, lse = c.attention(q, scale, [199])
    check_one_hot(c, q, kk, vv, win, out, lse, scale)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("top", [2.0 ** 112, 2.0 ** 120, 3.0e38])
def test_attention_values_near_the_end_of_the_range(top, hd, fmt, room):
    """A block of very large V that has no weight, one that has all of it, and equal weights over many."""
    c, q, kk, vv, win = one_hot(3, 300, hd, 1, fmt, 32, 64.0, 64.0, room, win=[100, 120])
    v = torch.from_numpy(vv)[None].clone()
    v[0, 160:224] *= top                                # values are within 1 here: blocks without weight
    v[0, 96:128, 1] *= top                              # head 1's winner
    v = v.to(torch.bfloat16).cuda()
    k = torch.from_numpy(kk)[None].to(torch.bfloat16).cuda()
    c = Cache(1, 2, hd, max(300, room), 32, fmt, 1)
    c.append(k, v, [0])
    kk, vv = expect(c, f64(k)[0], 300)[0], expect(c, f64(v)[0], 300)[0]
    for dtype in (torch.bfloat16, torch.float32):
        out, lse = c.attention(q, 1.0, [299], out=torch.full(q.shape, 7.0, dtype=dtype).cuda())
        check_one_hot(c, q, kk, vv, win, out, lse)
    # equal weights: the sum of 3000 values passes fp32, their mean does not
    v = (data(4, 1, 3000, 1, hd, 1, False).abs().clamp(0.25, 1.0).double() * top).to(torch.bfloat16)
    c = Cache(1, 1, hd, max(3000, room), 32, fmt, 1)
    c.append(torch.zeros_like(v), v, [0])
    vv = expect(c, f64(v)[0], 3000)[0]
    q = data(5, 1, 1, 4, hd, 1, False)
    out, lse = c.attention(q, 1.0, [2999])
    check_attention(c, [np.zeros_like(vv)], [vv], q, 1.0, [2999], None, out, lse)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_values_near_zero(hd, fmt, room):
    """V around the smallest scale, 2^-100: relative errors stay what they are elsewhere."""
    k, v = data(6, 1, 400, 2, hd, 1, False), data(7, 1, 400, 2, hd, 1, False) * 2.0 ** -96
    c = Cache(1, 2, hd, max(400, room), 64, fmt, 1)
    c.append(k, v, [0])
    kk, vv = expect(c, f64(k)[0], 400)[0], expect(c, f64(v)[0], 400)[0]
    q = data(8, 1, 1, 4, hd, 1, False)
    out, lse = c.attention(q, 0.1, [399], out=torch.full(q.shape, 7.0, dtype=torch.float32).cuda())
    up = [x * 2.0 ** 96 for x in (vv, f64(out))]         # by a power of two, so that the bound's absolute part means nothing
    for h in range(4):
        ref, rl, D, bound = attention(f64(q)[0, 0, h], kk[:, h // 2], up[0][:, h // 2], 0.1, 400, 64)
        assert (np.abs(up[1][0, 0, h] - ref) <= bound("float32")).all()


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("n,gap,quiet", [(30, 20.0, 1), (30, 24.0, 1), (30, 27.0, 1), (3000, 22.0, 1), (3000, 24.0, 1), (3000, 23.4, 64), (3000, 25.5, 64)])
def test_attention_first_token_that_takes_nearly_all(n, gap, quiet, hd, fmt, act, room):
    """A first token with 2^gap times the weight of each of the others, and V =
    0 in the first `quiet` tokens, so that the others make the output: their
    weights keep their bits far below the largest one's.  A weight w of a row
    whose largest is 1 is off by 2^-32 at most besides its relative rounding
    (fp16's smallest step is 2^-24, half of it 2^-25, and the largest weights
    stand at 2^7 or above)."""
    block = 64
    g = torch.Generator().manual_seed(9)
    k = torch.zeros(1, n, 1, hd)
    k[0, 0, 0, 0] = 1.0
    v = torch.rand(1, n, 1, hd, generator=g) * 0.5 + 0.5
    v[0, :quiet] = 0.0
    q = torch.zeros(1, 1, 2, hd)
    q[..., 0] = gap
    k, v, q = (x.to(ACT[act]).cuda() for x in (k, v, q))
    c = Cache(1, 1, hd, max(n, room), block, fmt, act)
    c.append(k, v, [0])
    kk, vv = expect(c, f64(k)[0], n)[0][:, 0], expect(c, f64(v)[0], n)[0][:, 0]
    scale = float(np.float32(math.log(2.0)))
    out, lse = c.attention(q, scale, [n - 1], out=torch.full(q.shape, 7.0, dtype=torch.float32).cuda())
    z = scale * (kk @ f64(q)[0, 0, 0])
    w = np.exp(z - z.max())
    ref = w @ vv / w.sum()
    d = scale * gap * 2.0 * np.abs(kk).max()
    tol = (2.0 ** -11 + 2.0 ** -12 + 2.0 * 2.0 ** -19 * d + 2.0 ** -23) * ref + n * 2.0 ** -32
    for h in range(2):
        err = np.abs(f64(out)[0, 0, h] - ref)
        assert (err <= tol).all(), (h, float((err / tol).max()), float((err / ref).max()))
        assert abs(float(lse[0, 0, h]) - (z.max() + math.log(w.sum()))) <= 2.0 ** -19 * d + 2.0 ** -13


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_attention_query_rows_that_are_not_finite(bad, fmt, room):
    """An infinity or a NaN in a query row makes that row NaN, whatever the keys' signs, and no other."""
    hd, n = 64, 100
    k = -data(11, 1, n, 1, hd, 1, False).abs()
    v = data(12, 1, n, 1, hd, 1, False)
    c = Cache(1, 1, hd, max(n, room), 32, fmt, 1)
    c.append(k, v, [0])
    q = data(13, 1, 3, 4, hd, 1, False)
    q[0, 1, 2, 5] = bad
    out, lse = c.attention(q, 0.125, [n - 3])
    hit = torch.zeros(1, 3, 4, dtype=torch.bool, device="cuda")
    hit[0, 1, 2] = True
    assert torch.isnan(lse[hit]).all() and torch.isnan(out[hit]).all()
    assert torch.isfinite(lse[~hit]).all() and torch.isfinite(out[~hit]).all()
