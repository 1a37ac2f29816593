"""The draw against the definition: tokens have to be equal, their logs to be
within fp32's half step and the weights' 2^-29 (both parts of the quotient)."""
import math

import numpy as np
import pytest
import torch

import token_level_early_gb300 as rv
from answers_util import draw

pytestmark = pytest.mark.gpu
DT = {torch.float32: 2, torch.bfloat16: 1, torch.float16: 0}


def call(x, t=None, k=None, p=None, m=None, u=None, logprob=True, stride=None, stream=None):
    """x [B][V] on the GPU (rows `stride` apart); settings as lists."""
    B, V = x.shape
    fl = [None if v is None else torch.tensor(v, dtype=torch.int32 if i == 1 else torch.float32).cuda() for i, v in enumerate((t, k, p, m, u))]
    ids = torch.full((B,), -7, dtype=torch.int32).cuda()
    lp = torch.full((B,), 7.0).cuda()
    torch.cuda.synchronize()
    a = [None if v is None else v.data_ptr() for v in fl]
    rv.sample(x.data_ptr(), DT[x.dtype], x.stride(0) if stride is None else stride, B, V, *a, ids.data_ptr(), lp.data_ptr() if logprob else None, stream)
    torch.cuda.synchronize()
    return ids.cpu().tolist(), lp.cpu().tolist()


def check(x, t=None, k=None, p=None, m=None, u=None):
    ids, lp = call(x, t, k, p, m, u)
    B = x.shape[0]
    for b in range(B):
        row = x[b].double().cpu().tolist()
        f32 = [None if v is None else float(np.float32(v[b])) for v in (t, p, m, u)]
        ref, rl = draw(row, 1.0 if t is None else f32[0], 0 if k is None else k[b], 1.0 if p is None else f32[1],
                       0.0 if m is None else f32[2], f32[3])
        assert ids[b] == ref, (b, ids[b], ref)
        if ref < 0:
            assert lp[b] == -math.inf
        else:
            # a small weight is a few whole units: half a unit of it on either side
            tol = 2.0 ** -24 * abs(rl) + 2.0 ** -28 + math.exp(min(-rl, 40.0)) * 2.0 ** -40
            assert abs(lp[b] - rl) <= tol, (b, lp[b], rl)


def logits(seed, B, V, dtype=torch.float32, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, V, generator=g) * spread
    up = torch.rand(B, V, generator=g) < 20.0 / V
    return torch.where(up, x + 6.0 + torch.rand(B, V, generator=g) * 4.0, x).to(dtype).cuda()


def uniform(seed, B):
    return torch.rand(B, generator=torch.Generator().manual_seed(seed)).tolist()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,V", [(1, 1), (3, 2), (2, 31), (5, 1000), (2, 4099), (3, 32000), (1, 50257), (2, 131075)])
def test_every_setting(B, V, dtype):
    x = logits(B * V, B, V, dtype)
    for seed, kw in enumerate((
            {}, dict(t=[0.7] * B), dict(k=[1] * B), dict(k=[5] * B), dict(k=[V] * B), dict(k=[max(V - 1, 1)] * B), dict(p=[0.9] * B), dict(p=[0.3] * B),
            dict(p=[0.999] * B), dict(m=[0.05] * B), dict(t=[1.5] * B, k=[40] * B, p=[0.8] * B, m=[0.01] * B))):
        check(x, u=uniform(seed, B), **kw)


def test_rows_with_settings_of_their_own():
    B, V = 40, 3001
    r = np.random.default_rng(3)
    x = logits(8, B, V)
    x[::5, ::2] = -math.inf
    x[3, 7], x[4, 1000:] = math.nan, math.nan
    check(x, t=[float(v) for v in r.choice([0.0, 0.3, 1.0, 2.0], B)], k=[int(v) for v in r.choice([-1, 0, 1, 3, 50, 3000, 9000], B)],
          p=[float(v) for v in r.choice([-0.5, 0.0, 0.2, 0.9, 1.0, 2.0, math.nan], B)], m=[float(v) for v in r.choice([-1.0, 0.0, 0.01, 0.3, 1.0, 5.0, math.nan], B)],
          u=[float(v) for v in r.random(B)])


@pytest.mark.parametrize("V", [1, 7, 64, 1000, 40000])
def test_equal_logits_are_cut_by_index(V):
    """All equal, and two values: every count, half the weight, exact ties of
    the random number with a border."""
    x = torch.full((8, V), 1.25).cuda()
    half = max(V // 2, 1)
    check(x, k=[1, half, V, 0, 0, 0, 0, half], p=[1.0, 1.0, 1.0, 0.5, 0.25, 1.0, 1.0, 0.5], u=[0.999, 0.999, 0.999, 0.999, 0.999, 0.5, 0.75, 0.75])
    y = x.clone()
    y[:, ::3] = 1.25 - math.log(4.0)
    check(y, k=[1, half, V, 0, 0, 0, 0, half], p=[1.0, 1.0, 1.0, 0.5, 0.9, 1.0, 0.7, 0.9], u=[0.999, 0.999, 0.3, 0.999, 0.999, 0.1, 0.2, 0.999])


def test_ends_of_the_random_number():
    x = logits(5, 6, 500)
    check(x, u=[0.0, -1.0, math.nan, 1.0, 7.0, 1.0 - 2.0 ** -24])
    check(x, k=[3] * 6, u=[0.0, -1.0, math.nan, 1.0, 7.0, 1.0 - 2.0 ** -24])


def test_special_logits():
    inf, nan = math.inf, math.nan
    rows = [[-inf] * 5, [nan] * 5, [nan, -inf, 3.0, nan, -inf], [inf, 0.0, inf, 1.0, nan], [-0.0, 0.0, -0.0, 0.0, -inf], [3e38, -3e38, 3e38, 0.0, 1.0],
            [1e-40, -1e-40, 0.0, 2e-45, 1.0], [-1e30, -2e30, -1e30, -inf, nan]]
    x = torch.tensor(rows).cuda()
    for kw in ({}, dict(k=[1] * 8), dict(k=[2] * 8), dict(p=[0.5] * 8), dict(t=[0.0] * 8), dict(t=[0.5] * 8, k=[3] * 8, p=[0.7] * 8, m=[0.2] * 8)):
        for u in (0.0, 0.49, 0.51, 0.99):
            check(x, u=[u] * 8, **kw)


def test_temperatures_at_their_ends():
    x = logits(6, 8, 300)
    check(x, t=[-1.0, math.nan, 1e-30, 1e-6, 0.01, 100.0, 1e6, math.inf], u=[0.7] * 8)


def test_rows_apart_and_unaligned():
    """Any stride and first element that the type allows; the rows' neighbours are poison."""
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        for off, V, stride in ((0, 100, 103), (1, 257, 300), (3, 5000, 5001), (7, 9, 11)):
            flat = torch.full((off + 4 * stride + 8,), 60000.0, dtype=dtype).cuda()
            x = flat[off:off + 4 * stride].view(4, stride)[:, :V]
            x.copy_(logits(V, 4, V, dtype))
            check(x, p=[0.9] * 4, u=uniform(9, 4))
    x = logits(11, 1, 700)
    ids, _ = call(x.expand(3, 700), u=[0.1, 0.5, 0.9], stride=0)
    assert ids == [draw(x[0].double().cpu().tolist(), 1.0, 0, 1.0, 0.0, float(np.float32(u)))[0] for u in (0.1, 0.5, 0.9)]


def test_without_logprob_and_many_rows():
    x = logits(12, 700, 257)
    u = uniform(1, 700)
    a, _ = call(x, u=u, k=[20] * 700, logprob=False)
    assert a == [draw(r, 1.0, 20, 1.0, 0.0, float(np.float32(v)))[0] for r, v in zip(x.double().cpu().tolist(), u)]


def test_draws_follow_their_probabilities():
    """200 numbers spread evenly over [0, 1) draw each token as often as its
    probability says, to one draw (the last number of a token's interval)."""
    x = torch.tensor([0.5, 2.0, -1.0, 1.0, 0.0])
    n = 200
    ids, _ = call(x.repeat(n, 1).cuda(), u=[(i + 0.5) / n for i in range(n)])
    prob = torch.softmax(x.double(), 0)
    for i in range(5):
        assert abs(ids.count(i) - n * float(prob[i])) <= 1.0
    assert ids == sorted(ids)


def test_captured_and_replayed():
    x = logits(13, 4, 9000)
    u = torch.zeros(4).cuda()
    t = torch.full((4,), 0.8).cuda()
    p = torch.full((4,), 0.9).cuda()
    ids = torch.zeros(4, dtype=torch.int32).cuda()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rv.sample(x.data_ptr(), rv.F32, 9000, 4, 9000, t.data_ptr(), None, p.data_ptr(), None, u.data_ptr(), ids.data_ptr(), None,
                  torch.cuda.current_stream().cuda_stream)
    for seed in range(3):
        v = uniform(seed, 4)
        y = logits(20 + seed, 4, 9000)
        x.copy_(y)
        u.copy_(torch.tensor(v))
        g.replay()
        torch.cuda.synchronize()
        assert ids.cpu().tolist() == [draw(r, float(np.float32(0.8)), 0, float(np.float32(0.9)), 0.0, float(np.float32(w)))[0]
                                      for r, w in zip(y.double().cpu().tolist(), v)]


def spaced(seed, B, V, centre, spread, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, V, generator=g) * spread + centre).to(dtype).cuda()


@pytest.mark.parametrize("centre,spread,t", [
    (-8.0, 1.5, 0.8), (0.0, 0.003, 0.001), (0.0, 0.003, 1.0), (0.001, 0.004, 0.002), (-0.02, 0.006, 0.01), (300.0, 40.0, 20.0), (0.0, 2000.0, 300.0),
    (-1e-3, 1e-4, 1.0), (0.0, 1e-30, 1e-30), (3.0, 0.02, 0.01)])
def test_bf16_values_small_large_and_of_one_sign(centre, spread, t):
    """Values share few numbers; the ones next to zero share a place, where the
    border may lie too; all negative; ranges beyond the places."""
    B, V = 12, 9001
    x = spaced(3, B, V, centre, spread)
    p = [0.3, 0.5, 0.7, 0.9, 0.99, 0.999, 1.0, 1.0, 1.0, 0.5, 0.8, 0.6]
    k = [0, 0, 0, 0, 0, 0, 7, 900, 5000, 2999, 20, 4000]
    check(x, t=[t] * B, k=k, p=p, m=[0.0] * 10 + [0.3, 0.01], u=uniform(4, B))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_many_equal_logits_at_the_border(dtype):
    """Logits that were bf16 before, of a large vocabulary: hundreds of elements in a step, at borders far down."""
    x = spaced(5, 6, 131072, 0.0, 2.0).to(dtype)
    x[:, 5] = 9.0
    check(x, t=[0.9, 1.0, 1.3, 0.6, 1.0, 1.0], p=[0.99, 0.9, 0.5, 0.95, 1.0, 0.7], k=[0, 0, 0, 0, 5000, 60000], u=uniform(6, 6))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_top_p_next_to_one_and_to_nothing(dtype):
    x = logits(7, 8, 20011, dtype)
    p = [0.9999, 0.99999, 1.0 - 2.0 ** -24, 0.9997, 1e-30, 2.0 ** -40, 1e-3, 0.99]
    check(x, p=p, u=uniform(8, 8))
    check(x, p=p, k=[17000] * 8, u=uniform(9, 8))


def test_draws_do_not_depend_on_the_rows_beside():
    """A row alone, and among many (other clusters, other shares): the same token and log."""
    x = logits(9, 300, 4001)
    u, t = uniform(10, 300), [0.3 + (b % 7) * 0.2 for b in range(300)]
    ids, lp = call(x, t=t, p=[0.9] * 300, u=u)
    for b in (0, 7, 151, 299):
        one, l1 = call(x[b:b + 1].contiguous(), t=t[b:b + 1], p=[0.9], u=u[b:b + 1])
        assert (one[0], l1[0]) == (ids[b], lp[b])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_more_rows_than_multiprocessors(dtype):
    """Many short rows take other blocks than few: the same definition."""
    B, V = 170, 2001
    r = np.random.default_rng(9)
    x = logits(17, B, V, dtype)
    x[::7, ::3] = -math.inf
    check(x, t=[float(v) for v in r.choice([0.0, 0.5, 1.0], B)], k=[int(v) for v in r.choice([0, 3, 50], B)],
          p=[float(v) for v in r.choice([0.2, 0.9, 1.0], B)], m=[float(v) for v in r.choice([0.0, 0.02], B)], u=[float(v) for v in r.random(B)])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,V", [(170, 5001), (160, 40001)])
def test_rows_alone_and_together(B, V, dtype):
    """However many rows there are (and so however a row's work is cut), its draw is the same."""
    r = np.random.default_rng(V)
    x = logits(V, B, V, dtype)
    kw = dict(t=[float(v) for v in r.choice([0.5, 1.0], B)], k=[int(v) for v in r.choice([0, 3, 50], B)],
              p=[float(v) for v in r.choice([0.2, 0.9, 1.0], B)], m=[float(v) for v in r.choice([0.0, 0.02], B)], u=[float(v) for v in r.random(B)])
    ids, lp = call(x, **kw)
    for n in (1, 20):
        for b in range(0, B - n + 1, 13):
            assert call(x[b:b + n], **{a: v[b:b + n] for a, v in kw.items()}) == (ids[b:b + n], lp[b:b + n]), b
