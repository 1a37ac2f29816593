"""Attention over a shared prefix and each row's own cache against the
definition in 64 bits; bounds are derived in answers_util."""
import math

import numpy as np
import pytest
import torch

import token_level_early_gb300 as rv
from answers_util import attention_parts
from kv8_util import lse_tolerance
from test_gpu_kv8 import ACT, Cache, data, expect, f64

pytestmark = pytest.mark.gpu


def filled(seed, rows, Hkv, hd, block, fmt, act, lens, max_seq):
    c = Cache(rows, Hkv, hd, max_seq, block, fmt, act)
    T = max(max(lens), 1)
    k, v = data(seed, rows, T, Hkv, hd, act), data(seed + 1, rows, T, Hkv, hd, act)
    c.append(k, v, [0] * rows, lens)
    values = [[expect(c, f64(x)[b], lens[b])[0] if lens[b] else np.zeros((0, Hkv, hd)) for b in range(rows)] for x in (k, v)]
    return c, values[0], values[1]


def call(pre, own, q, fan, scale, plen, pos, count=None, out=None, stream=None, work=None):
    B, T, H, _ = q.shape
    ints = [None if x is None else torch.tensor(x, dtype=torch.int32).cuda() for x in (plen, pos, count)]
    out = torch.full_like(q, 7.0) if out is None else out
    lse = torch.full((B, T, H), 7.0).cuda()
    need = rv.kv8_attention_shared_workspace(pre.c, own.c, B, T, fan, H)
    work = torch.full((need,), 0xFF, dtype=torch.uint8).cuda() if work is None else work
    torch.cuda.synchronize()
    rv.kv8_attention_shared(pre.c, own.c, rv.heads(q), rv.heads(out), B, T, fan, scale, *(None if x is None else x.data_ptr() for x in ints),
                            lse.data_ptr(), own.err.data_ptr(), work.data_ptr(), need, stream)
    torch.cuda.synchronize()
    assert int(own.err) == 0
    return out, lse


def check(pre, own, pk, pv, ok, ov, q, fan, scale, plen, pos, count, out, lse):
    B, T, H, hd = q.shape
    grp = H // own.Hkv
    name = str(out.dtype).split(".")[1]
    two = own.act == 0 or name == "float32"
    worst = 0.0
    for b in range(B):
        n = T if count is None else min(max(count[b], 0), T)
        assert (out[b, n:] == 7.0).all() and (lse[b, n:] == 7.0).all()
        for t in range(n):
            a = b // fan
            np_, no = min(max(plen[a], 0), pre.T), min(max(pos[b] + t + 1, 0), own.T)
            for h in range(H):
                g = h // grp
                ref, rl, D, bound = attention_parts(f64(q)[b, t, h], [(pk[a][:np_, g], pv[a][:np_, g], pre.block), (ok[b][:no, g], ov[b][:no, g], own.block)],
                                                    scale, two)
                got, gl = f64(out)[b, t, h], float(lse[b, t, h])
                if np_ + no == 0:
                    assert (got == 0).all() and gl == -math.inf
                    continue
                tol = bound(name)
                err = np.abs(got - ref)
                worst = max(worst, float((err / tol).max()))
                assert (err <= tol).all(), (b, t, h, np_, no, float((err / tol).max()))
                assert abs(gl - rl) <= lse_tolerance(rl, D), (b, t, h, gl, rl)
    return worst


def queries(seed, B, T, H, hd, act):
    return torch.randn(B, T, H, hd, generator=torch.Generator().manual_seed(seed)).to(ACT[act]).cuda()


CASES = [  # P, fan, T, H, Hkv, hd, block (prefix, own), format (prefix, own), act, prefix lengths, own positions, counts
    (1, 1, 1, 1, 1, 64, (16, 16), (0, 0), 1, [1], [0], None),
    (1, 4, 1, 8, 2, 128, (64, 64), (0, 0), 1, [200], [30, 0, -1, 63], None),
    (1, 4, 1, 8, 2, 128, (64, 16), (0, 1), 0, [0], [3, 0, -1, 20], None),
    (2, 3, 2, 6, 2, 64, (32, 32), (1, 1), 1, [127, 129], [5, -1, -2, 17, 31, 32], [2, 1, 2, 0, 2, 1]),
    (3, 2, 1, 4, 4, 128, (16, 128), (1, 0), 0, [128, 1, 300], [0, 1, 2, 3, 4, 100], None),
    (1, 40, 2, 8, 2, 64, (16, 16), (0, 0), 1, [150], [b % 7 - 1 for b in range(40)], [b % 3 for b in range(40)]),
    (1, 33, 2, 16, 2, 128, (64, 64), (0, 0), 1, [270], [b % 5 for b in range(33)], None),
    (2, 5, 3, 7, 1, 64, (128, 16), (0, 0), 0, [257, 500], [b for b in range(10)], None),
    (1, 2, 16, 16, 2, 128, (32, 32), (1, 1), 1, [385], [7, 40], [16, 9]),
    (2, 2, 1, 5, 1, 128, (128, 64), (0, 1), 0, [1000, 640], [50, 3, 0, 12], None),
    (4, 16, 1, 4, 1, 64, (64, 64), (1, 0), 1, [300, 0, 64, 700], [b % 9 for b in range(64)], None),
]


@pytest.mark.parametrize("q32,out32", [(False, False), (False, True), (True, False)])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c[:6]))
def test_against_the_definition(case, q32, out32):
    P, fan, T, H, Hkv, hd, block, fmt, act, plen, pos, count = case
    B = len(pos)
    pre, pk, pv = filled(1, P, Hkv, hd, block[0], fmt[0], act, plen, max(plen) + 9)
    own, ok, ov = filled(3, B, Hkv, hd, block[1], fmt[1], act, [max(p + T, 0) for p in pos], max(max(pos) + T, 1))
    q = queries(5, B, T, H, hd, act)
    out = torch.full(q.shape, 7.0, dtype=torch.float32 if out32 else q.dtype).cuda()
    out, lse = call(pre, own, q.float() if q32 else q, fan, hd ** -0.5, plen, pos, count, out)
    check(pre, own, pk, pv, ok, ov, q, fan, hd ** -0.5, plen, pos, count, out, lse)


def test_a_last_prefix_with_fewer_rows_and_lengths_out_of_range():
    pre, pk, pv = filled(1, 3, 2, 64, 16, 0, 1, [90, 90, 90], 90)
    own, ok, ov = filled(3, 8, 2, 64, 16, 0, 1, [5] * 8, 5)
    q = queries(5, 8, 1, 4, 64, 1)
    for plen in ([-4, 91, 2 ** 31 - 1], [90, -2 ** 31, 3]):
        out, lse = call(pre, own, q, 3, 0.125, plen, [4] * 8)
        check(pre, own, pk, pv, ok, ov, q, 3, 0.125, plen, [4] * 8, None, out, lse)
    out, lse = call(pre, own, q, 3, 0.125, None, [4] * 8)
    check(pre, own, pk, pv, ok, ov, q, 3, 0.125, [90] * 3, [4] * 8, None, out, lse)
    out, lse = call(pre, own, q, 100, 0.125, [50], [4] * 8)  # a fan above the batch
    check(pre, own, pk, pv, ok, ov, q, 100, 0.125, [50], [4] * 8, None, out, lse)


def test_the_same_prefix_copied_into_each_row_gives_the_same():
    """Forked caches and plain attention against the shared form, both within their bounds of the definition."""
    n, B, Hkv, hd, block, act = 331, 5, 2, 128, 32, 1
    pre, pk, pv = filled(1, 1, Hkv, hd, block, 0, act, [n], 400)
    new_k, new_v = data(7, B, 3, Hkv, hd, act, spread=False), data(8, B, 3, Hkv, hd, act, spread=False)
    q = queries(9, B, 1, 8, hd, act)
    own = Cache(B, Hkv, hd, 16, block, 0, act)
    own.append(new_k, new_v, [0] * B)
    a, la = call(pre, own, q, B, hd ** -0.5, [n], [2] * B)
    whole = Cache(B, Hkv, hd, 400, block, 0, act)
    f, t, m = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([0] * B, list(range(B)), [n] * B))
    rv.kv8_copy(pre.c, whole.c, B, f.data_ptr(), t.data_ptr(), m.data_ptr(), None)
    whole.append(new_k, new_v, [n] * B)
    b, lb = whole.attention(q, hd ** -0.5, [n + 2] * B)
    # the open block is quantised with the new tokens there: codes differ by up to a step of its scale, 1/127 of its largest value
    top = float(f64(whole.scale[1])[:, :, n // block].max())
    assert (a.float() - b.float()).abs().max() <= 4.0 * top + 2.0 ** -7 * float(b.float().abs().max())
    assert (la - lb).abs().max() < 0.5


def test_strides_and_inputs_left_alone():
    """Heads outside tokens, padded rows, a slice of a larger tensor."""
    P, fan, T, H, Hkv, hd = 2, 3, 2, 8, 2, 64
    pre, pk, pv = filled(1, P, Hkv, hd, 16, 0, 1, [77, 140], 160)
    own, ok, ov = filled(3, 6, Hkv, hd, 16, 0, 1, [9] * 6, 16)
    big = torch.randn(6, H, T + 3, hd + 8, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    q = big[:, :, 1:1 + T, :hd].transpose(1, 2)
    wide = torch.full((6, T, 2, H, hd + 16), 7.0, dtype=torch.bfloat16).cuda()
    out = wide[:, :, 1, :, 8:8 + hd]
    before = [x.clone() for x in pre.codes + own.codes + [big]]
    out, lse = call(pre, own, q, fan, 0.2, [77, 140], [7] * 6, None, out)
    check(pre, own, pk, pv, ok, ov, q, fan, 0.2, [77, 140], [7] * 6, None, out, lse)
    wide[:, :, 1, :, 8:8 + hd] = 7.0
    assert (wide == 7.0).all()
    for x, y in zip(before, pre.codes + own.codes + [big]):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("act", [0, 1])
def test_blocks_with_a_nan_reach_the_rows_that_see_them(act):
    P, fan, Hkv, hd, block = 2, 2, 2, 64, 16
    k, v = data(1, P, 200, Hkv, hd, act), data(2, P, 200, Hkv, hd, act)
    k[0, 150, 1, 3] = math.nan
    v[1, 160, 0, 5] = math.inf
    pre = Cache(P, Hkv, hd, 200, block, 0, act)
    pre.append(k, v, [0, 0])
    own, _, _ = filled(3, 4, Hkv, hd, 16, 0, act, [3] * 4, 16)
    q = queries(5, 4, 1, 4, hd, act)
    out, lse = call(pre, own, q, fan, 0.1, [144, 160], [2] * 4)  # the blocks at 144 and 160 are not seen
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    out, lse = call(pre, own, q, fan, 0.1, [145, 161], [2] * 4)
    bad = torch.isnan(out).all(-1)[:, 0]
    assert bad[:2].tolist() == [[False, False, True, True]] * 2 and bad[2:].tolist() == [[True, True, False, False]] * 2
    assert torch.isfinite(out[:2, :, :2]).all() and torch.isfinite(out[2:, :, 2:]).all()


def test_query_rows_with_infinities_and_nans():
    pre, pk, pv = filled(1, 1, 1, 64, 16, 0, 1, [40], 40)
    own, ok, ov = filled(3, 4, 1, 64, 16, 0, 1, [2] * 4, 16)
    q = queries(5, 4, 1, 2, 64, 1)
    q[0, 0, 0, 3], q[1, 0, 1, 0], q[2, 0, 0, 9] = math.nan, math.inf, -math.inf
    out, _ = call(pre, own, q, 4, 0.1, [40], [1] * 4)
    bad = torch.isnan(out)
    assert bad[0, 0, 0].all() and bad[1, 0, 1].all() and bad[2, 0, 0].all()
    bad[0, 0, 0] = bad[1, 0, 1] = bad[2, 0, 0] = False
    assert not bad.any()


@pytest.mark.parametrize("scale", [0.0, -0.3, 40.0])
def test_scales_of_any_sign_and_size(scale):
    pre, pk, pv = filled(1, 1, 2, 128, 64, 0, 1, [260], 300)
    own, ok, ov = filled(3, 3, 2, 128, 64, 0, 1, [4] * 3, 16)
    q = queries(5, 3, 1, 4, 128, 1)
    out, lse = call(pre, own, q, 3, scale, [260], [3] * 3)
    check(pre, own, pk, pv, ok, ov, q, 3, scale, [260], [3] * 3, None, out, lse)


@pytest.mark.parametrize("fmt", [0, 1])
def test_growing_scores_and_values(fmt):
    """Later blocks have ever larger keys and values (the references follow), then smaller ones."""
    n, Hkv, hd, block = 900, 1, 64, 16
    size = torch.exp2(torch.cat([torch.linspace(-20, 6, 600), torch.linspace(6, -14, 300)])).view(1, n, 1, 1).cuda()
    base = data(1, 1, n, Hkv, hd, 1, spread=False).float()
    k = (base * (size / size.max()) * 3).to(torch.bfloat16)
    v = (data(2, 1, n, Hkv, hd, 1, spread=False).float() * size).to(torch.bfloat16)
    pre = Cache(1, Hkv, hd, n, block, fmt, 1)
    pre.append(k, v, [0])
    pk, pv = ([expect(pre, f64(x)[0], n)[0]] for x in (k, v))
    own, ok, ov = filled(3, 3, Hkv, hd, 16, 0, 1, [1] * 3, 16)
    q = queries(5, 3, 1, 4, hd, 1)
    out, lse = call(pre, own, q, 3, 1.0, [n], [0] * 3)
    check(pre, own, pk, pv, ok, ov, q, 3, 1.0, [n], [0] * 3, None, out, lse)


def test_one_position_takes_nearly_all_the_weight():
    n, hd = 640, 128
    k, v = data(1, 1, n, 1, hd, 1, spread=False), data(2, 1, n, 1, hd, 1, spread=False)
    q = queries(5, 2, 1, 8, hd, 1)
    for at in (0, 130, n - 1):
        kk, vv = k.clone(), v.clone()
        kk[0, at, 0] = q[0, 0, 0] * 2
        vv[0, at, 0] *= 2.0 ** -9  # as first tokens of trained models have it
        pre = Cache(1, 1, hd, n, 64, 0, 1)
        pre.append(kk, vv, [0])
        pk, pv = ([expect(pre, f64(x)[0], n)[0]] for x in (kk, vv))
        own, ok, ov = filled(3, 2, 1, hd, 16, 0, 1, [1] * 2, 16)
        out, lse = call(pre, own, q, 2, 0.5, [n], [0] * 2)
        check(pre, own, pk, pv, ok, ov, q, 2, 0.5, [n], [0] * 2, None, out, lse)


def test_long_prefixes_and_every_split():
    """More tiles than blocks, pieces that end inside units, against the definition at a few rows."""
    P, fan, T, H, Hkv, hd, act = 3, 70, 1, 8, 2, 64, 1
    lens = [30011, 0, 20480]
    pre = Cache(P, Hkv, hd, 30011, 64, 0, act)
    k, v = data(1, P, 30011, Hkv, hd, act, spread=False), data(2, P, 30011, Hkv, hd, act, spread=False)
    pre.append(k, v, [0] * P, lens)
    own, ok, ov = filled(3, P * fan, Hkv, hd, 16, 0, act, [1] * (P * fan), 16)
    q = queries(5, P * fan, T, H, hd, act)
    out, lse = call(pre, own, q, fan, 0.125, lens, [0] * (P * fan))
    vals = {}
    for b in (0, 1, 31, 32, 63, 64, 69, 70, 139, 140, 173, 209):
        a = b // fan
        if a not in vals:
            vals[a] = [expect(pre, f64(x)[a], lens[a])[0] if lens[a] else np.zeros((0, Hkv, hd)) for x in (k, v)]
        for h in (0, 3, 4, 7):
            g = h // 4
            ref, rl, D, bound = attention_parts(f64(q)[b, 0, h], [(vals[a][0][:, g], vals[a][1][:, g], 64), (ok[b][:, g], ov[b][:, g], 16)], 0.125, False)
            assert (np.abs(f64(out)[b, 0, h] - ref) <= bound("bfloat16")).all(), (b, h)
            assert abs(float(lse[b, 0, h]) - rl) <= lse_tolerance(rl, D)


def test_many_short_prefixes():
    """More units than blocks, most of one tile (a stream has nothing of them), 80 rows each: the streams
    leave a unit's state at different times.  Every row against the definition, and the same bits again."""
    P, fan, T, H, Hkv, hd, act = 90, 5, 4, 8, 2, 64, 1
    lens = [(100, 128, 1, 300, 0, 64, 128)[p % 7] for p in range(P)]
    pre, pk, pv = filled(1, P, Hkv, hd, 32, 0, act, lens, 300)
    pos = [b % 4 - 2 for b in range(P * fan)]
    own, ok, ov = filled(3, P * fan, Hkv, hd, 16, 0, act, [max(p + T, 0) for p in pos], 16)
    q = queries(5, P * fan, T, H, hd, act)
    out, lse = call(pre, own, q, fan, 0.125, lens, pos)
    check(pre, own, pk, pv, ok, ov, q, fan, 0.125, lens, pos, None, out, lse)
    for _ in range(20):
        again, l2 = call(pre, own, q, fan, 0.125, lens, pos)
        assert torch.equal(again, out) and torch.equal(l2, lse)


def test_captured_and_replayed_beside_another_stream():
    """One graph per workspace on two streams at once, with lengths and positions that change between replays."""
    P, fan, T, H, Hkv, hd, act = 2, 8, 1, 8, 2, 128, 1
    pre, pk, pv = filled(1, P, Hkv, hd, 64, 0, act, [900, 700], 1000)
    own, ok, ov = filled(3, 16, Hkv, hd, 64, 0, act, [40] * 16, 64)
    need = rv.kv8_attention_shared_workspace(pre.c, own.c, 16, T, fan, H)
    sides = []
    for i in range(2):
        s = torch.cuda.Stream()
        d = dict(s=s, q=queries(5 + i, 16, T, H, hd, act), out=torch.zeros(16, T, H, hd, dtype=torch.bfloat16).cuda(), lse=torch.zeros(16, T, H).cuda(),
                 plen=torch.zeros(P, dtype=torch.int32).cuda(), pos=torch.zeros(16, dtype=torch.int32).cuda(),
                 work=torch.full((need,), 0xFF, dtype=torch.uint8).cuda(), g=torch.cuda.CUDAGraph())
        torch.cuda.synchronize()
        with torch.cuda.graph(d["g"], stream=s):
            rv.kv8_attention_shared(pre.c, own.c, rv.heads(d["q"]), rv.heads(d["out"]), 16, T, fan, 0.1, d["plen"].data_ptr(), d["pos"].data_ptr(), None,
                                    d["lse"].data_ptr(), None, d["work"].data_ptr(), need, torch.cuda.current_stream().cuda_stream)
        sides.append(d)
    for plen, at in (([900, 700], 39), ([1, 0], 0), ([128, 513], 20)):
        for d in sides:
            d["plen"].copy_(torch.tensor(plen, dtype=torch.int32))
            d["pos"].fill_(at)
        torch.cuda.synchronize()
        for _ in range(3):
            for d in sides:
                with torch.cuda.stream(d["s"]):
                    d["g"].replay()
        torch.cuda.synchronize()
        for d in sides:
            check(pre, own, pk, pv, ok, ov, d["q"], fan, 0.1, plen, [at] * 16, None, d["out"], d["lse"])


def test_workspace_of_the_largest_serves_the_smaller():
    pre, _, _ = filled(1, 2, 2, 64, 16, 0, 1, [50, 60], 64)
    own, _, _ = filled(3, 12, 2, 64, 16, 0, 1, [4] * 12, 32)
    big = rv.kv8_attention_shared_workspace(pre.c, own.c, 12, 16, 6, 32)
    for B, T in ((1, 1), (5, 3), (6, 16), (7, 16), (12, 1)):
        assert 0 < rv.kv8_attention_shared_workspace(pre.c, own.c, B, T, 6, 32) <= big
    q = queries(5, 12, 1, 4, 64, 1)
    with pytest.raises(rv.RVError):
        rv.kv8_attention_shared(pre.c, own.c, rv.heads(q), rv.heads(q), 12, 1, 6, 0.1, None, None, None, None, None,
                                torch.zeros(64, dtype=torch.uint8).cuda().data_ptr(), 64)


@pytest.mark.parametrize("long", [64, 40000])
def test_both_caches_are_read_as_the_call_before_left_them(long):
    """Appends to the prefix and to the own rows, each followed at once by the attention that reads
    them, chained in a graph: the bits of the same calls one at a time.  `long`: room in the own
    rows, which decides whether their part is one kernel or two."""
    Hkv, hd, B, n, steps = 2, 128, 6, 1500, 8
    pre, own = Cache(1, Hkv, hd, n, 64, 0, 1), Cache(B, Hkv, hd, long, 16, 0, 1)
    ks, vs = ([data(10 * i + j, 1, n, Hkv, hd, 1) for i in range(steps)] for j in (1, 2))
    ko, vo = ([data(10 * i + j, B, 5, Hkv, hd, 1) for i in range(steps)] for j in (3, 4))
    qs = [queries(i, B, 1, 8, hd, 1) for i in range(steps)]
    zero, pos = torch.zeros(B, dtype=torch.int32).cuda(), torch.full((B,), 4, dtype=torch.int32).cuda()
    need = rv.kv8_attention_shared_workspace(pre.c, own.c, B, 1, B, 8)
    work = torch.full((need,), 0xFF, dtype=torch.uint8).cuda()

    def steps_of(outs, stream, wait):
        for i in range(steps):
            rv.kv8_append(own.c, rv.heads(ko[i]), rv.heads(vo[i]), B, 5, zero.data_ptr(), None, own.err.data_ptr(), stream)
            rv.kv8_append(pre.c, rv.heads(ks[i]), rv.heads(vs[i]), 1, n, zero.data_ptr(), None, pre.err.data_ptr(), stream)
            wait()
            rv.kv8_attention_shared(pre.c, own.c, rv.heads(qs[i]), rv.heads(outs[i]), B, 1, B, 0.1, None, pos.data_ptr(), None, None, own.err.data_ptr(),
                                    work.data_ptr(), need, stream)
            wait()

    want, got = [torch.zeros_like(q) for q in qs], [torch.zeros_like(q) for q in qs]
    torch.cuda.synchronize()
    steps_of(want, None, torch.cuda.synchronize)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        steps_of(got, stream.cuda_stream, lambda: None)
    for _ in range(30):
        for x in got:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, got))
    assert int(pre.err) == 0 and int(own.err) == 0
