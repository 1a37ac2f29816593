"""The rotary operator against its formula in 64 bits.

Tolerance: cos and sin come from a half-turn fraction rounded to 24 bits (the
angle is off by at most pi 2^-25 < 2^-23.3) through sincospif (2 units in the
last place, below 2^-22) and one rounding with the attention factor, so each
is off by less than 2^-21.4; an element is the sum of two products of inputs
with them, each rounded: |error| <= 2^-21 (|x0| + |x1|) x factor + half a step
of the output type."""
import numpy as np
import pytest
import torch

import token_level_early_gb300 as rv
from kv8_util import U, rope, rope_frequencies

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
KIND = {"plain": rv.ROPE_PLAIN, "linear": rv.ROPE_LINEAR, "base": rv.ROPE_BASE, "bands": rv.ROPE_BANDS, "ramp": rv.ROPE_RAMP}


def f64(t):
    return t.detach().double().cpu().numpy()


def check(y, x, ref, att, dtype):
    mag = np.abs(f64(x)).max(axis=-1, keepdims=True)
    tol = 2.0 ** -20 * mag * max(att, 1.0) + U[str(dtype).split(".")[1]] * np.abs(ref) + 2.0 ** -25
    err = np.abs(f64(y) - ref)
    assert (err <= tol).all(), float((err / tol).max())


def plan_of(hd, rot, inter, scaling="plain", **kw):
    names = {"low": "low_freq_factor", "high": "high_freq_factor", "original": "original_max_position", "fast": "beta_fast", "slow": "beta_slow"}
    return rv.rope_plan(hd, rot, rv.ROPE_INTERLEAVED if inter else rv.ROPE_HALF, 500000.0, KIND[scaling],
                        **{names.get(k, k): v for k, v in kw.items()})


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dt_in,dt_out", [("fp16", "fp16"), ("bf16", "bf16"), ("fp32", "fp32"), ("fp32", "fp16"), ("fp32", "bf16")])
@pytest.mark.parametrize("B,T,H,Hkv,hd,rot", [(1, 1, 32, 8, 128, 128), (3, 5, 4, 2, 64, 32), (2, 37, 7, 1, 80, 16), (1, 300, 3, 3, 256, 256), (65, 1, 1, 1, 16, 16)])
def test_rope_matches_formula(B, T, H, Hkv, hd, rot, dt_in, dt_out, inter):
    g = torch.Generator().manual_seed(B * 131 + T + hd)
    q = torch.randn(B, T, H, hd, generator=g).to(DT[dt_in]).cuda()
    k = torch.randn(B, T, Hkv, hd, generator=g).to(DT[dt_in]).cuda()
    pos = torch.randint(0, 100000, (B,), generator=g, dtype=torch.int32).cuda()
    qo, ko = torch.empty_like(q, dtype=DT[dt_out]), torch.empty_like(k, dtype=DT[dt_out])
    rv.rope(plan_of(hd, rot, inter), rv.heads(q), rv.heads(qo), rv.heads(k), rv.heads(ko), B, T, pos.data_ptr())
    torch.cuda.synchronize()
    at = pos.cpu().numpy()[:, None] + np.arange(T)
    freq, _ = rope_frequencies(rot, 500000.0)
    check(qo, q, rope(f64(q), at, freq, rot, inter), 1.0, DT[dt_out])
    check(ko, k, rope(f64(k), at, freq, rot, inter), 1.0, DT[dt_out])


@pytest.mark.parametrize("scaling,kw", [("linear", dict(factor=4.0)), ("linear", dict(factor=0.5)), ("base", dict(factor=8.0)),
                                        ("bands", dict(factor=8.0, low=1.0, high=4.0, original=8192)),
                                        ("ramp", dict(factor=16.0, original=4096)), ("ramp", dict(factor=2.0, original=64, fast=2.0, slow=1.5))])
def test_rope_scaled_frequencies_and_far_positions(scaling, kw):
    """Positions up to the largest int32 and negative ones; a product of 31 and
    53 bits is exact to 2^-22 turns in the double reference at the far end, so
    the reference is taken with an exact reduction (python integers)."""
    hd, B = 64, 6
    g = torch.Generator().manual_seed(3)
    x = torch.randn(B, 1, 2, hd, generator=g).cuda()
    at = [0, 1, 131071, 2 ** 31 - 1, -1, -70000]
    pos = torch.tensor(at, dtype=torch.int32).cuda()
    plan = plan_of(hd, hd, False, scaling, **kw)
    y = torch.empty_like(x)
    rv.rope(plan, rv.heads(x), rv.heads(y), None, None, B, 1, pos.data_ptr())
    freq, att = rope_frequencies(hd, 500000.0, scaling, **kw)
    assert abs(plan.attention_factor - att) <= 2.0 ** -23 * att
    turns = np.array([plan.turns[i] / 2.0 ** 64 for i in range(hd // 2)])
    assert np.abs(turns - freq / (2 * np.pi) % 1.0).max() <= 1e-13
    exact = np.array([[(p * plan.turns[i]) % 2 ** 64 / 2.0 ** 64 * 2 * np.pi for i in range(hd // 2)] for p in at])
    ref = np.zeros((B, 1, 2, hd))
    for b in range(B):
        ref[b:b + 1] = rope(f64(x[b:b + 1]), [[1.0]], exact[b], hd, False, att)
    check(y, x, ref, att, torch.float32)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_strides_counts_and_in_place(inter):
    B, T, H, hd, rot = 3, 9, 5, 64, 48
    g = torch.Generator().manual_seed(11)
    big = torch.randn(B, H, T + 2, hd + 8, generator=g).to(torch.bfloat16).cuda()  # heads outside tokens, padded rows
    x = big[:, :, 1:T + 1, :hd].transpose(1, 2)
    before = big.clone()
    pos = torch.tensor([5, 0, 77], dtype=torch.int32).cuda()
    count = torch.tensor([4, 0, 50], dtype=torch.int32).cuda()  # 50 is taken as T
    k = torch.randn(B, T, 1, hd, generator=g).to(torch.bfloat16).cuda()
    ko = torch.full_like(k, 7.0)
    rv.rope(plan_of(hd, rot, inter), rv.heads(x), rv.heads(x), rv.heads(k), rv.heads(ko), B, T, pos.data_ptr(), count.data_ptr())
    torch.cuda.synchronize()
    at = np.array([5, 0, 77])[:, None] + np.arange(T)
    freq, _ = rope_frequencies(rot, 500000.0)
    x0 = before[:, :, 1:T + 1, :hd].transpose(1, 2)
    ref, refk = rope(f64(x0), at, freq, rot, inter), rope(f64(k), at, freq, rot, inter)
    for b, n in enumerate([4, 0, T]):
        if n:
            check(x[b, :n], x0[b, :n], ref[b, :n], 1.0, torch.bfloat16)
            check(ko[b, :n], k[b, :n], refk[b, :n], 1.0, torch.bfloat16)
        assert torch.equal(x[b, n:], x0[b, n:]) and (ko[b, n:] == 7.0).all()
    after = big.clone()
    after[:, :, 1:T + 1, :hd] = before[:, :, 1:T + 1, :hd]
    assert torch.equal(after, before)  # nothing outside the tensor was touched


@pytest.mark.parametrize("inter", [False, True])
def test_rope_inverse_is_the_gradient(inter):
    """The rotation is linear, so its gradient is its transpose: against the
    formula, and against differences of L = sum g rope(x) along random
    directions (exact for a linear map up to fp32 rounding)."""
    B, T, H, hd, rot = 2, 7, 3, 64, 32
    kw = dict(factor=16.0, original=4096)
    plan = plan_of(hd, rot, inter, "ramp", **kw)
    g = torch.Generator().manual_seed(5)
    x, w = (torch.randn(B, T, H, hd, generator=g).cuda() for _ in range(2))
    pos = torch.tensor([3, 12345], dtype=torch.int32).cuda()

    def call(t, inverse):
        y = torch.empty_like(t)
        rv.rope(plan, rv.heads(t), rv.heads(y), None, None, B, T, pos.data_ptr(), None, inverse)
        return y

    freq, att = rope_frequencies(rot, 500000.0, "ramp", **kw)
    at = pos.cpu().numpy()[:, None] + np.arange(T)
    grad = call(w, True)
    check(grad, w, rope(f64(w), at, freq, rot, inter, att, inverse=True), att, torch.float32)
    for _ in range(3):
        d = torch.randn(B, T, H, hd, generator=g).cuda()
        diff = float((f64(w) * (f64(call(x + d, False)) - f64(call(x - d, False)))).sum()) / 2
        dot = float((f64(grad) * f64(d)).sum())
        size = float((np.abs(f64(w)) * np.abs(f64(d))).sum()) + float((np.abs(f64(w)) * np.abs(f64(x))).sum())
        assert abs(diff - dot) <= 2.0 ** -18 * size


def test_rope_captures_into_a_graph():
    B, T, H, hd = 2, 3, 4, 128
    x = torch.randn(B, T, H, hd).to(torch.float16).cuda()
    y = torch.zeros_like(x)
    pos = torch.tensor([4, 9], dtype=torch.int32).cuda()
    plan = plan_of(hd, hd, False)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        rv.rope(plan, rv.heads(x), rv.heads(y), None, None, B, T, pos.data_ptr(), stream=torch.cuda.current_stream().cuda_stream)
    freq, _ = rope_frequencies(hd, 500000.0)
    for start in (4, 1000):
        pos.copy_(torch.tensor([start, 9], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        at = np.array([start, 9])[:, None] + np.arange(T)
        check(y, x, rope(f64(x), at, freq, hd, False), 1.0, torch.float16)


@pytest.mark.parametrize("B,T,H,hd,rot", [(1, 200003, 1, 16, 16), (70001, 3, 1, 64, 64), (2, 40000, 2, 128, 128)])
def test_rope_many_tokens_of_few_heads(B, T, H, hd, rot):
    """Runs of tokens that end inside a row and blocks that hold many rows."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(B, T, H, hd, generator=g, device="cuda")
    pos = torch.randint(0, 1000, (B,), generator=g, device="cuda").to(torch.int32)
    y = torch.empty_like(x)
    rv.rope(plan_of(hd, rot, False), rv.heads(x), rv.heads(y), None, None, B, T, pos.data_ptr())
    freq, _ = rope_frequencies(rot, 500000.0)
    rows = sorted({0, B - 1, B // 2, min(B - 1, 1)})
    at = pos.cpu().numpy()[rows][:, None] + np.arange(T)
    check(y[rows], x[rows], rope(f64(x[rows]), at, freq, rot, False), 1.0, torch.float32)


def test_rope_one_token_of_many_heads():
    x = torch.randn(1, 2, 4096, 128).to(torch.bfloat16).cuda()
    y = torch.empty_like(x)
    rv.rope(plan_of(128, 64, True), rv.heads(x), rv.heads(y), None, None, 1, 2, None)
    freq, _ = rope_frequencies(64, 500000.0)
    check(y, x, rope(f64(x), [[0, 1]], freq, 64, True), 1.0, torch.bfloat16)


def test_memory_that_is_not_the_devices_is_refused():
    plan, x = plan_of(64, 64, False), torch.zeros(1, 1, 2, 64).cuda()
    host = torch.zeros(1, 1, 2, 64)
    pos = torch.zeros(1, dtype=torch.int32)
    for a in ((host, x, None), (x, host, None), (x, x, pos.data_ptr())):
        with pytest.raises(rv.RVError) as e:
            rv.rope(plan, rv.heads(a[0]), rv.heads(a[1]), None, None, 1, 1, a[2])
        assert e.value.code == rv.RV_EINVAL
