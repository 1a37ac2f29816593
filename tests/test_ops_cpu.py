"""The operators' host side: plans, and every refusal, before any GPU work.
The pointers here are numbers that no call may dereference."""
import math

import numpy as np
import pytest

import token_level_early_gb300 as rv
from kv8_util import QMAX, block_scale, quantise, rope, rope_frequencies, to_code, up8

OK = 0x10000


def refused(f, *a, code=rv.RV_EINVAL, **k):
    with pytest.raises(rv.RVError) as e:
        f(*a, **k)
    assert e.value.code == code and len(str(e.value)) > 20, str(e.value)


def heads(data=OK, dtype=rv.BF16, n=8, sb=8192, st=1024, sh=128):
    return rv.Heads(data, dtype, n, sb, st, sh)


def cache(**kw):
    d = dict(max_batch=4, n_kv_heads=8, head_dim=128, max_seq=1000, block=64, format=rv.KV8_INT8, act_dtype=rv.BF16,
             k_codes=OK, v_codes=OK, k_scale=OK, v_scale=OK, k_tail=OK, v_tail=OK)
    d.update(kw)
    return rv.KV8(*d.values())


# ------------------------------------------------------------------ plans

@pytest.mark.parametrize("scaling,kw", [
    ("plain", {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
    ("bands", dict(factor=8.0, low=1.0, high=4.0, original=8192)),
    ("ramp", dict(factor=16.0, original=4096)), ("ramp", dict(factor=0.5, original=4096)),
    ("ramp", dict(factor=2.0, original=1, fast=2.0, slow=1.5))])
@pytest.mark.parametrize("rot", [16, 64, 128])
def test_plan_holds_the_frequencies_in_turns(scaling, kw, rot):
    kind = dict(plain=rv.ROPE_PLAIN, linear=rv.ROPE_LINEAR, base=rv.ROPE_BASE, bands=rv.ROPE_BANDS, ramp=rv.ROPE_RAMP)[scaling]
    names = {"low": "low_freq_factor", "high": "high_freq_factor", "original": "original_max_position", "fast": "beta_fast", "slow": "beta_slow"}
    p = rv.rope_plan(128, rot, rv.ROPE_HALF, 500000.0, kind, **{names.get(k, k): v for k, v in kw.items()})
    f, att = rope_frequencies(rot, 500000.0, scaling, **kw)
    got = np.array([p.turns[i] / 2.0 ** 64 for i in range(rot // 2)])
    # pow, log and the quotients are a few steps of 2^-53 each, times the exponent's size (up to 13 in ln)
    assert np.abs(got - f / (2 * math.pi)).max() <= 2.0 ** -44
    assert abs(p.attention_factor - att) <= 2.0 ** -23 * att
    assert all(p.turns[i] == 0 for i in range(rot // 2, 128))
    assert (p.head_dim, p.rotary_dim, p.layout) == (128, rot, rv.ROPE_HALF)


def test_plan_attention_factor_given():
    assert rv.rope_plan(64, attention_factor=1.25).attention_factor == 1.25
    assert rv.rope_plan(64, scaling=rv.ROPE_RAMP, factor=4.0, original_max_position=100, attention_factor=0.5).attention_factor == 0.5


@pytest.mark.parametrize("kw", [
    dict(head_dim=0), dict(head_dim=24), dict(head_dim=272), dict(rotary_dim=0), dict(rotary_dim=8), dict(rotary_dim=80),
    dict(layout=2), dict(layout=-1), dict(scaling=5), dict(scaling=-1), dict(theta=1.0), dict(theta=math.inf), dict(theta=math.nan),
    dict(scaling=rv.ROPE_LINEAR, factor=0.0), dict(scaling=rv.ROPE_LINEAR, factor=math.nan), dict(scaling=rv.ROPE_BASE, factor=-2.0),
    dict(scaling=rv.ROPE_BASE, factor=1e308, theta=1e300), dict(scaling=rv.ROPE_BANDS, factor=2.0),
    dict(scaling=rv.ROPE_BANDS, factor=2.0, original_max_position=10, low_freq_factor=4.0, high_freq_factor=4.0),
    dict(scaling=rv.ROPE_BANDS, factor=2.0, original_max_position=10, low_freq_factor=0.0),
    dict(scaling=rv.ROPE_RAMP, factor=2.0), dict(scaling=rv.ROPE_RAMP, factor=2.0, original_max_position=10, beta_fast=1.0),
    dict(scaling=rv.ROPE_RAMP, factor=2.0, original_max_position=10, beta_slow=0.0), dict(attention_factor=-1.0),
    dict(attention_factor=math.nan), dict(scaling=rv.ROPE_LINEAR, factor=1e-30)])
def test_plan_refusals(kw):
    d = dict(head_dim=64)
    d.update(kw)
    refused(rv.rope_plan, **d)


def test_null_arguments():
    import ctypes as C

    lib, E = rv.lib(), rv.RV_EINVAL
    h, c, p = heads(), cache(), rv.rope_plan(128)
    assert lib.rv_rope_init(None, C.byref(p)) == E and lib.rv_rope_init(C.byref(rv.RopeConfig()), None) == E
    assert lib.rv_rope(None, h, h, None, None, 1, 1, None, None, 0, None) == E
    assert lib.rv_rope(p, None, h, None, None, 1, 1, None, None, 0, None) == E
    assert lib.rv_rope(p, h, None, None, None, 1, 1, None, None, 0, None) == E
    assert lib.rv_kv8_append(None, h, h, 1, 1, None, None, None, None) == E
    assert lib.rv_kv8_append(c, None, h, 1, 1, None, None, None, None) == E
    assert lib.rv_kv8_append(c, h, None, 1, 1, None, None, None, None) == E
    assert lib.rv_kv8_read(None, h, h, 1, 1, None, None, None, None) == E
    assert lib.rv_kv8_read(c, None, None, 1, 1, None, None, None, None) == E
    assert lib.rv_kv8_attention(None, h, h, 1, 1, 1.0, None, None, None, OK, 1 << 30, None) == E
    assert lib.rv_kv8_attention(c, None, h, 1, 1, 1.0, None, None, None, OK, 1 << 30, None) == E
    assert lib.rv_kv8_attention(c, h, None, 1, 1, 1.0, None, None, None, OK, 1 << 30, None) == E
    assert lib.rv_kv8_attention_workspace(None, 1, 1, 8) == 0 and lib.rv_last_error()


# ------------------------------------------------------------------ tensors

BAD_HEADS = [dict(data=0), dict(data=OK + 8), dict(dtype=3), dict(dtype=-1), dict(n=0), dict(sb=8196), dict(st=1020), dict(sh=132),
             dict(sb=-8192), dict(st=-1024), dict(sh=-128), dict(sb=1 << 62)]
OVERLAP = [dict(sh=0), dict(sh=64), dict(st=512), dict(st=0), dict(sb=1024), dict(sb=0)]


@pytest.mark.parametrize("kw", BAD_HEADS)
def test_bad_tensors_are_refused_everywhere(kw):
    p, c, h, bad = rv.rope_plan(128), cache(), heads(), heads(**kw)
    for a in ((bad, h, None, None), (h, bad, None, None), (h, h, bad, h), (h, h, h, bad)):
        refused(rv.rope, p, *a, 4, 3, None)
    refused(rv.kv8_append, c, bad, h, 4, 3, None)
    refused(rv.kv8_append, c, h, bad, 4, 3, None)
    refused(rv.kv8_read, c, bad, None, 4, 3, None)
    refused(rv.kv8_read, c, None, bad, 4, 3, None)
    refused(rv.kv8_attention, c, bad, h, 4, 3, 1.0, None, None, None, OK, 1 << 40)
    refused(rv.kv8_attention, c, h, bad, 4, 3, 1.0, None, None, None, OK, 1 << 40)


@pytest.mark.parametrize("kw", OVERLAP)
def test_outputs_whose_rows_overlap_are_refused(kw):
    p, c, h, bad = rv.rope_plan(128), cache(), heads(), heads(**kw)
    refused(rv.rope, p, h, bad, None, None, 4, 3, None)
    refused(rv.kv8_read, c, bad, None, 4, 3, None)
    refused(rv.kv8_attention, c, h, bad, 4, 3, 1.0, None, None, None, OK, 1 << 40)


@pytest.mark.parametrize("B,T", [(0, 1), (1, 0), (-1, 1), (1 << 20, 1 << 20)])
def test_bad_batches(B, T):
    h = heads()
    refused(rv.rope, rv.rope_plan(128), h, h, None, None, B, T, None)
    refused(rv.kv8_append, cache(max_batch=65535), h, h, B, T, None)
    refused(rv.kv8_read, cache(max_batch=65535), h, h, B, T, None)
    refused(rv.kv8_attention, cache(max_batch=65535), h, h, B, T, 1.0, None, None, None, OK, 1 << 40)


def test_rope_refusals():
    p, h, f = rv.rope_plan(128), heads(), heads(dtype=rv.F32)
    refused(rv.rope, rv.RopePlan(), h, h, None, None, 1, 1, None)       # not made by rope_plan
    refused(rv.rope, p, h, h, h, None, 1, 1, None)
    refused(rv.rope, p, h, h, None, h, 1, 1, None)
    refused(rv.rope, p, h, heads(n=4), None, None, 1, 1, None)
    refused(rv.rope, p, h, h, h, heads(n=4), 1, 1, None)
    refused(rv.rope, p, h, heads(dtype=rv.F16), None, None, 1, 1, None)
    refused(rv.rope, p, h, f, None, None, 1, 1, None)                   # 16-bit inputs keep their type
    refused(rv.rope, p, f, h, None, None, 1, 1, None)                   # in place with two types
    refused(rv.rope, p, h, h, f, f, 1, 1, None)
    refused(rv.rope, p, h, h, None, None, 1, 1, OK + 2)
    big = heads(n=4096)
    refused(rv.rope, p, big, big, h, h, 1, 1, None)                     # 4104 heads of 128
    refused(rv.rope, p, h, h, None, None, 1, 1, None, OK + 1)


BAD_CACHES = [dict(max_batch=0), dict(max_batch=65536), dict(n_kv_heads=1025), dict(n_kv_heads=0), dict(max_seq=0), dict(max_seq=2 ** 31 - 1), dict(head_dim=96), dict(block=48),
              dict(block=256), dict(block=0), dict(format=2), dict(act_dtype=rv.F32), dict(k_codes=0), dict(v_codes=0), dict(k_scale=0),
              dict(v_scale=0), dict(k_tail=0), dict(v_tail=0), dict(k_codes=OK + 4), dict(v_tail=OK + 8)]


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_bad_caches(kw):
    c, h = cache(**kw), heads()
    refused(rv.kv8_append, c, h, h, 1, 1, None)
    refused(rv.kv8_read, c, h, h, 1, 1, None)
    refused(rv.kv8_attention, c, h, h, 1, 1, 1.0, None, None, None, OK, 1 << 40)


def test_cache_call_refusals():
    c, h = cache(), heads()
    refused(rv.kv8_append, c, h, h, 5, 1, None)                          # above max_batch
    refused(rv.kv8_append, c, heads(n=4), h, 1, 1, None)
    refused(rv.kv8_append, c, heads(dtype=rv.F16), heads(dtype=rv.F16), 1, 1, None)
    refused(rv.kv8_append, c, h, heads(dtype=rv.F32), 1, 1, None)
    refused(rv.kv8_append, c, h, h, 1, 1, OK + 1)
    refused(rv.kv8_append, c, h, h, 1, 1, None, None, OK + 2)
    refused(rv.kv8_read, c, heads(n=9), None, 1, 1, None)
    refused(rv.kv8_read, c, h, heads(dtype=rv.F32), 1, 1, None)
    refused(rv.kv8_read, c, h, h, 5, 1, None)
    for a in (dict(T=17), dict(B=5), dict(scale=math.nan), dict(scale=math.inf), dict(q=heads(n=12)), dict(out=heads(n=16)),
              dict(q=heads(dtype=rv.F16)), dict(out=heads(dtype=rv.F16)), dict(lse=OK + 2), dict(pos=OK + 1), dict(work=OK + 8)):
        d = dict(q=h, out=h, B=1, T=1, scale=1.0, pos=None, count=None, lse=None, work=OK, size=1 << 40)
        d.update(a)
        refused(rv.kv8_attention, c, *d.values())


# ------------------------------------------------------------------ the plain forms themselves

def test_plain_forms():
    """Closed forms that the 64-bit reference must satisfy."""
    assert up8(1.0) == 1.0 and up8(1.0 + 2.0 ** -20) == 1.0 + 2.0 ** -7 and up8(255.0) == 255.0 and up8(255.5) == 256.0
    assert block_scale(np.zeros(4), 0) == 2.0 ** -100 and math.isnan(block_scale(np.array([1.0, math.inf]), 1))
    assert list(to_code(np.array([0.5, 1.5, -2.5, 126.5]), 0)) == [0.0, 2.0, -2.0, 126.0]
    assert list(to_code(np.array([17.0, 19.0, 448.0, 2.0 ** -10, 3 * 2.0 ** -10]), 1)) == [16.0, 20.0, 448.0, 0.0, 2.0 ** -8]
    for fmt in (0, 1):
        x = np.random.default_rng(0).standard_normal((64, 8))
        v, s = quantise(x, fmt, 16)
        step = np.repeat(s, 16)[:, None] / 2 if fmt == 0 else np.maximum(np.abs(x) * 2.0 ** -4, np.repeat(s, 16)[:, None] * 2.0 ** -10)
        assert (np.abs(v - x) <= step * (1 + 1e-12)).all() and s.max() * QMAX[fmt] <= np.abs(x).max() * (1 + 2.0 ** -7)
    f, _ = rope_frequencies(8, 10000.0)
    x = np.random.default_rng(1).standard_normal((1, 3, 2, 8))
    for inter in (False, True):
        y = rope(x, [[5, 6, 7]], f, 8, inter)
        assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
        assert np.allclose(rope(y, [[5, 6, 7]], f, 8, inter, inverse=True), x)


def test_model_calls_reject_a_null_handle():
    import ctypes as C

    lib = rv.lib()
    assert lib.rv_set_rope(None, C.byref(rv.RopeConfig())) == rv.RV_EINVAL
    assert lib.rv_set_option(None, rv.OPT_KV_CACHE, rv.KV_INT8) == rv.RV_EINVAL
    assert lib.rv_kv_cache_bytes(None) == 0


@pytest.mark.parametrize("factor", [1e39, math.inf])
def test_attention_factor_beyond_fp32_is_refused(factor):
    refused(rv.rope_plan, 64, attention_factor=factor)
    assert rv.rope_plan(64, attention_factor=3e38).attention_factor == np.float32(3e38)
