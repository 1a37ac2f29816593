"""The operators for several answers to one prompt, host side: every refusal,
before any GPU work.  The pointers here are numbers that no call may
dereference.  And the plain draw against closed forms."""
import math

import pytest

import test_ops_sources_cpu as sources
import token_level_early_gb300 as rv
from answers_util import draw
from test_ops_cpu import OK, cache, heads, refused


# ------------------------------------------------------------------ copy

def copy(src=None, dst=None, n=1, first=OK, to=OK, length=OK, err=None):
    rv.kv8_copy(src or cache(), dst or cache(), n, first, to, length, err)


@pytest.mark.parametrize("kw", [
    dict(n=0), dict(n=-1), dict(n=1025), dict(first=None), dict(to=None), dict(first=OK + 2), dict(to=OK + 1), dict(length=OK + 3), dict(err=OK + 2),
    dict(src=cache(head_dim=64)), dict(src=cache(block=32)), dict(dst=cache(format=rv.KV8_E4M3)), dict(dst=cache(act_dtype=rv.F16)),
    dict(src=cache(n_kv_heads=4)), dict(src=cache(k_codes=None)), dict(dst=cache(v_tail=OK + 8)), dict(dst=cache(v_scale=2 * OK)),
    dict(src=cache(max_seq=999)), dict(src=cache(max_batch=3)), dict(src=cache(max_seq=0)),
    dict(src=cache(k_codes=3 * OK, v_codes=4 * OK, k_scale=5 * OK, v_scale=6 * OK, k_tail=7 * OK)), dict(dst=cache(max_batch=0)),
    dict(src=cache(max_seq=2 ** 28), dst=cache(max_seq=2 ** 28))])
def test_copy_refusals(kw):
    refused(copy, **kw)


def test_copy_null_caches():
    lib, c = rv.lib(), cache()
    assert lib.rv_kv8_copy(None, c, 1, OK, OK, None, None, None) == rv.RV_EINVAL
    assert lib.rv_kv8_copy(c, None, 1, OK, OK, None, None, None) == rv.RV_EINVAL


# ------------------------------------------------------------------ shared prefix

def shared(prefix=None, own=None, q=None, out=None, B=4, T=1, fan=2, scale=1.0, plen=None, pos=None, count=None, lse=None, err=None,
           work=OK, n=1 << 40):
    rv.kv8_attention_shared(prefix or cache(), own or cache(), q or heads(n=32), out or heads(n=32), B, T, fan, scale, plen, pos, count, lse, err,
                            work, n)


@pytest.mark.parametrize("kw", [
    dict(B=0), dict(B=5), dict(T=0), dict(T=17), dict(fan=0), dict(fan=-3), dict(prefix=cache(max_batch=1)), dict(prefix=cache(head_dim=64)),
    dict(prefix=cache(n_kv_heads=4)), dict(prefix=cache(act_dtype=rv.F16)), dict(prefix=cache(v_codes=None)), dict(own=cache(k_scale=OK + 4)),
    dict(own=cache(block=48)), dict(q=heads(n=12)), dict(q=heads(n=16)), dict(q=heads(n=32, dtype=rv.F16)), dict(out=heads(n=32, dtype=rv.F16)),
    dict(q=heads(n=32, data=OK + 2)), dict(q=heads(n=32, sb=8196)), dict(out=heads(n=32, sb=1024)), dict(out=heads(n=32, dtype=7)),
    dict(scale=math.inf), dict(scale=math.nan), dict(plen=OK + 1), dict(pos=OK + 2), dict(count=OK + 1), dict(lse=OK + 2), dict(err=OK + 3),
    dict(work=OK + 8)])
def test_shared_refusals(kw):
    refused(shared, **kw)


def test_shared_null_and_workspace():
    lib, c, h, E = rv.lib(), cache(), heads(n=32), rv.RV_EINVAL
    a = (1, 1, 1, 1.0, None, None, None, None, None, OK, 1 << 40, None)
    assert lib.rv_kv8_attention_shared(None, c, h, h, *a) == E
    assert lib.rv_kv8_attention_shared(c, None, h, h, *a) == E
    assert lib.rv_kv8_attention_shared(c, c, None, h, *a) == E
    assert lib.rv_kv8_attention_shared(c, c, h, None, *a) == E
    for args in ((None, c, 1, 1, 1, 8), (c, None, 1, 1, 1, 8), (c, c, 5, 1, 2, 8), (c, c, 4, 17, 2, 8), (c, c, 4, 1, 0, 8), (c, c, 4, 1, 2, 12),
                 (c, cache(head_dim=64), 4, 1, 2, 8)):
        assert lib.rv_kv8_attention_shared_workspace(*args) == 0 and lib.rv_last_error()


# ------------------------------------------------------------------ sample

def sample(logits=OK, dtype=rv.F32, stride=1000, B=2, vocab=1000, t=None, k=None, p=None, m=None, u=OK, ids=OK, lp=None):
    rv.sample(logits, dtype, stride, B, vocab, t, k, p, m, u, ids, lp)


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(u=None), dict(ids=None), dict(dtype=3), dict(dtype=-1), dict(B=0), dict(B=65536), dict(vocab=0), dict(vocab=262145),
    dict(stride=-1), dict(stride=2 ** 62), dict(logits=OK + 2), dict(logits=OK + 1, dtype=rv.BF16), dict(t=OK + 1), dict(k=OK + 2), dict(p=OK + 3),
    dict(m=OK + 1), dict(u=OK + 2), dict(ids=OK + 2), dict(lp=OK + 1)])
def test_sample_refusals(kw):
    refused(sample, **kw)


# ------------------------------------------------------------------ the plain draw

def test_draw_closed_forms():
    x = [math.log(v) for v in (1.0, 4.0, 2.0, 1.0)]
    assert [draw(x, 1.0, 0, 1.0, 0.0, u)[0] for u in (0.0, 0.1249, 0.126, 0.62, 0.63, 0.87, 0.88, 1.0)] == [0, 0, 1, 1, 2, 2, 3, 3]
    i, lp = draw(x, 1.0, 2, 1.0, 0.0, 0.9)
    assert i == 2 and abs(lp - math.log(1 / 3)) < 1e-9
    assert draw(x, 1.0, 0, 0.5, 0.0, 0.99)[0] == 1   # half of the weight lies on the first: the second is cut
    assert draw(x, 1.0, 0, 0.5001, 0.0, 0.99)[0] == 2
    assert draw(x, 1.0, 0, 1.0, 0.4, 0.99)[0] == 2 and draw(x, 1.0, 0, 1.0, 0.6, 0.99)[0] == 1
    assert draw(x, 0.0, 0, 1.0, 0.0, 0.99) == (1, 0.0)
    assert draw([1.0, 1.0, 1.0, 1.0], 0.7, 3, 1.0, 0.0, 0.999)[0] == 2  # equal ones by index
    assert draw([1.0, 1.0, 1.0, 1.0], 0.7, 0, 0.5, 0.0, 0.999)[0] == 1
    assert draw([-math.inf, math.nan], 1.0, 0, 1.0, 0.0, 0.5) == (-1, -math.inf)
    assert draw([0.0, math.inf, 3.0, math.inf], 1.0, 0, 1.0, 0.0, 0.6)[0] == 3


# ------------------------------------------------------------------ sources

@pytest.mark.parametrize("name", ["kv8_copy.cu", "kv8_shared.cuh", "kv8_shared.cu", "kv8_shared_e4m3.cu", "sample.cu"])
def test_no_read_only_loads(name):
    sources.test_no_read_only_loads_in_chained_kernels(name)
