"""The model on an 8-bit K/V cache (RV_OPT_KV_CACHE) and with scaled rotary
frequencies (rv_set_rope).

The first layer's K/V do not depend on any cache, so there the 8-bit cache has
to hold exactly the definition's codes of what the 16-bit cache holds.  Every
layer is checked against the oracle from the GPU's own inputs and the cache's
own values (which differ from what the step used only in the rounding of
code x scale to 16 bits and in the token's own K/V, one of many positions)."""
import numpy as np
import pytest
import torch

import oracle
import synth
import token_level_early_gb300 as rv
from gpu_util import TOL_HIDDEN, TOL_LOGIT, cos64, kv_values, rel_l2
from kv8_util import quantise, rope_frequencies

pytestmark = pytest.mark.gpu

SMALL = synth.ModelShape("kv8-hd128", 3, 512, 8, 2, 128, 512, 1024, 0, synth.BF16, 1e-5, 500000.0)
KINDS = [(rv.KV_INT8, 0), (rv.KV_E4M3, 1)]


def to16(x, act):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16 if act else torch.float16).view(torch.int16).numpy().view(np.uint16)


def expect_layer(bits, lens, act, fmt):
    """16-bit image [2][B][Hkv][T][hd] -> what the 8-bit cache reads back."""
    x = kv_values(bits, act).astype(np.float64)
    out = np.full(bits.shape, 0x7FFF, dtype=np.uint16)
    for i in range(2):
        for b, n in enumerate(lens):
            for h in range(bits.shape[2]):
                if n:
                    out[i, b, h, :n] = to16(quantise(x[i, b, h, :n], fmt, 64)[0], act)
    return out


def same(a, b):
    """Equal 16-bit values (a code 0 has no sign in int8: both zeros are one value)."""
    return np.array_equal(np.where(a == 0x8000, 0, a), np.where(b == 0x8000, 0, b))


def pair(shape, B, T, group=64):
    w = synth.make_weights(shape)
    ms = []
    for cls in (rv.Model, rv.Model, oracle.Model):
        m = cls(shape, w, B, T)
        m.quantize_river(group, 1)
        ms.append(m)
    for m in ms[:2]:
        m.set_debug(True)
    return ms


def check_step(gm, om, shape, lens_pre, g_next, g_exit, B):
    """Layer by layer against the oracle (see the module's text)."""
    L = shape.n_layers
    hid = gm.dump(rv.DUMP_HIDDEN)[:, :B].astype(np.float64)
    s_gpu = gm.dump(rv.DUMP_S)[:, :B]
    kv = gm.dump(rv.DUMP_KV)
    om.set_kv(kv, lens_pre)
    for l in range(1, L + 1):
        river = [1 if int(g_exit[b]) < l else 0 for b in range(B)]
        out = om.layer_forward(l, hid[l - 1], river)
        for b in range(B):
            r = rel_l2(hid[l, b], out[b])
            assert r <= TOL_HIDDEN, (l, b, r)
            if not river[b]:
                assert abs(float(s_gpu[l - 1, b]) - cos64(hid[l - 1, b], hid[l, b])) <= 1e-5
    for b in range(B):
        p = int(lens_pre[b]) + 1
        assert not (kv[:, :, b, :, :p] == 0x7FFF).any() and (kv[:, :, b, :, p:] == 0x7FFF).all()
    ol, _ = om.head(hid[L])
    assert np.abs(gm.dump(rv.DUMP_LOGITS)[:B] - ol).max() <= TOL_LOGIT
    for b in range(B):
        assert ol[b].max() - ol[b][int(g_next[b])] <= 2 * TOL_LOGIT


@pytest.mark.parametrize("kind,fmt", KINDS)
@pytest.mark.parametrize("shape,B", [(synth.TINY, 1), (SMALL, 1), (synth.TINY, 3), (SMALL, 5)])
def test_decode_on_the_8bit_cache(shape, B, kind, fmt):
    """Prefill, then decode across a block's border, forced exits at every
    layer: batch 1 (the GEMV chain) and batches (the rows path)."""
    T0, steps = 60, 9
    g16, g8, om = pair(shape, B, T0 + steps + 3)
    prompt = synth.make_prompt(shape.vocab, B, T0)
    g8.set_kv_cache(kind)
    L = shape.n_layers
    g8.prefill(prompt, 0.9, L)
    nxt, _ = g16.prefill(prompt, 0.9, L)
    act = shape.act_dtype
    ref = g16.dump(rv.DUMP_KV)
    got = g8.dump(rv.DUMP_KV)
    lens = [T0] * B
    # the prefill attends over its own 16-bit K/V: all layers hold the same values before quantisation
    for l in range(L):
        assert same(got[l], expect_layer(ref[l], lens, act, fmt)), l
    tok = nxt
    for step in range(steps):
        forced = np.array([(step + b) % (L + 1) for b in range(B)], dtype=np.int32)
        lens_pre = g8.dump(rv.DUMP_LENS).copy()
        g_next, g_exit = g8.decode_step(tok, 0.9, forced)
        assert np.array_equal(g_exit, forced)
        g16.decode_step(tok, 0.9, forced)
        check_step(g8, om, shape, lens_pre, g_next, g_exit, B)
        lens = [T0 + step + 1] * B
        if B == 1:  # the same kernels made the 16-bit K/V: the first layer's cache is exact
            assert same(g8.dump(rv.DUMP_KV)[0], expect_layer(g16.dump(rv.DUMP_KV)[0], lens, act, fmt))
        else:       # V is; K was turned by the rotary operator, whose sines differ in the last bits
            assert same(g8.dump(rv.DUMP_KV)[0, 1], expect_layer(g16.dump(rv.DUMP_KV)[0], lens, act, fmt)[1])
            a, b = kv_values(g8.dump(rv.DUMP_KV)[0, 0][:, :, :lens[0]], act), kv_values(expect_layer(g16.dump(rv.DUMP_KV)[0], lens, act, fmt)[0][:, :, :lens[0]], act)
            # a last bit of K before quantisation moves a code by one at most: a step of int8 (scale = amax / 127) or of e4m3
            assert np.abs(a - b).max() <= np.abs(b).max() * (1.1 / 127 if fmt == 0 else 2.0 ** -3)
        tok = g_next
    assert list(g8.dump(rv.DUMP_LENS)[:B]) == [T0 + steps] * B
    for m in (g16, g8, om):
        m.close()


def test_tau_rule_from_an_empty_cache_and_capacity():
    shape = synth.TINY
    _, g8, om = pair(shape, 2, 8)
    g8.set_kv_cache(rv.KV_INT8)
    tok = np.array([3, 900], dtype=np.int32)
    for step in range(8):
        lens_pre = g8.dump(rv.DUMP_LENS).copy()
        nxt, ex = g8.decode_step(tok, 0.9)
        check_step(g8, om, shape, lens_pre, nxt, ex, 2)
        tok = nxt
    with pytest.raises(rv.RVError) as e:
        g8.decode_step(tok, 0.9)
    assert e.value.code == rv.RV_ECAPACITY
    g8.kv_reset([0, 1])
    assert (g8.dump(rv.DUMP_KV) == 0x7FFF).all()
    one, _ = g8.prefill(np.array([[5], [6]], dtype=np.int32), 0.9, shape.n_layers)  # a prompt of one token
    assert (g8.dump(rv.DUMP_KV)[:, :, :, :, 0] != 0x7FFF).all() and (g8.dump(rv.DUMP_KV)[:, :, :, :, 1:] == 0x7FFF).all()
    ms, by = g8.time_kernel(rv.TIME_ATTN, 1, False, 3)
    assert ms > 0 and by == 2.0 * shape.n_kv_heads * (2 * shape.head_dim + 4)


def test_switching_caches():
    """There and back again: positions are forgotten, results of the 16-bit
    cache are what they were, memory follows, and what cannot be is refused."""
    shape = synth.TINY
    w = synth.make_weights(shape)
    m = rv.Model(shape, w, 2, 100)
    m.quantize_river(64)
    full = m.kv_bytes()
    assert m.kv_cache_bytes() == full
    prompt = synth.make_prompt(shape.vocab, 2, 70)

    def run():
        nxt, _ = m.prefill(prompt, 0.9)
        out = [nxt]
        for _ in range(5):
            nxt, ex = m.decode_step(nxt, 0.9)
            out += [nxt, ex]
        return np.concatenate(out), m.dump(rv.DUMP_KV).copy()

    ids, kv = run()
    m.set_kv_cache(rv.KV_E4M3)
    assert m.kv_bytes() == full and m.kv_cache_bytes() == shape.n_layers * 2 * 2 * shape.n_kv_heads * (128 * 64 + 2 * 4 + 128 * 64 * 2)
    assert (m.dump(rv.DUMP_LENS) == 0).all() and (m.dump(rv.DUMP_KV) == 0x7FFF).all()
    run()
    m.set_kv_cache(rv.KV_INT8)
    a = run()
    for bad in (3, -1):
        with pytest.raises(rv.RVError) as e:
            m.set_kv_cache(bad)
        assert e.value.code == rv.RV_EINVAL
    with pytest.raises(rv.RVError) as e:
        m.set_engine(rv.ENGINE_PERSISTENT)
    assert e.value.code == rv.RV_ESTATE
    for after in range(5):  # out of memory: nothing changes
        rv.debug_fail_alloc(after if after else 0)
        with pytest.raises(rv.RVError) as e:
            m.set_kv_cache(rv.KV_E4M3 if after else rv.KV_16BIT)
        rv.debug_fail_alloc(-1)
        assert e.value.code == rv.RV_ENOMEM
    b = run()
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    m.set_kv_cache(rv.KV_16BIT)
    assert m.kv_cache_bytes() == full and (m.dump(rv.DUMP_KV) == 0x7FFF).all()
    ids2, kv2 = run()
    assert np.array_equal(ids, ids2) and np.array_equal(kv, kv2)
    m.set_engine(rv.ENGINE_PERSISTENT)
    with pytest.raises(rv.RVError) as e:
        m.set_kv_cache(rv.KV_INT8)
    assert e.value.code == rv.RV_ESTATE
    m.close()


def test_offloaded_river_on_the_8bit_cache():
    shape = synth.TINY
    _, g8, om = pair(shape, 1, 40)
    g8.set_kv_cache(rv.KV_INT8)
    g8.offload_backbone(2)
    g8.prefill(synth.make_prompt(shape.vocab, 1, 20), 0.9, 2)
    lens = g8.dump(rv.DUMP_LENS).copy()
    nxt, ex = g8.decode_step([7], 2.0)  # no similarity passes 2: the cap ends the backbone
    assert ex[0] == 2
    check_step(g8, om, shape, lens, nxt, ex, 1)


@pytest.mark.parametrize("kind", [rv.KV_16BIT, rv.KV_INT8])
@pytest.mark.parametrize("scaling", ["linear", "ramp"])
def test_scaled_rotary_frequencies(kind, scaling):
    """With frequencies divided by 4 a model at position 4 p turns as the plain
    one at p; here: the first layer's K of a prefill against the plain K turned
    by the difference in 64 bits, and a decode step that follows it."""
    shape = synth.TINY
    hd, T0 = shape.head_dim, 33
    w = synth.make_weights(shape)
    m = rv.Model(shape, w, 2, 64)
    prompt = synth.make_prompt(shape.vocab, 2, T0)
    L = shape.n_layers
    m.prefill(prompt, 0.9, L)
    plain = kv_values(m.dump(rv.DUMP_KV)[0, 0][:, :, :T0], shape.act_dtype).astype(np.float64)
    kw = dict(factor=4.0) if scaling == "linear" else dict(factor=4.0, original=32, fast=4.0, slow=1.0)
    cfg = rv.RopeConfig(hd, hd, rv.ROPE_HALF, rv.ROPE_LINEAR if scaling == "linear" else rv.ROPE_RAMP, kw.get("original", 0),
                        shape.rope_theta, kw["factor"], 0.0, 0.0, kw.get("fast", 0.0), kw.get("slow", 0.0), 0.0)
    m.set_kv_cache(kind)
    m.set_rope(cfg)
    assert (m.dump(rv.DUMP_LENS) == 0).all()
    m.prefill(prompt, 0.9, L)
    nxt, _ = m.decode_step(prompt[:, 0], 0.9, [L, L])  # position T0: the first token again
    got = kv_values(m.dump(rv.DUMP_KV)[0, 0][:, :, :T0 + 1], shape.act_dtype).astype(np.float64)
    f0, _ = rope_frequencies(hd, shape.rope_theta)
    f1, att = rope_frequencies(hd, shape.rope_theta, scaling, **kw)
    n = hd // 2
    at = np.arange(T0 + 1)[:, None]
    before = np.concatenate([plain, plain[:, :, :1]], 2)                   # what was turned by f0 at its place (the last at 0)
    ang = att * np.exp(1j * (at * f1 - np.concatenate([at[:-1], [[0]]]) * f0))
    z = (before[..., :n] + 1j * before[..., n:]) * ang
    ref = np.concatenate([z.real, z.imag], -1)
    # both were rounded to fp16 (2 x 2^-11 of a pair's size) and, in 8 bits, to steps of amax / 127 per block (up8: x 1 + 2^-7)
    size = np.abs(z).max() * (2.0 ** -10 + (0.51 / 127 if kind else 0.0))
    assert np.abs(got - ref).max() <= size
    m.set_rope(None)
    m.set_kv_cache(rv.KV_16BIT)
    m.prefill(prompt, 0.9, L)
    assert np.array_equal(kv_values(m.dump(rv.DUMP_KV)[0, 0][:, :, :T0], shape.act_dtype), plain)
    for bad in (dict(head_dim=128), dict(rotary_dim=32), dict(layout=rv.ROPE_INTERLEAVED), dict(scaling=9)):
        c = rv.RopeConfig.from_buffer_copy(cfg)
        for k, v in bad.items():
            setattr(c, k, v)
        with pytest.raises(rv.RVError) as e:
            m.set_rope(c)
        assert e.value.code == rv.RV_EINVAL
    m.close()


def test_plain_frequencies_that_the_8bit_cache_lacks():
    """rope_theta 1 has no plan: the 8-bit cache works on frequencies that were set, and they cannot be taken away."""
    shape = synth.ModelShape("kv8-theta1", 2, 256, 4, 2, 64, 256, 512, 0, synth.BF16, 1e-5, 1.0)
    m = rv.Model(shape, synth.make_weights(shape), 2, 64)
    with pytest.raises(rv.RVError) as e:
        m.set_kv_cache(rv.KV_INT8)
    assert e.value.code == rv.RV_EINVAL
    cfg = rv.RopeConfig(64, 64, rv.ROPE_HALF, rv.ROPE_PLAIN, 0, 10000.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0)
    m.set_rope(cfg)
    m.set_kv_cache(rv.KV_INT8)
    L, prompt = shape.n_layers, synth.make_prompt(shape.vocab, 2, 5)
    m.prefill(prompt, 0.9, L)
    with pytest.raises(rv.RVError) as e:
        m.set_rope(None)
    assert e.value.code == rv.RV_ESTATE
    assert list(m.dump(rv.DUMP_LENS)[:2]) == [5, 5]  # nothing changed
    m.decode_step(prompt[:, 0], 0.9, [L, L])
    m.set_kv_cache(rv.KV_16BIT)
    m.set_rope(None)
    m.prefill(prompt, 0.9, L)
    m.close()
