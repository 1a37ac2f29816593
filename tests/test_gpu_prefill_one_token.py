"""A prompt of one token, on every K/V cache: the oracle's layers and greedy
pick from the GPU's own states, the same hidden states whichever cache is
filled (a prefill attends over its own 16-bit K/V), the cache's values, and the
decode step that follows."""
import numpy as np
import pytest

import oracle
import synth
import token_level_early_gb300 as rv
from gpu_util import TIE_LOGIT, TOL_HIDDEN, TOL_LOGIT, check_ids, rel_l2
from test_gpu_kv8_model import KINDS, SMALL, check_step, expect_layer, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("exit_layer", [1, 99])
@pytest.mark.parametrize("shape,B", [(synth.TINY, 1), (synth.TINY, 3), (SMALL, 1), (SMALL, 2)])
def test_one_token_prompt(shape, B, exit_layer):
    L = shape.n_layers
    exit_layer = min(exit_layer, L)
    w = synth.make_weights(shape)
    prompt = synth.make_prompt(shape.vocab, B, 1)
    om = oracle.Model(shape, w, B, 8)
    om.quantize_river(64, 1)
    m = rv.Model(shape, w, B, 8)
    m.quantize_river(64, 1)
    m.set_debug(True)

    # 16 bits
    nxt, ex = m.prefill(prompt, 0.9, exit_layer)
    hid, kv = m.dump(rv.DUMP_HIDDEN)[:, :B].copy(), m.dump(rv.DUMP_KV).copy()
    assert list(ex) == [exit_layer] * B and list(m.dump(rv.DUMP_LENS)[:B]) == [1] * B
    assert not (kv[:, :, :, :, 0] == 0x7FFF).any() and (kv[:, :, :, :, 1:] == 0x7FFF).all()
    om.set_kv(np.full_like(kv, 0x7FFF), np.zeros(B, dtype=np.int32))
    for l in range(1, L + 1):
        out = om.layer_forward(l, hid[l - 1].astype(np.float64), [1 if l > exit_layer else 0] * B)
        for b in range(B):
            assert rel_l2(hid[l, b], out[b]) <= TOL_HIDDEN, (l, b)
    ol, _ = om.head(hid[L].astype(np.float64))
    assert np.abs(m.dump(rv.DUMP_LOGITS)[:B] - ol).max() <= TOL_LOGIT
    check_ids(nxt, ol, TIE_LOGIT)
    n2, _ = m.decode_step(nxt, 0.9, [L] * B)
    kv2 = m.dump(rv.DUMP_KV).copy()
    assert np.array_equal(kv2[:, :, :, :, 0], kv[:, :, :, :, 0])
    check_step(m, om, shape, [1] * B, n2, [L] * B, B)

    # 8 bits: the same states, and every layer holds the codes of the 16-bit values
    for kind, fmt in KINDS:
        m.set_kv_cache(kind)
        n8, _ = m.prefill(prompt, 0.9, exit_layer)
        assert np.array_equal(m.dump(rv.DUMP_HIDDEN)[:, :B], hid) and np.array_equal(n8, nxt)
        got = m.dump(rv.DUMP_KV)
        for l in range(L):
            assert same(got[l], expect_layer(kv[l], [1] * B, shape.act_dtype, fmt)), (kind, l)
        # The step that follows quantises the block anew from the prompt's originals.  The first layer's V depend on
        # the tokens alone (K of a batch is turned by another kernel, whose sines differ in the last bits).  No oracle
        # step here: its own token is not quantised, and that is one of two positions.
        m.decode_step(n8, 0.9, [L] * B)
        got, want = m.dump(rv.DUMP_KV)[0], expect_layer(kv2[0], [2] * B, shape.act_dtype, fmt)
        assert same(got[1], want[1]) and (B > 1 or same(got[0], want[0]))
    m.close()
    om.close()
