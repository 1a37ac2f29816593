"""Several answers to one prompt from end to end: the prompt cached once, rows
that share it and rows that hold copies of it, tokens drawn, kept rows put into a
new order, and on."""
import math

import numpy as np
import pytest
import torch

import token_level_early_gb300 as rv
from answers_util import attention_parts, draw
from test_gpu_kv8 import Cache, data, expect, f64

pytestmark = pytest.mark.gpu
ACT = {0: torch.float16, 1: torch.bfloat16}


def ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def copy(src, dst, pairs):
    f, t, n = (ints([p[i] for p in pairs]) for i in range(3))
    rv.kv8_copy(src.c, dst.c, len(pairs), f.data_ptr(), t.data_ptr(), n.data_ptr(), dst.err.data_ptr())
    torch.cuda.synchronize()
    assert int(dst.err) == 0


def shared(pre, own, q, fan, n, pos, scale):
    B, T, H, _ = q.shape
    need = rv.kv8_attention_shared_workspace(pre.c, own.c, B, T, fan, H)
    work = torch.full((need,), 0xFF, dtype=torch.uint8).cuda()
    out, pl, po = torch.zeros_like(q), ints(n), ints(pos)
    rv.kv8_attention_shared(pre.c, own.c, rv.heads(q), rv.heads(out), B, T, fan, scale, pl.data_ptr(), po.data_ptr(), None, None, own.err.data_ptr(),
                            work.data_ptr(), need)
    torch.cuda.synchronize()
    assert int(own.err) == 0
    return out


@pytest.mark.parametrize("act,fmt,hd", [(1, 0, 128), (0, 1, 64)])
def test_answers_to_a_prompt(act, fmt, hd):
    """Five steps of six rows: the attention within its bounds of the definition
    on what the caches hold, the tokens those of the plain draw on the same
    logits, a new order of the rows carried along by every later step."""
    n, rows, Hkv, H, V, block, steps = 389, 6, 2, 8, 501, 32, 5
    g = torch.Generator().manual_seed(7)
    embed = torch.randn(V, Hkv, hd, generator=g).to(ACT[act]).cuda()
    mix = (torch.randn(H * hd, V, generator=g) / math.sqrt(hd)).cuda()
    pk, pv = data(1, 1, n, Hkv, hd, act, spread=False), data(2, 1, n, Hkv, hd, act, spread=False)
    pre = Cache(1, Hkv, hd, n, block, fmt, act)
    pre.append(pk, pv, [0])
    vals = [expect(pre, f64(x)[0], n)[0] for x in (pk, pv)]
    own = Cache(rows, Hkv, hd, 32, block, fmt, act)
    whole = Cache(rows, Hkv, hd, n + 32, block, fmt, act)   # each row its own copy of the prompt
    copy(pre, whole, [(0, b, n) for b in range(rows)])
    new_k, new_v = (torch.zeros(rows, steps, Hkv, hd, dtype=ACT[act]).cuda() for _ in range(2))
    tokens = list(range(rows))
    scale, rng = hd ** -0.5, np.random.default_rng(3)
    for step in range(steps):
        k = embed[tokens].unsqueeze(1).contiguous()
        v = embed[[(t * 7 + 1) % V for t in tokens]].unsqueeze(1).contiguous()
        q = embed[[(t * 3 + 2) % V for t in tokens]].repeat_interleave(H // Hkv, dim=1).unsqueeze(1).contiguous()
        new_k[:, step], new_v[:, step] = k[:, 0], v[:, 0]
        own.append(k, v, [step] * rows)
        whole.append(k, v, [n + step] * rows)
        out = shared(pre, own, q, rows, [n], [step] * rows, scale)
        plain, _ = whole.attention(q, scale, [n + step] * rows)
        for b in range(rows):
            ok, ov = (expect(own, f64(x)[b], step + 1)[0] for x in (new_k, new_v))
            for h in range(H):
                j = h * Hkv // H
                ref, _, _, bound = attention_parts(f64(q)[b, 0, h], [(vals[0][:, j], vals[1][:, j], block), (ok[:, j], ov[:, j], block)], scale, act == 0)
                assert (np.abs(f64(out)[b, 0, h] - ref) <= bound(str(out.dtype).split(".")[1])).all(), (step, b, h)
        # the copies' open block has one scale for the prompt's end and the new tokens: within a step of its codes
        top = max(float(f64(s)[:, :, n // block:(n + step) // block + 1].max()) for s in whole.scale)
        assert (plain.float() - out.float()).abs().max() <= 16 * top + 0.02 * float(out.float().abs().max())
        logits = out.float().reshape(rows, -1) @ mix
        u = torch.tensor(rng.random(rows), dtype=torch.float32).cuda()
        t, kk, p, m = torch.full((rows,), 0.9).cuda(), ints([50] * rows), torch.full((rows,), 0.9).cuda(), torch.full((rows,), 0.01).cuda()
        ids, lp = torch.zeros(rows, dtype=torch.int32).cuda(), torch.zeros(rows).cuda()
        torch.cuda.synchronize()
        rv.sample(logits.data_ptr(), rv.F32, V, rows, V, t.data_ptr(), kk.data_ptr(), p.data_ptr(), m.data_ptr(), u.data_ptr(), ids.data_ptr(), lp.data_ptr())
        torch.cuda.synchronize()
        want = [draw(r, float(np.float32(0.9)), 50, float(np.float32(0.9)), float(np.float32(0.01)), float(x))
                for r, x in zip(logits.double().cpu().tolist(), u.double().cpu().tolist())]
        assert ids.cpu().tolist() == [i for i, _ in want]
        tokens = ids.cpu().tolist()
        order = [int(x) for x in rng.integers(0, rows, rows)] if step % 2 else [int(x) for x in rng.permutation(rows)]
        copy(own, own, [(a, b, step + 1) for b, a in enumerate(order)])
        copy(whole, whole, [(a, b, n + step + 1) for b, a in enumerate(order)])
        new_k, new_v, tokens = new_k[order].contiguous(), new_v[order].contiguous(), [tokens[a] for a in order]


def test_rows_in_a_new_order_give_the_same_bits():
    Hkv, hd, block, rows, n = 2, 64, 16, 5, 210
    pre = Cache(1, Hkv, hd, n, block, 0, 1)
    pre.append(data(1, 1, n, Hkv, hd, 1), data(2, 1, n, Hkv, hd, 1), [0])
    own = Cache(rows, Hkv, hd, 64, block, 0, 1)
    own.append(data(3, rows, 37, Hkv, hd, 1), data(4, rows, 37, Hkv, hd, 1), [0] * rows)
    q = torch.randn(rows, 1, 8, hd, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    a = shared(pre, own, q, rows, [n], [36] * rows, 0.1)
    order = [3, 0, 4, 1, 2]
    copy(own, own, [(x, b, 37) for b, x in enumerate(order)])
    b = shared(pre, own, q[order].contiguous(), rows, [n], [36] * rows, 0.1)
    assert torch.equal(a[order], b)


def test_a_cache_may_be_prefix_and_own_at_once():
    """Rows of one cache: row 0's prompt, read by rows that also hold positions there."""
    Hkv, hd, block, rows = 2, 128, 64, 4
    c = Cache(rows, Hkv, hd, 300, block, 0, 1)
    k, v = data(1, rows, 200, Hkv, hd, 1, spread=False), data(2, rows, 200, Hkv, hd, 1, spread=False)
    c.append(k, v, [0] * rows, [200, 3, 4, 5])
    q = torch.randn(rows, 1, 4, hd, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    out = shared(c, c, q, rows, [200], [-1, 2, 3, 4], 0.1)
    kk, vv = (expect(c, f64(x)[0], 200)[0] for x in (k, v))
    for b, m in enumerate((0, 3, 4, 5)):
        ok, ov = (expect(c, f64(x)[b], m)[0] if m else np.zeros((0, Hkv, hd)) for x in (k, v))
        for h in range(4):
            ref, _, _, bound = attention_parts(f64(q)[b, 0, h], [(kk[:, h // 2], vv[:, h // 2], block), (ok[:, h // 2], ov[:, h // 2], block)], 0.1, False)
            assert (np.abs(f64(out)[b, 0, h] - ref) <= bound("bfloat16")).all()
