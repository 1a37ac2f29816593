"""The 8-bit K/V cache and its attention against the definition in 64 bits.

Codes and scales have to be equal to the definition's bit for bit: x / s is
either exactly a midpoint between codes or too far from one for fp32 to
round it the other way (see kv8.cu), and a scale is exact.  The attention's
bounds are derived in kv8_util."""
import math

import numpy as np
import pytest
import torch

import token_level_early_gb300 as rv
from kv8_util import attention, lse_tolerance, quantise

pytestmark = pytest.mark.gpu

ACT = {0: torch.float16, 1: torch.bfloat16}


def f64(t):
    return t.detach().double().cpu().numpy()


class Cache:
    """A cache of one layer in torch memory, filled with bytes that no call may rely on."""

    def __init__(self, B, Hkv, hd, max_seq, block, fmt, act, junk=0x7F):
        n = -(-max_seq // block) * block
        self.B, self.Hkv, self.hd, self.T, self.block, self.fmt, self.act, self.N = B, Hkv, hd, max_seq, block, fmt, act, n
        self.codes = [torch.full((B, Hkv, n, hd), junk, dtype=torch.uint8).cuda() for _ in range(2)]
        self.scale = [torch.full((B, Hkv, n // block), math.nan).cuda() for _ in range(2)]
        self.tail = [torch.full((B, Hkv, 2 * block, hd), math.nan, dtype=ACT[act]).cuda() for _ in range(2)]
        self.err = torch.zeros(1, dtype=torch.int32).cuda()
        self.c = rv.KV8(B, Hkv, hd, max_seq, block, fmt, act, *(t.data_ptr() for x in (self.codes, self.scale, self.tail) for t in x))

    def append(self, k, v, pos, count=None, err=True):
        p = torch.tensor(pos, dtype=torch.int32).cuda()
        n = None if count is None else torch.tensor(count, dtype=torch.int32).cuda()
        rv.kv8_append(self.c, rv.heads(k), rv.heads(v), k.shape[0], k.shape[1], p.data_ptr(), None if n is None else n.data_ptr(),
                      self.err.data_ptr() if err else None)
        torch.cuda.synchronize()

    def read(self, pos, T, dtype=torch.float32, count=None, fill=7.0):
        p = torch.tensor(pos, dtype=torch.int32).cuda()
        n = None if count is None else torch.tensor(count, dtype=torch.int32).cuda()
        out = [torch.full((len(pos), T, self.Hkv, self.hd), fill, dtype=dtype).cuda() for _ in range(2)]
        rv.kv8_read(self.c, rv.heads(out[0]), rv.heads(out[1]), len(pos), T, p.data_ptr(), None if n is None else n.data_ptr(), self.err.data_ptr())
        torch.cuda.synchronize()
        return out

    def attention(self, q, scale, pos, count=None, out=None, lse=True, stream=None):
        B, T, H, _ = q.shape
        p = torch.tensor(pos, dtype=torch.int32).cuda()
        n = None if count is None else torch.tensor(count, dtype=torch.int32).cuda()
        out = torch.full_like(q, 7.0) if out is None else out
        ls = torch.full((B, T, H), 7.0).cuda()
        need = rv.kv8_attention_workspace(self.c, B, T, H)
        work = torch.full((max(need, 16),), 0xFF, dtype=torch.uint8).cuda()  # NaNs: nothing may be read before it is written
        rv.kv8_attention(self.c, rv.heads(q), rv.heads(out), B, T, scale, p.data_ptr(), None if n is None else n.data_ptr(),
                         ls.data_ptr() if lse else None, work.data_ptr(), need)
        torch.cuda.synchronize()
        return out, ls


def data(seed, B, T, H, hd, act, spread=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, T, H, hd, generator=g)
    if spread:
        x = x * (torch.rand(hd, generator=g) * 2 + 0.05) * torch.exp2(torch.randint(-6, 6, (B, T, H, 1), generator=g).float())
    return x.to(ACT[act]).cuda()


def expect(cache, x, n):
    """values and scales of row tokens x [n][Hkv][hd] (float64 numpy)."""
    val = np.zeros((n, cache.Hkv, cache.hd))
    sc = np.zeros((cache.Hkv, -(-n // cache.block)))
    for h in range(cache.Hkv):
        val[:, h], sc[h] = quantise(x[:n, h], cache.fmt, cache.block)
    return val, sc


def check_cache(cache, rows_k, rows_v, lens):
    """The cache's rows hold rows_k / rows_v [B][T][Hkv][hd] up to lens."""
    T = max(max(lens), 1)
    got = cache.read([0] * len(lens), T, count=lens)
    for x, rows, sc in zip(got, (rows_k, rows_v), cache.scale):
        for b, n in enumerate(lens):
            val, s = expect(cache, f64(rows)[b], n)
            assert np.array_equal(f64(x)[b, :n], val), (b, n)
            assert np.array_equal(f64(sc)[b, :, :s.shape[1]], s), (b, n)
            assert (x[b, n:] == 7.0).all()


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("block,hd", [(16, 64), (32, 128), (64, 64), (64, 128), (128, 128), (16, 128), (128, 64)])
def test_append_at_once_and_in_pieces(block, hd, act, fmt):
    """However the tokens come in, the cache is the same function of them."""
    B, Hkv, T = 2, 3, 3 * block + 5
    k, v = data(1, B, T, Hkv, hd, act), data(2, B, T, Hkv, hd, act)
    whole = Cache(B, Hkv, hd, T + 3, block, fmt, act)
    whole.append(k, v, [0] * B)
    check_cache(whole, k, v, [T] * B)
    parts = Cache(B, Hkv, hd, T + 3, block, fmt, act, junk=0xFF)
    at = 0
    for n in (1, 1, block - 3, 2, block + 1, 7, T):
        n = min(n, T - at)
        if n:
            parts.append(k[:, at:at + n].contiguous(), v[:, at:at + n].contiguous(), [at] * B)
            at += n
            check_cache(parts, k, v, [at] * B)
    assert at == T
    for a, b in zip(whole.codes + whole.scale, parts.codes + parts.scale):
        assert torch.equal(a.reshape(B, Hkv, -1)[..., :T * hd if a.dtype == torch.uint8 else -(-T // block)],
                           b.reshape(B, Hkv, -1)[..., :T * hd if a.dtype == torch.uint8 else -(-T // block)])
    for a, b in zip(whole.tail, parts.tail):
        for p in range(max(0, T - 2 * block), T):
            assert torch.equal(a[:, :, p % (2 * block)], b[:, :, p % (2 * block)])
    assert int(whole.err) == 0 and int(parts.err) == 0


def test_append_ragged_rows_strides_and_types():
    """Rows at different positions with different counts, [B][heads][T][hd]
    inputs, fp32 inputs (rounded first), rows beyond B left alone."""
    B, Hkv, hd, block = 4, 2, 64, 16
    lens, add = [0, 13, 16, 40], [21, 0, 1, 9]
    old_k, old_v = data(3, B, 40, Hkv, hd, 1), data(4, B, 40, Hkv, hd, 1)
    wide = torch.randn(2, B, Hkv, 25, hd + 4, generator=torch.Generator().manual_seed(9)).cuda()
    new = [w[:, :, 2:23, :hd].transpose(1, 2) for w in wide]  # fp32, heads outside tokens, padded rows
    c = Cache(B + 1, Hkv, hd, 64, block, 0, 1)
    c.append(old_k, old_v, [0] * B, lens)
    before = [t[B].clone() for t in c.codes + c.scale + c.tail]
    c.append(new[0], new[1], lens, add)
    full = []
    for old, n in ((old_k, new[0]), (old_v, new[1])):
        f = torch.zeros(B, 64, Hkv, hd, dtype=torch.bfloat16).cuda()
        for b in range(B):
            f[b, :lens[b]] = old[b, :lens[b]]
            f[b, lens[b]:lens[b] + add[b]] = n[b, :add[b]].to(torch.bfloat16)
        full.append(f)
    check_cache(c, full[0], full[1], [a + b for a, b in zip(lens, add)])
    for a, b in zip(before, [t[B] for t in c.codes + c.scale + c.tail]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert int(c.err) == 0


@pytest.mark.parametrize("back", [1, 5, 16])
def test_append_goes_back_and_continues(back):
    """Drafted tokens refused: up to `block` positions are taken back, across a
    block border, and the cache forgets them."""
    B, Hkv, hd, block, act = 1, 2, 64, 16, 1
    T = 35
    k, v = data(5, B, T, Hkv, hd, act), data(6, B, T, Hkv, hd, act)
    k[:, T - back:] *= 64.0  # the refused tokens would have set the scale
    k2, v2 = data(7, B, 9, Hkv, hd, act), data(8, B, 9, Hkv, hd, act)
    c = Cache(B, Hkv, hd, 64, block, 0, act)
    c.append(k, v, [0])
    c.append(k2, v2, [T - back])
    kk, vv = torch.cat([k[:, :T - back], k2], 1), torch.cat([v[:, :T - back], v2], 1)
    check_cache(c, kk, vv, [T - back + 9])


@pytest.mark.parametrize("fmt", [0, 1])
def test_append_special_values(fmt):
    """All-zero blocks, the smallest and largest magnitudes, and blocks with an
    infinity or a NaN, which poison themselves and no other block or head."""
    Hkv, hd, block = 2, 64, 16
    x = torch.zeros(1, 6 * block, Hkv, hd)
    x[0, block:2 * block, 0] = 1e-39              # below the smallest scale's half step
    x[0, block + 1, 1, 3] = 2.0 ** 126
    x[0, 2 * block:3 * block] = torch.randn(block, Hkv, hd, generator=torch.Generator().manual_seed(1))
    x[0, 2 * block + 4, 0, 5] = math.inf
    x[0, 3 * block:4 * block] = 0.25
    x[0, 3 * block + 2, 1, 63] = math.nan
    x[0, 4 * block:5 * block, 0] = -3.0
    x[0, 5 * block:, 1] = 2.0 ** -99
    k = x.to(torch.bfloat16).cuda()
    c = Cache(1, Hkv, hd, 6 * block, block, fmt, 1)
    c.append(k, k, [0])
    got = c.read([0], 6 * block)
    for y in got:
        y = f64(y)[0]
        for h in range(Hkv):
            ref, s = quantise(f64(k)[0, :, h], fmt, block)
            np.testing.assert_array_equal(y[:, h], ref)
            np.testing.assert_array_equal(f64(c.scale[0])[0, h], s)
        assert np.isnan(y[2 * block:3 * block, 0]).all() and np.isfinite(y[2 * block:3 * block, 1]).all()
        assert np.isnan(y[3 * block:4 * block, 1]).all() and np.isfinite(y[3 * block:4 * block, 0]).all()


def test_codes_take_every_tie_to_even():
    """Values that lie exactly between two codes, and next to them."""
    for fmt, act in ((0, 0), (0, 1), (1, 0), (1, 1)):
        for top in (127.0, 448.0, 1.0, 3.140625):
            grid = torch.arange(-255, 256) / 2.0 if fmt == 0 else torch.tensor(
                [s * (m / 16.0) * 2.0 ** e for s in (-1, 1) for e in range(-9, 9) for m in range(16, 32)])
            s = float(quantise(np.array([[top]]), fmt, 16)[1][0])
            x = (grid.double() * s).to(ACT[act]).double()
            x = x[x.abs() <= top]
            x = torch.cat([x, torch.tensor([top], dtype=torch.float64)])
            n = -(-len(x) // 64) * 64
            x = torch.cat([x, torch.zeros(n - len(x), dtype=torch.float64)]).view(-1, 64)
            for i in range(0, x.shape[0], 16):
                y = x[i:i + 16]
                k = torch.zeros(1, 16, 1, 64, dtype=torch.float64)
                k[0, :y.shape[0], 0] = y
                k[0, 15, 0, 63] = top
                k = k.to(ACT[act]).cuda()
                c = Cache(1, 1, 64, 16, 16, fmt, act)
                c.append(k, k, [0])
                check_cache(c, k, k, [16])


def test_append_and_read_report_positions_outside():
    c = Cache(3, 1, 64, 20, 16, 0, 0)
    k = data(1, 3, 8, 1, 64, 0)
    c.append(k, k, [-1, 16, 0])       # row 0 is refused, row 1 loses its last 4 tokens
    assert int(c.err) == 64
    c.err.zero_()
    assert torch.isnan(c.tail[0][0]).all()
    got = c.read([16, 16, -2], 8)     # only positions 16..19 of rows 0, 1 and 0..5 of row 2 exist
    assert int(c.err) == 64
    ref, _ = quantise(f64(k)[1, :4, 0], 0, 16)
    assert np.array_equal(f64(got[0])[1, :4, 0], ref)
    assert (got[0][:2, 4:] == 7.0).all() and (got[0][2, :2] == 7.0).all()
    val, _ = expect(c, f64(k)[2], 6)
    # row 2's first block holds 8 tokens: its scale is theirs
    val8, _ = expect(c, f64(k)[2], 8)
    assert np.array_equal(f64(got[0])[2, 2:], val8[:6]) and val.shape == (6, 1, 64)


def test_append_at_the_caches_end_changes_nothing():
    """A first position at or behind max_seq, in the last open block's range too."""
    c = Cache(2, 2, 64, 20, 16, 0, 0)
    k = data(1, 2, 20, 2, 64, 0)
    c.append(k, k, [0, 0])
    before = [t.clone() for t in c.codes + c.scale + c.tail]
    for pos in (20, 21, 31, 32, 2 ** 31 - 1):
        c.append(k[:, :3].contiguous() * 5, k[:, :3].contiguous() * 5, [pos, pos])
        assert int(c.err) == 64
        c.err.zero_()
    c.append(k, k, [20, 20], [0, 0])  # no tokens: no error either
    assert int(c.err) == 0
    for a, b in zip(before, c.codes + c.scale + c.tail):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("act", [0, 1])
def test_read_rounds_once_and_saturates(act):
    c = Cache(1, 1, 64, 48, 16, 0, act)
    k = data(3, 1, 48, 1, 64, act)
    big = torch.finfo(ACT[act]).max
    k[0, 32, 0, 0], k[0, 33, 0, 1] = big, -big
    c.append(k, k, [0])
    val, _ = expect(c, f64(k)[0], 48)
    for dtype in (torch.float16, torch.bfloat16):
        got = c.read([0], 48, dtype=dtype)[0]
        top = torch.finfo(dtype).max
        ref = torch.from_numpy(val).clamp(-top, top).to(dtype)
        assert torch.equal(got[0].cpu(), ref)
        assert torch.isfinite(got).all()
    only = torch.zeros(1, 48, 1, 64).cuda()
    rv.kv8_read(c.c, None, rv.heads(only), 1, 48, None)
    torch.cuda.synchronize()
    assert np.array_equal(f64(only)[0], val)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (16, 8), (24, 16)])
def test_read_into_strided_outputs(dtype, pad, shift):
    """Rows on 16-byte and on 32-byte boundaries, heads outside tokens, ragged
    counts, a head count that does not fill a block's threads; nothing else is
    touched."""
    B, Hkv, hd, T, block = 2, 5, 128, 37, 32
    c = Cache(B, Hkv, hd, 64, block, 1, 1)
    k, v = data(51, B, 40, Hkv, hd, 1), data(52, B, 40, Hkv, hd, 1)
    c.append(k, v, [0] * B)
    pos, count = [3, 11], [T, 20]
    p, n = (torch.tensor(x, dtype=torch.int32).cuda() for x in (pos, count))
    big = [torch.full((B, Hkv, T, hd + pad + shift), 7.0, dtype=dtype).cuda() for _ in range(2)]
    out = [x[..., shift:shift + hd].transpose(1, 2) for x in big]
    rv.kv8_read(c.c, rv.heads(out[0]), rv.heads(out[1]), B, T, p.data_ptr(), n.data_ptr(), c.err.data_ptr())
    torch.cuda.synchronize()
    top = torch.finfo(dtype).max
    for x, full, src in zip(out, big, (k, v)):
        for b in range(B):
            ref = torch.from_numpy(expect(c, f64(src)[b], 40)[0][pos[b]:pos[b] + count[b]]).clamp(-top, top).to(dtype)
            assert torch.equal(x[b, :count[b]].cpu(), ref)
            assert (x[b, count[b]:] == 7.0).all()
        full[..., shift:shift + hd] = 7.0
        assert (full == 7.0).all()
    assert int(c.err) == 0


# ------------------------------------------------------------------ attention

def check_attention(c, kk, vv, q, scale, pos, count, out, lse):
    """out, lse of query rows over the values the cache stands for (kk, vv [B][n][Hkv][hd] float64)."""
    B, T, H, hd = q.shape
    grp = H // c.Hkv
    name = str(out.dtype).split(".")[1]
    for b in range(B):
        nq = T if count is None else min(max(count[b], 0), T)
        assert (out[b, nq:] == 7.0).all() and (lse[b, nq:] == 7.0).all()
        for t in range(nq):
            n = min(max(pos[b] + t + 1, 0), c.T)
            for h in range(H):
                k, v = kk[b][:, h // grp], vv[b][:, h // grp]
                ref, rl, D, bound = attention(f64(q)[b, t, h], k, v, scale, n, c.block)
                got, gl = f64(out)[b, t, h], float(lse[b, t, h])
                if n == 0:
                    assert (got == 0).all() and gl == -math.inf
                    continue
                tol = bound(name)
                err = np.abs(got - ref)
                assert (err <= tol).all(), (b, t, h, n, float((err / tol).max()))
                assert abs(gl - rl) <= lse_tolerance(rl, D), (b, t, h, gl, rl)


@pytest.fixture(params=[0, 70000], ids=["cluster", "line"])
def room(request):
    """Smallest max_seq of a test's caches: small caches run the attention's
    cluster plan, large ones (however little they hold) the cut line."""
    return request.param


def filled(B, Hkv, hd, block, fmt, act, lens, max_seq, seed=1, room=0):
    c = Cache(B, Hkv, hd, max(max_seq, room), block, fmt, act)
    T = max(max(lens), 1)
    k, v = data(seed, B, T, Hkv, hd, act, False), data(seed + 1, B, T, Hkv, hd, act, False)
    k[..., 3] *= 6.0
    c.append(k, v, [0] * B, lens)
    kk = [expect(c, f64(k)[b], lens[b])[0] for b in range(B)]
    vv = [expect(c, f64(v)[b], lens[b])[0] for b in range(B)]
    return c, kk, vv


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_attention_types_and_blocks(block, hd, fmt, act, room):
    lens = [1, 31, 200, 130]
    B, Hkv, H = 4, 2, 8
    c, kk, vv = filled(B, Hkv, hd, block, fmt, act, lens, 205, room=room)
    q = data(9, B, 1, H, hd, act, False)
    pos = [n - 1 for n in lens]
    out, lse = c.attention(q, hd ** -0.5, pos)
    check_attention(c, kk, vv, q, hd ** -0.5, pos, None, out, lse)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 3), (8, 1), (7, 1), (16, 1), (20, 1), (10, 2), (32, 8)])
@pytest.mark.parametrize("T", [1, 2, 5, 16])
def test_attention_head_layouts_and_drafted_tokens(T, H, Hkv, room):
    """Query rows of every count per KV head (T x H / Hkv from 1 to 320), with
    ragged counts and rows that see little or nothing."""
    lens, act, hd = [300, 17, T, 97], 1, 64
    B = 4
    c, kk, vv = filled(B, Hkv, hd, 32, 0, act, lens, 320, room=room)
    q = data(10, B, T, H, hd, act, False)
    pos = [300 - T, 17 - T, -2, 97 - T]
    count = [T, max(T - 1, 1), T, 0]
    out, lse = c.attention(q, 0.2, pos, count)
    check_attention(c, kk, vv, q, 0.2, pos, count, out, lse)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 511, 1000, 2047, 2049, 5000])
def test_attention_lengths(n, room):
    c, kk, vv = filled(1, 1, 128, 64, 0, 1, [n], n, room=room)
    q = data(11, 1, 1, 4, 128, 1, False)
    out, lse = c.attention(q, 128 ** -0.5, [n - 1])
    check_attention(c, kk, vv, q, 128 ** -0.5, [n - 1], None, out, lse)


def test_attention_many_rows_of_unequal_length(room):
    B, Hkv, H, hd = 37, 3, 6, 64
    g = np.random.default_rng(2)
    lens = [int(x) for x in g.integers(1, 400, B)]
    lens[5], lens[20] = 1, 1900
    c, kk, vv = filled(B, Hkv, hd, 16, 1, 0, lens, 1900, room=room)
    q = data(12, B, 1, H, hd, 0, False)
    pos = [n - 1 for n in lens]
    out, lse = c.attention(q, 0.125, pos)
    check_attention(c, kk, vv, q, 0.125, pos, None, out, lse)


def test_attention_ignores_what_lies_behind(room):
    """Codes and scales behind a row's last visible position are junk (NaN
    codes, NaN scales in this cache's first filling); a block poisoned by a
    NaN reaches the rows that see it and no others."""
    Hkv, hd, block = 2, 64, 32
    c, kk, vv = filled(2, Hkv, hd, block, 1, 1, [40, 70], 96, room=room)
    q = data(13, 2, 2, 4, hd, 1, False)
    out, lse = c.attention(q, 0.125, [38, 68])
    check_attention(c, kk, vv, q, 0.125, [38, 68], None, out, lse)
    # a NaN in block 1 of KV head 1: query tokens that see only block 0 stay clean
    v = data(17, 1, 64, Hkv, hd, 1, False)
    k = data(18, 1, 64, Hkv, hd, 1, False)
    k[0, 33, 1, 0] = math.inf
    c2 = Cache(1, Hkv, hd, max(64, room), block, 0, 1)
    c2.append(k, v, [0])
    q = data(19, 1, 4, 4, hd, 1, False)
    out, lse = c2.attention(q, 0.125, [30])                                # tokens see 31, 32, 33, 34 positions
    assert torch.isfinite(out[:, :2]).all() and torch.isfinite(out[:, :, :2]).all()
    assert torch.isnan(out[:, 2:, 2:]).all() and torch.isnan(lse[:, 2:, 2:]).all()
    val = [[expect(c2, f64(x)[0], 64)[0]] for x in (k, v)]
    ok = f64(q)[:, :2]
    for t in range(2):
        for h in range(4):
            ref, rl, D, bound = attention(ok[0, t, h], np.nan_to_num(val[0][0][:, h // 2]), val[1][0][:, h // 2], 0.125, 31 + t, block)
            assert (np.abs(f64(out)[0, t, h] - ref) <= bound("bfloat16")).all() and abs(float(lse[0, t, h]) - rl) <= lse_tolerance(rl, D)


def test_attention_blocks_of_very_different_scales(room):
    """Scales of neighbouring blocks that differ by 2^60: the weights decide,
    not the sizes of the scales."""
    hd, block = 64, 16
    k = data(20, 1, 64, 1, hd, 1, False)
    v = data(21, 1, 64, 1, hd, 1, False)
    k[0, 16:32] *= 2.0 ** -60
    v[0, 16:32] *= 2.0 ** -40
    v[0, 32:48] *= 2.0 ** 40
    k[0, 32:48, 0, 0] = -1e4   # so that what is large has no weight
    q = data(22, 1, 1, 2, hd, 1, False)
    q[..., 0] = 4.0
    c = Cache(1, 1, hd, max(64, room), block, 0, 1)
    c.append(k, v, [0])
    kk, vv = [expect(c, f64(k)[0], 64)[0]], [expect(c, f64(v)[0], 64)[0]]
    out, lse = c.attention(q, 0.5, [63])
    check_attention(c, kk, vv, q, 0.5, [63], None, out, lse)


def test_attention_large_and_small_queries(room):
    """Queries near the ends of bf16's range, scale 0 and a negative scale."""
    c, kk, vv = filled(1, 1, 64, 16, 0, 1, [50], 64, room=room)
    for mul, scale in ((2.0 ** 100, 2.0 ** -103), (2.0 ** -100, 2.0 ** 97), (1.0, 0.0), (1.0, -0.125)):
        q = data(23, 1, 2, 3, 64, 1, False) * mul
        out, lse = c.attention(q, scale, [48])
        check_attention(c, kk, vv, q, scale, [48], None, out, lse)


def test_attention_scores_far_from_zero(room):
    """Scores around +-1e4 and rows whose maxima rise from tile to tile: the
    reference of the weights has to follow."""
    hd, n, block = 64, 700, 32
    for sign in (1.0, -1.0):
        k = torch.zeros(1, n, 1, hd)
        k[0, :, 0, 0] = sign * torch.linspace(1.0, 200.0, n)
        k[0, :, 0, 1:] = torch.randn(n, hd - 1, generator=torch.Generator().manual_seed(3)) * 0.1
        v = data(31, 1, n, 1, hd, 1, False)
        q = data(32, 1, 2, 2, hd, 1, False)
        q[..., 0] = 50.0
        c = Cache(1, 1, hd, max(n, room), block, 1, 1)
        k = k.to(torch.bfloat16).cuda()
        c.append(k, v, [0])
        kk, vv = [expect(c, f64(k)[0], n)[0]], [expect(c, f64(v)[0], n)[0]]
        out, lse = c.attention(q, 1.0, [n - 2])
        check_attention(c, kk, vv, q, 1.0, [n - 2], None, out, lse)


def test_calls_refuse_what_is_not_device_memory():
    c = Cache(1, 2, 64, 32, 16, 0, 1)
    x = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    d = x.cuda()
    need = rv.kv8_attention_workspace(c.c, 1, 1, 2)
    w = torch.zeros(need, dtype=torch.uint8).cuda()
    bad = rv.KV8.from_buffer_copy(c.c)
    host = torch.zeros(4096, dtype=torch.uint8)
    bad.k_scale = (host.data_ptr() + 15) // 16 * 16
    h, g = rv.heads(x), rv.heads(d)
    for f in (lambda: rv.kv8_append(c.c, h, g, 1, 1, None), lambda: rv.kv8_append(c.c, g, h, 1, 1, None),
              lambda: rv.kv8_append(bad, g, g, 1, 1, None), lambda: rv.kv8_read(c.c, h, None, 1, 1, None),
              lambda: rv.kv8_attention(c.c, h, g, 1, 1, 1.0, None, None, None, w.data_ptr(), need),
              lambda: rv.kv8_attention(c.c, g, g, 1, 1, 1.0, None, None, None, w.data_ptr(), need - 1),
              lambda: rv.kv8_attention(c.c, g, g, 1, 1, 1.0, None, None, None, None, need),
              lambda: rv.kv8_attention(c.c, g, g, 1, 1, 1.0, None, None, None, bad.k_scale, need)):
        with pytest.raises(rv.RVError) as e:
            f()
        assert e.value.code == rv.RV_EINVAL
    for T in range(1, 17):  # the workspace of a larger call serves every smaller one
        assert rv.kv8_attention_workspace(c.c, 1, T, 16) <= rv.kv8_attention_workspace(c.c, 1, 16, 16)


def test_attention_strides_fp32_and_no_lse(room):
    B, T, H, hd = 2, 3, 4, 64
    c, kk, vv = filled(B, 2, hd, 16, 0, 1, [90, 33], 96, room=room)
    wide = torch.randn(B, H, T, hd + 8, generator=torch.Generator().manual_seed(1)).cuda()
    q = wide[..., :hd].transpose(1, 2)          # fp32, rounded to bf16 by the call
    qr = q.to(torch.bfloat16)
    out = torch.full((B, H, T, hd + 8), 7.0).cuda()
    o = out[..., :hd].transpose(1, 2)
    pos = [87, 30]
    _, lse = c.attention(q, 0.125, pos, out=o)
    check_attention(c, kk, vv, qr, 0.125, pos, None, o, lse)
    assert (out[..., hd:] == 7.0).all()
    o2 = torch.full((B, T, H, hd), 7.0).cuda()
    _, lse = c.attention(qr, 0.125, pos, out=o2, lse=False)
    assert (lse == 7.0).all() and torch.equal(o2, o.contiguous())


def test_attention_repeats_bit_for_bit(room):
    c, _, _ = filled(3, 2, 128, 64, 0, 1, [3000, 700, 64], 3000, room=room)
    q = data(24, 3, 2, 8, 128, 1, False)
    a = c.attention(q, 0.1, [2998, 698, 62])
    for _ in range(3):
        b = c.attention(q, 0.1, [2998, 698, 62])
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_run_with_all_operators_and_graphs(room):
    """A generation as a program runs it: rotate, append, attend, one token at
    a time, the three calls captured once into a graph per stream and replayed
    with positions that move on the device; two such programs run at the same
    time on two streams with their own caches and workspaces."""
    H, Hkv, hd, block, act, steps, T0 = 4, 2, 64, 16, 1, 20, 30
    plan = rv.rope_plan(hd, hd, rv.ROPE_HALF, 10000.0)
    progs = []
    for i in range(2):
        p = {"c": Cache(1, Hkv, hd, max(T0 + steps, room), block, i, act), "pos": torch.zeros(1, dtype=torch.int32).cuda(), "s": torch.cuda.Stream()}
        kv = data(30 + i, 1, T0 + steps, Hkv, hd, act, False), data(40 + i, 1, T0 + steps, Hkv, hd, act, False)
        q = data(50 + i, 1, T0 + steps, H, hd, act, False)
        p.update(kv=kv, q=q, in_q=q[:, :1].clone(), in_k=kv[0][:, :1].clone(), in_v=kv[1][:, :1].clone())
        p["out"], p["lse"] = torch.zeros(1, 1, H, hd, dtype=ACT[act]).cuda(), torch.zeros(1, 1, H).cuda()
        p["rq"], p["rk"] = torch.zeros_like(p["in_q"]), torch.zeros_like(p["in_k"])
        need = rv.kv8_attention_workspace(p["c"].c, 1, 1, H)
        p["work"] = torch.zeros(max(need, 16), dtype=torch.uint8).cuda()
        rk = torch.zeros_like(kv[0])
        rv.rope(plan, rv.heads(kv[0]), rv.heads(rk), None, None, 1, T0 + steps, None)
        torch.cuda.synchronize()
        p["rot"] = rk
        p["c"].append(rk[:, :T0], kv[1][:, :T0], [0])
        p["need"] = need
        progs.append(p)
    torch.cuda.synchronize()
    for p in progs:
        p["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(p["graph"], stream=p["s"]):
            st = torch.cuda.current_stream().cuda_stream
            at = p["pos"].data_ptr()
            rv.rope(plan, rv.heads(p["in_q"]), rv.heads(p["rq"]), rv.heads(p["in_k"]), rv.heads(p["rk"]), 1, 1, at, stream=st)
            rv.kv8_append(p["c"].c, rv.heads(p["rk"]), rv.heads(p["in_v"]), 1, 1, at, stream=st)
            rv.kv8_attention(p["c"].c, rv.heads(p["rq"]), rv.heads(p["out"]), 1, 1, hd ** -0.5, at, None, p["lse"].data_ptr(),
                             p["work"].data_ptr(), p["need"], st)
    got = [[], []]
    for i in range(steps):
        for p in progs:
            with torch.cuda.stream(p["s"]):
                t = T0 + i
                p["pos"].fill_(t)
                p["in_q"].copy_(p["q"][:, t:t + 1]), p["in_k"].copy_(p["kv"][0][:, t:t + 1]), p["in_v"].copy_(p["kv"][1][:, t:t + 1])
                p["graph"].replay()
        for j, p in enumerate(progs):
            with torch.cuda.stream(p["s"]):
                got[j].append((p["rq"].clone(), p["out"].clone(), p["lse"].clone()))
    torch.cuda.synchronize()
    for j, p in enumerate(progs):
        for i in range(steps):
            n = T0 + i + 1
            kk = [expect(p["c"], f64(p["rot"])[0], n)[0]]
            vv = [expect(p["c"], f64(p["kv"][1])[0], n)[0]]
            rq, out, lse = got[j][i]
            check_attention(p["c"], kk, vv, rq, hd ** -0.5, [n - 1], None, out, lse)


def test_rows_behind_32_bit_offsets():
    """A cache of 5.4 GB of K codes: its last row lies behind every 32-bit
    offset; the rows before it see one position each or nothing."""
    B, Hkv, hd, block, n = 40, 8, 128, 64, 150
    c = Cache(B, Hkv, hd, 131072, block, 0, 1)
    assert c.codes[0].numel() > 2 ** 32
    k, v = data(41, 1, n, Hkv, hd, 1, False), data(42, 1, n, Hkv, hd, 1, False)
    kb, vb = (x.expand(B, n, Hkv, hd) for x in (k, v))          # every row the same tokens, stride 0
    count = [1] * (B - 2) + [0, n]
    c.append(kb, vb, [0] * B, count)
    got = c.read([0] * B, n, count=count)
    for x, src in zip(got, (k, v)):
        assert np.array_equal(f64(x)[B - 1], expect(c, f64(src)[0], n)[0])
        assert np.array_equal(f64(x)[0, :1], expect(c, f64(src)[0], 1)[0])
    del got
    q = data(43, B, 1, 2 * Hkv, hd, 1, False)
    pos = [0] * (B - 2) + [-1, n - 1]
    kk = [expect(c, f64(k)[0], max(m, 1))[0] for m in count]
    vv = [expect(c, f64(v)[0], max(m, 1))[0] for m in count]
    out, lse = c.attention(q, 0.1, pos)
    check_attention(c, kk, vv, q, 0.1, pos, None, out, lse)
