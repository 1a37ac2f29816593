"""The cache attention where its line of tiles is long: pieces that count the
beginning of a unit, several units in a piece, units over many pieces, more
units than pieces, every number of query columns.

V marks where a position lies: element d of position p is 1 where p / 16 is d
modulo head_dim (small numbers elsewhere), so an element of the output is the
weight of a handful of 16-position steps, and one step too few or too many
moves it by far more than its bound."""
import math

import pytest
import torch

import token_level_early_gb300 as rv
from kv8_util import U
from test_gpu_kv8 import ACT, Cache

pytestmark = pytest.mark.gpu


def marked(seed, B, T, Hkv, hd, act):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.randn(B, T, Hkv, hd, generator=g, device="cuda")
    v = 0.01 * torch.rand(B, T, Hkv, hd, generator=g, device="cuda")
    p = torch.arange(T, device="cuda")
    v[:, p, :, (p // 16) % hd] = 1.0
    return k.to(ACT[act]), v.to(ACT[act])


def reference(q, k, v, scale, n, block):
    """Query rows q [m][hd] that see n positions each, over k, v [N][hd] of one KV head, all in 64 bits:
    (out, lse, bound, lse's bound).  Weights: 2^-11 and 2^-32 of the largest (test_gpu_kv8_range), 2^-12 for the
    exponential, the fp32 sums and the joins, 2^-18 D for the scores (kv8_util)."""
    N = k.shape[0]
    z = scale * (q @ k.T)
    see = torch.arange(N, device="cuda")[None] < n[:, None]
    z = torch.where(see, z, -math.inf)
    lse = torch.logsumexp(z, -1)
    w = torch.exp(z - torch.where(n > 0, lse, 0.0)[:, None])
    d = abs(scale) * q.abs().sum(-1) * 2.0 * k.abs().max()
    out = w @ v
    tol = (2.0 ** -11 + 2.0 ** -12 + 2.0 ** -18 * d)[:, None] * (w @ v.abs()) + (n * 2.0 ** -32)[:, None]
    return out, lse, tol, 2.0 ** -19 * d + 2.0 ** -13 + 2.0 ** -22 * lse.abs()


CASES = {  # B, T, Hkv, heads per group, head_dim, block, format, act, longest, ragged
    "one row": (1, 1, 8, 4, 128, 64, 0, 1, 10007, False),
    "one unit": (1, 1, 1, 8, 128, 64, 1, 1, 90001, False),
    "more units than pieces": (64, 2, 8, 4, 128, 32, 1, 1, 600, True),
    "more units than pieces, heads of 64": (100, 1, 8, 4, 64, 16, 0, 0, 900, True),
    "two columns": (2, 1, 4, 16, 64, 128, 1, 1, 30011, True),
    "three columns": (9, 6, 4, 4, 128, 64, 0, 0, 6007, True),
    "three columns in groups": (3, 16, 8, 4, 128, 16, 0, 1, 4003, True),
}


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("name", CASES)
def test_attention_on_a_long_line(name, f32):
    B, T, Hkv, grp, hd, block, fmt, act, longest, ragged = CASES[name]
    g = torch.Generator().manual_seed(5)
    see = [longest] * B
    count = [T] * B
    if ragged:
        see = [longest] + [int(x) for x in torch.randint(longest // 3, longest, (B - 1,), generator=g)]
        count = [T] + [int(x) for x in torch.randint(1, T + 1, (B - 1,), generator=g)]
        if B > 3:
            see[1], see[2], count[3] = 1, 0, 0      # one position, nothing, no tokens
    pos = [n - m for n, m in zip(see, count)]
    # the line is long enough for pieces to count beginnings, and taken (a cache with room for far more)
    tile = 32 if hd == 128 else 64
    rows = T * grp
    cols = -(-rows // 8)
    nt = -(-cols // -(-cols // 3))
    blocks = (3 if nt == 1 and hd == 64 else 2) * torch.cuda.get_device_properties(0).multi_processor_count
    assert sum(-(-n // tile) * Hkv * -(-m * grp // (8 * nt)) for n, m in zip(see, count)) >= 8 * blocks
    c = Cache(B, Hkv, hd, max(longest, 9000), block, fmt, act)
    k, v = marked(6, B, longest, Hkv, hd, act)
    c.append(k, v, [0] * B, see)
    kk, vv = c.read([0] * B, longest, count=see, fill=0.0)
    q = (0.3 * torch.randn(B, T, Hkv * grp, hd, generator=g)).to(ACT[act]).cuda()
    scale = hd ** -0.5
    out, lse = c.attention(q, scale, pos, count, out=torch.full(q.shape, 7.0, dtype=torch.float32).cuda() if f32 else None)
    again = c.attention(q, scale, pos, count, out=torch.full(q.shape, 7.0, dtype=torch.float32).cuda() if f32 else None)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    u = U[str(out.dtype).split(".")[1]]
    for b in range(B):
        m = count[b]
        assert (out[b, m:] == 7.0).all() and (lse[b, m:] == 7.0).all()
        n = (pos[b] + 1 + torch.arange(m)).clamp(min=0).repeat_interleave(grp).cuda()
        for h in range(Hkv if m else 0):
            at = slice(h * grp, (h + 1) * grp)
            N = max(see[b], 1)
            ref, rl, tol, lt = reference(q[b, :m, at].reshape(-1, hd).double(), kk[b, :N, h].double(), vv[b, :N, h].double(), scale, n, block)
            got, gl = out[b, :m, at].reshape(-1, hd).double(), lse[b, :m, at].reshape(-1).double()
            some = n > 0
            assert (got[~some] == 0).all() and (gl[~some] == -math.inf).all()
            err = (got - ref)[some].abs()
            assert (err <= (tol + u * ref.abs())[some]).all(), (b, h, float((err / tol[some]).max()))
            assert ((gl - rl)[some].abs() <= lt[some]).all(), (b, h)
