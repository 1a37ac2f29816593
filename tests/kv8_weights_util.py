"""What a row of few positions may be off by where the attention's weights enter
the product with V as two fp16 terms (fp16 caches, fp32 outputs), and numpy
models of that product."""
import numpy as np


def case(seed, H, n, hd):
    """Scores within [-1, 1]: q [H][hd] has one element, k [n][hd] is read in that column; v [n][hd]."""
    g = np.random.default_rng(seed)
    q = np.zeros((H, hd))
    q[:, 0] = g.uniform(0.25, 1.0, H)
    k = g.uniform(-1.0, 1.0, (n, hd))
    return q, k, g.uniform(-1.0, 1.0, (n, hd))


def bound(q, k, v, block, scale=1.0):
    """(out, bound) of one query row over values k, v [n][hd], n <= 40, in 64 bits:
    - a weight is off by 2^-22 in its two terms (2^-11 of what 2^-11 left), by
      2^-22 in the exponential, and by twice its score's 2^-19 x D (kv8_util);
    - the sum over V has at most n products twice, cut off at the last of 24
      bits of the largest, the weights' sum n terms, and the joins of 4 warps
      and 8 blocks, the division and the scaling are below 40 steps: (2 n + n +
      40) x 2^-23 of sum w |v|;
    - the fp32 output's half step."""
    n = k.shape[0]
    assert n <= 40
    ktop = np.array([np.abs(k[i:i + block]).max() for i in range(0, n, block)]).repeat(block)[:n]
    z = scale * (k @ q)
    d = abs(scale) * float((2.0 * ktop * np.abs(q).sum()).max())
    w = np.exp(z - z.max())
    w /= w.sum()
    rel = 2.0 ** -22 + 2.0 ** -22 + 2.0 * 2.0 ** -19 * d + (3 * n + 40) * 2.0 ** -23
    out = w @ v
    return out, rel * (w @ np.abs(v)) + 2.0 ** -24 * np.abs(out)


def product(q, k, v, terms, scale=1.0):
    """The row with its weights rounded to fp16: one term, two, or the second with its sign turned (terms = -2)."""
    z = scale * (k @ q) / np.log(2.0)
    w = np.exp2((z - z.max() + 7.0).astype(np.float32)).astype(np.float32)
    hi = w.astype(np.float16).astype(np.float64)
    lo = (w - hi.astype(np.float32)).astype(np.float16).astype(np.float64)
    return (hi + {1: 0.0, 2: 1.0, -2: -1.0}[terms] * lo) @ v / w.astype(np.float64).sum()
