"""Plain forms of the operators for several answers to one prompt (include/rv.h):
row copies, attention over a shared prefix, the draw.  numpy in 64 bits; nothing
here calls the library."""
import math

import numpy as np

from kv8_util import U


def copy_rows(src, dst, pairs, per):
    """src, dst [rows][heads][n]..: dst after the pairs (from, to, length), all at once; `per` positions to an entry (None: all entries)."""
    out, last = dst.copy(), {}
    for a, b, m in pairs:
        if 0 <= a < src.shape[0] and 0 <= b < dst.shape[0]:
            last[b] = (a, m)
    for b, (a, m) in last.items():
        e = src.shape[2] if per is None else -(-m // per)
        out[b, :, :e] = src[a, :, :e]
    return out


def attention_parts(q, parts, scale, two_terms):
    """q [hd]; parts: (k [n][hd], v [n][hd], block) with all n seen -> (out, lse, D, bound).  bound(dtype), from arithmetic:
    - a score: as in kv8_util.attention, at most 2^-19 relative to D = scale x sum |q| x 2 x the block's largest |k| (the
      prefix's products have no bias and up to 8 sums of 16: less);
    - a weight (the prefix: times its block's V scale) as one fp16: half a step, 2^-11, or 2^-25 absolute at a reference that
      stands 2^-7 or less of the largest; as two terms 2^-22;
    - sums: exponentials to 2^-22, fp32 sums of n / 16 products one after another, each cut at 2^-23 of the sum at most, and a few
      more for the joins: (n / 16 + 64) 2^-23 of A = sum of weights x |v|;
    - the own cache's int8 V codes with a bias of 128: 2^-20 x sum of weights x the block's largest |v| (kv8_util.attention);
    - the output's own half step."""
    hd = q.shape[-1]
    parts = [p for p in parts if p[0].shape[0]]
    if not parts:
        return np.zeros(hd), -math.inf, 0.0, lambda dtype: 1e-30
    tops = [[np.array([np.abs(x[i:i + b]).max() for i in range(0, x.shape[0], b)]).repeat(b)[:x.shape[0]] for x in (k, v)] for k, v, b in parts]
    k, v = (np.concatenate([p[i] for p in parts]) for i in (0, 1))
    ktop, top = (np.concatenate([t[i] for t in tops]) for i in (0, 1))
    z = scale * (k @ q)
    d = abs(scale) * float((2.0 * ktop * np.abs(q).sum()).max())
    m = z.max()
    w = np.exp(z - m)
    l = w.sum()
    w /= l
    out, A, S, n = w @ v, w @ np.abs(v), float(w @ top), v.shape[0]
    rel = (2.0 ** -22 if two_terms else 2.0 ** -11) + 2.0 ** -22 + (n / 16 + 64) * 2.0 ** -23 + 2.0 * 2.0 ** -19 * d
    tiny = n * 2.0 ** -32 * np.abs(v).max(axis=0)

    def bound(dtype):
        return rel * A + 2.0 ** -20 * S + tiny + U[dtype] * np.abs(out) + 1e-30

    return out, m + math.log(l), d, bound


def draw(x, t, k, p, lowest, u):
    """One row: (token, log of its part of the kept weight), with whole numbers of Python."""
    x = [-math.inf if v != v else float(v) for v in x]
    order = sorted(range(len(x)), key=lambda i: (-x[i], i))
    best = x[order[0]]
    if best == -math.inf:
        return -1, -math.inf
    if not t > 0:
        return order[0], 0.0
    w = [1 << 40 if v == best else int(round(math.exp(max(-1e4, (v - best) / t)) * 2.0 ** 40)) for v in x]
    if k > 0:
        for i in order[k:]:
            w[i] = 0
    kept = set(order)
    if p < 1:
        total, before, kept = sum(w), 0, set()
        num, den = float(max(p, 0.0)).as_integer_ratio()
        for j, i in enumerate(order):
            if j and before * den >= num * total:
                break
            kept.add(i)
            before += w[i]
    if lowest > 0:
        kept = {i for i in kept if x[i] == best or math.exp(max(-1e4, (x[i] - best) / t)) >= min(lowest, 1.0)}
    total = sum(w[i] for i in kept)
    u = 0.0 if not u > 0 else min(u, 1.0 - 2.0 ** -24)
    num, den = float(u).as_integer_ratio()
    run = 0
    for i in range(len(x)):
        if i in kept:
            run += w[i]
            if run * den > num * total:
                return i, math.log(w[i] / total)
    raise AssertionError("no token")
