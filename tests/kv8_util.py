"""Plain 64-bit forms of the 8-bit K/V cache, its attention and the rotary
operator (include/rv.h), for the operator tests.  numpy on the CPU; nothing
here calls the library."""
import math

import numpy as np

QMAX = {0: 127.0, 1: 448.0}  # RV_KV8_INT8, RV_KV8_E4M3
U = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8, "float32": 2.0 ** -24}  # half a step, relative


def up8(x):
    """Smallest number of 8 significant bits not below x > 0."""
    m, e = math.frexp(x)
    return math.ldexp(math.ceil(m * 256.0) / 256.0, e)


def block_scale(x, fmt):
    """Scale of one block's present values (any shape)."""
    x = np.asarray(x, dtype=np.float64)
    if not np.isfinite(x).all():
        return math.nan
    top = float(np.abs(x).max()) / QMAX[fmt] if x.size else 0.0
    return max(up8(top), 2.0 ** -100) if top > 0 else 2.0 ** -100


def to_code(y, fmt):
    """Nearest code value, ties to even."""
    if fmt == 0:
        return np.rint(y)
    a = np.maximum(np.abs(y), 2.0 ** -40)
    _, e = np.frexp(a)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.rint(y / step) * step


def quantise(x, fmt, block):
    """x [n][hd] -> (values [n][hd], scales [ceil(n / block)]): what the cache stands for."""
    x = np.asarray(x, dtype=np.float64)
    out, sc = np.zeros_like(x), []
    for i in range(0, x.shape[0], block):
        s = block_scale(x[i:i + block], fmt)
        sc.append(s)
        out[i:i + block] = to_code(x[i:i + block] / s, fmt) * s if s == s else math.nan
    return out, np.array(sc)


def attention(q, k, v, scale, n, block):
    """q [hd], k and v [N][hd], n visible -> (out, lse, bound): bound(dtype) is what the kernel's
    output may be off by, from arithmetic:
    - a score is a sum of up to 128 products, exact each, added to an fp32 sum
      16 at a time, and two scalings: at most 2 x 8 + 4 roundings of 2^-24,
      below 2^-19, relative to the sum of magnitudes.  int8 K codes enter as
      code + 128 and -128 x sum q is taken off in the same sum, so the
      magnitudes are those of 2 x the block's largest |k| for every element:
      D = max scale x sum |q| x 2 ktop.  A weight is off by a factor exp(2 x
      2^-19 D) at most (its score and the maximum);
    - a weight enters the product as fp16: half a step 2^-11 relative, or
      2^-25 absolute for weights below 2^-14 of the largest;
    - the exponential, the fp32 sums over at most a few thousand partial
      products in order and the joins: below 2^-12 relative to A = sum of
      weights x |v| together;
    - int8 V codes enter the products as code + 128, and -128 x the sum of the
      weights is taken off in the same fp32 sum: up to 6 roundings per tile of
      sums below 256 x (sum of weights), each 2^-24 relative, is less than
      2^-13.4 of a code step, and a step is the block's largest magnitude /
      127: 2^-20 x sum of weights x (largest |v| of its block);
    - the output's own half step."""
    hd = q.shape[-1]
    if n <= 0:
        return np.zeros(hd), -math.inf, 0.0, None
    ktop, top = (np.array([np.abs(x[i:i + block]).max() for i in range(0, x.shape[0], block)]).repeat(block)[:n] for x in (k, v))
    k, v = k[:n], v[:n]
    z = scale * (k @ q)
    d = abs(scale) * float((2.0 * ktop * np.abs(q).sum()).max())
    m = z.max()
    w = np.exp(z - m)
    l = w.sum()
    w /= l
    out, A, S = w @ v, w @ np.abs(v), float(w @ top)
    rel = 2.0 ** -11 + 2.0 ** -12 + 2.0 * 2.0 ** -19 * d

    def bound(dtype):
        return rel * A + 2.0 ** -20 * S + n * 2.0 ** -24 * np.abs(v).max(axis=0) + U[dtype] * np.abs(out) + 1e-30

    return out, m + math.log(l), d, bound


def lse_tolerance(lse, D):
    """fp32: the score's error, the sum's (below 2^-13 for up to a few thousand terms) and the result's steps."""
    return 2.0 ** -19 * D + 2.0 ** -13 + 2.0 ** -22 * abs(lse)


def rope_frequencies(rotary_dim, theta, scaling="plain", factor=1.0, low=1.0, high=4.0, original=0, fast=32.0, slow=1.0):
    """Angle per position of each pair (list of floats) and the default attention factor."""
    r, out, att = rotary_dim, [], 1.0
    base = theta * factor ** (r / (r - 2.0)) if scaling == "base" else theta
    if scaling == "ramp":
        def c(n):
            return r * math.log(original / (2 * math.pi * n)) / (2 * math.log(theta))
        lo, hi = max(0, math.floor(c(fast))), min(r - 1, math.ceil(c(slow)))
        lo, hi = min(lo, r - 1), max(hi, 0)
        hi = lo + 0.001 if hi <= lo else hi
        att = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    for i in range(r // 2):
        f = base ** (-2.0 * i / r)
        if scaling == "linear":
            f = f / factor
        elif scaling == "bands":
            k = min(1.0, max(0.0, (original * f / (2 * math.pi) - low) / (high - low)))
            f = k * f + (1 - k) * f / factor
        elif scaling == "ramp":
            u = min(1.0, max(0.0, (i - lo) / (hi - lo)))
            f = (1 - u) * f + u * f / factor
        out.append(f)
    return np.array(out), att


def rope(x, pos, freq, rotary_dim, interleaved, att=1.0, inverse=False):
    """x [B][T][heads][hd], pos [B][T] -> rotated, in 64 bits."""
    y = np.array(x, dtype=np.float64)
    n = rotary_dim // 2
    ang = np.asarray(pos, dtype=np.float64)[..., None] * freq * (-1.0 if inverse else 1.0)
    c, s = np.cos(ang)[:, :, None] * att, np.sin(ang)[:, :, None] * att
    lo = slice(0, rotary_dim, 2) if interleaved else slice(0, n)
    hi = slice(1, rotary_dim, 2) if interleaved else slice(n, rotary_dim)
    a, b = np.array(x[..., lo], dtype=np.float64), np.array(x[..., hi], dtype=np.float64)
    y[..., lo], y[..., hi] = a * c - b * s, a * s + b * c
    return y
