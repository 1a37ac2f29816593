"""What the operators for several answers to one prompt cost, and what they have to give.

Three operators of serving many rows that come from few prompts:

  copy     rows of an 8-bit K/V cache copied to other rows: forked, reordered, compacted (include/rv.h, rv_kv8_copy)
  shared   attention of new tokens over a prefix that several rows share, read once for all of them, and over each row's own
           cache (rv_kv8_attention_shared)
  sample   the next token drawn from logits with temperature, top-k, top-p and min-p, from given random numbers (rv_sample)

Cache blocks, scales and tails are those of the 8-bit cache (rv_kv8 in include/rv.h): `block` consecutive positions of a row and KV
head share a scale for K and one for V, the last 2 x block originals stay in 16 bits.

Row b of a shared batch belongs to prefix b // fan and sees its first `prefix` positions, and of its own cache positions
0 .. pos[b] + t with query token t.

A draw: weights are whole multiples of 2^-40 of the row's largest, w_i = round(2^40 exp((x_i - max x) / temperature)); NaN and
-infinity are absent, temperature 0 leaves the largest logit alone.  In descending order of logits, equal ones by index, top-k keeps
the first k; top-p keeps of those the ones before which less than p of their weight lies; min-p keeps the ones of at least min_p of
the largest.  The token is the first, by index, up to which more than u of the kept weight lies.
"""
import math
import random

import numpy as np
import torch

own = False

ACT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
QMAX = {"int8": 127.0, "e4m3": 448.0}
SMIN = 2.0 ** -100
ONE = 2.0 ** 40


# ------------------------------------------------------------------ cases

def _copy(name, n, rows, Hkv, hd, act, fmt, block, length, how):
    """n pairs into a cache of `rows` rows; how: "fork" (one row of the same cache to n others) or "order" (rows of one cache
    into another in a new order); length: positions of the longest."""
    return dict(name=name, op="copy", n=n, rows=rows, Hkv=Hkv, hd=hd, act=act, fmt=fmt, block=block, length=length, how=how)


def _shared(name, P, fan, T, H, Hkv, hd, act, fmt, block, prefix, ctx):
    """P prefixes of up to `prefix` positions with `fan` rows each; ctx: own positions before the call (the longest row's)."""
    return dict(name=name, op="shared", P=P, fan=fan, T=T, H=H, Hkv=Hkv, hd=hd, act=act, fmt=fmt, block=block, prefix=prefix, ctx=ctx)


def _sample(name, B, V, act, how):
    """how: "temp" (temperature alone), "top_k", "top_p", or "mixed" (every row its own, some greedy, some with banned tokens)."""
    return dict(name=name, op="sample", B=B, V=V, act=act, how=how)


def listed():
    return [
        # a short prompt of the 8B shape to three more rows: latency
        _copy("copy_fork_short", 3, 4, 8, 128, "bf16", "int8", 64, 300, "fork"),
        # kept beams in their new order, ragged rows of the 1B shape
        _copy("copy_order", 48, 48, 8, 64, "fp16", "e4m3", 32, 2101, "order"),
        # a long prompt to 16 rows that will go on from it
        _copy("copy_fork_long", 16, 17, 8, 128, "bf16", "int8", 64, 32768, "fork"),
        # four answers to a short prompt, as they begin: latency
        _shared("shared_short", 1, 4, 1, 32, 8, 128, "bf16", "int8", 64, 200, 30),
        # 64 answers to one long document, 8B shape
        _shared("shared_batch", 1, 64, 1, 32, 8, 128, "bf16", "int8", 64, 32768, 400),
        # eight answers to each of sixteen prompts, 1B shape, ragged
        _shared("shared_prompts", 16, 8, 1, 32, 8, 64, "bf16", "e4m3", 32, 6001, 300),
        # drafted tokens of many rows behind one prompt
        _shared("shared_draft", 1, 32, 5, 32, 8, 128, "fp16", "int8", 64, 16000, 700),
        # one row, the next token: latency
        _sample("sample_one", 1, 32000, "fp32", "top_p"),
        # a decoded batch whose rows ask for different things
        _sample("sample_batch", 64, 128256, "fp32", "mixed"),
        # nothing but a temperature, an odd vocabulary, 16-bit logits
        _sample("sample_temp", 200, 50257, "fp16", "temp"),
        # a large batch under top-p alone
        _sample("sample_large", 256, 128256, "bf16", "top_p"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["copy", "shared", "shared", "sample", "sample"])
    if op == "sample":
        B = _log_int(rng, 1, 512)
        V = _log_int(rng, 100, min(200000, 256 * 128256 // B))
        return _sample("", B, V, rng.choice(["fp32", "fp32", "bf16", "fp16"]), rng.choice(["temp", "top_k", "top_p", "mixed"]))
    hd = rng.choice([64, 128])
    Hkv, grp = rng.choice([(1, 8), (2, 2), (8, 4), (8, 1), (4, 8), (8, 4), (2, 7)])
    act, fmt = rng.choice(["bf16", "fp16"]), rng.choice(["int8", "e4m3"])
    block = rng.choice([16, 32, 64, 128])
    if op == "copy":
        n = _log_int(rng, 1, 64)
        length = _log_int(rng, 1, 17 * 32768 * 8 * 128 // (2 * (n + 1) * Hkv * hd))
        return _copy("", n, n + 1 + rng.randrange(4), Hkv, hd, act, fmt, block, min(length, 65536), rng.choice(["fork", "order"]))
    P = _log_int(rng, 1, 16)
    fan = _log_int(rng, 1, 128 // P)
    T = 1 if rng.random() < 0.6 else rng.randint(2, 8)
    most = 16000 * 32 * 5 * 32 * 128 // (P * fan * T * Hkv * grp * hd)
    return _shared("", P, fan, T, Hkv * grp, Hkv, hd, act, fmt, block, _log_int(rng, 1, max(1, min(65536, most, 65536 * 8 // (P * Hkv)))),
                   _log_int(rng, 1, 1000) - 1)


# ------------------------------------------------------------------ inputs

def _lengths(n, top, salt):
    """A length per row: the longest row at top, the others spread below it, by the case alone."""
    r = random.Random(n * 1000003 + top * 101 + salt)
    return [top] + [min(top, int(top * r.uniform(0.2, 1.0))) for _ in range(n - 1)]


def _pairs(c):
    """(from, to, length) of each pair."""
    if c["how"] == "fork":
        return [(0, 1 + i, c["length"]) for i in range(c["n"])]
    r = random.Random(c["n"] * 7919 + c["length"])
    lens = _lengths(c["rows"], c["length"], 5)
    to = r.sample(range(c["rows"]), c["n"])
    src = [r.randrange(c["rows"]) for _ in to]  # some rows twice, some not at all, as beams go
    return [(a, b, lens[a]) for a, b in zip(src, to)]


def _counts(c):
    """Query tokens of each row: all T in the first, 1..T in the others."""
    B, T = c["P"] * c["fan"], c["T"]
    r = random.Random(B * 7919 + T)
    return [T] + [r.randint(1, T) for _ in range(B - 1)]


def _up8(x):
    """Smallest float32 of 8 significant bits that is not below x (x > 0)."""
    return ((x.view(torch.int32) + 0xFFFF) & ~0xFFFF).view(torch.float32)


def _quantise(x, fmt, block):
    """x [..., tokens, hd] (tokens a multiple of block; absent values are 0) -> (codes as bytes, scales [..., blocks])."""
    lead, n, hd = x.shape[:-2], x.shape[-2], x.shape[-1]
    y = x.float().reshape(*lead, n // block, block * hd)
    top = y.abs().amax(-1)
    s = _up8((top / torch.full_like(top, QMAX[fmt])).clamp_min(2.0 ** -120)).clamp_min(SMIN)
    y = y / s.unsqueeze(-1)
    q = (y.round().to(torch.int8) if fmt == "int8" else y.to(torch.float8_e4m3fn)).view(torch.uint8)
    return q.reshape(x.shape), s


def _code_values(codes, fmt):
    return codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).float()


def _kv(g, shape, act):
    """Keys or values [..., hd]: channels of unequal size, a few of them large, as trained models have them."""
    hd = shape[-1]
    ch = torch.rand(hd, generator=g, device="cuda") * 0.9 + 0.1
    ch[torch.randint(0, hd, (3,), generator=g, device="cuda")] *= 8.0
    return (torch.randn(shape, generator=g, device="cuda") * ch).to(ACT[act])


def _pad(n, m):
    return -(-n // m) * m


def _fill(s, name, g, rows, seen, max_seq, c):
    """A cache whose rows hold `seen` positions each; behind them lies whatever was there before."""
    n, block, hd = _pad(max_seq, c["block"]), c["block"], c["hd"]
    some = (torch.arange(n, device="cuda") < torch.tensor(seen, device="cuda").view(-1, 1)).view(rows, 1, n, 1)
    for x in "kv":
        codes = torch.empty(rows, c["Hkv"], n, hd, dtype=torch.uint8, device="cuda")
        scale = torch.empty(rows, c["Hkv"], n // block, device="cuda")
        for b in range(rows):  # row by row: a long cache's values in 32 bits take much room
            v = _kv(g, (c["Hkv"], n, hd), c["act"])
            q, scale[b] = _quantise(torch.where(some[b], v, torch.zeros_like(v)), c["fmt"], block)
            codes[b] = torch.where(some[b], q, torch.randint(0, 256, (n, hd), generator=g, device="cuda").to(torch.uint8))
        s[name + x + "_codes"], s[name + x + "_scale"] = codes, scale
        s[name + x + "_tail"] = _kv(g, (rows, c["Hkv"], 2 * block, hd), c["act"])


def _junk(s, name, g, rows, max_seq, c):
    """A cache of any contents: copying does not look at them."""
    n, block, hd = _pad(max_seq, c["block"]), c["block"], c["hd"]
    for x in "kv":
        s[name + x + "_codes"] = torch.randint(-2 ** 62, 2 ** 62, (rows, c["Hkv"], n, hd // 8), generator=g, device="cuda").view(torch.uint8)
        s[name + x + "_scale"] = torch.rand(rows, c["Hkv"], n // block, generator=g, device="cuda") + 0.01
        s[name + x + "_tail"] = torch.randn(rows, c["Hkv"], 2 * block, hd, generator=g, device="cuda").to(ACT[c["act"]])


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev, s = "cuda", {"case": c}

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    if c["op"] == "copy":
        pairs = _pairs(c)
        s["from"], s["to"], s["len"] = (ints(list(v)) for v in zip(*pairs))
        _junk(s, "dst_", g, c["rows"], c["length"] + 70, c)
        if c["how"] == "order":
            _junk(s, "src_", g, c["rows"], c["length"], c)
    elif c["op"] == "shared":
        P, B, T, hd, H = c["P"], c["P"] * c["fan"], c["T"], c["hd"], c["H"]
        plen, pos, count = _lengths(P, c["prefix"], 3), _lengths(B, c["ctx"], 4), _counts(c)
        s["plen"], s["pos"], s["count"] = ints(plen), ints(pos), ints(count)
        _fill(s, "pre_", g, P, plen, c["prefix"], c)
        _fill(s, "own_", g, B, [p + m for p, m in zip(pos, count)], c["ctx"] + T, c)
        s["q"] = torch.randn(B, T, H, hd, generator=g, device=dev).to(ACT[c["act"]])
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(B, T, H, device=dev)
    else:
        B, V, how = c["B"], c["V"], c["how"]

        def some(*values):
            v = torch.tensor(values, device=dev)
            return v[torch.randint(0, len(values), (B,), generator=g, device=dev)].contiguous()

        # a bell of many unlikely tokens and some tens of likely ones, more or less of them by the row
        x = torch.randn(B, V, generator=g, device=dev) * 2.0
        at = torch.randint(0, V, (B, 40), generator=g, device=dev)
        up = torch.rand(B, 40, generator=g, device=dev) * (torch.rand(B, 1, generator=g, device=dev) * 9.0)
        x.scatter_reduce_(1, at, x.gather(1, at) + 5.0 + up, "amax")  # (a place drawn twice takes the larger)
        s["temperature"] = torch.rand(B, generator=g, device=dev) * 0.9 + 0.4
        s["top_k"], s["top_p"], s["min_p"] = ints([0] * B), torch.ones(B, device=dev), torch.zeros(B, device=dev)
        if how in ("top_k", "mixed"):
            s["top_k"] = some(1, 20, 50, 200, 0 if how == "mixed" else 1000).to(torch.int32)
        if how in ("top_p", "mixed"):
            s["top_p"] = some(0.5, 0.8, 0.9, 0.95, 1.0 if how == "mixed" else 0.99)
        if how == "mixed":
            s["min_p"] = some(0.0, 0.0, 0.02, 0.1)
            s["temperature"] = torch.where(some(0, 1, 1, 1, 1, 1, 1, 1) == 0, torch.zeros_like(s["temperature"]), s["temperature"])
            banned = (torch.rand(B, V, generator=g, device=dev) < 0.3) & (some(0, 0, 1) == 1).unsqueeze(1)
            x = torch.where(banned, torch.full_like(x, float("-inf")), x)
        s["logits"] = x.to(ACT[c["act"]])
        s["u"] = torch.rand(B, generator=g, device=dev)
        s["id"], s["logprob"] = ints([0] * B), torch.zeros(B, device=dev)
    if own:
        _handles(s)
    return s


# ------------------------------------------------------------------ plain forms

def _run_copy(s):
    c, src = s["case"], "dst_" if s["case"]["how"] == "fork" else "src_"
    a, b = s["from"].long(), s["to"].long()
    res = {}
    for x in "kv":
        for y, unit in (("_codes", 1), ("_scale", c["block"]), ("_tail", None)):
            old, new = s["dst_" + x + y], s[src + x + y]
            if unit is None:
                old[b] = new[a]
            else:
                m = min(old.shape[2], new.shape[2])
                some = (torch.arange(m, device="cuda") * unit < s["len"].view(-1, 1)).view(-1, 1, m, *([1] * (old.dim() - 3)))
                old[b, :, :m] = torch.where(some, new[a, :, :m], old[b, :, :m])
            res[x + y] = old
    return res


def _plain_values(s, name, x, c):
    y = _code_values(s[name + x + "_codes"], c["fmt"])
    return (y.view(*y.shape[:2], -1, c["block"], c["hd"]) * s[name + x + "_scale"][..., None, None]).view(y.shape)


def _run_shared(s):
    c = s["case"]
    P, fan, T, H, Hkv, hd = c["P"], c["fan"], c["T"], c["H"], c["Hkv"], c["hd"]
    B, grp, low = P * fan, H // Hkv, torch.full((), float("-inf"), device="cuda")
    j = torch.arange(T, device="cuda")
    q = s["q"].float().view(B, T, Hkv, grp, hd).permute(0, 2, 1, 3, 4)                    # [B, Hkv, T, grp, hd]
    zero = torch.zeros((), device="cuda")
    n = s["pre_k_codes"].shape[2]
    on = torch.arange(n, device="cuda") < s["plen"].view(P, 1)                            # [P, n]
    k, v = (torch.where(on.view(P, 1, n, 1), _plain_values(s, "pre_", x, c), zero) for x in "kv")
    qp = q.reshape(P, fan, Hkv, T * grp, hd).transpose(1, 2).reshape(P, Hkv, fan * T * grp, hd)
    z1 = torch.where(on.view(P, 1, 1, n), (qp @ k.transpose(-1, -2)) * hd ** -0.5, low)   # [P, Hkv, fan T grp, n]
    m = s["own_k_codes"].shape[2]
    seen = (s["pos"].view(B, 1) + j + 1).view(B, 1, T, 1, 1)
    some = (torch.arange(m, device="cuda") < (s["pos"] + s["count"]).view(B, 1)).view(B, 1, m, 1)
    k2, v2 = (torch.where(some, _plain_values(s, "own_", x, c), zero) for x in "kv")
    z2 = (q.reshape(B, Hkv, T * grp, hd) @ k2.transpose(-1, -2)).view(B, Hkv, T, grp, m) * hd ** -0.5
    z2 = torch.where(torch.arange(m, device="cuda") < seen, z2, low).view(B, Hkv, T * grp, m)

    def rows(t):  # [P, Hkv, fan T grp, e] -> [B, Hkv, T grp, e]
        return t.reshape(P, Hkv, fan, T * grp, -1).transpose(1, 2).reshape(B, Hkv, T * grp, -1)

    top = torch.maximum(rows(z1.amax(-1, keepdim=True)), z2.amax(-1, keepdim=True))
    at = top.view(P, fan, Hkv, T * grp, 1).transpose(1, 2).reshape(P, Hkv, -1, 1)
    w1, w2 = (z1 - at).exp(), (z2 - top).exp()
    total = rows(w1.sum(-1, keepdim=True)) + w2.sum(-1, keepdim=True)
    o = (rows(w1 @ v) + w2 @ v2) / total
    lse = (total.log() + top).view(B, Hkv, T, grp).transpose(1, 2).reshape(B, T, H)
    o = o.view(B, Hkv, T, grp, hd).transpose(1, 2).reshape(B, T, H, hd)
    valid = (j < s["count"].view(B, 1)).view(B, T, 1)
    return {"out": torch.where(valid.unsqueeze(-1), o, zero).to(s["q"].dtype), "lse": torch.where(valid, lse, zero)}


def _run_sample(s):
    c = s["case"]
    B, V = c["B"], c["V"]
    x = s["logits"].double()
    x = torch.where(x.isnan(), torch.full((), float("-inf"), dtype=torch.float64, device="cuda"), x)
    t = s["temperature"].double().view(B, 1)
    z, order = torch.sort(x, dim=1, descending=True, stable=True)
    top = z[:, :1]
    rank = torch.arange(V, device="cuda")
    gap = torch.where(z == top, torch.zeros_like(z), z - top) / torch.where(t > 0, t, torch.ones_like(t))
    ratio = torch.where(t > 0, gap.exp(), (rank == 0).double())
    w = (ratio * ONE).round().to(torch.int64)
    k = s["top_k"].view(B, 1)
    w = torch.where((k <= 0) | (rank < k), w, torch.zeros_like(w))
    p = s["top_p"].double().view(B, 1)
    before, total = w.cumsum(1) - w, w.sum(1, keepdim=True)
    keep = ((p >= 1) | (before.double() < p * total.double()) | (rank == 0)) & (ratio >= s["min_p"].double().clamp_max(1.0).view(B, 1))
    w = torch.where(keep, w, torch.zeros_like(w))
    total = w.sum(1, keepdim=True)
    up = torch.zeros_like(w).scatter_(1, order, w).cumsum(1)
    pick = (up.double() <= s["u"].double().view(B, 1) * total.double()).sum(1, keepdim=True).clamp_max(V - 1)
    mine = up.gather(1, pick) - torch.where(pick > 0, up.gather(1, (pick - 1).clamp_min(0)), torch.zeros_like(pick))
    logprob = (mine.double() / total.double()).log()
    return {"id": pick.view(B).to(torch.int32), "logprob": logprob.view(B).float()}


# ------------------------------------------------------------------ the framework's calls

def _handles(s):
    """What a program keeps between calls: the caches' descriptors, the tensors' layouts, a workspace."""
    import token_level_early_gb300 as rv

    c = s["case"]
    s["rv"], s["stream"] = rv, torch.cuda.current_stream().cuda_stream
    if c["op"] == "sample":
        return

    def cache(name, rows, max_seq):
        return rv.KV8(rows, c["Hkv"], c["hd"], max_seq, c["block"], rv.KV8_INT8 if c["fmt"] == "int8" else rv.KV8_E4M3,
                      rv.BF16 if c["act"] == "bf16" else rv.F16,
                      *(s[name + x + "_" + y].data_ptr() for y in ("codes", "scale", "tail") for x in "kv"))

    if c["op"] == "copy":
        s["dst"] = cache("dst_", c["rows"], c["length"] + 70)
        s["src"] = s["dst"] if c["how"] == "fork" else cache("src_", c["rows"], c["length"])
        return
    B = c["P"] * c["fan"]
    s["prefix"], s["cache"] = cache("pre_", c["P"], c["prefix"]), cache("own_", B, c["ctx"] + c["T"])
    s["h"] = {x: rv.heads(s[x]) for x in ("q", "out")}
    need = rv.kv8_attention_shared_workspace(s["prefix"], s["cache"], B, c["T"], c["fan"], c["H"])
    s["work"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")


def _run_own(s):
    c, rv, stream = s["case"], s["rv"], s["stream"]
    if c["op"] == "copy":
        rv.kv8_copy(s["src"], s["dst"], c["n"], s["from"].data_ptr(), s["to"].data_ptr(), s["len"].data_ptr(), None, stream)
        return {x + y: s["dst_" + x + y] for x in "kv" for y in ("_codes", "_scale", "_tail")}
    if c["op"] == "shared":
        rv.kv8_attention_shared(s["prefix"], s["cache"], s["h"]["q"], s["h"]["out"], c["P"] * c["fan"], c["T"], c["fan"], c["hd"] ** -0.5,
                                s["plen"].data_ptr(), s["pos"].data_ptr(), s["count"].data_ptr(), s["lse"].data_ptr(), None,
                                s["work"].data_ptr(), s["work"].numel(), stream)
        return {"out": s["out"], "lse": s["lse"]}
    dtype = {"fp32": rv.F32, "bf16": rv.BF16, "fp16": rv.F16}[c["act"]]
    rv.sample(s["logits"].data_ptr(), dtype, c["V"], c["B"], c["V"], s["temperature"].data_ptr(), s["top_k"].data_ptr(),
              s["top_p"].data_ptr(), s["min_p"].data_ptr(), s["u"].data_ptr(), s["id"].data_ptr(), s["logprob"].data_ptr(), stream)
    return {"id": s["id"], "logprob": s["logprob"]}


def run(state):
    if own:
        return _run_own(state)
    return {"copy": _run_copy, "shared": _run_shared, "sample": _run_sample}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "sample":
        n = c["B"] * c["V"]
        return {"bytes": n * (4 if c["act"] == "fp32" else 2) + 28 * c["B"], "flops": 2 * n}
    Hkv, hd, block = c["Hkv"], c["hd"], c["block"]
    if c["op"] == "copy":
        def row(m):
            return 2 * Hkv * (m * hd + 4 * -(-m // block) + 2 * 2 * block * hd)

        pairs = _pairs(c)
        read = sum(row(m) for m in {a: m for a, _, m in pairs}.values())
        by = read + sum(row(m) for _, _, m in pairs) + 12 * c["n"]
        return {"bytes": by, "flops": by}
    P, B, H = c["P"], c["P"] * c["fan"], c["H"]
    plen, pos, count = _lengths(P, c["prefix"], 3), _lengths(B, c["ctx"], 4), _counts(c)
    by, fl = 8 * B + 4 * P, 0
    for n in plen + [p + m for p, m in zip(pos, count)]:
        by += 2 * Hkv * (n * hd + 4 * -(-n // block))
    for b, (p, m) in enumerate(zip(pos, count)):
        by += m * H * (2 * hd * 2 + 4)
        fl += sum(4 * H * hd * (plen[b // c["fan"]] + p + t + 1) for t in range(m))
    return {"bytes": by, "flops": fl}


# ------------------------------------------------------------------ the definition in 64 bits

def _two_to(e):
    """2^e in 64 bits for whole e."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_draw(x, t, k, p, lowest, u):
    """One row: logits as a numpy array of doubles -> (token, log of its part of the kept weight)."""
    x = np.where(np.isnan(x), -np.inf, x)
    order = np.argsort(-x, kind="stable")
    best = x[order[0]]
    if t > 0:
        share = np.exp((x - best) / t)
        weight = np.rint(share * ONE).astype(np.int64)
        allowed = np.ones(x.size, dtype=bool)
        if k > 0:
            allowed[order[k:]] = False
        if p < 1:
            lined = np.where(allowed, weight, 0)[order]
            sums = np.cumsum(lined)
            out = (sums - lined).astype(np.float64) >= p * float(sums[-1])
            out[0] = False
            allowed[order[out]] = False
        allowed &= share >= min(lowest, 1.0)
        weight = np.where(allowed, weight, 0)
    else:
        weight = np.zeros(x.size, dtype=np.int64)
        weight[order[0]] = 1
    sums = np.cumsum(weight)
    i = min(int(np.searchsorted(sums.astype(np.float64), u * float(sums[-1]), side="right")), x.size - 1)
    return i, math.log(int(weight[i])) - math.log(int(sums[-1]))


def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    c = s["case"]
    if c["op"] == "sample":
        if c["B"] * c["V"] > 40000000:
            return None
        rows = [v.double().cpu().numpy() for v in (s["logits"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], s["u"])]
        got = [_exact_draw(x, float(t), int(k), float(p), float(m), float(u)) for x, t, k, p, m, u in zip(*rows)]
        return {"id": torch.tensor([i for i, _ in got], dtype=torch.int32, device="cuda"),
                "logprob": torch.tensor([v for _, v in got], dtype=torch.float64, device="cuda")}
    block, fmt, Hkv, hd = c["block"], c["fmt"], c["Hkv"], c["hd"]
    if c["op"] == "copy":
        src, res = "dst_" if c["how"] == "fork" else "src_", {}
        for x in "kv":
            for y in ("_codes", "_scale", "_tail"):
                new, old = s["dst_" + x + y].clone(), s[src + x + y]
                for a, b, m in _pairs(c):
                    e = {"_codes": m, "_scale": -(-m // block), "_tail": 2 * block}[y]
                    new[b, :, :e] = old[a, :, :e]
                res[x + y] = new if y == "_codes" else new.double()
        return res
    P, fan, T, H = c["P"], c["fan"], c["T"], c["H"]
    plen, pos, count = _lengths(P, c["prefix"], 3), _lengths(P * fan, c["ctx"], 4), _counts(c)

    def value(name, x, b, n):
        """Values of row b's first n positions, [Hkv, n, hd]."""
        codes = s[name + x + "_codes"][b, :, :n]
        if fmt == "int8":
            v = codes.to(torch.int16).double()
            v = torch.where(v > 127, v - 256, v)
        else:
            i = codes.to(torch.int64)
            e, m = (i >> 3) & 15, (i & 7).double()
            v = torch.where(e > 0, (1 + m / 8) * _two_to(e - 7), m * 2.0 ** -9)
            v = torch.where(i > 127, -v, v)
        return v * s[name + x + "_scale"][b].double().repeat_interleave(block, 1)[:, :n, None]

    out = torch.zeros(P * fan, T, H, hd, dtype=torch.float64, device="cuda")
    lse = torch.zeros(P * fan, T, H, dtype=torch.float64, device="cuda")
    for a in range(P):
        k, v = value("pre_", "k", a, plen[a]), value("pre_", "v", a, plen[a])
        for b in range(a * fan, a * fan + fan):
            k2, v2 = value("own_", "k", b, pos[b] + count[b]), value("own_", "v", b, pos[b] + count[b])
            for t in range(count[b]):
                m = pos[b] + t + 1
                q = s["q"][b, t].double().view(Hkv, H // Hkv, hd)
                z = torch.cat([q @ k.transpose(1, 2), q @ k2[:, :m].transpose(1, 2)], -1) / math.sqrt(hd)
                w = torch.softmax(z, -1)
                lse[b, t] = torch.logsumexp(z, -1).view(H)
                out[b, t] = (w[..., :plen[a]] @ v + w[..., plen[a]:] @ v2[:, :m]).reshape(H, hd)
    return {"out": out, "lse": lse}
