"""What the 8-bit K/V cache operators and the rotary operator cost, and what they have to give.

Four operators of long-context serving:

  rope       rotary positions of query and key heads (include/rv.h, rv_rope)
  write      quantise new K/V into the 8-bit cache, then read back the blocks it touched (rv_kv8_append, rv_kv8_read)
  read       read a stretch of the 8-bit cache back as values (rv_kv8_read)
  attention  attention of a few new tokens over the 8-bit cache (rv_kv8_attention)

A cache block is `block` consecutive positions of one sequence and one KV
head; its K (and its V) share one scale

  s = max(up8(amax / QMAX), 2^-100),   QMAX = 127 (int8) or 448 (e4m3),

where amax is the largest magnitude of the block's present values and up8
rounds up to 8 significant bits; a code is x / s rounded to the nearest code,
ties to even.  The last 2 x block originals of a sequence stay in 16 bits
(`tail`, slot = position mod 2 block), so the open block is always quantised
from originals.
"""
import math
import random

import torch

own = False

ACT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
QMAX = {"int8": 127.0, "e4m3": 448.0}
SMIN = 2.0 ** -100


# ------------------------------------------------------------------ cases

def _rope(name, B, T, H, Hkv, hd, act, layout, rot, scaling, far, back):
    """rot: rotated part of the head; far: the largest position; back: the gradient's direction."""
    return dict(name=name, op="rope", B=B, T=T, H=H, Hkv=Hkv, hd=hd, act=act, layout=layout, rot=rot, scaling=scaling,
                far=far, back=back)


def _write(name, B, T, Hkv, hd, act, fmt, block, max_seq, ctx):
    """ctx: positions cached before the call (the longest row's)."""
    return dict(name=name, op="write", B=B, T=T, Hkv=Hkv, hd=hd, act=act, fmt=fmt, block=block, max_seq=max_seq, ctx=ctx)


def _read(name, B, T, Hkv, hd, act, fmt, block, max_seq, ctx):
    """ctx: the position (of the longest row) that the read starts at."""
    return dict(name=name, op="read", B=B, T=T, Hkv=Hkv, hd=hd, act=act, fmt=fmt, block=block, max_seq=max_seq, ctx=ctx)


def _attention(name, B, T, H, Hkv, hd, act, fmt, block, max_seq, ctx):
    """ctx: the largest visible length of a first query token; rows are ragged where B > 1."""
    return dict(name=name, op="attention", B=B, T=T, H=H, Hkv=Hkv, hd=hd, act=act, fmt=fmt, block=block, max_seq=max_seq,
                ctx=ctx)


def listed():
    return [
        # one decoded token of the 8B shape: latency
        _rope("rope_decode", 1, 1, 32, 8, 128, "bf16", "half", 128, "none", 1024, False),
        # a batch of 1B-shape prompts with frequencies stretched for long contexts
        _rope("rope_prefill", 16, 511, 32, 8, 64, "bf16", "half", 64, "bands", 65536, False),
        # the gradient of a partly rotated, interleaved head
        _rope("rope_grad", 2, 4096, 32, 8, 128, "fp16", "interleaved", 64, "linear", 8192, True),
        # one decoded token per row: the open block of each row
        _write("write_decode", 64, 1, 8, 64, "bf16", "int8", 64, 4096, 2048),
        # chunks of prompts that begin and end inside blocks
        _write("write_chunk", 8, 509, 8, 128, "fp16", "e4m3", 16, 4096, 1500),
        # a whole long prompt of the 8B shape
        _write("write_prompt", 1, 65536, 8, 128, "bf16", "int8", 64, 65792, 0),
        # a short stretch read back while decoding
        _read("read_short", 4, 100, 2, 64, "fp16", "e4m3", 32, 2048, 900),
        # a long cache read back whole
        _read("read_long", 2, 32701, 8, 128, "bf16", "int8", 128, 65536, 77),
        # batch-1 decode at a prompt's end
        _attention("attn_decode", 1, 1, 32, 8, 128, "bf16", "int8", 64, 2048, 1024),
        # batched decode of the 1B shape, ragged rows
        _attention("attn_batch", 64, 1, 32, 8, 64, "bf16", "e4m3", 32, 8192, 8000),
        # batch-1 decode over a very long cache
        _attention("attn_long", 1, 1, 32, 8, 128, "bf16", "int8", 64, 131072, 131000),
        # drafted tokens of several rows in one pass
        _attention("attn_draft", 16, 6, 32, 8, 128, "fp16", "int8", 64, 16384, 9000),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attention", "attention"])
    hd = rng.choice([64, 128])
    Hkv, grp = rng.choice([(1, 8), (2, 2), (8, 4), (8, 1), (4, 8), (8, 4), (2, 7)])
    act, fmt = rng.choice(["bf16", "fp16"]), rng.choice(["int8", "e4m3"])
    block = rng.choice([16, 32, 64, 128])
    if op == "rope":
        B = _log_int(rng, 1, 64)
        T = _log_int(rng, 1, 8192 // B)
        rot = rng.choice([hd, hd, hd // 2, hd // 4])
        return _rope("", B, T, Hkv * grp, Hkv, hd, act, rng.choice(["half", "interleaved"]), rot,
                     rng.choice(["none", "linear", "bands"]), T + _log_int(rng, 1, 131072), rng.random() < 0.4)
    B = _log_int(rng, 1, 64)
    if op in ("write", "read"):
        T = 1 if rng.random() < 0.25 else _log_int(rng, 1, 65536 // B)
        ctx = _log_int(rng, 1, 4096) - 1
        return (_write if op == "write" else _read)("", B, T, Hkv, hd, act, fmt, block, ctx + T + rng.randrange(64), ctx)
    ctx = _log_int(rng, 1, min(131072, 64 * 8000 // B))
    T = 1 if rng.random() < 0.5 else rng.randint(2, 16)
    while T > 1 and B * ctx * T * Hkv * grp * hd > 16 * 9000 * 6 * 32 * 128:
        T //= 2
    return _attention("", B, T, Hkv * grp, Hkv, hd, act, fmt, block, ctx + T + rng.randrange(64), ctx)


# ------------------------------------------------------------------ inputs

def _starts(c):
    """First position of each row: the longest row at ctx, the others spread below it, by the case alone."""
    top = c["ctx"]
    if c["B"] == 1:
        return [top]
    r = random.Random(c["B"] * 1000003 + top * 101 + c["T"])
    return [top] + [min(top, int(top * r.uniform(0.05, 1.0))) for _ in range(c["B"] - 1)]


def _counts(c):
    """Tokens of each row: all T in the first row, 0..T in the others of a ragged batch."""
    if c["T"] == 1 or c["B"] == 1:
        return [c["T"]] * c["B"]
    r = random.Random(c["B"] * 7919 + c["T"])
    return [c["T"]] + [r.randint(0, c["T"]) for _ in range(c["B"] - 1)]


def _frequencies(c):
    """Angle per position of each pair, in 64 bits (plain python floats)."""
    theta, n = 500000.0, c["rot"] // 2
    out = []
    for i in range(n):
        f = theta ** (-2.0 * i / c["rot"])
        if c["scaling"] == "linear":
            f /= 4.0
        elif c["scaling"] == "bands":  # long waves stretched by 8, short ones kept, a ramp between
            turns = 8192.0 * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - 1.0) / (4.0 - 1.0)))
            f = keep * f + (1 - keep) * f / 8.0
        out.append(f)
    return out


def _up8(x):
    """Smallest float32 of 8 significant bits that is not below x (x > 0)."""
    return ((x.view(torch.int32) + 0xFFFF) & ~0xFFFF).view(torch.float32)


def _quantise(x, fmt, block):
    """x [..., tokens, hd] (tokens a multiple of block; absent values are 0) -> (codes as values, scales [..., blocks])."""
    lead, n, hd = x.shape[:-2], x.shape[-2], x.shape[-1]
    y = x.float().reshape(*lead, n // block, block * hd)
    top = y.abs().amax(-1)
    s = _up8((top / torch.full_like(top, QMAX[fmt])).clamp_min(2.0 ** -120)).clamp_min(SMIN)  # a division, not x * (1 / QMAX)
    y = y / s.unsqueeze(-1)
    y = y.round() if fmt == "int8" else y.to(torch.float8_e4m3fn).float()
    return y.reshape(x.shape), s


def _bits(q, fmt):
    """Codes as the bytes that the cache holds."""
    return (q.to(torch.int8) if fmt == "int8" else q.to(torch.float8_e4m3fn)).view(torch.uint8)


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


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev, B, T, hd = "cuda", c["B"], c["T"], c["hd"]
    act = ACT[c["act"]]
    s = {"case": c}
    if c["op"] == "rope":
        top = c["far"] - T
        s["pos"] = torch.randint(0, top + 1, (B,), generator=g, device=dev).to(torch.int32)
        s["q"] = torch.randn(B, T, c["H"], hd, generator=g, device=dev).to(act)
        s["k"] = torch.randn(B, T, c["Hkv"], hd, generator=g, device=dev).to(act)
        s["q_out"], s["k_out"] = torch.zeros_like(s["q"]), torch.zeros_like(s["k"])
        s["freq"] = torch.tensor(_frequencies(c), dtype=torch.float64, device=dev)
    else:
        Hkv, block, fmt, n = c["Hkv"], c["block"], c["fmt"], _pad(c["max_seq"], c["block"])
        start, count = _starts(c), _counts(c)
        s["pos"] = torch.tensor(start, dtype=torch.int32, device=dev)
        s["count"] = torch.tensor(count, dtype=torch.int32, device=dev)
        if c["op"] == "write":
            s["first"] = s["pos"] // block * block            # the read-back begins with the open block
            s["span"] = torch.where(s["count"] > 0, s["pos"] + s["count"] - s["first"], torch.zeros_like(s["pos"]))
            s["longest"] = max(p % block + m if m else 0 for p, m in zip(start, count))
            for x in "kv":
                s[x] = _kv(g, (B, T, Hkv, hd), c["act"])
                s[x + "_tail"] = _kv(g, (B, Hkv, 2 * block, hd), c["act"])
                s[x + "_codes"] = torch.zeros(B, Hkv, n, hd, dtype=torch.uint8, device=dev)
                s[x + "_scale"] = torch.ones(B, Hkv, n // block, device=dev)
                # the open block as the calls before this one left it
                j = torch.arange(block, device=dev)
                at = s["first"].view(B, 1) + j
                b = torch.arange(B, device=dev).view(B, 1)
                old = s[x + "_tail"][b, :, at % (2 * block)].transpose(1, 2)
                old = torch.where((at < s["pos"].view(B, 1)).view(B, 1, block, 1), old, torch.zeros_like(old))
                q, sc = _quantise(old, fmt, block)
                s[x + "_codes"][b, :, at] = _bits(q, fmt).transpose(1, 2)
                s[x + "_scale"][b, :, (s["first"] // block).view(B, 1)] = sc.transpose(1, 2)
                s[x + "_out"] = torch.zeros(B, s["longest"], Hkv, hd, dtype=act, device=dev)
        else:
            seen = (s["pos"] + s["count"]).view(B, 1, 1, 1)
            for x in "kv":
                v = _kv(g, (B, Hkv, n, hd), c["act"])
                v = torch.where(torch.arange(n, device=dev).view(1, 1, n, 1) < seen, v, torch.zeros_like(v))
                q, s[x + "_scale"] = _quantise(v, fmt, block)
                codes = _bits(q, fmt)
                # what lies behind a row's last token is whatever was there before
                junk = torch.randint(0, 256, (n, hd), generator=g, device=dev).to(torch.uint8)
                s[x + "_codes"] = torch.where(torch.arange(n, device=dev).view(1, 1, n, 1) < seen, codes, junk)
                s[x + "_tail"] = torch.zeros(B, Hkv, 2 * block, hd, dtype=act, device=dev)
                if c["op"] == "read":
                    s[x + "_out"] = torch.zeros(B, T, Hkv, hd, dtype=act, device=dev)
                del v, q, codes
            if c["op"] == "attention":
                s["q"] = torch.randn(B, T, c["H"], hd, generator=g, device=dev).to(act)
                s["out"] = torch.zeros_like(s["q"])
                s["lse"] = torch.zeros(B, T, c["H"], device=dev)
    if own:
        _handles(s)
    return s


# ------------------------------------------------------------------ plain forms

def _run_rope(s):
    c = s["case"]
    T, n = c["T"], c["rot"] // 2
    at = s["pos"].view(-1, 1).double() + torch.arange(T, device="cuda")
    angle = at.unsqueeze(-1) * s["freq"]
    if c["back"]:
        angle = -angle
    cos, sin = angle.cos().float().unsqueeze(2), angle.sin().float().unsqueeze(2)
    res = {}
    for x in "qk":
        y = s[x].float()
        rot, rest = y[..., :c["rot"]], y[..., c["rot"]:]
        if c["layout"] == "half":
            a, b = rot[..., :n], rot[..., n:]
            rot = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        else:
            a, b = rot[..., 0::2], rot[..., 1::2]
            rot = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        res[x] = torch.cat([rot, rest], -1).to(s[x].dtype)
    return res


def _run_write(s):
    c = s["case"]
    B, T, block, n = c["B"], c["T"], c["block"], _pad(c["max_seq"], c["block"])
    dev, ring = "cuda", 2 * c["block"]
    b = torch.arange(B, device=dev).view(B, 1)
    pos, end, first = s["pos"].view(B, 1), (s["pos"] + s["count"]).view(B, 1), s["first"].view(B, 1)
    at = first + torch.arange(_pad(s["longest"], block), device=dev)
    slot = torch.arange(ring, device=dev).view(1, ring)
    last = end - 1 - (end - 1 - slot) % ring                     # the latest position of each tail slot
    blk = torch.arange(n // block, device=dev).view(1, -1) - first // block
    touched = (blk >= 0) & (blk * block + first < end) & (end > pos)
    res = {}
    for x in "kv":
        new, tail = s[x].transpose(1, 2), s[x + "_tail"]
        old = tail[b, :, at % ring].transpose(1, 2)
        fresh = new[b, :, (at - pos).clamp(0, T - 1)].transpose(1, 2)
        v = torch.where((at < pos).view(B, 1, -1, 1), old, fresh)
        v = torch.where(((at < end) & (end > pos)).view(B, 1, -1, 1), v, torch.zeros_like(v))
        q, sc = _quantise(v, c["fmt"], block)
        back = (q.view(*sc.shape, block, -1) * sc[..., None, None]).view(q.shape)
        top = torch.finfo(v.dtype).max
        res[x] = back.clamp(-top, top).to(v.dtype).transpose(1, 2)[:, :s["longest"]]
        res[x + "_scale"] = torch.where(touched.unsqueeze(1), sc[b, :, blk.clamp(0, sc.shape[-1] - 1)].transpose(1, 2),
                                        s[x + "_scale"])
        kept = new[b, :, (last - pos).clamp(0, T - 1)].transpose(1, 2)
        res[x + "_tail"] = torch.where((last >= pos).view(B, 1, -1, 1), kept, tail)
    return res


def _run_read(s):
    c = s["case"]
    B, T, block = c["B"], c["T"], c["block"]
    b, j = torch.arange(B, device="cuda").view(B, 1), torch.arange(T, device="cuda")
    at = (s["pos"].view(B, 1) + j).clamp_max(_pad(c["max_seq"], block) - 1)
    res = {}
    for x in "kv":
        y = _code_values(s[x + "_codes"][b, :, at], c["fmt"]) * s[x + "_scale"][b, :, at // block].unsqueeze(-1)
        top = torch.finfo(ACT[c["act"]]).max
        y = y.clamp(-top, top).to(ACT[c["act"]])
        res[x] = torch.where((j < s["count"].view(B, 1)).view(B, T, 1, 1), y, torch.zeros_like(y))
    return res


def _run_attention(s):
    c = s["case"]
    B, T, H, Hkv, hd, block, n = c["B"], c["T"], c["H"], c["Hkv"], c["hd"], c["block"], _pad(c["max_seq"], c["block"])
    j = torch.arange(T, device="cuda")
    seen = (s["pos"].view(B, 1) + j + 1).view(B, 1, 1, T, 1)
    mask = torch.arange(n, device="cuda") < seen                                         # [B, 1, 1, T, n]
    some = (torch.arange(n, device="cuda") < (s["pos"] + s["count"]).view(B, 1)).view(B, 1, n, 1)
    kv = []
    for x in "kv":
        y = _code_values(s[x + "_codes"], c["fmt"]).view(B, Hkv, n // block, block, hd) * s[x + "_scale"][..., None, None]
        kv.append(torch.where(some, y.view(B, Hkv, n, hd), torch.zeros((), device="cuda")))
    q = s["q"].float().view(B, T, Hkv, H // Hkv, hd).permute(0, 2, 3, 1, 4)              # [B, Hkv, grp, T, hd]
    p = (q.reshape(B, Hkv, -1, hd) @ kv[0].transpose(-1, -2)).view(B, Hkv, -1, T, n) * (hd ** -0.5)
    p = torch.where(mask, p, torch.full((), float("-inf"), device="cuda"))
    top = p.amax(-1, keepdim=True)
    p = (p - torch.where(top.isinf(), torch.zeros_like(top), top)).exp()
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(B, Hkv, -1, n) @ kv[1]).view(B, Hkv, -1, T, hd) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (total.log() + top).squeeze(-1)
    valid = (j < s["count"].view(B, 1)).view(B, T, 1)
    o, lse = o.permute(0, 3, 1, 2, 4).reshape(B, T, H, hd), lse.permute(0, 3, 1, 2).reshape(B, T, H)
    return {"out": torch.where(valid.unsqueeze(-1), o, torch.zeros_like(o)).to(s["q"].dtype),
            "lse": torch.where(valid, lse, torch.zeros_like(lse))}


# ------------------------------------------------------------------ the framework's calls

def _handles(s):
    """What a program keeps between calls: the cache's descriptor, the tensors' layouts, the plan, a workspace."""
    import token_level_early_gb300 as rv

    c = s["case"]
    B, T = c["B"], c["T"]
    s["rv"], s["stream"] = rv, torch.cuda.current_stream().cuda_stream
    if c["op"] == "rope":
        kind = {"none": rv.ROPE_PLAIN, "linear": rv.ROPE_LINEAR, "bands": rv.ROPE_BANDS}[c["scaling"]]
        s["plan"] = rv.rope_plan(c["hd"], c["rot"], rv.ROPE_HALF if c["layout"] == "half" else rv.ROPE_INTERLEAVED,
                                 500000.0, scaling=kind, factor=4.0 if c["scaling"] == "linear" else 8.0,
                                 low_freq_factor=1.0, high_freq_factor=4.0, original_max_position=8192)
        s["h"] = {x: rv.heads(s[x]) for x in ("q", "k", "q_out", "k_out")}
        return
    if c["op"] == "write" and T > c["block"]:
        # a row may go back by `block` positions only: a pass that appends more begins from the tail as it was
        s["tails"] = torch.stack([s["k_tail"], s["v_tail"]])
        s["k_tail"], s["v_tail"], s["tails_before"] = s["tails"][0], s["tails"][1], s["tails"].clone()
    s["cache"] = rv.KV8(B, c["Hkv"], c["hd"], c["max_seq"], c["block"],
                        rv.KV8_INT8 if c["fmt"] == "int8" else rv.KV8_E4M3, rv.BF16 if c["act"] == "bf16" else rv.F16,
                        *(s[x + "_" + y].data_ptr() for y in ("codes", "scale", "tail") for x in "kv"))
    s["h"] = {x: rv.heads(s[x]) for x in ("q", "k", "v", "k_out", "v_out", "out") if x in s}
    if c["op"] == "attention":
        need = rv.kv8_attention_workspace(s["cache"], B, T, c["H"])
        s["work"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")


def _run_own(s):
    c, rv, h, stream = s["case"], s["rv"], s["h"], s["stream"]
    B, T, pos = c["B"], c["T"], s["pos"].data_ptr()
    if c["op"] == "rope":
        rv.rope(s["plan"], h["q"], h["q_out"], h["k"], h["k_out"], B, T, pos, None, c["back"], stream)
        return {"q": s["q_out"], "k": s["k_out"]}
    count = s["count"].data_ptr()
    if c["op"] == "write":
        if "tails" in s:
            s["tails"].copy_(s["tails_before"])
        rv.kv8_append(s["cache"], h["k"], h["v"], B, T, pos, count, None, stream)
        rv.kv8_read(s["cache"], h["k_out"], h["v_out"], B, s["longest"], s["first"].data_ptr(), s["span"].data_ptr(), None,
                    stream)
        return {"k": s["k_out"], "v": s["v_out"], "k_scale": s["k_scale"], "v_scale": s["v_scale"], "k_tail": s["k_tail"],
                "v_tail": s["v_tail"]}
    if c["op"] == "read":
        rv.kv8_read(s["cache"], h["k_out"], h["v_out"], B, T, pos, count, None, stream)
        return {"k": s["k_out"], "v": s["v_out"]}
    rv.kv8_attention(s["cache"], h["q"], h["out"], B, T, c["hd"] ** -0.5, pos, count, s["lse"].data_ptr(),
                     s["work"].data_ptr(), s["work"].numel(), stream)
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _run_own(state)
    return {"rope": _run_rope, "write": _run_write, "read": _run_read, "attention": _run_attention}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    B, T, hd = c["B"], c["T"], c["hd"]
    if c["op"] == "rope":
        tokens = B * T * (c["H"] + c["Hkv"])
        return {"bytes": tokens * hd * 2 * 2 + 4 * B, "flops": tokens * c["rot"] * 3}
    Hkv, block = c["Hkv"], c["block"]
    start, count = _starts(c), _counts(c)
    if c["op"] == "write":
        by = 0
        for p, m in zip(start, count):
            if m:
                held, row = p % block, 2 * Hkv * hd
                # new values and the open block's originals in; codes, scales, tail and values back out
                by += row * (2 * (m + held) + (held + m) + 2 * min(m, 2 * block) + 2 * (held + m))
                by += 2 * Hkv * 4 * -(-(held + m) // block)
        return {"bytes": by + 8 * B, "flops": by}
    if c["op"] == "read":
        row = 2 * Hkv * hd
        by = sum(row * 3 * m + 2 * Hkv * 4 * -(-m // block) for m in count)
        return {"bytes": by + 8 * B, "flops": row * sum(count)}
    by, fl = 8 * B, 0
    for p, m in zip(start, count):
        if m:
            n = p + m
            by += 2 * Hkv * (n * hd + 4 * -(-n // block)) + m * c["H"] * (2 * hd * 2 + 4)
            fl += sum(4 * c["H"] * hd * (p + t + 1) for t in range(m))
    return {"bytes": by, "flops": fl}


# ------------------------------------------------------------------ the definition in 64 bits

def _two_to(e):
    """2^e in 64 bits for whole e, without a power function's last-bit error (which would move ties)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_code(y, fmt):
    if fmt == "int8":
        return torch.round(y)
    _, e = torch.frexp(y.abs().clamp_min(2.0 ** -60))
    step = _two_to((e - 1).clamp_min(-6) - 3)
    return torch.round(y / step) * step


def _exact_block(x, fmt):
    """One block's values [..., block, hd] in 64 bits -> (values it stands for, scale [...])."""
    top = x.abs().amax((-1, -2)) / QMAX[fmt]
    m, e = torch.frexp(top.clamp_min(2.0 ** -130))
    s = (torch.ceil(m * 256.0) / 256.0 * _two_to(e)).clamp_min(SMIN)
    return _exact_code(x / s[..., None, None], fmt) * s[..., None, None], s


def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    c = s["case"]
    B, T, hd = c["B"], c["T"], c["hd"]
    if c["op"] == "rope":
        res = {"q": s["q"].double(), "k": s["k"].double()}
        n, f = c["rot"] // 2, torch.tensor(_frequencies(c), dtype=torch.float64, device="cuda")
        t = torch.arange(T, device="cuda", dtype=torch.float64)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           (s["pos"].double().view(B, 1, 1, 1) + t.view(1, T, 1, 1)) * f * (-1.0 if c["back"] else 1.0))
        for x in res:
            y = res[x]
            lo = slice(0, n) if c["layout"] == "half" else slice(0, c["rot"], 2)
            hi = slice(n, c["rot"]) if c["layout"] == "half" else slice(1, c["rot"], 2)
            z = torch.complex(y[..., lo].contiguous(), y[..., hi].contiguous()) * turn
            y[..., lo], y[..., hi] = z.real, z.imag
        return res
    block, fmt, Hkv = c["block"], c["fmt"], c["Hkv"]
    start, count = _starts(c), _counts(c)
    if c["op"] == "write":
        if sum(count) // block + B > 5000:
            return None
        res = {}
        for x in "kv":
            sc, tail = s[x + "_scale"].double().clone(), s[x + "_tail"].double().clone()
            out = torch.zeros(B, s["longest"], Hkv, hd, dtype=torch.float64, device="cuda")
            for b in range(B):
                p, m = start[b], count[b]
                if not m:
                    continue
                f = p // block * block
                old = tail[b][:, [i % (2 * block) for i in range(f, p)]]
                v = torch.cat([old, s[x][b, :m].double().transpose(0, 1)], 1)
                for i in range(0, v.shape[1], block):
                    y, one = _exact_block(v[:, i:i + block], fmt)
                    out[b, i:i + y.shape[1]] = y.transpose(0, 1)
                    sc[b, :, (f + i) // block] = one
                for i in range(max(p, p + m - 2 * block), p + m):
                    tail[b, :, i % (2 * block)] = s[x][b, i - p].double()
            res[x], res[x + "_scale"], res[x + "_tail"] = out, sc, tail
        return res

    def value(x, b, lo, hi):
        """Values of row b's positions lo..hi-1, [Hkv, hi - lo, hd]."""
        codes = s[x + "_codes"][b, :, lo:hi]
        if fmt == "int8":
            v = codes.to(torch.int16).double()
            v = torch.where(v > 127, v - 256, v)
        else:
            i = codes.to(torch.int64)
            e, m = (i >> 3) & 15, (i & 7).double()
            v = torch.where(e > 0, (1 + m / 8) * _two_to(e - 7), m * 2.0 ** -9)
            v = torch.where(i > 127, -v, v)
        return v * s[x + "_scale"][b].double().repeat_interleave(block, 1)[:, lo:hi, None]

    if c["op"] == "read":
        res = {x: torch.zeros(B, T, Hkv, hd, dtype=torch.float64, device="cuda") for x in "kv"}
        for x in "kv":
            for b in range(B):
                res[x][b, :count[b]] = value(x, b, start[b], start[b] + count[b]).transpose(0, 1)
        return res
    H = c["H"]
    out = torch.zeros(B, T, H, hd, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, T, H, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = start[b] + count[b]
        if not count[b]:
            continue
        k, v = value("k", b, 0, n), value("v", b, 0, n)
        for t in range(count[b]):
            m = start[b] + t + 1
            q = s["q"][b, t].double().view(Hkv, H // Hkv, hd)
            z = torch.einsum("ghd,gnd->ghn", q, k[:, :m]) / math.sqrt(hd)
            lse[b, t] = torch.logsumexp(z, -1).view(H)
            out[b, t] = torch.einsum("ghn,gnd->ghd", torch.softmax(z, -1), v[:, :m]).reshape(H, hd)
    return {"out": out, "lse": lse}
