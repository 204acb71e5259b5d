"""Measured cases of the 8-bit serving operators: the INT8 matrix product, the
append of new tokens to a paged 8-bit key/value cache, and attention over that
cache.

The three belong together: a projection's output is appended to the cache, the
cache is read by attention, and attention's output is quantized for the next
projection.  With ``own`` false, ``run`` computes the plain form of an operator
from elementary torch operations; with ``own`` true it makes the framework's
calls.

Cache layout (both forms): K codes [blocks, kv heads, tokens, head dim], V
codes [blocks, kv heads, head dim, tokens], one fp32 scale per block and kv
head for each; int8 codes, or e4m3 codes as uint8.  Position p of sequence b
lives in block table[b, p // tokens].
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
QMAX = {"int8": 127.0, "fp8": 448.0}
TINY = 2.0 ** -64          # absolute maxima below this get scale 0


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # one token through an attention output projection: latency
        {"name": "gemm one token", "op": "gemm", "m": 1, "n": 4096, "k": 4096, "out": "bf16",
         "bias": False},
        # a decoding batch through an MLP up projection
        {"name": "gemm decode batch", "op": "gemm", "m": 48, "n": 14336, "k": 4096, "out": "bf16",
         "bias": True},
        # a short odd prompt, odd width, ragged reduction, fp32 output
        {"name": "gemm odd", "op": "gemm", "m": 777, "n": 1031, "k": 2064, "out": "f32",
         "bias": True},
        # a 4096-token prompt through an MLP up projection
        {"name": "gemm prompt", "op": "gemm", "m": 4096, "n": 14336, "k": 4096, "out": "bf16",
         "bias": False},
        # one new token for each of 64 sequences: every decode step does this
        {"name": "append decode", "op": "append", "seqs": 64, "lo": 5, "hi": 2047, "new": 1,
         "mix": 0, "kv": 8, "d": 128, "tokens": 64, "fmt": "int8", "dtype": "bf16"},
        # ragged chunks that begin and end inside blocks, small blocks, fp32 rows
        {"name": "append ragged", "op": "append", "seqs": 23, "lo": 40, "hi": 1900, "new": 333,
         "mix": 5, "kv": 4, "d": 64, "tokens": 16, "fmt": "fp8", "dtype": "f32"},
        # a 16384-token prompt
        {"name": "append prompt", "op": "append", "seqs": 1, "lo": 16384, "hi": 16384,
         "new": 16384, "mix": 0, "kv": 8, "d": 128, "tokens": 64, "fmt": "fp8", "dtype": "bf16"},
        # one user, short context: latency
        {"name": "attend short", "op": "attend", "seqs": 1, "lo": 129, "hi": 129, "new": 1,
         "mix": 0, "heads": 32, "kv": 8, "d": 128, "tokens": 64, "fmt": "int8", "dtype": "bf16",
         "window": 0, "lse": False},
        # a decoding batch of 64 sequences of very different lengths
        {"name": "attend decode", "op": "attend", "seqs": 64, "lo": 300, "hi": 16384, "new": 1,
         "mix": 0, "heads": 32, "kv": 8, "d": 128, "tokens": 64, "fmt": "int8", "dtype": "bf16",
         "window": 0, "lse": False},
        # one user with a long context, the work split along it
        {"name": "attend long", "op": "attend", "seqs": 1, "lo": 131071, "hi": 131071, "new": 1,
         "mix": 0, "heads": 32, "kv": 8, "d": 128, "tokens": 128, "fmt": "fp8", "dtype": "bf16",
         "window": 0, "lse": True},
        # chunks of prompts next to decoding sequences in one call, a sliding
        # window, small heads and blocks, fp16
        {"name": "attend mixed", "op": "attend", "seqs": 24, "lo": 70, "hi": 3500, "new": 501,
         "mix": 3, "heads": 16, "kv": 4, "d": 64, "tokens": 16, "fmt": "fp8", "dtype": "f16",
         "window": 1000, "lse": True},
        # a whole prompt attending to itself
        {"name": "attend prompt", "op": "attend", "seqs": 1, "lo": 8192, "hi": 8192, "new": 8192,
         "mix": 0, "heads": 32, "kv": 8, "d": 128, "tokens": 64, "fmt": "int8", "dtype": "bf16",
         "window": 0, "lse": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gemm", "append", "attend", "attend"))
    if op == "gemm":
        while True:
            c = {"op": "gemm", "m": _log(rng, 1, 4096), "n": _log(rng, 64, 16384),
                 "k": 16 * _log(rng, 4, 1024), "out": rng.choice(("bf16", "f16", "f32")),
                 "bias": rng.random() < 0.5}
            if c["m"] * c["n"] * c["k"] <= 4096 * 14336 * 4096:
                return c
    shape = {"tokens": rng.choice((16, 32, 64, 128, 256)), "fmt": rng.choice(("int8", "fp8"))}
    if op == "append":
        while True:
            seqs, new = _log(rng, 1, 128), _log(rng, 1, 4096)
            hi = new + _log(rng, 1, 4096)
            c = {"op": "append", "seqs": seqs, "lo": rng.randint(new, hi), "hi": hi, "new": new,
                 "mix": rng.randint(0, 9), "kv": rng.choice((1, 2, 3, 4, 8)),
                 "d": rng.choice((64, 128, 192, 256)), **shape,
                 "dtype": rng.choice(("bf16", "f16", "f32"))}
            if seqs * hi * c["kv"] * c["d"] <= 1 << 26 and seqs * new <= 16384:
                return c
    while True:
        seqs = _log(rng, 1, 96)
        new = 1 if rng.random() < 0.4 else _log(rng, 1, 2048)
        hi = new + _log(rng, 1, 32768)
        kv, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 5, 8, 16))
        c = {"op": "attend", "seqs": seqs, "lo": rng.randint(new, hi), "hi": hi, "new": new,
             "mix": rng.randint(0, 9), "heads": kv * group, "kv": kv,
             "d": rng.choice((64, 128, 192, 256)), **shape, "dtype": rng.choice(("bf16", "f16")),
             "window": rng.choice((0, 0, 0, _log(rng, 16, 4096))), "lse": rng.random() < 0.5}
        # the plain form's padded scores and gathered cache stay within the card
        if (seqs * c["heads"] * new * hi <= 1 << 31 and seqs * hi * kv * c["d"] <= 1 << 29
                and work(c)["flops"] <= 4e11):
            return c


def _sizes(c):
    """Context lengths (new tokens included) and new tokens of each sequence,
    from the case alone.  mix 0: every sequence has `new` tokens; else some
    have none, some one, some a part of `new`, the last all of it."""
    n, lens, news = c["seqs"], [], []
    for i in range(n):
        f = 1.0 if i == n - 1 else (0.37 + 0.6180339887498949 * i) % 1.0
        lens.append(c["lo"] + int((c["hi"] - c["lo"]) * f))
        if c["mix"] == 0 or i == n - 1:
            w = c["new"]
        else:
            w = (0, 1, 1, 1, 1 + c["new"] // 7, 1, 1 + c["new"] // 3, 1)[(i * 5 + c["mix"]) % 8]
        news.append(min(w, lens[-1], c["new"]))
    return lens, news


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------


def _scale(amax, fmt, base=0.0):
    """Scale of an absolute maximum, at least `base`, and its reciprocal (fp32
    divisions by tensors: a division by a number multiplies by its rounded
    reciprocal)."""
    s = torch.where(amax < TINY, torch.zeros_like(amax), amax / torch.full_like(amax, QMAX[fmt]))
    s = torch.maximum(s, torch.zeros_like(s) + base)
    return s, torch.where(s > 0, torch.ones_like(s) / s, torch.zeros_like(s))


def _quantized(x, fmt, dims):
    """Codes and scales of x with one scale over `dims`."""
    amax = x.abs().amax(dims)
    s, inv = _scale(amax, fmt)
    for d in sorted(dims):
        inv = inv.unsqueeze(d)
    return _encode(x * inv, fmt), s


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rows(g, total, heads, d, outliers):
    """N(0, 1) rows with four dims of each head times 8 for queries and keys."""
    x = _normal(g, total, heads, d)
    if outliers:
        x[..., ::d // 4] *= 8.0
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    if c["op"] == "gemm":
        # an activation with a few strong channels, one scale per token; a
        # weight with one scale per output channel
        x = _normal(g, c["m"], c["k"])
        x[:, ::c["k"] // 4] *= 50.0
        w = _normal(g, c["n"], c["k"]) * 0.02
        w *= torch.exp(0.5 * _normal(g, c["n"], 1))
        a, sa = _quantized(x, "int8", (1,))
        b, sb = _quantized(w, "int8", (1,))
        bias = _normal(g, c["n"]) if c["bias"] else None
        return {"case": c, "a": a, "sa": sa, "b": b, "sb": sb, "bias": bias}
    lens, news = _sizes(c)
    t, kv, d, fmt = c["tokens"], c["kv"], c["d"], c["fmt"]
    need = [(n + t - 1) // t for n in lens]
    blocks = sum(need) + 3                       # a few that no sequence owns
    # the pool's blocks in any order
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(c["seqs"], max(need), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    kc, ks = _quantized(_rows(g, blocks * kv, t, d, True).view(blocks, kv, t, d), fmt, (2, 3))
    vc, vs = _quantized(_normal(g, blocks, kv, d, t), fmt, (2, 3))
    st = {"case": c, "k": kc, "ks": ks, "v": vc, "vs": vs, "table": table,
          "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    total = sum(news)
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    # one length for all: no offsets are kept, the rows are [sequences, new]
    st["cu"] = None if c["mix"] == 0 else torch.tensor(cu, dtype=torch.int32, device="cuda")
    lead = (c["seqs"], c["new"]) if c["mix"] == 0 else (total,)
    dt = DTYPES[c["dtype"]]
    if c["op"] == "append":
        st["new_k"] = _rows(g, total, kv, d, True).to(dt).view(*lead, kv, d)
        st["new_v"] = _normal(g, total, kv, d).to(dt).view(*lead, kv, d)
    else:
        st["q"] = _rows(g, total, c["heads"], d, True).to(dt).view(*lead, c["heads"], d)
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------


def run(st):
    c = st["case"]
    if own:
        import pruning_quantization_amd as S

        if c["op"] == "gemm":
            return S.int8_gemm(st["a"], st["sa"], st["b"], st["sb"], bias=st["bias"],
                               dtype=DTYPES[c["out"]])
        cache = S.KVCache(st["k"], st["ks"], st["v"], st["vs"])
        if c["op"] == "append":
            S.kv_append(cache, st["new_k"], st["new_v"], st["table"], st["lens"],
                        cu_tokens=st["cu"])
            return _cache_values(st)
        return S.kv_attention(st["q"], cache, st["table"], st["lens"], cu_tokens=st["cu"],
                              window=c["window"], return_lse=c["lse"])
    if c["op"] == "gemm":
        y = (st["a"].float() @ st["b"].float().T) * st["sa"][:, None] * st["sb"]
        y = y if st["bias"] is None else y + st["bias"]
        return y.to(DTYPES[c["out"]])
    if c["op"] == "append":
        return _plain_append(st)
    return _plain_attend(st)


def _cache_values(st):
    """The whole cache: int8 codes are the whole numbers they stand for, e4m3
    codes are seen as their type."""
    see = (lambda x: x) if st["case"]["fmt"] == "int8" else (lambda x: x.view(torch.float8_e4m3fn))
    return {"k": see(st["k"]), "ks": st["ks"], "v": see(st["v"]), "vs": st["vs"]}


def _encode(y, fmt):
    """fp32 values in code units -> codes: nearest, ties to even, saturating."""
    y = y.clamp(-QMAX[fmt], QMAX[fmt])
    if fmt == "int8":
        return y.round().to(torch.int8)
    return y.to(torch.float8_e4m3fn).view(torch.uint8)


def _decode(codes, fmt):
    return codes.float() if fmt == "int8" else codes.view(torch.float8_e4m3fn).float()


def _token_places(st, total):
    """Sequence and position of every new token."""
    c, lens = st["case"], st["lens"].long()
    rows = torch.arange(total, device="cuda")
    if st["cu"] is None:
        b = rows // c["new"]
        first, n = b * c["new"], c["new"]
    else:
        cu = st["cu"].long()
        b = torch.searchsorted(cu[1:], rows, right=True)
        first, n = cu[b], (cu[1:] - cu[:-1])[b]
    return b, lens[b] - n + rows - first


def _plain_append(st):
    c = st["case"]
    t, kv, d, fmt = c["tokens"], c["kv"], c["d"], c["fmt"]
    k, v = st["new_k"].reshape(-1, kv, d).float(), st["new_v"].reshape(-1, kv, d).float()
    b, pos = _token_places(st, k.shape[0])
    blk, off = st["table"][b, pos // t].long(), pos % t
    blocks = st["k"].shape[0]
    # first new offset of each block: what lies before it is kept
    first = torch.full((blocks,), t, device="cuda").scatter_reduce(0, blk, off, "amin")
    kept = torch.where(first == t, torch.zeros_like(first), first)
    touched = torch.unique(blk)
    old = torch.arange(t, device="cuda") < kept[touched, None]          # [touched, t]
    _plain_side(st["k"], st["ks"], k, blk, off, first, touched, old[:, None, :, None], fmt, False)
    _plain_side(st["v"], st["vs"], v, blk, off, first, touched, old[:, None, None, :], fmt, True)
    return _cache_values(st)


def _plain_side(codes, scales, x, blk, off, first, touched, old, fmt, transposed):
    blocks, kv = scales.shape
    amax = torch.zeros(blocks, kv, device="cuda")
    amax.scatter_reduce_(0, blk[:, None].expand(-1, kv), x.abs().amax(-1), "amax")
    base = torch.where((first > 0)[:, None], scales, torch.zeros_like(scales))
    s, inv = _scale(amax, fmt, base)
    # codes kept in a block whose scale grows are coded again
    r = (base * inv)[touched][:, :, None, None]
    grew = (s > base)[touched][:, :, None, None]
    was = codes[touched]
    codes[touched] = torch.where(old & grew, _encode(_decode(was, fmt) * r, fmt), was)
    scales[touched] = s[touched]
    new = _encode(x * inv[blk][:, :, None], fmt)
    if transposed:
        codes[blk, :, :, off] = new
    else:
        codes[blk, :, off] = new


def _plain_attend(st):
    c = st["case"]
    t, kv, d, fmt, heads = c["tokens"], c["kv"], c["d"], c["fmt"], c["heads"]
    q = st["q"].reshape(-1, heads, d)
    total, n, seqs, width = q.shape[0], c["new"], c["seqs"], st["table"].shape[1]
    b, pos = _token_places(st, total)
    # padded: queries [seqs, n], keys [seqs, width * t]
    lens = st["lens"].long()
    slot = pos - lens[b] + n
    qp = torch.zeros(seqs, n, heads, d, device="cuda")
    qp[b, slot] = q.float()
    where = torch.full((seqs, n), -1, device="cuda")
    where[b, slot] = pos
    blk = st["table"].long()
    kk = (_decode(st["k"][blk], fmt) * st["ks"][blk][..., None, None])   # [seqs, width, kv, t, d]
    kk = kk.permute(0, 2, 4, 1, 3).reshape(seqs, kv, d, width * t)
    qp = qp.view(seqs, n, kv, heads // kv, d).permute(0, 2, 3, 1, 4).reshape(seqs, kv, -1, d)
    s = (qp @ kk).view(seqs, kv, heads // kv, n, width * t)
    del kk
    s *= d ** -0.5
    key = torch.arange(width * t, device="cuda")
    see = (key <= where[:, :, None]) & (key < lens[:, None, None])
    if c["window"]:
        see &= key > where[:, :, None] - c["window"]
    s.masked_fill_(~see[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = s.sub_(top).exp_()
    z = p.sum(-1, keepdim=True)
    vv = (_decode(st["v"][blk], fmt) * st["vs"][blk][..., None, None])   # [seqs, width, kv, d, t]
    vv = vv.permute(0, 2, 1, 4, 3).reshape(seqs, kv, width * t, d)
    o = p.view(seqs, kv, -1, width * t) @ vv
    o = o.view(seqs, kv, heads // kv, n, d) / torch.where(z > 0, z, torch.ones_like(z))
    o = o.permute(0, 3, 1, 2, 4).reshape(seqs, n, heads, d)[b, slot]
    o = o.to(st["q"].dtype).view(st["q"].shape)
    if not c["lse"]:
        return o
    lse = (z.log() + top).squeeze(-1).permute(0, 3, 1, 2).reshape(seqs, n, heads)[b, slot]
    return o, lse.view(st["q"].shape[:-1])


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    c = case
    if c["op"] == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        size = 4 if c["out"] == "f32" else 2
        return {"bytes": m * k + n * k + 4 * (m + n) + (4 * n if c["bias"] else 0) + size * m * n,
                "flops": 2 * m * n * k}
    lens, news = _sizes(c)
    t, kv, d, total = c["tokens"], c["kv"], c["d"], sum(news)
    if c["op"] == "append":
        size = 4 if c["dtype"] == "f32" else 2
        touched = sum((le - 1) // t - (le - n) // t + 1 for le, n in zip(lens, news) if n)
        # rows in, codes out (K and V), one scale read and written per touched block and head
        return {"bytes": 2 * (size + 1) * total * kv * d + 16 * touched * kv,
                "flops": 4 * total * kv * d}
    pairs = kept = 0
    w = c["window"]
    for le, n in zip(lens, news):
        if not n:
            continue
        if w:
            pairs += sum(min(le - n + i + 1, w) for i in range(n))
            kept += le - max(0, le - n - w + 1)
        else:
            pairs += n * (le - n) + n * (n + 1) // 2
            kept += le
    # the visible cache once, queries in, outputs (and lse) out
    return {"bytes": 2 * kept * kv * d + 4 * total * c["heads"] * d
            + (4 * total * c["heads"] if c["lse"] else 0),
            "flops": 4 * pairs * c["heads"] * d}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------


def _f32(x):
    """One rounding to 32 bits of a value held in 64."""
    return x.float().double()


def _nearest(y, fmt):
    """Nearest code value of y (64 bits), ties to even, saturating."""
    if fmt == "int8":
        return torch.round(y).clamp(-127, 127)
    y = y.clamp(-448, 448)
    exponent = torch.frexp(y)[1].long().clamp_min(-5) - 4     # of a step: 3 bits below the first
    step = ((exponent + 1023) << 52).view(torch.float64)      # an exact power of two
    return torch.round(y / step) * step


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    if c["op"] == "gemm":
        y = st["a"].double() @ st["b"].double().T * (st["sa"].double()[:, None] * st["sb"].double())
        return y if st["bias"] is None else y + st["bias"].double()
    lens, news = _sizes(c)
    t, kv, d, fmt, group = c["tokens"], c["kv"], c["d"], c["fmt"], c.get("heads", c["kv"]) // c["kv"]
    values = (lambda x: x.double()) if fmt == "int8" else (
        lambda x: x.view(torch.float8_e4m3fn).double())
    table = st["table"].tolist()
    k, v, ks, vs = values(st["k"]), values(st["v"]).transpose(2, 3), st["ks"].double(), st["vs"].double()
    start = 0
    if c["op"] == "append":
        for side, scale, rows in ((k, ks, st["new_k"]), (v, vs, st["new_v"])):
            rows, start = rows.reshape(-1, kv, d).double(), 0
            for b, (le, n) in enumerate(zip(lens, news)):
                p = le - n
                while p < le:                       # one block after the other
                    e = min(le, (p // t + 1) * t)
                    x = rows[start + p - (le - n):start + e - (le - n)].transpose(0, 1)
                    blk, o = table[b][p // t], p % t
                    amax = x.abs().amax((1, 2))
                    s = torch.where(amax < TINY, 0.0, _f32(amax / QMAX[fmt]))
                    before = scale[blk] if o else torch.zeros_like(s)
                    s = torch.maximum(s, before)
                    inv = torch.where(s > 0, _f32(1.0 / s), 0.0)[:, None, None]
                    if o:
                        again = _nearest(_f32(side[blk, :, :o] * _f32(before[:, None, None] * inv)), fmt)
                        side[blk, :, :o] = torch.where((s > before)[:, None, None], again, side[blk, :, :o])
                    side[blk, :, o:e - p + o] = _nearest(_f32(x * inv), fmt)
                    scale[blk] = s
                    p = e
                start += n
        return {"k": k, "ks": ks, "v": v.transpose(2, 3).contiguous(), "vs": vs}
    k, v = k * ks[:, :, None, None], v * vs[:, :, None, None]
    q = st["q"].reshape(-1, kv, group, d).double()
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], dtype=torch.float64, device="cuda")
    for b, (le, n) in enumerate(zip(lens, news)):
        if not n:
            continue
        own_blocks = st["table"][b, :(le + t - 1) // t].long()
        i = torch.arange(le - n, le, device="cuda")[:, None]
        j = torch.arange(le, device="cuda")
        hide = (j > i) if not c["window"] else (j > i) | (j <= i - c["window"])
        for h in range(kv):
            kb = k[own_blocks, h].reshape(-1, d)[:le]
            vb = v[own_blocks, h].reshape(-1, d)[:le]
            for r in range(group):
                s = q[start:start + n, h, r] @ kb.T / math.sqrt(d)
                s = s.masked_fill(hide, -math.inf)
                z = torch.logsumexp(s, 1)
                out[start:start + n, h, r] = torch.exp(s - z[:, None]) @ vb
                lse[start:start + n, h, r] = z
        start += n
    out = out.view(st["q"].shape)
    return (out, lse.view(st["q"].shape[:-1])) if c["lse"] else out
