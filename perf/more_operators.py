"""Measured cases of the serving operators around 4-bit data: RMS norm with the
residual's addition and a quantized output, the MXFP4 matrix product, the append
of new tokens to a paged MXFP4 key/value cache, and attention over that cache.

The four are one layer's step: the norm's codes go into the product, the
product's rows are appended to the cache, and the cache is attended to.  With
``own`` false, ``run`` computes the plain form of an operator from elementary
torch operations; with ``own`` true it makes the framework's calls.

MXFP4: E2M1 codes, two to a byte (the even element in the low nibble), and one
power of two per 32 elements as a biased exponent byte.  Codes come back as the
bytes that hold them: equal bytes are equal values, two to a byte.

Cache layout (both forms): K and V codes [blocks, kv heads, tokens, head dim / 2],
exponents [blocks, kv heads, head dim / 32, tokens].  Position p of sequence b
lives in block table[b, p // tokens].
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
QMAX = {"int8": 127.0, "fp8": 448.0}
TINY = 2.0 ** -64          # absolute maxima of a row below this get scale 0
EPS = 1e-5
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # one token before a projection: latency
        {"name": "norm one token", "op": "norm", "rows": 1, "k": 4096, "dtype": "bf16",
         "weight": "bf16", "residual": True, "fmt": "int8"},
        # odd width and count, fp16, no residual, 4-bit codes for the next product
        {"name": "norm odd", "op": "norm", "rows": 333, "k": 5152, "dtype": "f16",
         "weight": "f32", "residual": False, "fmt": "mxfp4"},
        # a long prompt with its residual stream
        {"name": "norm prompt", "op": "norm", "rows": 16384, "k": 4096, "dtype": "bf16",
         "weight": "bf16", "residual": True, "fmt": "fp8"},
        # one token through an attention output projection: latency
        {"name": "product one token", "op": "product", "m": 1, "n": 4096, "k": 4096,
         "out": "bf16", "bias": False},
        # a decoding batch through an MLP up projection
        {"name": "product decode batch", "op": "product", "m": 48, "n": 14336, "k": 4096,
         "out": "bf16", "bias": True},
        # a short odd prompt, odd width, ragged reduction, fp32 output
        {"name": "product odd", "op": "product", "m": 777, "n": 1031, "k": 2080, "out": "f32",
         "bias": True},
        # a 4096-token prompt through an MLP up projection
        {"name": "product prompt", "op": "product", "m": 4096, "n": 14336, "k": 4096,
         "out": "bf16", "bias": False},
        # one new token for each of 64 sequences: every decode step does this
        {"name": "append decode", "op": "append", "seqs": 64, "lo": 5, "hi": 2047, "new": 1,
         "mix": 0, "kv": 8, "d": 128, "tokens": 64, "dtype": "bf16"},
        # ragged chunks of prompts that begin and end inside small blocks
        {"name": "append ragged", "op": "append", "seqs": 23, "lo": 700, "hi": 3000, "new": 1500,
         "mix": 5, "kv": 4, "d": 64, "tokens": 16, "dtype": "f32"},
        # a decoding batch of 64 sequences of very different lengths
        {"name": "attend decode", "op": "attend", "seqs": 64, "lo": 300, "hi": 16384, "new": 1,
         "mix": 0, "heads": 32, "kv": 8, "d": 128, "tokens": 64, "dtype": "bf16",
         "window": 0, "lse": False},
        # chunks of prompts next to decoding sequences in one call, a sliding
        # window, small heads and blocks, fp16
        {"name": "attend mixed", "op": "attend", "seqs": 24, "lo": 70, "hi": 3500, "new": 501,
         "mix": 3, "heads": 16, "kv": 4, "d": 64, "tokens": 16, "dtype": "f16",
         "window": 1000, "lse": True},
        # a whole prompt attending to itself
        {"name": "attend prompt", "op": "attend", "seqs": 1, "lo": 8192, "hi": 8192, "new": 8192,
         "mix": 0, "heads": 32, "kv": 8, "d": 128, "tokens": 64, "dtype": "bf16",
         "window": 0, "lse": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "product", "append", "attend", "attend"))
    if op == "norm":
        while True:
            fmt = rng.choice(("int8", "fp8", "mxfp4"))
            step = 32 if fmt == "mxfp4" else 8
            c = {"op": "norm", "rows": _log(rng, 1, 16384), "k": step * _log(rng, 64 // step, 16384 // step),
                 "dtype": rng.choice(("bf16", "f16", "f32")), "residual": rng.random() < 0.6, "fmt": fmt}
            c["weight"] = rng.choice(("f32", c["dtype"]))
            if c["rows"] * c["k"] * SIZE[c["dtype"]] <= 16384 * 4096 * 2:
                return c
    if op == "product":
        while True:
            c = {"op": "product", "m": _log(rng, 1, 4096), "n": _log(rng, 64, 16384),
                 "k": 32 * _log(rng, 2, 512), "out": rng.choice(("bf16", "f16", "f32")),
                 "bias": rng.random() < 0.5}
            if c["m"] * c["n"] * c["k"] <= 4096 * 14336 * 4096:
                return c
    tokens = rng.choice((16, 32, 64, 128, 256))
    if op == "append":
        while True:
            seqs, new = _log(rng, 1, 128), _log(rng, 1, 4096)
            hi = new + _log(rng, 1, 4096)
            c = {"op": "append", "seqs": seqs, "lo": rng.randint(new, hi), "hi": hi, "new": new,
                 "mix": rng.randint(0, 9), "kv": rng.choice((1, 2, 3, 4, 8)),
                 "d": rng.choice((64, 128, 192, 256)), "tokens": tokens,
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
             "d": rng.choice((64, 128, 192, 256)), "tokens": tokens,
             "dtype": rng.choice(("bf16", "f16")),
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
    if c["op"] == "norm":
        # a layer's output (a few strong channels, tokens of different size) and
        # the residual stream that it is added to
        dt = DTYPES[c["dtype"]]
        x = _normal(g, c["rows"], c["k"])
        x[:, ::c["k"] // 4] *= 20.0
        x *= torch.exp(0.5 * _normal(g, c["rows"], 1))
        residual = (_normal(g, c["rows"], c["k"]) * 3.0).to(dt) if c["residual"] else None
        weight = (1.0 + 0.2 * _normal(g, c["k"])).to(DTYPES[c["weight"]])
        return {"case": c, "x": x.to(dt), "residual": residual, "weight": weight}
    if c["op"] == "product":
        # an activation with a few strong channels; a weight whose channels differ
        x = _normal(g, c["m"], c["k"])
        x[:, ::c["k"] // 4] *= 50.0
        w = _normal(g, c["n"], c["k"]) * 0.02
        w *= torch.exp(0.5 * _normal(g, c["n"], 1))
        a, sa = _mx(x)
        b, sb = _mx(w)
        bias = _normal(g, c["n"]) if c["bias"] else None
        return {"case": c, "a": a, "sa": sa, "b": b, "sb": sb, "bias": bias}
    lens, news = _sizes(c)
    t, kv, d = c["tokens"], c["kv"], c["d"]
    need = [(n + t - 1) // t for n in lens]
    blocks = sum(need) + 3                       # a few that no sequence owns
    # the pool's blocks in any order
    order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(c["seqs"], max(need), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    kc, ks = _mx(_rows(g, blocks * kv, t, d, True).view(blocks, kv, t, d))
    vc, vs = _mx(_normal(g, blocks, kv, t, d))
    st = {"case": c, "k": kc, "ks": ks.transpose(2, 3).contiguous(),
          "v": vc, "vs": vs.transpose(2, 3).contiguous(), "table": table,
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

        if c["op"] == "norm":
            q = ("int", 8) if c["fmt"] == "int8" else c["fmt"]
            return _norm_outputs(c, S.rmsnorm_quantize(st["x"], st["weight"], q, eps=EPS,
                                                       residual=st["residual"]))
        if c["op"] == "product":
            return S.mxfp4_gemm(st["a"], st["sa"], st["b"], st["sb"], bias=st["bias"],
                                dtype=DTYPES[c["out"]])
        cache = S.KVCache(st["k"], st["ks"], st["v"], st["vs"])
        if c["op"] == "append":
            S.kv_append(cache, st["new_k"], st["new_v"], st["table"], st["lens"],
                        cu_tokens=st["cu"])
            return _cache_values(st)
        return S.kv_attention(st["q"], cache, st["table"], st["lens"], cu_tokens=st["cu"],
                              window=c["window"], return_lse=c["lse"])
    if c["op"] == "norm":
        return _plain_norm(st)
    if c["op"] == "product":
        y = _mx_values(st["a"], st["sa"]) @ _mx_values(st["b"], st["sb"]).T
        y = y if st["bias"] is None else y + st["bias"]
        return y.to(DTYPES[c["out"]])
    if c["op"] == "append":
        return _plain_append(st)
    return _plain_attend(st)


def _norm_outputs(c, got):
    """e4m3 codes are seen as their type; int8 codes are whole numbers."""
    codes = got[0].view(torch.float8_e4m3fn) if c["fmt"] == "fp8" else got[0]
    out = {"codes": codes, "scales": got[1]}
    if c["residual"]:
        out["residual"] = got[2]
    return out


def _cache_values(st):
    """The whole cache: codes two to a byte, exponent bytes."""
    return {"k": st["k"], "ks": st["ks"], "v": st["v"], "vs": st["vs"]}


def _power(e):
    """fp32 powers of two from biased exponents 0 .. 254 (2^-127 is subnormal), exactly."""
    e = e.int()
    return torch.where(e > 0, e << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _mx(x):
    """MXFP4 of x [..., d]: codes [..., d / 2] and exponent bytes [..., d / 32]."""
    x = x.float()
    blocks = x.reshape(*x.shape[:-1], -1, 32)
    e = (torch.frexp(blocks.abs().amax(-1))[1] - 3).clamp(-127, 127)
    e = torch.where(blocks.abs().amax(-1) > 0, e, torch.full_like(e, -127))
    y = (blocks * _power(127 - e)[..., None]).reshape(x.shape)
    a = y.abs()
    # nearest value, ties to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0) + 8 * torch.signbit(y).to(torch.uint8))
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _mx_values(codes, e):
    """fp32 values of MXFP4 codes [..., d / 2] with exponent bytes [..., d / 32]."""
    values = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    x = values[torch.stack((codes & 15, codes >> 4), -1).int()]
    x = x.reshape(*codes.shape[:-1], -1, 32)
    return (x * _power(e)[..., None]).reshape(*codes.shape[:-1], -1)


def _plain_norm(st):
    c = st["case"]
    h = st["x"]
    if c["residual"]:
        h = (h.float() + st["residual"].float()).to(h.dtype)
    mean = h.double().square().sum(-1, keepdim=True) / c["k"]
    r = (1.0 / (mean + float(torch.tensor(EPS))).sqrt()).float()
    y = h.float() * r * st["weight"].float()
    if c["fmt"] == "mxfp4":
        codes, scales = _mx(y)
    else:
        # divisions by tensors: a division by a number multiplies by its rounded reciprocal
        amax = y.abs().amax(-1)
        top, there = torch.full_like(amax, QMAX[c["fmt"]]), amax >= TINY
        scales = torch.where(there, amax / top, torch.zeros_like(amax))
        inv = torch.where(there, top / amax, torch.zeros_like(amax))
        codes = (y * inv[:, None]).clamp(-QMAX[c["fmt"]], QMAX[c["fmt"]])
        codes = (codes.round().to(torch.int8) if c["fmt"] == "int8"
                 else codes.to(torch.float8_e4m3fn).view(torch.uint8))
    return _norm_outputs(c, (codes, scales, h))


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
    t, kv, d = c["tokens"], c["kv"], c["d"]
    for codes, scales, rows in ((st["k"], st["ks"], st["new_k"]), (st["v"], st["vs"], st["new_v"])):
        rows = rows.reshape(-1, kv, d)
        b, pos = _token_places(st, rows.shape[0])
        blk, off = st["table"][b, pos // t].long(), pos % t
        codes[blk, :, off], scales[blk, :, :, off] = _mx(rows)
    return _cache_values(st)


def _plain_attend(st):
    c = st["case"]
    t, kv, d, heads = c["tokens"], c["kv"], c["d"], c["heads"]
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
    kk = _mx_values(st["k"][blk], st["ks"][blk].transpose(3, 4))         # [seqs, width, kv, t, d]
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
    vv = _mx_values(st["v"][blk], st["vs"][blk].transpose(3, 4))         # [seqs, width, kv, t, d]
    vv = vv.permute(0, 2, 1, 3, 4).reshape(seqs, kv, width * t, d)
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
    if c["op"] == "norm":
        rows, k, size = c["rows"], c["k"], SIZE[c["dtype"]]
        streams = 3 if c["residual"] else 1      # x, and the residual in and out
        out = rows * (k // 2 + k // 32) if c["fmt"] == "mxfp4" else rows * (k + 4)
        return {"bytes": streams * rows * k * size + k * SIZE[c["weight"]] + out,
                "flops": (6 if c["residual"] else 5) * rows * k}
    if c["op"] == "product":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": (m + n) * (k // 2 + k // 32) + (4 * n if c["bias"] else 0) + SIZE[c["out"]] * m * n,
                "flops": 2 * m * n * k}
    lens, news = _sizes(c)
    kv, d, total = c["kv"], c["d"], sum(news)
    if c["op"] == "append":
        # rows in, codes and exponents out (K and V)
        return {"bytes": 2 * total * kv * (SIZE[c["dtype"]] * d + d // 2 + d // 32),
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
    return {"bytes": 2 * kept * kv * (d // 2 + d // 32) + 4 * total * c["heads"] * d
            + (4 * total * c["heads"] if c["lse"] else 0),
            "flops": 4 * pairs * c["heads"] * d}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------


def _f32(x):
    """One rounding to 32 bits of a value held in 64."""
    return x.float().double()


def _nearest_e4m3(y):
    """Nearest e4m3 value of y (64 bits), ties to even, saturating."""
    y = y.clamp(-448, 448)
    exponent = torch.frexp(y)[1].long().clamp_min(-5) - 4     # of a step: 3 bits below the first
    step = ((exponent + 1023) << 52).view(torch.float64)      # an exact power of two
    return torch.round(y / step) * step


def _two(e):
    """Exact powers of two, in 64 bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _four_bits(x):
    """MXFP4 of x [..., d] (64 bits): packed codes and exponent bytes."""
    g = x.unflatten(-1, (-1, 32))
    top = g.abs().amax(-1)
    e = torch.where(top > 0, torch.frexp(top)[1].long() - 3, -127).clamp(-127, 127)
    y = (g / _two(e)[..., None]).flatten(-2)
    a = y.abs().clamp_max(6.0)
    # spacing of the grid around a: 1/2 below 2, 1 below 4, 2 above; half to even
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    near = torch.round(a / step) * step
    code = torch.where(near < 2, near * 2, torch.where(near < 4, near + 2, near / 2 + 4)).long()
    code = code + 8 * torch.signbit(y).long()
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), (e + 127).to(torch.uint8)


def _of_four_bits(codes, e):
    """64-bit values of packed codes [..., d / 2] with exponent bytes [..., d / 32]."""
    c = torch.stack((codes % 16, codes // 16), -1).flatten(-2).long()
    low, up = c % 2, (c % 8) // 2                               # mantissa bit, exponent
    mag = torch.where(up == 0, 0.5 * low, (1 + 0.5 * low) * _two(up - 1))
    x = torch.where(c >= 8, -mag, mag)
    return x * _two(e.long() - 127).repeat_interleave(32, -1)


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    if c["op"] == "norm":
        h = st["x"].double()
        if c["residual"]:
            h = (h + st["residual"].double()).float().to(st["x"].dtype).double()
        r = _f32(torch.rsqrt((h * h).mean(-1) + float(torch.tensor(EPS))))
        y = _f32(_f32(h * r[:, None]) * st["weight"].double())
        if c["fmt"] == "mxfp4":
            codes, scales = _four_bits(y)
        else:
            amax, top = y.abs().amax(-1), QMAX[c["fmt"]]
            scales = torch.where(amax < TINY, 0.0, _f32(amax / top))
            z = _f32(y * torch.where(amax < TINY, 0.0, _f32(top / amax))[:, None])
            codes = torch.round(z).clamp(-127, 127).to(torch.int8) if c["fmt"] == "int8" else _nearest_e4m3(z)
        out = {"codes": codes, "scales": scales}
        if c["residual"]:
            out["residual"] = h
        return out
    if c["op"] == "product":
        y = _of_four_bits(st["a"], st["sa"]) @ _of_four_bits(st["b"], st["sb"]).T
        return y if st["bias"] is None else y + st["bias"].double()
    lens, news = _sizes(c)
    t, kv, d = c["tokens"], c["kv"], c["d"]
    table, start = st["table"].tolist(), 0
    if c["op"] == "append":
        for codes, scales, rows in ((st["k"], st["ks"], st["new_k"]), (st["v"], st["vs"], st["new_v"])):
            rows, start = rows.reshape(-1, kv, d).double(), 0
            for b, (le, n) in enumerate(zip(lens, news)):
                p = le - n
                while p < le:                       # one block after the other
                    end = min(le, (p // t + 1) * t)
                    x = rows[start + p - (le - n):start + end - (le - n)].transpose(0, 1)
                    blk, o = table[b][p // t], p % t
                    x, e = _four_bits(x)
                    codes[blk, :, o:o + end - p] = x
                    scales[blk, :, :, o:o + end - p] = e.transpose(1, 2)
                    p = end
                start += n
        return {"k": st["k"], "ks": st["ks"], "v": st["v"], "vs": st["vs"]}
    group = c["heads"] // kv
    k, v = (_of_four_bits(x, e.transpose(2, 3)) for x, e in ((st["k"], st["ks"]), (st["v"], st["vs"])))
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
