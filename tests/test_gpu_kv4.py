"""GPU parity of the paged MXFP4 key/value cache: append (bit for bit) and attention
(against the oracle in 64 bits), alone and in a run with the norm, the MXFP4 product
and the quantizer.

Bound of an attention output, with P = sum_t p_t |V_t| / sum_t p_t:
* a score is off by the fp32 sum of D exact products, at most (D + 8) 2^-24 of scale *
  sum_d |q_d K_td|, and its exponent (below 2^3 in units of log2 here, or 2^bits) by the
  factor's and the fma's roundings and an instruction of one unit in the last place:
  2^(bits - 22) of the weight; a score that is off by e changes its weight by e, in the
  numerator and in the sum;
* a weight is rounded to the queries' type: 2^-8 (bf16) or 2^-11 (fp16), and below fp16's
  2^-14, where the largest stands at 2^8 or more, by 2^-25: 2^-33 of the largest |V| a token;
* the fp32 sums over the tokens: len * 2^-23, in the numerator and in the sum;
* the output's rounding: half a step, and 2^-24 (of fp16's subnormals).
A log-sum is off by a score's error, the fp32 sum and its own rounding."""
import numpy as np
import pytest

import oracle as O
import oracle.serving4 as V

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU, skipped there
    pytest.skip("no GPU", allow_module_level=True)

import pruning_quantization_amd as S  # noqa: E402
from gpu_util import DEV, raw_np  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def stored(x, dtype):
    """x rounded to the type: a device tensor and its exact float64 values."""
    t = torch.from_numpy(np.asarray(x, np.float32)).to(DT[dtype])
    return t.to(DEV), t.to(torch.float64).numpy()


class Pool:
    """A cache in use: random codes and exponents in every block, tables in any order,
    lens tokens in each sequence.  wide: tables that allow more than the 1024 tokens up
    to which a call splits no sequence."""

    def __init__(self, seed, lens, kv=2, dim=64, tokens=16, width=None, spare=2, wide=False):
        rng = self.rng = np.random.default_rng(seed)
        self.lens, self.tokens, self.kv, self.dim = list(lens), tokens, kv, dim
        need = [-(-max(n, 0) // tokens) for n in lens]
        blocks = max(1, sum(need) + spare)
        width = width or max(max(need), 1025 // tokens + 1 if wide else 1)
        order = rng.permutation(blocks).astype(np.int32)
        self.table = np.full((len(lens), width), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        codes = lambda: rng.integers(0, 256, (blocks, kv, tokens, dim // 2)).astype(np.uint8)  # noqa: E731
        exps = lambda: rng.integers(122, 127, (blocks, kv, dim // 32, tokens)).astype(np.uint8)  # noqa: E731
        self.ref = (codes(), exps(), codes(), exps())

    def dev(self, ref=None):
        return S.KVCache(*(torch.from_numpy(x.copy()).to(DEV) for x in ref or self.ref))

    def args(self):
        return (torch.from_numpy(self.table).to(DEV),
                torch.tensor(self.lens, dtype=torch.int32, device=DEV))


def offsets(news):
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    return cu, torch.from_numpy(cu).to(DEV)


def check_attention(got, lse, pool, q64, cu, dtype, scale, ref=None, bits=4, **kw):
    ref = ref or pool.ref
    out, want_lse, spread, reach = V.kv_attention(q64, ref, pool.table, pool.lens, cu, scale, **kw)
    n = max(max(pool.lens), 1)
    vmax = 6 * 2.0 ** (float(ref[3][ref[3] < 255].max()) - 127)
    ds = (pool.dim + 8) * 2.0 ** -24 * reach + 2.0 ** (bits - 22)
    weight = torch.finfo(DT[dtype]).eps / 2
    tol = (spread * (weight + 2 * ds[..., None] + 2 * n * 2.0 ** -23) + (n * 2.0 ** -33 * vmax if dtype == "f16" else 0)
           + np.abs(out) * weight + 2.0 ** -24)
    got = got.cpu().to(torch.float64).numpy().reshape(out.shape)
    ok = np.abs(got - out) <= tol
    assert ok.all(), f"{(~ok).sum()} of {ok.size} outside; worst {np.nanmax(np.abs(got - out) / tol):.3g}"
    if lse is not None:
        l64 = lse.cpu().to(torch.float64).numpy().reshape(want_lse.shape)
        none = np.isneginf(want_lse)
        assert np.array_equal(none, np.isneginf(l64))
        with np.errstate(invalid="ignore"):
            ok = np.abs(l64 - want_lse) <= ds + n * 2.0 ** -23 + 2.0 ** -21 * np.abs(want_lse)
        assert ok[~none].all()


def unchanged(cache, ref):
    for t, x in zip(cache, ref):
        assert np.array_equal(t.cpu().numpy(), x)


# --- append ------------------------------------------------------------------


@pytest.mark.parametrize("dtype,dim,tokens,kv", [
    ("bf16", 128, 64, 8), ("f16", 64, 16, 3), ("f32", 192, 32, 1), ("bf16", 256, 256, 2), ("f32", 128, 128, 2),
    ("f16", 64, 64, 1)])
def test_append(dtype, dim, tokens, kv):
    # whole prompts, ends inside blocks, single tokens, nothing, one that fills its block
    news = [tokens * 2 + 5, 1, 0, 3, tokens, 1, 7, 1]
    lens = [tokens * 2 + 5, 40, 9, 3, tokens * 3, tokens, tokens + 3, tokens * 2 + 1]
    p = Pool(dim + tokens, lens, kv, dim, tokens)
    cu, dcu = offsets(news)
    size = np.exp(p.rng.normal(0.5, 3.0, (cu[-1], kv, 1)))
    k, k64 = stored(p.rng.standard_normal((cu[-1], kv, dim)) * size, dtype)
    v, v64 = stored(p.rng.standard_normal((cu[-1], kv, dim)) * size[::-1], dtype)
    cache = p.dev()
    want = V.kv_append(p.ref, k64, v64, p.table, lens, cu)
    S.kv_append(cache, k, v, *p.args(), cu_tokens=dcu)
    unchanged(cache, want)
    S.kv_append(cache, k, v, *p.args(), cu_tokens=dcu)       # again: nothing changes
    unchanged(cache, want)
    # the codes are those of the quantizer
    codes, exps = S.quantize(k.contiguous(), "mxfp4")
    for b, n in enumerate(news):
        for i in range(n):
            pos = lens[b] - n + i
            blk = p.table[b, pos // tokens]
            assert torch.equal(cache.k[blk, :, pos % tokens], codes[cu[b] + i])
            assert torch.equal(cache.k_scale[blk, :, :, pos % tokens], exps[cu[b] + i])


@pytest.mark.parametrize("n", [1, 5, 33])
def test_append_same_count_strided(n):
    # rows cut out of a fused projection [tokens, (q, k, v) heads, dim]
    lens = [n, 50, 64, n + 31, 200]
    p = Pool(n, lens, 2, 64, 32)
    fused, f64 = stored(p.rng.standard_normal((5, n, 8, 64)) * 3, "bf16")
    cu, _ = offsets([n] * 5)
    cache = p.dev()
    S.kv_append(cache, fused[:, :, 4:6], fused[:, :, 6:8], *p.args())
    f64 = f64.reshape(5 * n, 8, 64)
    unchanged(cache, V.kv_append(p.ref, f64[:, 4:6], f64[:, 6:8], p.table, lens, cu))


def test_append_special_values():
    x = np.zeros((4, 20, 1, 64), np.float32)
    x[0] = 2.0 ** -140
    x[1, 3, 0, 5], x[1, 9], x[1, 4, 0, 32:], x[1, 5, 0, 40] = np.nan, 3e38, np.inf, -np.inf
    x[1, 6], x[1, 7, 0, ::2] = np.nan, np.nan
    x[1, :, 0, 1] += 1.0
    x[2] = -0.0
    x[3] = 2.0 ** -126 * np.arange(64)
    lens, cu = [16, 20, 5, 33], [0, 16, 36, 41, 61]
    rows = np.concatenate([x[0, :16], x[1], x[2, :5], x[3]])
    k, k64 = stored(rows, "f32")
    p = Pool(5, lens, 1, 64, 16)
    cache = p.dev()
    S.kv_append(cache, k, k, *p.args(), cu_tokens=torch.tensor(cu, dtype=torch.int32, device=DEV))
    unchanged(cache, V.kv_append(p.ref, k64, k64, p.table, lens, cu))


def test_append_stays_out_of_what_is_not_named():
    # entries outside the pool, positions past the table, more rows than tokens, spare rows
    p = Pool(8, [40, 40, 30, 5], 1, 64, 16)
    p.table[0, 1], p.table[1, 2] = -7, 10 ** 6
    p.lens = [40, 40, 100, 5]                # 100 tokens, a table of 48
    news = [40, 20, 70, 9]
    cu, dcu = offsets(news)
    k, k64 = stored(p.rng.standard_normal((cu[-1] + 6, 1, 64)), "bf16")
    cache = p.dev()
    S.kv_append(cache, k, k, *p.args(), cu_tokens=dcu)
    unchanged(cache, V.kv_append(p.ref, k64, k64, p.table, p.lens, cu))


def test_append_two_sequences_to_one_block():
    # a block shared by two sequences, each at positions of its own
    p = Pool(9, [16, 16], 2, 64, 16)
    p.table[:] = 1
    p.lens = [8, 16]
    cu, dcu = offsets([8, 5])
    k, k64 = stored(p.rng.standard_normal((13, 2, 64)), "bf16")
    cache = p.dev()
    S.kv_append(cache, k, k, *p.args(), cu_tokens=dcu)
    unchanged(cache, V.kv_append(p.ref, k64, k64, p.table, p.lens, cu))


@pytest.mark.parametrize("uniform", [False, True])
def test_append_to_thousands(uniform):
    rng = np.random.default_rng(13)
    lens = [int(x) for x in rng.integers(2, 40, 4200)]
    news = [2] * 4200 if uniform else [min(n, int(x)) for n, x in zip(lens, rng.integers(0, 4, 4200))]
    p = Pool(14, lens, 1, 64, 16)
    cu, dcu = offsets(news)
    k, k64 = stored(p.rng.standard_normal((cu[-1], 1, 64)) * 2, "bf16")
    cache = p.dev()
    if uniform:
        S.kv_append(cache, k.view(4200, 2, 1, 64), k.view(4200, 2, 1, 64), *p.args())
    else:
        S.kv_append(cache, k, k, *p.args(), cu_tokens=dcu)
    unchanged(cache, V.kv_append(p.ref, k64, k64, p.table, lens, cu))


# --- attention ----------------------------------------------------------------


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,tokens,kv,group", [
    (64, 16, 2, 1), (128, 64, 2, 4), (128, 32, 1, 5), (192, 128, 1, 3), (256, 256, 1, 2), (256, 16, 2, 16),
    (64, 64, 1, 48), (128, 256, 1, 71), (192, 16, 1, 20), (256, 64, 1, 33)])
def test_decode(dim, tokens, kv, group, dtype, wide):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 129, 511, 700]
    p = Pool(dim + group, lens, kv, dim, tokens, wide=wide)
    q, q64 = stored(p.rng.standard_normal((len(lens), 1, kv * group, dim)), dtype)
    cu = np.arange(len(lens) + 1)
    out, lse = S.kv_attention(q, p.dev(), *p.args(), return_lse=True)
    assert out.shape == q.shape and lse.shape == q.shape[:-1]
    check_attention(out, lse, p, q64[:, 0], cu, dtype, dim ** -0.5)
    assert torch.equal(out, S.kv_attention(q, p.dev(), *p.args()))          # the same bits without lse
    S.kv_attention(q, p.dev(), *p.args(), out=q)                            # over its own queries
    assert torch.equal(out, q)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("kw", [{}, {"window": 1}, {"window": 37}, {"window": 200}, {"causal": False}])
@pytest.mark.parametrize("dim,tokens,group,dtype", [(64, 16, 4, "bf16"), (128, 64, 3, "f16"), (256, 32, 1, "bf16"),
                                                    (192, 64, 2, "bf16"), (64, 128, 2, "f16"), (128, 16, 2, "bf16"),
                                                    (192, 32, 1, "f16"), (256, 64, 1, "f16")])
def test_chunks(dim, tokens, group, dtype, kw, wide):
    # whole prompts, chunks behind a context, decoding, nothing, in one call
    lens = [130, 400, 77, 9, 64, 300, 1]
    news = [130, 90, 1, 0, 64, 2, 1]
    p = Pool(dim, lens, 2, dim, tokens, wide=wide)
    cu, dcu = offsets(news)
    q, q64 = stored(p.rng.standard_normal((cu[-1], 2 * group, dim)) * 1.5, dtype)
    out, lse = S.kv_attention(q, p.dev(), *p.args(), cu_tokens=dcu, return_lse=True, scale=0.11, **kw)
    check_attention(out, lse, p, q64, cu, dtype, np.float32(0.11), **kw)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("n", [2, 16, 70, 257])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_same_count_strided(n, dtype, wide):
    # queries cut out of a fused projection; n tokens of each sequence
    lens = [n, n + 1, n + 300]
    p = Pool(n, lens, 2, 128, 64, wide=wide)
    fused, f64 = stored(p.rng.standard_normal((3, n, 12, 128)), dtype)
    cu = np.arange(4) * n
    out = S.kv_attention(fused[:, :, :8], p.dev(), *p.args())
    check_attention(out, None, p, f64.reshape(3 * n, 12, 128)[:, :8], cu, dtype, 128 ** -0.5)


@pytest.mark.parametrize("seqs,dim,n", [(9, 128, 270), (13, 64, 270), (25, 64, 200)])
def test_prompts_of_the_same_count(seqs, dim, n):
    # two row tiles a CU (three, one), all resident at once: the second from the shortest up
    p = Pool(seqs, [n + (7 * i) % 30 for i in range(seqs)], 8, dim, 32)
    q, q64 = stored(p.rng.standard_normal((seqs, n, 16, dim)), "bf16")
    out, lse = S.kv_attention(q, p.dev(), *p.args(), return_lse=True)
    check_attention(out, lse, p, q64.reshape(seqs * n, 16, dim), np.arange(seqs + 1) * n, "bf16", dim ** -0.5)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,tokens,kv,group,n,kw", [
    (64, 16, 2, 4, 5, {}), (128, 64, 1, 4, 8, {}), (192, 32, 2, 3, 6, {"window": 70}), (256, 128, 1, 8, 3, {}),
    (128, 16, 1, 1, 17, {"causal": False}), (64, 64, 1, 32, 1, {}), (256, 16, 2, 2, 16, {"window": 5}),
    (192, 64, 1, 7, 4, {})])
def test_two_row_tiles(dim, tokens, kv, group, n, kw, dtype, wide):
    # 17 to 32 rows per kv head: more tokens than the sequence has, ends in a tile, many tiles
    lens = [n, n + 1, max(n - 2, 0), 64, 65, 700, 1023]
    p = Pool(dim + n, lens, kv, dim, tokens, wide=wide)
    p.ref[1][:, :, 0, :3], p.ref[3][:, :, -1, 5:7] = 255, 255
    q, q64 = stored(p.rng.standard_normal((len(lens), n, kv * group, dim)), dtype)
    clean = tuple(np.where(x == 255, 120, x).astype(np.uint8) if i % 2 else x for i, x in enumerate(p.ref))
    cu = np.arange(len(lens) + 1) * n
    out, lse = S.kv_attention(q, p.dev(clean), *p.args(), return_lse=True, **kw)
    check_attention(out, lse, p, q64.reshape(-1, kv * group, dim), cu, dtype, dim ** -0.5, ref=clean, **kw)
    # NaN scales of tokens that a row sees, and only they, make it NaN
    nan = S.kv_attention(q, p.dev(), *p.args(), **kw).cpu()
    seen = torch.zeros(len(lens), n, dtype=torch.bool)
    for b, length in enumerate(lens):
        for i in range(n):
            pos = length - n + i
            hi = min(pos + 1, length) if kw.get("causal", True) else length
            lo = max(pos - kw["window"] + 1, 0) if kw.get("window") else 0
            seen[b, i] = any(t % tokens in (0, 1, 2, 5, 6) for t in range(lo, hi))
    assert nan[seen].isnan().all() and torch.equal(nan[~seen], out.cpu()[~seen])


@pytest.mark.parametrize("dim", [64, 128])
def test_counts_around_two_row_tiles(dim):
    # offsets: 17 to 32 rows on average, from none to many in a sequence
    news, lens = [5, 1, 0, 8, 4, 21, 7, 2], [900, 3, 50, 8, 1500, 21, 70, 2000]
    p = Pool(dim, lens, 2, dim, 32)
    cu, dcu = offsets(news)
    q, q64 = stored(p.rng.standard_normal((cu[-1], 8, dim)), "bf16")
    out, lse = S.kv_attention(q, p.dev(), *p.args(), cu_tokens=dcu, return_lse=True)
    check_attention(out, lse, p, q64, cu, "bf16", dim ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_split_along_the_tokens(dtype):
    # far more tiles than one workgroup takes; a width that allows much more
    p = Pool(21, [6001, 40, 0, 1500], 1, 64, 32, width=400)
    q, q64 = stored(p.rng.standard_normal((4, 1, 3, 64)), dtype)
    out, lse = S.kv_attention(q, p.dev(), *p.args(), return_lse=True)
    check_attention(out, lse, p, q64[:, 0], np.arange(5), dtype, 0.125)
    assert not out[2].any()


@pytest.mark.parametrize("wide", [False, True])
def test_rows_that_see_nothing(wide):
    p = Pool(4, [0, 3, 50, 40], 1, 64, 16, wide=wide)
    p.table[2, 1:], p.table[3, :] = 10 ** 6, -1      # a part of a table, a whole table outside the pool
    news = [2, 6, 5, 2]                               # more queries than tokens: the first see nothing
    cu, dcu = offsets(news)
    q, q64 = stored(p.rng.standard_normal((cu[-1], 2, 64)), "bf16")
    out, lse = S.kv_attention(q, p.dev(), *p.args(), cu_tokens=dcu, return_lse=True)
    check_attention(out, lse, p, q64, cu, "bf16", 0.125)
    assert not out[:5].any() and torch.isinf(lse[:5]).all() and not out[13:].any()
    out, lse = S.kv_attention(q, p.dev(), *p.args(), cu_tokens=dcu, return_lse=True, window=20)
    check_attention(out, lse, p, q64, cu, "bf16", 0.125, window=20)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,dim,group", [(16, 64, 2), (64, 128, 2), (128, 192, 1), (64, 256, 12), (32, 128, 12)])
def test_garbage_in_unseen_places(tokens, dim, group, dtype, wide):
    # NaN and huge scales behind the sequences, before the windows and in foreign blocks
    lens = [tokens + 3, 5, 200, 3 * tokens]
    p = Pool(tokens, lens, 2, dim, tokens, spare=4, wide=wide)
    q, q64 = stored(p.rng.standard_normal((4, 2, 2 * group, dim)), dtype)
    cu = np.arange(5) * 2
    for window in (0, 30):
        dirty = [x.copy() for x in p.ref]
        seen = np.zeros((p.ref[0].shape[0], tokens), bool)
        for b, n in enumerate(lens):
            for pos in range(max(0, n - 2 - window + 1) if window else 0, n):
                seen[p.table[b, pos // tokens], pos % tokens] = True
        for i, byte in ((1, 255), (3, 255)):
            dirty[i][np.broadcast_to(~seen[:, None, None, :], dirty[i].shape)] = byte
        dirty[3][:, :, 0, ::3][np.broadcast_to(~seen[:, None, ::3], dirty[3][:, :, 0, ::3].shape)] = 254
        out, lse = S.kv_attention(q, p.dev(dirty), *p.args(), return_lse=True, window=window)
        check_attention(out, lse, p, q64.reshape(8, 2 * group, dim), cu, dtype, dim ** -0.5, window=window)
        clean, cl = S.kv_attention(q, p.dev(), *p.args(), return_lse=True, window=window)
        assert torch.equal(out, clean) and torch.equal(lse, cl)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("side", [1, 3])
@pytest.mark.parametrize("dim,tokens,group,n", [(64, 16, 2, 1), (128, 64, 4, 3), (192, 32, 1, 40), (256, 128, 2, 20),
                                                (128, 16, 2, 70), (64, 64, 2, 70)])
def test_nan_scales_reach_the_rows_that_see_them(dim, tokens, group, n, side, dtype, wide):
    lens = [200, 150]
    p = Pool(dim + n, lens, 2, dim, tokens, wide=wide)
    q, q64 = stored(p.rng.standard_normal((2, n, 2 * group, dim)), dtype)
    bad = 200 - n // 2 - 1                       # position in the first sequence, kv head 1
    want, wl = S.kv_attention(q, p.dev(), *p.args(), return_lse=True)
    dirty = [x.copy() for x in p.ref]
    dirty[side][p.table[0, bad // tokens], 1, dim // 32 - 1, bad % tokens] = 255
    out, lse = S.kv_attention(q, p.dev(dirty), *p.args(), return_lse=True)
    hit = torch.zeros(2, n, 2 * group, dtype=torch.bool, device=DEV)
    hit[0, max(0, bad - (200 - n)):, group:] = True
    assert out[hit].isnan().all() and lse[hit].isnan().all()
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], wl[~hit])


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("dtype,low,high", [("bf16", 90, 133), ("f16", 108, 131)])
def test_exponents_far_apart(dtype, low, high, n, wide):
    # exponents over many binades on both sides (fp16: within its normal range), and zeros
    lens = [500, 64, 300]
    p = Pool(31, lens, 2, 128, 16, wide=wide)
    k, ks, v, vs = (x.copy() for x in p.ref)
    ks[:] = p.rng.integers(low, 127, ks.shape)
    vs[:] = p.rng.integers(low, high, vs.shape)
    zero = p.rng.random(vs.shape) < 0.2
    vs[zero] = 0
    v.reshape(*v.shape[:3], -1, 16)[zero.transpose(0, 1, 3, 2)] = 0
    p.ref = (k, ks, v, vs)
    q, q64 = stored(p.rng.standard_normal((3, n, 4, 128)) * np.exp2(p.rng.integers(-3, 3, (3, n, 4, 1))), dtype)
    out, lse = S.kv_attention(q, p.dev(), *p.args(), return_lse=True)
    check_attention(out, lse, p, q64.reshape(3 * n, 4, 128), np.arange(4) * n, dtype, 128 ** -0.5, bits=7)
    p.ref = (k, ks, np.zeros_like(v), np.zeros_like(vs))
    out, lse = S.kv_attention(q, p.dev(), *p.args(), return_lse=True)
    assert not out.any()


@pytest.mark.parametrize("n", [1, 40])
def test_scales_past_fp16_saturate(n):
    p = Pool(33, [100, 70], 1, 64, 16)
    q, _ = stored(p.rng.standard_normal((2, n, 2, 64)), "f16")
    for byte in (141, 254):
        got = []
        for b in (140, byte):
            ref = [x.copy() for x in p.ref]
            ref[3][:] = b                    # the values; keys as they were
            got.append(S.kv_attention(q, p.dev(ref), *p.args()))
        assert torch.equal(*got) and got[0].isfinite().all() and got[0].any()


@pytest.mark.parametrize("n", [1, 40])
def test_large_scores(n):
    # scores are exact multiples of 2^12: the largest takes all (or several share it), past
    # the range in which one fma forms the exponent; the weights are powers of two
    p = Pool(35, [300, 200], 1, 64, 32)
    p.ref[1][:] = 126
    q, q64 = stored(np.sign(p.rng.standard_normal((2, n, 2, 64))) * 2.0 ** 12, "bf16")
    out, lse = S.kv_attention(q, p.dev(), *p.args(), return_lse=True, scale=4.0)
    o, want, spread, _ = V.kv_attention(q64.reshape(2 * n, 2, 64), p.ref, p.table, p.lens, np.arange(3) * n, 4.0)
    assert np.abs(want).max() > 2.0 ** 17
    got = out.cpu().double().numpy().reshape(o.shape)
    assert (np.abs(got - o) <= spread * 600 * 2.0 ** -23 + np.abs(o) * 2.0 ** -8).all()
    got = lse.cpu().double().numpy().reshape(want.shape)
    assert (np.abs(got - want) <= np.abs(want) * 2.0 ** -21).all()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n", [1, 30])
def test_queries_that_are_no_numbers(n, dtype, wide):
    p = Pool(41, [300, 300, 300], 1, 128, 64, wide=wide)
    q, _ = stored(p.rng.standard_normal((3, n, 2, 128)), dtype)
    out, lse = S.kv_attention(q, p.dev(), *p.args(), return_lse=True)
    q[2, 0, 1, 7], q[0, n - 1, 0, 127] = float("nan"), float("inf")
    out2, lse2 = S.kv_attention(q, p.dev(), *p.args(), return_lse=True)
    hit = torch.zeros(3, n, 2, dtype=torch.bool, device=DEV)
    hit[2, 0, 1] = hit[0, n - 1, 0] = True
    assert out2[hit].isnan().all() and lse2[hit].isnan().all()
    assert torch.equal(out[~hit], out2[~hit]) and torch.equal(lse[~hit], lse2[~hit])
    # a row that sees nothing is zeros whatever its query
    out3 = S.kv_attention(q, p.dev(), p.args()[0], torch.zeros(3, dtype=torch.int32, device=DEV))
    assert not out3.any()


def test_rows_of_no_sequence_stay():
    p = Pool(2, [20, 70], 1, 64, 16)
    cu, dcu = offsets([1, 3])
    q, q64 = stored(p.rng.standard_normal((9, 2, 64)), "bf16")
    out = torch.full((9, 2, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((9, 2), 3.0, device=DEV)
    S.kv_attention(q, p.dev(), *p.args(), cu_tokens=dcu, out=out, lse=lse)
    check_attention(out[:4], lse[:4], p, q64[:4], cu, "bf16", 0.125)
    assert (out[4:] == 3).all() and (lse[4:] == 3).all()


@pytest.mark.parametrize("uniform", [False, True])
@pytest.mark.parametrize("count,kv", [(66, 1), (129, 1), (300, 2)])
def test_many_sequences_some_split(count, kv, uniform):
    # more sequences than a workgroup adds up by itself, a few of them split
    rng = np.random.default_rng(count + uniform)
    lens = [int(x) for x in rng.integers(1, 90, count)]
    for b, n in ((0, 2500), (count // 2, 1100), (count - 1, 1700)):
        lens[b] = n
    p = Pool(count, lens, kv, 64, 16)
    news = [1] * count if uniform else [min(n, int(x)) for n, x in zip(lens, rng.integers(0, 3, count))]
    if not uniform:
        news[3], news[count - 1] = min(lens[3], 40), 200                 # the second: prompt rows
    cu, dcu = offsets(news)
    q, q64 = stored(rng.standard_normal((cu[-1], 2 * kv, 64)), "f16")
    x, kw = (q[:, None], {}) if uniform else (q, {"cu_tokens": dcu})
    out, lse = S.kv_attention(x, p.dev(), *p.args(), return_lse=True, **kw)
    check_attention(out, lse, p, q64, cu, "f16", 0.125)


def test_offsets_past_32_bits():
    # a pool of more than 2^32 code bytes on each side; the last blocks are used
    blocks, kv, T, D = 130 * 1024 + 8, 4, 64, 256
    cache = S.kv_cache(blocks, kv, D, T, "mxfp4")
    assert cache.k.numel() > 2 ** 32
    rng = np.random.default_rng(2)
    table = np.array([[blocks - 1, blocks - 3]], np.int32)
    rows, r64 = stored(rng.standard_normal((1, 100, kv, D)), "bf16")
    args = torch.from_numpy(table).to(DEV), torch.tensor([100], dtype=torch.int32, device=DEV)
    S.kv_append(cache, rows, rows, *args)
    small = tuple(np.zeros(s, np.uint8) for s in ((3, kv, T, D // 2), (3, kv, D // 32, T)) * 2)
    want = V.kv_append(small, r64[0], r64[0], np.array([[2, 0]]), [100], [0, 100])
    for t, x in zip(cache, want):
        assert np.array_equal(t[blocks - 3:].cpu().numpy(), x)
        assert not t[:blocks - 3].any()
    for n in (1, 30):
        q, q64 = stored(rng.standard_normal((1, n, 8, D)), "bf16")
        out = S.kv_attention(q, cache, *args)
        o, _, spread, _ = V.kv_attention(q64[0], want, np.array([[2, 0]]), [100], [0, n], D ** -0.5)
        assert (np.abs(out[0].cpu().double().numpy() - o) <= spread * 2.0 ** -7 + np.abs(o) * 2.0 ** -8).all()


def test_refusals():
    p = Pool(2, [20, 70], 2, 64, 16)
    c, (table, lens) = p.dev(), p.args()
    q = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16, device=DEV)
    for bad in (lambda: S.kv_attention(q, c, table.cpu(), lens),
                lambda: S.kv_attention(q, c._replace(v_scale=c.v_scale[:, :1]), table, lens),
                lambda: S.kv_append(c, q[:, :, :2], q[:, :, :1], table, lens)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: S.kv_attention(q.float(), c, table, lens), lambda: S.kv_attention(q[:, :, :3], c, table, lens),
                lambda: S.kv_attention(q, c, table, lens, causal=False, window=4),
                lambda: S.kv_append(c, q, q, table, lens)):
        with pytest.raises(S.Sparq24Error):
            bad()


# --- together -------------------------------------------------------------------


def layer(x, res, norm, w, wo, cache, table, lens, cu, heads, kv, dim, ws=None):
    """One attention layer of a serving step on 4-bit operands."""
    cx, sx, res = S.rmsnorm_quantize(x, norm, "mxfp4", residual=res)
    y = S.mxfp4_gemm(cx, sx, *w, dtype=torch.bfloat16).view(-1, heads + 2 * kv, dim)
    q, k, v = y[:, :heads], y[:, heads:heads + kv], y[:, heads + kv:]
    S.kv_append(cache, k, v, table, lens, cu_tokens=cu)
    o = S.kv_attention(q, cache, table, lens, cu_tokens=cu, workspace=ws)
    co, so = S.quantize(o.view(-1, heads * dim), "mxfp4")
    return cx, sx, res, y, o, S.mxfp4_gemm(co, so, *wo)


def test_a_serving_step():
    rng = np.random.default_rng(17)
    heads, kv, dim, hidden, T = 8, 2, 64, 256, 16
    p = Pool(18, [90, 33, 70], kv, dim, T, width=8)
    news = [90, 1, 5]
    cu, dcu = offsets(news)
    x, _ = stored(rng.standard_normal((cu[-1], hidden)), "bf16")
    res, _ = stored(rng.standard_normal((cu[-1], hidden)) * 3, "bf16")
    norm, _ = stored(rng.random(hidden) + 0.5, "f32")
    w, _ = stored(rng.standard_normal(((heads + 2 * kv) * dim, hidden)) * 0.05, "bf16")
    wo, _ = stored(rng.standard_normal((hidden, heads * dim)) * 0.05, "bf16")
    w4, wo4 = S.quantize(w, "mxfp4"), S.quantize(wo, "mxfp4")
    cache = p.dev()
    cx, sx, total, y, o, z = layer(x, res, norm, w4, wo4, cache, *p.args(), dcu, heads, kv, dim)
    # each stage against the oracle on what the stage before gave
    want = V.rmsnorm_quantize(raw_np(x), "bf16", raw_np(norm), 1e-6, O.QSpec("mxfp4"), raw_np(res))
    for a, b in zip((cx, sx, total), want):
        assert np.array_equal(raw_np(a), b)
    product, size = V.mxfp4_gemm(raw_np(cx), raw_np(sx), raw_np(w4[0]), raw_np(w4[1]))
    y64 = y.cpu().double().numpy()
    assert (np.abs(y64.reshape(product.shape) - product) <= size * 16 * 2.0 ** -23 + np.abs(product) * 2.0 ** -8).all()
    ref = V.kv_append(p.ref, y64[:, heads:heads + kv], y64[:, heads + kv:], p.table, p.lens, cu)
    unchanged(cache, ref)
    check_attention(o, None, p, y64[:, :heads], cu, "bf16", dim ** -0.5, ref=ref)
    co, so = O.quantize_mxfp4(raw_np(o.reshape(-1, heads * dim)), "bf16")
    product, size = V.mxfp4_gemm(co, so, raw_np(wo4[0]), raw_np(wo4[1]))
    assert (np.abs(z.cpu().double().numpy() - product) <= size * 24 * 2.0 ** -23 + np.abs(product) * 2.0 ** -23).all()


def test_captured_steps_replay():
    # two captured decode steps that share nothing but the cache, replayed with other inputs,
    # eager work and synchronizations in between; workspaces of their own
    rng = np.random.default_rng(19)
    heads, kv, dim, hidden, T = 4, 2, 64, 128, 16
    p = Pool(20, [1300, 30, 5], kv, dim, T, width=120)
    mk = lambda *s: stored(rng.standard_normal(s) * 0.1, "bf16")[0]  # noqa: E731
    w4 = S.quantize(mk((heads + 2 * kv) * dim, hidden), "mxfp4")
    wo4 = S.quantize(mk(hidden, heads * dim), "mxfp4")
    x, res, norm = mk(3, hidden), mk(3, hidden), torch.ones(hidden, device=DEV)
    table, lens = p.args()
    dcu = torch.arange(4, dtype=torch.int32, device=DEV)
    cache = p.dev()
    ws = [torch.empty(8 << 20, dtype=torch.uint8, device=DEV) for _ in range(2)]
    run = lambda c, w: layer(x, res, norm, w4, wo4, c, table, lens, dcu, heads, kv, dim, w)  # noqa: E731
    run(cache, ws[0])     # warm
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(cache, ws[i]))
        graphs.append(g)
    for step in range(5):
        x.copy_(mk(3, hidden))
        lens += 1
        eager = S.KVCache(*(t.clone() for t in cache))
        want = [t.clone() for t in run(eager, ws[0])]
        ws[0].fill_(0xFF)
        torch.cuda.synchronize()
        graphs[step % 2].replay()
        if step % 2:
            torch.cuda.synchronize()
        for a, b in zip(outs[step % 2], want):
            assert torch.equal(a, b)
        for a, b in zip(cache, eager):
            assert torch.equal(a, b)


def test_captured_many_sequences_follow_their_lengths():
    # the work list of a replay comes from the lengths and offsets of that replay
    rng = np.random.default_rng(23)
    count = 140
    lens = [int(x) for x in rng.integers(1, 90, count)]
    lens[7] = 1900
    p = Pool(24, lens, 1, 64, 16)
    table, dlens = p.args()
    cu, dcu = offsets(np.ones(count, int))
    q, q64 = stored(rng.standard_normal((count, 2, 64)), "f16")
    cache = p.dev()
    S.kv_attention(q, cache, table, dlens, cu_tokens=dcu)                # warm
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = S.kv_attention(q, cache, table, dlens, cu_tokens=dcu, return_lse=True)
    for step in range(4):
        now = [max(1, n - 13 * step * (b % 3)) for b, n in enumerate(lens)]
        take = np.ones(count, int)
        take[3 * step], take[3 * step + 1] = 2, 0
        cu, fresh = offsets(take)
        dlens.copy_(torch.tensor(now, dtype=torch.int32))
        dcu.copy_(fresh)
        eager, elens = S.kv_attention(q, cache, table, dlens, cu_tokens=dcu, return_lse=True)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(lse, elens)
        check_attention(out, lse, type("P", (), dict(vars(p), lens=now))(), q64, cu, "f16", 0.125)


def test_two_streams_at_once():
    # calls on side streams with their own data give what the calls give one after the other
    ps = [Pool(50 + i, [900 + 100 * i, 64], 2, 64, 16, wide=True) for i in range(2)]
    qs = [stored(p.rng.standard_normal((2, 1, 4, 64)), "bf16")[0] for p in ps]
    caches, args = [p.dev() for p in ps], [p.args() for p in ps]
    want = [S.kv_attention(q, c, *a) for q, c, a in zip(qs, caches, args)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in ps], [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(S.kv_attention(qs[i], caches[i], *args[i]))
    torch.cuda.synchronize()
    for w, gs in zip(want, got):
        assert all(torch.equal(w, g) for g in gs)
