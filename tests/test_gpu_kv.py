"""GPU parity of the paged 8-bit key/value cache: append (bit for bit) and
attention (against the oracle in 64 bits), alone and in a run with the
quantizers and the INT8 product.

Bound of an attention output, with P = sum_t p_t |V_t| / sum_t p_t:
* weights are rounded to fp16 (half a step: 2^-11 relative; below 2^-14 of the
  scale at which the largest weight stands at 2^8 or more, 2^-25 absolute, so
  at most len * 2^-33 of the largest |V|);
* a score is off by the fp32 sum of D exact products, at most (D + 8) 2^-24 of
  scale * sum_d |q_d K_td|, and by the fp32 steps of its exponent, 2^-20; a
  score that is off by e changes its weight by e, in numerator and sum;
* the fp32 sums over the tokens: len * 2^-23;
* the output's rounding: half a step.
A log-sum is off by a score's error, the fp32 sum and its own rounding."""
import numpy as np
import pytest

import oracle as O
import oracle.serving as V

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU, skipped there
    pytest.skip("no GPU", allow_module_level=True)

import pruning_quantization_amd as S  # noqa: E402
from gpu_util import DEV  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def stored(x, dtype):
    """x rounded to the type: a device tensor and its exact float64 values."""
    t = torch.from_numpy(np.asarray(x, np.float32)).to(DT[dtype])
    return t.to(DEV), t.to(torch.float64).numpy()


class Pool:
    """A cache in use: random codes and scales in every block, tables in any
    order, lens tokens in each sequence.  wide: tables that allow more than the
    1024 tokens up to which a call splits no sequence."""

    def __init__(self, seed, lens, kv=2, dim=64, tokens=16, fmt="int8", width=None, spare=2, wide=False):
        rng = self.rng = np.random.default_rng(seed)
        self.lens, self.fmt, self.tokens, self.kv, self.dim = list(lens), fmt, tokens, kv, dim
        need = [-(-max(n, 0) // tokens) for n in lens]
        blocks = max(1, sum(need) + spare)
        width = width or max(max(need), 1025 // tokens + 1 if wide else 1)
        order = rng.permutation(blocks).astype(np.int32)
        self.table = np.full((len(lens), width), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (blocks, kv, tokens, dim)
        if fmt == "int8":
            k, v = (np.clip(np.rint(rng.standard_normal(s) * 40), -127, 127).astype(np.int8)
                    for s in (shape, (blocks, kv, dim, tokens)))
        else:
            k, v = (O.e4m3_encode(np.clip(rng.standard_normal(s) * 120, -448, 448))
                    for s in (shape, (blocks, kv, dim, tokens)))
        self.ref = (k, (rng.random((blocks, kv)) * 0.02 + 0.01).astype(np.float32),
                    v, (rng.random((blocks, kv)) * 0.02 + 0.01).astype(np.float32))
        if fmt == "fp8":
            self.ref = (k, self.ref[1] / 3, v, self.ref[3] / 3)

    def dev(self):
        return S.KVCache(*(torch.from_numpy(x.copy()).to(DEV) for x in self.ref))

    def args(self):
        return (torch.from_numpy(self.table).to(DEV),
                torch.tensor(self.lens, dtype=torch.int32, device=DEV))


def offsets(news):
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    return cu, torch.from_numpy(cu).to(DEV)


def check_attention(got, lse, pool, q64, cu, dtype, scale, ref=None, **kw):
    out, want_lse, spread, reach = V.kv_attention(q64, ref or pool.ref, pool.table, pool.lens, cu,
                                                  pool.fmt, scale, **kw)
    n = max(max(pool.lens), 1)
    vmax = (ref or pool.ref)[3].max() * (127 if pool.fmt == "int8" else 448)
    ds = (pool.dim + 8) * 2.0 ** -24 * reach + 2.0 ** -20
    tol = (spread * (2.0 ** -11 + 2 * ds[..., None] + n * 2.0 ** -23) + n * 2.0 ** -33 * vmax
           + np.abs(out) * torch.finfo(DT[dtype]).eps / 2 + 2.0 ** -24)
    got = got.cpu().to(torch.float64).numpy().reshape(out.shape)
    err = np.abs(got - out)
    assert (err <= tol).all(), f"{(err > tol).sum()} of {err.size} outside; worst {np.nanmax(err / tol):.3g}"
    if lse is not None:
        l64 = lse.cpu().to(torch.float64).numpy().reshape(want_lse.shape)
        none = np.isneginf(want_lse)
        assert np.array_equal(none, np.isneginf(l64))
        with np.errstate(invalid="ignore"):
            bad = np.abs(l64 - want_lse) > ds + n * 2.0 ** -23 + 2.0 ** -21 * np.abs(want_lse)
        assert not bad[~none].any()


def unchanged(cache, ref):
    for t, x in zip(cache, ref):
        assert np.array_equal(t.cpu().numpy().view(np.uint8), x.view(np.uint8))


# --- append ------------------------------------------------------------------


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("dtype,dim,tokens,kv", [
    ("bf16", 128, 64, 8), ("f16", 64, 16, 3), ("f32", 192, 32, 1), ("bf16", 256, 256, 2), ("f32", 128, 128, 2)])
def test_append(fmt, dtype, dim, tokens, kv):
    # whole prompts, ends inside blocks, single tokens, nothing, one that fills its block
    news = [tokens * 2 + 5, 1, 0, 3, tokens, 1, 7, 1]
    lens = [tokens * 2 + 5, 40, 9, 3, tokens * 3, tokens, tokens + 3, tokens * 2 + 1]
    p = Pool(dim + tokens, lens, kv, dim, tokens, fmt)
    cu, dcu = offsets(news)
    # rows whose size differs from block to block, so that scales grow and stay
    size = np.exp(p.rng.normal(0.5, 1.0, (cu[-1], kv, 1)))
    k, k64 = stored(p.rng.standard_normal((cu[-1], kv, dim)) * size, dtype)
    v, v64 = stored(p.rng.standard_normal((cu[-1], kv, dim)) * size[::-1], dtype)
    cache = p.dev()
    want = V.kv_append(p.ref, k64, v64, p.table, lens, cu, fmt)
    S.kv_append(cache, k, v, *p.args(), cu_tokens=dcu)
    unchanged(cache, want)
    S.kv_append(cache, k, v, *p.args(), cu_tokens=dcu)       # again: nothing changes
    unchanged(cache, want)
    assert not np.array_equal(want[1], p.ref[1])


@pytest.mark.parametrize("n", [1, 5, 33])
def test_append_same_count_strided(n):
    # rows cut out of a fused projection [tokens, (q, k, v) heads, dim]
    lens = [n, 50, 64, n + 31, 200]
    p = Pool(n, lens, 2, 64, 32, "int8")
    fused, f64 = stored(p.rng.standard_normal((5, n, 8, 64)) * 3, "bf16")
    cu, _ = offsets([n] * 5)
    cache = p.dev()
    S.kv_append(cache, fused[:, :, 4:6], fused[:, :, 6:8], *p.args())
    f64 = f64.reshape(5 * n, 8, 64)
    unchanged(cache, V.kv_append(p.ref, f64[:, 4:6], f64[:, 6:8], p.table, lens, cu, "int8"))


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_append_token_by_token_grows_scales(fmt):
    lens, T = [0, 0, 0], 16
    p = Pool(3, [40, 40, 40], 2, 64, T, fmt)
    cache, ref = p.dev(), p.ref
    for step in range(40):
        k, k64 = stored(p.rng.standard_normal((3, 1, 2, 64)) * 1.07 ** step, "bf16")
        v, v64 = stored(p.rng.standard_normal((3, 1, 2, 64)) * 1.3 ** (step % 7), "bf16")
        lens = [step + 1] * 3
        S.kv_append(cache, k, v, p.args()[0], torch.tensor(lens, dtype=torch.int32, device=DEV))
        ref = V.kv_append(ref, k64[:, 0], v64[:, 0], p.table, lens, [0, 1, 2, 3], fmt)
    unchanged(cache, ref)


def test_append_special_values():
    p = Pool(5, [16, 20, 5, 33], 1, 64, 16, "fp8")
    x = np.zeros((4, 20, 1, 64), np.float32)
    x[0] = 2.0 ** -66                       # under the smallest scaled maximum: scale 0
    x[1, 3, 0, 5], x[1, 9] = np.nan, 1e30
    x[2] = -0.0
    x[3] = 2.0 ** -126 * np.arange(64)
    lens, cu = [16, 20, 5, 33], [0, 16, 36, 41, 61]
    rows = np.concatenate([x[0, :16], x[1], x[2, :5], x[3]])
    k, k64 = stored(rows, "f32")
    for fmt in ("fp8", "int8"):
        p = Pool(5, lens, 1, 64, 16, fmt)
        cache = p.dev()
        S.kv_append(cache, k, k, *p.args(), cu_tokens=torch.tensor(cu, dtype=torch.int32, device=DEV))
        unchanged(cache, V.kv_append(p.ref, k64, k64, p.table, lens, cu, fmt))


def test_append_stays_out_of_what_is_not_named():
    # entries outside the pool, positions past the table, more rows than tokens, spare rows
    p = Pool(8, [40, 40, 30, 5], 1, 64, 16, "int8")
    p.table[0, 1], p.table[1, 2] = -7, 10 ** 6
    p.lens = [40, 40, 100, 5]                # 100 tokens, a table of 48
    news = [40, 20, 70, 9]
    cu, dcu = offsets(news)
    k, k64 = stored(p.rng.standard_normal((cu[-1] + 6, 1, 64)), "bf16")
    cache = p.dev()
    S.kv_append(cache, k, k, *p.args(), cu_tokens=dcu)
    unchanged(cache, V.kv_append(p.ref, k64, k64, p.table, p.lens, cu, "int8"))


def test_append_many_sequences():
    rng = np.random.default_rng(11)
    lens = [int(x) for x in rng.integers(0, 60, 300)]
    news = [min(n, int(x)) for n, x in zip(lens, rng.integers(0, 4, 300))]
    p = Pool(12, lens, 1, 64, 16, "int8")
    cu, dcu = offsets(news)
    k, k64 = stored(p.rng.standard_normal((cu[-1], 1, 64)) * 2, "f16")
    v, v64 = stored(p.rng.standard_normal((cu[-1], 1, 64)) * 2, "f16")
    cache = p.dev()
    S.kv_append(cache, k, v, *p.args(), cu_tokens=dcu)
    unchanged(cache, V.kv_append(p.ref, k64, v64, p.table, lens, cu, "int8"))


# --- attention ----------------------------------------------------------------


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,tokens,kv,group", [
    (64, 16, 2, 1), (128, 64, 2, 4), (128, 32, 1, 5), (192, 128, 1, 3), (256, 256, 1, 2), (256, 16, 2, 16),
    (64, 64, 1, 48), (128, 256, 1, 71)])
def test_decode(dim, tokens, kv, group, dtype, fmt, wide):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 129, 511, 700]
    p = Pool(dim + group, lens, kv, dim, tokens, fmt, wide=wide)
    q, q64 = stored(p.rng.standard_normal((len(lens), 1, kv * group, dim)), dtype)
    cu = np.arange(len(lens) + 1)
    out, lse = S.kv_attention(q, p.dev(), *p.args(), return_lse=True)
    assert out.shape == q.shape and lse.shape == q.shape[:-1]
    check_attention(out, lse, p, q64[:, 0], cu, dtype, dim ** -0.5)
    assert torch.equal(out, S.kv_attention(q, p.dev(), *p.args()))          # the same bits without lse


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("kw", [{}, {"window": 1}, {"window": 37}, {"window": 200}, {"causal": False}])
@pytest.mark.parametrize("dim,tokens,group,fmt", [(64, 16, 4, "fp8"), (128, 64, 3, "int8"), (256, 32, 1, "fp8"),
                                                  (192, 64, 2, "int8")])
def test_chunks(dim, tokens, group, fmt, kw, wide):
    # whole prompts, chunks behind a context, decoding, nothing, in one call
    lens = [130, 400, 77, 9, 64, 300, 1]
    news = [130, 90, 1, 0, 64, 2, 1]
    p = Pool(dim, lens, 2, dim, tokens, fmt, wide=wide)
    cu, dcu = offsets(news)
    q, q64 = stored(p.rng.standard_normal((cu[-1], 2 * group, dim)) * 1.5, "bf16")
    out, lse = S.kv_attention(q, p.dev(), *p.args(), cu_tokens=dcu, return_lse=True, scale=0.11, **kw)
    check_attention(out, lse, p, q64, cu, "bf16", np.float32(0.11), **kw)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("n", [2, 16, 70, 257])
@pytest.mark.parametrize("dtype,fmt", [("bf16", "int8"), ("f16", "fp8")])
def test_same_count_strided(n, dtype, fmt, wide):
    # queries cut out of a fused projection; n tokens of each sequence
    lens = [n, n + 1, n + 300]
    p = Pool(n, lens, 2, 128, 64, fmt, wide=wide)
    fused, f64 = stored(p.rng.standard_normal((3, n, 12, 128)), dtype)
    cu = np.arange(4) * n
    out = S.kv_attention(fused[:, :, :8], p.dev(), *p.args())
    check_attention(out, None, p, f64.reshape(3 * n, 12, 128)[:, :8], cu, dtype, 128 ** -0.5)


@pytest.mark.parametrize("seqs,dim,n", [(9, 128, 270), (13, 64, 270)])
def test_prompts_of_the_same_count(seqs, dim, n):
    # two row tiles a CU (three, one), all resident at once: the second from the shortest up
    p = Pool(seqs, [n + (7 * i) % 30 for i in range(seqs)], 8, dim, 32, "fp8")
    q, q64 = stored(p.rng.standard_normal((seqs, n, 16, dim)), "bf16")
    out, lse = S.kv_attention(q, p.dev(), *p.args(), return_lse=True)
    check_attention(out, lse, p, q64.reshape(seqs * n, 16, dim), np.arange(seqs + 1) * n, "bf16", dim ** -0.5)


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_split_along_the_tokens(fmt):
    # far more tiles than one workgroup takes; a width that allows much more
    p = Pool(21, [6001, 40, 0, 1500], 1, 64, 32, fmt, width=400)
    q, q64 = stored(p.rng.standard_normal((4, 1, 3, 64)), "f16")
    out, lse = S.kv_attention(q, p.dev(), *p.args(), return_lse=True)
    check_attention(out, lse, p, q64[:, 0], np.arange(5), "f16", 0.125)
    assert not out[2].any()


@pytest.mark.parametrize("wide", [False, True])
def test_rows_that_see_nothing(wide):
    p = Pool(4, [0, 3, 50, 40], 1, 64, 16, "int8", wide=wide)
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
@pytest.mark.parametrize("tokens", [16, 64, 128])
def test_garbage_in_unseen_places(tokens, wide):
    # NaN codes behind the sequences, before the windows and in foreign blocks; NaN and
    # infinite scales in blocks that no row sees
    lens = [tokens + 3, 5, 200, 3 * tokens]
    p = Pool(tokens, lens, 2, 64, tokens, "fp8", spare=4, wide=wide)
    q, q64 = stored(p.rng.standard_normal((4, 2, 4, 64)), "bf16")
    cu = np.arange(5) * 2
    for window in (0, 30):
        want = [x.copy() for x in p.ref]
        dirty = [x.copy() for x in p.ref]
        seen = np.zeros((p.ref[0].shape[0], tokens), bool)
        for b, n in enumerate(lens):
            for pos in range(max(0, n - 2 - window + 1) if window else 0, n):
                seen[p.table[b, pos // tokens], pos % tokens] = True
        dirty[0][np.broadcast_to(~seen[:, None, :, None], dirty[0].shape)] = 0x7F
        dirty[2][np.broadcast_to(~seen[:, None, None, :], dirty[2].shape)] = 0xFF
        none = ~seen.any(1)
        dirty[1][none], dirty[3][none] = np.nan, np.inf
        cache = S.KVCache(*(torch.from_numpy(x).to(DEV) for x in dirty))
        out, lse = S.kv_attention(q, cache, *p.args(), return_lse=True, window=window)
        check_attention(out, lse, p, q64.reshape(8, 4, 64), cu, "bf16", 0.125, ref=tuple(want), window=window)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_scales_far_apart(fmt, wide):
    # block scales over 40 binades and zeros, queries over many more
    lens = [500, 64, 300]
    p = Pool(31, lens, 2, 64, 16, fmt, wide=wide)
    k, ks, v, vs = (x.copy() for x in p.ref)
    vs *= np.exp2(p.rng.integers(-40, 1, vs.shape)).astype(np.float32)
    ks *= np.exp2(p.rng.integers(-20, 1, ks.shape)).astype(np.float32)
    zero = p.rng.random(vs.shape) < 0.2
    v[zero], vs[zero] = 0, 0
    zero = p.rng.random(ks.shape) < 0.2
    k[zero], ks[zero] = 0, 0
    p.ref = (k, ks, v, vs)
    q = p.rng.standard_normal((3, 1, 4, 64)) * np.exp2(p.rng.integers(-3, 3, (3, 1, 4, 1)))
    q[0, 0, 1] = 0
    q[1, 0, 0] *= 2.0 ** -9
    q, q64 = stored(q, "f16")
    out, lse = S.kv_attention(q, p.dev(), *p.args(), return_lse=True)
    check_attention(out, lse, p, q64[:, 0], np.arange(4), "f16", 0.125)
    # all values zero with zero scales: zeros
    p.ref = (k, ks, np.zeros_like(v), np.zeros_like(vs))
    out, lse = S.kv_attention(q, p.dev(), *p.args(), return_lse=True)
    assert not out.any()
    check_attention(out, lse, p, q64[:, 0], np.arange(4), "f16", 0.125)


@pytest.mark.parametrize("wide", [False, True])
def test_extreme_queries(wide):
    # bf16 rows at both ends of the range, peaked and flat weights
    p = Pool(41, [300, 300, 300, 300], 1, 128, 64, "int8", wide=wide)
    q = p.rng.standard_normal((4, 1, 2, 128))
    q[0] *= 1e30
    q[1] *= 1e-30
    q[2] *= 50
    q[3, :, :, 1:] *= 1e-6
    dq, q64 = stored(q, "bf16")
    cu = np.arange(5)
    out, lse = S.kv_attention(dq, p.dev(), *p.args(), return_lse=True, scale=0.1)
    # of the first the largest score takes all; its bound on scores is vast, so look at the value itself
    o, _, _, _ = V.kv_attention(q64[:, 0], p.ref, p.table, p.lens, cu, "int8", np.float32(0.1))
    assert np.allclose(out[0, 0].cpu().float().numpy(), o[0], rtol=2.0 ** -8, atol=1e-6)
    check_attention(out[1:], lse[1:], _rest(p, 1), q64[1:, 0], cu[:4], "bf16", np.float32(0.1))
    dq[2, 0, 1, 7] = float("nan")
    out2 = S.kv_attention(dq, p.dev(), *p.args(), scale=0.1)
    assert out2[2, 0, 1].isnan().all()
    out2[2, 0, 1] = out[2, 0, 1]
    assert torch.equal(out, out2), "a NaN query reached other rows"


def _rest(p, n):
    r = Pool.__new__(Pool)
    r.__dict__.update(p.__dict__)
    r.table, r.lens = p.table[n:], p.lens[n:]
    return r


def test_rows_of_no_sequence_stay():
    p = Pool(2, [20, 70], 1, 64, 16, "int8")
    cu, dcu = offsets([1, 3])
    q, q64 = stored(p.rng.standard_normal((9, 2, 64)), "bf16")
    out = torch.full((9, 2, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((9, 2), 3.0, device=DEV)
    S.kv_attention(q, p.dev(), *p.args(), cu_tokens=dcu, out=out, lse=lse)
    check_attention(out[:4], lse[:4], p, q64[:4], cu, "bf16", 0.125)
    assert (out[4:] == 3).all() and (lse[4:] == 3).all()


def test_many_sequences():
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 150, 333)]
    news = [min(max(n, 1), int(x)) for n, x in zip(lens, rng.integers(0, 3, 333))]
    p = Pool(6, lens, 1, 64, 16, "fp8", width=40)
    cu, dcu = offsets(news)
    q, q64 = stored(rng.standard_normal((cu[-1], 2, 64)), "bf16")
    out, lse = S.kv_attention(q, p.dev(), *p.args(), cu_tokens=dcu, return_lse=True)
    check_attention(out, lse, p, q64, cu, "bf16", 0.125)


@pytest.mark.parametrize("uniform", [False, True])
@pytest.mark.parametrize("count,kv", [(66, 1), (129, 1), (300, 2)])
def test_many_sequences_some_split(count, kv, uniform):
    # more sequences than a workgroup adds up by itself, a few of them split; 600 sequences and heads fill
    # the card, so their chunks are longer
    rng = np.random.default_rng(count + uniform)
    lens = [int(x) for x in rng.integers(1, 90, count)]
    for b, n in ((0, 2500), (count // 2, 1100), (count - 1, 1700)):
        lens[b] = n
    p = Pool(count, lens, kv, 64, 16, "int8")
    news = [1] * count if uniform else [min(n, int(x)) for n, x in zip(lens, rng.integers(0, 3, count))]
    if not uniform:
        news[3], news[count - 1] = min(lens[3], 40), 200                 # the second: prompt rows
    cu, dcu = offsets(news)
    q, q64 = stored(rng.standard_normal((cu[-1], 2 * kv, 64)), "f16")
    x, kw = (q[:, None], {}) if uniform else (q, {"cu_tokens": dcu})
    out, lse = S.kv_attention(x, p.dev(), *p.args(), return_lse=True, **kw)
    check_attention(out, lse, p, q64, cu, "f16", 0.125)


@pytest.mark.parametrize("uniform", [False, True])
def test_append_to_thousands(uniform):
    rng = np.random.default_rng(13)
    lens = [int(x) for x in rng.integers(2, 40, 4200)]
    news = [2] * 4200 if uniform else [min(n, int(x)) for n, x in zip(lens, rng.integers(0, 4, 4200))]
    p = Pool(14, lens, 1, 64, 16, "int8")
    cu, dcu = offsets(news)
    k, k64 = stored(p.rng.standard_normal((cu[-1], 1, 64)) * 2, "bf16")
    cache = p.dev()
    if uniform:
        S.kv_append(cache, k.view(4200, 2, 1, 64), k.view(4200, 2, 1, 64), *p.args())
    else:
        S.kv_append(cache, k, k, *p.args(), cu_tokens=dcu)
    unchanged(cache, V.kv_append(p.ref, k64, k64, p.table, lens, cu, "int8"))


def test_offsets_past_32_bits():
    # a pool of more than 2^31 (and K more than 2^32) code bytes; the last blocks are used
    blocks, kv, T, D = 65 * 1024 + 8, 4, 64, 256
    k = torch.zeros(blocks, kv, T, D, dtype=torch.int8, device=DEV)
    v = torch.zeros(blocks, kv, D, T, dtype=torch.int8, device=DEV)
    assert k.numel() > 2 ** 32
    ks, vs = (torch.zeros(blocks, kv, device=DEV) for _ in range(2))
    cache = S.KVCache(k, ks, v, vs)
    rng = np.random.default_rng(2)
    table = np.array([[blocks - 1, blocks - 3]], np.int32)
    rows, r64 = stored(rng.standard_normal((1, 100, kv, D)), "bf16")
    args = torch.from_numpy(table).to(DEV), torch.tensor([100], dtype=torch.int32, device=DEV)
    S.kv_append(cache, rows, rows, *args)
    small = tuple(np.zeros(s, t) for s, t in (((3, kv, T, D), np.int8), ((3, kv), np.float32),
                                              ((3, kv, D, T), np.int8), ((3, kv), np.float32)))
    want = V.kv_append(small, r64[0], r64[0], np.array([[2, 0]]), [100], [0, 100], "int8")
    for t, x in zip(cache, want):
        assert np.array_equal(t[blocks - 3:].cpu().numpy(), x)
        assert not t[:blocks - 3].any()
    q, q64 = stored(rng.standard_normal((1, 1, 8, D)), "bf16")
    out = S.kv_attention(q, cache, *args)
    o, _, spread, _ = V.kv_attention(q64[0], want, np.array([[2, 0]]), [100], [0, 1], "int8", D ** -0.5)
    assert (np.abs(out[0].cpu().double().numpy() - o) <= spread * 2.0 ** -10 + np.abs(o) * 2.0 ** -8).all()


def test_refusals():
    p = Pool(2, [20, 70], 2, 64, 16, "int8")
    c, (table, lens) = p.dev(), p.args()
    q = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16, device=DEV)
    for bad in (lambda: S.kv_attention(q, c, table, lens, out=torch.empty(2, 4, 64, device=DEV)),
                lambda: S.kv_attention(q, c, table.cpu(), lens),
                lambda: S.kv_attention(q, c, table, lens, lse=torch.empty(2, 4, device=DEV)),
                lambda: S.kv_append(c, q[:, :, :2], q[:, :, :1], table, lens)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: S.kv_attention(q.float(), c, table, lens), lambda: S.kv_attention(q[:, :, :3], c, table, lens),
                lambda: S.kv_attention(q, c, table, lens, scale=-1.0),
                lambda: S.kv_attention(q, c, table, lens, causal=False, window=4),
                lambda: S.kv_append(c, q, q, table, lens)):
        with pytest.raises(S.Sparq24Error):
            bad()


# --- together -------------------------------------------------------------------


def layer(x, w, wo, cache, table, lens, cu, heads, kv, dim, ws=None):
    """One attention layer of a serving step on 8-bit operands."""
    cx, sx = S.quantize(x, ("int", 8))
    y = S.int8_gemm(cx, sx, *w, dtype=torch.bfloat16).view(-1, heads + 2 * kv, dim)
    q, k, v = y[:, :heads], y[:, heads:heads + kv], y[:, heads + kv:]
    S.kv_append(cache, k, v, table, lens, cu_tokens=cu)
    o = S.kv_attention(q, cache, table, lens, cu_tokens=cu, workspace=ws)
    co, so = S.quantize(o.view(-1, heads * dim), ("int", 8))
    return y, o, S.int8_gemm(co, so, *wo)


def test_a_serving_step():
    rng = np.random.default_rng(17)
    heads, kv, dim, hidden, T = 8, 2, 64, 256, 16
    p = Pool(18, [90, 33, 70], kv, dim, T, "fp8", width=8)
    news = [90, 1, 5]
    cu, dcu = offsets(news)
    x, _ = stored(rng.standard_normal((cu[-1], hidden)), "bf16")
    w, _ = stored(rng.standard_normal(((heads + 2 * kv) * dim, hidden)) * 0.05, "bf16")
    wo, _ = stored(rng.standard_normal((hidden, heads * dim)) * 0.05, "bf16")
    w8, wo8 = S.quantize(w, ("int", 8)), S.quantize(wo, ("int", 8))
    cache = p.dev()
    y, o, z = layer(x, w8, wo8, cache, *p.args(), dcu, heads, kv, dim)
    # each stage against the oracle on what the stage before gave
    raw = lambda t: t.cpu().view(torch.int16).numpy().view(np.uint16)  # noqa: E731
    q8 = O.QSpec("int", 8)
    cx, sx = O.quantize_rows(raw(x), "bf16", q8)
    cw, sw = O.quantize_rows(raw(w), "bf16", q8)
    want = torch.from_numpy(V.int8_gemm(cx, sx, cw, sw)).to(torch.bfloat16)
    assert torch.equal(y.cpu().view(want.shape), want)
    y64 = y.cpu().double().numpy()
    ref = V.kv_append(p.ref, y64[:, heads:heads + kv], y64[:, heads + kv:], p.table, p.lens, cu, "fp8")
    unchanged(cache, ref)
    check_attention(o, None, p, y64[:, :heads], cu, "bf16", dim ** -0.5, ref=ref)
    co, so = O.quantize_rows(raw(o.reshape(-1, heads * dim)), "bf16", q8)
    cwo, swo = O.quantize_rows(raw(wo), "bf16", q8)
    assert np.array_equal(z.cpu().numpy(), V.int8_gemm(co, so, cwo, swo))


def test_captured_steps_replay():
    # two captured decode steps that share nothing but the cache, replayed with other inputs,
    # eager work and synchronizations in between; workspaces of their own
    rng = np.random.default_rng(19)
    heads, kv, dim, hidden, T = 4, 2, 64, 128, 16
    p = Pool(20, [700, 30, 5], kv, dim, T, "int8", width=80)
    mk = lambda *s: stored(rng.standard_normal(s) * 0.1, "bf16")[0]  # noqa: E731
    w8, wo8 = S.quantize(mk((heads + 2 * kv) * dim, hidden), ("int", 8)), S.quantize(mk(hidden, heads * dim), ("int", 8))
    x = mk(3, hidden)
    table, lens = p.args()
    dcu = torch.arange(4, dtype=torch.int32, device=DEV)
    cache = p.dev()
    ws = [torch.empty(8 << 20, dtype=torch.uint8, device=DEV) for _ in range(2)]
    layer(x, w8, wo8, cache, table, lens, dcu, heads, kv, dim, ws[0])     # warm
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer(x, w8, wo8, cache, table, lens, dcu, heads, kv, dim, ws[i]))
        graphs.append(g)
    for step in range(5):
        x.copy_(mk(3, hidden))
        lens += 1
        eager = S.KVCache(*(t.clone() for t in cache))
        want = [t.clone() for t in layer(x, w8, wo8, eager, table, lens, dcu, heads, kv, dim)]
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
    p = Pool(24, lens, 1, 64, 16, "int8")
    table, dlens = p.args()
    news = np.ones(count, int)
    cu, dcu = offsets(news)
    q, q64 = stored(rng.standard_normal((count, 2, 64)), "f16")
    k, _ = stored(rng.standard_normal((count, 1, 64)), "f16")
    cache, other = p.dev(), p.dev()
    S.kv_append(other, k, k, table, dlens, cu_tokens=dcu)                # warm
    S.kv_attention(q, cache, table, dlens, cu_tokens=dcu)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        S.kv_append(other, k, k, table, dlens, cu_tokens=dcu)
        out, lse = S.kv_attention(q, cache, table, dlens, cu_tokens=dcu, return_lse=True)
    for step in range(4):
        now = [max(1, n - 13 * step * (b % 3)) for b, n in enumerate(lens)]
        take = np.ones(count, int)
        take[3 * step], take[3 * step + 1] = 2, 0
        cu, fresh = offsets(take)
        dlens.copy_(torch.tensor(now, dtype=torch.int32))
        dcu.copy_(fresh)
        for a, b in zip(other, p.dev()):
            a.copy_(b)
        want = p.dev()
        S.kv_append(want, k, k, table, dlens, cu_tokens=dcu)
        eager, elens = S.kv_attention(q, cache, table, dlens, cu_tokens=dcu, return_lse=True)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(lse, elens)
        for a, b in zip(other, want):
            assert torch.equal(a, b)
        check_attention(out, lse, type("P", (), dict(vars(p), lens=now))(), q64, cu, "f16", 0.125)


def test_two_streams_at_once():
    # calls on side streams with their own data give what the calls give one after the other
    ps = [Pool(50 + i, [900 + 100 * i, 64], 2, 64, 16, "int8", wide=True) for i in range(2)]
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
