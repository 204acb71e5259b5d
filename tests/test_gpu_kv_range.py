"""The cache's calls at the ends of their numbers' ranges."""
import numpy as np
import pytest

import oracle.serving as V

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU, skipped there
    pytest.skip("no GPU", allow_module_level=True)

import pruning_quantization_amd as S  # noqa: E402
from gpu_util import DEV  # noqa: E402
from kv_check import bounds, check_attention  # noqa: E402
from test_gpu_kv import Pool, offsets, stored, unchanged  # noqa: E402

I32 = dict(dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("wide", [False, True])
def test_scores_of_any_size_leave_single_tokens_whole(n, wide):
    # one visible token gives its value whatever its score is, here from 2^10 to 2^40, where the step of a
    # score passes the distance between a reference and the largest weight: out = V, a whole number up to 64
    # off by fp16's 2^-11 of it at most, which bf16 rounds back
    heads, dim = 64, 64
    k = torch.zeros(2, 1, 16, dim, dtype=torch.int8, device=DEV)
    v = torch.zeros(2, 1, dim, 16, dtype=torch.int8, device=DEV)
    k[..., 0] = 1
    v[1, 0, :, 0] = torch.arange(1, dim + 1, device=DEV)
    one = torch.ones(2, 1, device=DEV)
    q = torch.zeros(1, n, heads, dim, dtype=torch.bfloat16, device=DEV)
    rng = np.random.default_rng(n)
    size = 2.0 ** np.linspace(10, 40, n * heads) * rng.uniform(1, 2, n * heads)
    q[..., 0] = torch.from_numpy(size).to(DEV).view(1, n, heads)
    table = torch.full((1, 80 if wide else 1), -1, **I32)
    table[0, 0] = 1
    lens = torch.tensor([1], **I32)
    out = S.kv_attention(q, S.KVCache(k, one, v, one), table, lens, scale=1.0, causal=False)
    bad = (out != v[1, 0, :, 0]).any(-1).flatten().cpu().numpy()
    assert not bad.any(), f"wrong at log2 q = {np.log2(size[bad])}"


# exponents of the V scales, dealt to runs of blocks in order; None: a scale of zero over codes of zero
FAR = [(None, 0), (None, 46), (None, 48), (None, 100), (48, None), (100, None), (-70, 60), (60, -70),
       (None, -70, 0, 100), (100, 0, -70, None)]


@pytest.mark.parametrize("far", FAR, ids=str)
@pytest.mark.parametrize("place", ["wave", "waves", "chunks", "prompt", "long prompt"])
@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_v_scales_over_the_whole_range(fmt, place, far):
    # the softmax does not know the V scales: a block of small or no values counts in the sum beside one whose
    # values are up to 2^170 times larger, in a wave, across the waves and chunks, and in the prompt kernel
    lens, news, wide = {"wave": ([64, 40], [1, 1], False), "waves": ([700, 300], [1, 2], False),
                        "chunks": ([2600, 300], [1, 1], True), "prompt": ([150, 90], [90, 20], False),
                        "long prompt": ([1500, 200], [30, 40], True)}[place]
    p = Pool(len(far), lens, 1, 64, 16, fmt, wide=wide)
    k, ks, v, vs = (x.copy() for x in p.ref)
    for row, n in zip(p.table, lens):
        blocks = row[:-(-n // 16)]
        for i, blk in enumerate(blocks):
            e = far[i * len(far) // len(blocks)]
            vs[blk] = 0 if e is None else np.exp2(e + p.rng.random())
            if e is None:
                v[blk] = 0
    p.ref = (k, ks, v, vs)
    cu, dcu = offsets(news)
    q, q64 = stored(p.rng.standard_normal((cu[-1], 4, 64)), "bf16")
    out, lse = S.kv_attention(q, p.dev(), *p.args(), cu_tokens=dcu, return_lse=True)
    check_attention(out, lse, p.ref, p.table, lens, cu, q64, fmt, 0.125, 2.0 ** -8, bits=8)


def rows_apart(out, lse, sees, p, ref, cu, q64, fmt, **kw):
    """Rows that see what is not a number are NaN throughout, the others as if it were not there."""
    sees = np.asarray(sees)
    o, l = out.cpu().double().numpy().reshape(len(sees), -1), lse.cpu().double().numpy().reshape(len(sees), -1)
    assert np.isnan(o[sees]).all() and np.isnan(l[sees]).all()
    clean = torch.from_numpy(np.where(sees[:, None], 0, o)).view(out.shape)
    want = [x.copy() for x in ref]
    q64 = q64.copy()
    o64, l64, spread, reach = V.kv_attention(q64, want, p.table, p.lens, cu, fmt, 0.125, **kw)
    tol, own = bounds(want, p.lens, fmt, q64.shape[-1], spread, reach, o64, 2.0 ** -8)
    assert (np.abs(clean.numpy().reshape(o64.shape) - o64) <= tol)[~sees].all()
    assert (np.abs(l.reshape(l64.shape) - l64) <= own + 2.0 ** -21 * np.abs(l64))[~sees].all()


# first query position, queries, window: a decoding step's rows, a prompt's, a window that has left the block
SEEING = [(78, 4, 0), (40, 70, 0), (70, 60, 10)]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("first,n,window", SEEING)
@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("what", [np.inf, np.nan])
@pytest.mark.parametrize("tokens,fmt", [(16, "int8"), (16, "fp8"), (64, "int8"), (64, "fp8")])
def test_scales_that_are_no_numbers_stay_with_rows_that_see_them(tokens, fmt, what, side, first, n, window, wide):
    p = Pool(n, [first + n], 1, 64, tokens, fmt, wide=wide)
    page = 80 // tokens                        # positions 80 .. 95, or 64 .. 127
    q, q64 = stored(p.rng.standard_normal((n, 4, 64)), "bf16")
    ref = [x.copy() for x in p.ref]
    blk = p.table[0, page]
    p.ref[0][blk], p.ref[2][blk] = 0, 0        # as an append leaves such a block
    p.ref[1 if side == "k" else 3][blk] = what
    pos = np.arange(first, first + n)
    sees = pos >= page * tokens
    if window:
        sees &= pos - window + 1 < (page + 1) * tokens
    assert sees.any() and not (sees.all() and tokens == 16)
    out, lse = S.kv_attention(q[None], p.dev(), *p.args(), return_lse=True, window=window)
    ref[0][blk], ref[2][blk] = 0, 0
    rows_apart(out, lse, sees, p, ref, [0, n], q64, fmt, window=window)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("first,n,window", SEEING)
@pytest.mark.parametrize("dim,tokens", [(64, 16), (64, 64), (128, 16), (128, 128), (192, 32), (192, 64), (256, 16),
                                        (256, 256)])
def test_nan_codes_stay_with_rows_that_see_them(dim, tokens, first, n, window, wide):
    # e4m3 NaN codes of values at two positions, in some dims each: those dims of the rows that see them are NaN,
    # the rest is as without them; of a key's at a third: the rows that see it are NaN throughout
    p = Pool(n + dim, [first + n], 1, dim, tokens, "fp8", wide=wide)
    q, q64 = stored(p.rng.standard_normal((n, 4, dim)), "bf16")
    ref = [x.copy() for x in p.ref]
    pos = np.arange(first, first + n)
    sees = lambda at: (pos >= at) & (pos < at + window if window else True)  # noqa: E731
    nan = np.zeros((n, dim), bool)
    last = first + n - 1
    for at, dims in ((80, [3, 17, dim - 1]), (last - 1, [0, 17, 40])):
        blk = p.table[0, at // tokens]
        ref[2][blk, 0, dims, at % tokens] = 0
        p.ref[2][blk, 0, dims, at % tokens] = [0x7F, 0xFF, 0x7F]
        nan[np.ix_(sees(at), dims)] = True
    p.ref[0][p.table[0, last // tokens], 0, last % tokens, 5] = 0xFF
    out, lse = S.kv_attention(q[None], p.dev(), *p.args(), return_lse=True, window=window)
    o, l = out.cpu().double().numpy().reshape(n, 4, dim), lse.cpu().double().numpy().reshape(n, 4)
    assert np.isnan(o[-1]).all() and np.isnan(l[-1]).all()
    o, l, nan = o[:-1], l[:-1], np.broadcast_to(nan[:-1, None], (n - 1, 4, dim))
    assert np.array_equal(np.isnan(o), nan)
    want, want_lse, spread, reach = V.kv_attention(q64, ref, p.table, p.lens, [0, n], "fp8", dim ** -0.5,
                                                   window=window)
    tol, own = bounds(ref, p.lens, "fp8", dim, spread, reach, want, 2.0 ** -8)
    assert (np.abs(o - want[:-1]) <= tol[:-1])[~nan].all()
    assert (np.abs(l - want_lse[:-1]) <= (own + 2.0 ** -21 * np.abs(want_lse))[:-1]).all()


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("dtype,dim,tokens", [("bf16", 64, 16), ("f16", 128, 64), ("f32", 64, 256), ("f32", 256, 128)])
def test_append_of_infinities(dtype, dim, tokens, fmt):
    # single infinities, rows and blocks of them, next to kept tokens and alone; blocks whose rows a workgroup
    # holds and larger ones
    lens, news = [2 * tokens + 5, tokens + 3, 7, tokens], [tokens + 9, 3, 7, 5]
    p = Pool(tokens + dim, lens, 2, dim, tokens, fmt)
    cu, dcu = offsets(news)
    rows = [p.rng.standard_normal((cu[-1], 2, dim)) * 3 for _ in range(2)]
    for x in rows:
        x[3, 0, 5], x[3, 1, 7], x[cu[1], :, :2], x[cu[1] + 1, 0] = np.inf, -np.inf, np.nan, -np.inf
        x[cu[2]:cu[3], 1] = np.inf
        x[cu[3]:, 0] = -np.inf
        x[tokens // 2, 1, ::3] = np.inf
    (k, k64), (v, v64) = (stored(x, dtype) for x in rows)
    cache = p.dev()
    S.kv_append(cache, k, v, *p.args(), cu_tokens=dcu)
    want = V.kv_append(p.ref, k64, v64, p.table, lens, cu, fmt)
    assert all(np.isfinite(x).all() for x in (want[1], want[3]))
    unchanged(cache, want)


def test_an_empty_workspace():
    # enough where a call needs none, refused where it needs one: never outputs that nothing wrote
    p = Pool(3, [20, 70], 1, 64, 16, "int8")
    q, _ = stored(p.rng.standard_normal((2, 1, 2, 64)), "bf16")
    want = S.kv_attention(q, p.dev(), *p.args())
    for empty in (torch.empty(0, dtype=torch.uint8, device=DEV), torch.empty(0, 4, device=DEV)):
        out = torch.full_like(q, 7.0)
        S.kv_attention(q, p.dev(), *p.args(), out=out, workspace=empty)
        assert torch.equal(out, want)
        p_wide = Pool(3, [20, 70], 1, 64, 16, "int8", wide=True)
        out = torch.full_like(q, 7.0)
        with pytest.raises(S.Sparq24Error, match="workspace"):
            S.kv_attention(q, p_wide.dev(), *p_wide.args(), out=out, workspace=empty)
        assert (out == 7).all()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("n", [1, 30])
@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_infinite_queries(fmt, n, wide):
    # every score is infinite or NaN: a row that sees a token is NaN whatever the signs, one that sees none gives
    # zeros, others are as they were
    p = Pool(n, [70, 70, 0], 1, 64, 16, fmt, wide=wide)
    p.ref[0][..., 3] = 1 if fmt == "int8" else 0x38          # keys of one sign along a dim
    q, _ = stored(p.rng.standard_normal((3, n, 4, 64)), "bf16")
    want, want_lse = S.kv_attention(q, p.dev(), *p.args(), return_lse=True)
    q[0, 0, 0, 3], q[0, 0, 1, 3], q[1, n - 1, 2, 9], q[2, 0, 0, 3] = -np.inf, np.inf, np.inf, -np.inf
    out, lse = S.kv_attention(q, p.dev(), *p.args(), return_lse=True)
    for b, i, h in ((0, 0, 0), (0, 0, 1), (1, n - 1, 2)):
        assert out[b, i, h].isnan().all() and lse[b, i, h].isnan()
        out[b, i, h], lse[b, i, h] = want[b, i, h], want_lse[b, i, h]
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert not out[2].any() and torch.isneginf(lse[2]).all()


def test_thousands_of_sequences():
    # more than the work list's workgroup has threads: each adds up several sequences
    rng = np.random.default_rng(3)
    count = 2500
    lens = [int(x) for x in rng.integers(0, 40, count)]
    news = [min(n, int(x)) for n, x in zip(lens, rng.integers(0, 3, count))]
    for b, n, w in ((0, 1500, 1), (1024, 1300, 2), (1301, 60, 30), (2499, 2000, 1)):
        lens[b], news[b] = n, w
    p = Pool(4, lens, 1, 64, 16, "int8")
    cu, dcu = offsets(news)
    q, q64 = stored(rng.standard_normal((cu[-1], 2, 64)), "bf16")
    out, lse = S.kv_attention(q, p.dev(), *p.args(), cu_tokens=dcu, return_lse=True)
    check_attention(out, lse, p.ref, p.table, lens, cu, q64, "int8", 0.125, 2.0 ** -8, bits=4)
    q, q64 = stored(rng.standard_normal((count, 1, 2, 64)), "bf16")
    out, lse = S.kv_attention(q, p.dev(), *p.args(), return_lse=True)
    check_attention(out, lse, p.ref, p.table, lens, np.arange(count + 1), q64[:, 0], "int8", 0.125, 2.0 ** -8, bits=4)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_the_largest_weight_is_exact(fmt, wide, n):
    # a row's largest weight is a power of two in fp16, so a softmax that one token has gives its value to the
    # output's own rounding: fp16's half step, and the exponent's 2^(4 - 22) in the sum, twice
    p = Pool(n, [1, 1, 1, 1], 4, 64, 16, fmt, wide=wide)
    q, _ = stored(p.rng.standard_normal((4, n, 32, 64)), "f16")
    out = S.kv_attention(q, p.dev(), *p.args(), causal=False).cpu().double().numpy()
    for b in range(4):
        blk = p.table[b, 0]
        v = V.kv_decode(p.ref[2][blk, :, :, 0], fmt) * p.ref[3][blk].astype(np.float64)[:, None]
        want = np.repeat(v, 8, 0)
        assert (np.abs(out[b] - want) <= np.abs(want) * (2.0 ** -11 + 2.0 ** -17) + 2.0 ** -25).all()
