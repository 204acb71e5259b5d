"""CPU pins of the INT8 product, cache append and cache attention oracles, and
the host-side refusals of the three C entry points."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

import oracle.serving as V

B = pytest.importorskip("pruning_quantization_amd.binding")

FAKE = 0x7F0000000000          # 16-byte aligned, never dereferenced on the host
OK, INVALID, UNSUPPORTED, SHAPE, ALIGN, WORKSPACE, DEVICE = 0, 1, 2, 3, 4, 5, 6


# --- oracles ---------------------------------------------------------------


def test_int8_gemm_by_hand():
    a = np.array([[1, -2, 3, 127] + [0] * 12], dtype=np.int8)
    b = np.array([[4, 5, -6, 127] + [0] * 12, [-128] * 16], dtype=np.int8)
    y = V.int8_gemm(a, np.float32([0.5]), b, np.float32([2.0, 0.25]), np.float32([1.0, -1.0]))
    # 4 - 10 - 18 + 16129 = 16105; -128 * 129 = -16512
    assert y.tolist() == [[16105.0 + 1.0, -16512 * 0.125 - 1.0]]


def test_append_by_hand():
    # one head, T = 16, D = 64: two tokens, then a third that doubles the maximum
    cache = (np.full((2, 1, 16, 64), 9, np.int8), np.full((2, 1), 7, np.float32),
             np.full((2, 1, 64, 16), 9, np.int8), np.full((2, 1), 7, np.float32))
    table = np.array([[1]], np.int32)
    x = np.zeros((2, 1, 64), np.float32)
    x[0, 0, :3] = (127.0, 63.0, -1.0)
    x[1, 0, 0] = 2.5                                   # tie: rounds to the even code
    k, ks, v, vs = V.kv_append(cache, x, x, table, [2], [0, 2], "int8")
    assert ks[1, 0] == 1.0 and ks[0, 0] == 7.0
    assert k[1, 0, :3, :4].tolist() == [[127, 63, -1, 0], [2, 0, 0, 0], [9, 9, 9, 9]]
    assert v[1, 0, :4, :3].tolist() == [[127, 2, 9], [63, 0, 9], [-1, 0, 9], [0, 0, 9]]
    y = np.zeros((1, 1, 64), np.float32)
    y[0, 0, 5] = -254.0
    k, ks, v, vs = V.kv_append((k, ks, v, vs), y, y, table, [3], [0, 1], "int8")
    assert ks[1, 0] == 2.0
    # 127 / 2 = 63.5 -> 64, 63 / 2 = 31.5 -> 32, -1 / 2 -> 0 (ties to even), 2 / 2 = 1
    assert k[1, 0, :3, :4].tolist() == [[64, 32, 0, 0], [1, 0, 0, 0], [0, 0, 0, 0]]
    assert k[1, 0, 2, 5] == -127 and v[1, 0, 5, 2] == -127 and k[1, 0, 3, 0] == 9
    # the same call again changes nothing
    again = V.kv_append((k, ks, v, vs), y, y, table, [3], [0, 1], "int8")
    assert all(np.array_equal(p, q) for p, q in zip(again, (k, ks, v, vs)))


def test_append_scales_and_nan():
    cache = (np.zeros((1, 1, 16, 64), np.uint8), np.zeros((1, 1), np.float32),
             np.zeros((1, 1, 64, 16), np.uint8), np.zeros((1, 1), np.float32))
    x = np.full((1, 1, 64), 2.0 ** -70, np.float32)    # below the smallest scaled maximum
    k, ks, _, _ = V.kv_append(cache, x, x, np.array([[0]], np.int32), [1], [0, 1], "fp8")
    assert ks[0, 0] == 0 and not k.any()
    x[0, 0, 0], x[0, 0, 1] = np.nan, 896.0
    k, ks, _, _ = V.kv_append(cache, x, x, np.array([[0]], np.int32), [1], [0, 1], "fp8")
    assert ks[0, 0] == 2.0 and k[0, 0, 0, 0] == 0 and k[0, 0, 0, 1] == 0x7E


def test_attention_by_hand():
    # two visible tokens with scores ln 3 and 0: weights 3/4 and 1/4
    d, t = 64, 16
    k = np.zeros((1, 1, t, d), np.int8)
    v = np.zeros((1, 1, d, t), np.int8)
    k[0, 0, 0, 0], v[0, 0, 0, :2], k[0, 0, 2] = 1, (4, 8), 100
    ones = np.ones((1, 1), np.float32)
    q = np.zeros((2, 1, d))
    q[:, 0, 0] = math.log(3.0)
    out, lse, spread, _ = V.kv_attention(q, (k, ones, v, ones * 2, ), np.array([[0]]), [2], [0, 2],
                                         "int8", 1.0)
    assert math.isclose(out[0, 0, 0], 8.0) and math.isclose(lse[0, 0], math.log(3.0))
    assert math.isclose(out[1, 0, 0], 2 * (4 * 0.75 + 8 * 0.25)) and math.isclose(lse[1, 0], math.log(4.0))
    out, lse, _, _ = V.kv_attention(q, (k, ones, v, ones * 2), np.array([[0]]), [2], [0, 2], "int8",
                                    1.0, window=1)
    assert math.isclose(out[1, 0, 0], 16.0) and abs(lse[1, 0]) < 1e-12
    out, lse, _, _ = V.kv_attention(q, (k, ones, v, ones), np.array([[-1]]), [2], [0, 2], "int8", 1.0)
    assert not out.any() and np.isneginf(lse).all()


def test_attention_in_exact_arithmetic():
    # equal scores: plain means of the values, in rationals
    rng = np.random.default_rng(1)
    k = np.zeros((3, 1, 16, 64), np.int8)
    v = rng.integers(-127, 128, (3, 1, 64, 16)).astype(np.int8)
    sc = np.float32([[0.5], [0.25], [2.0]])
    table = np.array([[2, 0]])
    out, lse, _, _ = V.kv_attention(rng.standard_normal((1, 1, 64)), (k, sc, v, sc), table, [21],
                                    [0, 1], "int8", 0.125)
    for d in range(64):
        want = (sum(Fraction(2) * int(x) for x in v[2, 0, d]) +
                sum(Fraction(1, 2) * int(x) for x in v[0, 0, d, :5])) / 21
        assert math.isclose(out[0, 0, d], float(want), rel_tol=1e-13, abs_tol=1e-13)
    assert math.isclose(lse[0, 0], math.log(21))


# --- refusals on the host ---------------------------------------------------


@pytest.fixture(scope="module")
def L():
    try:
        return B.lib()
    except ImportError as e:
        pytest.skip(str(e))


def gemm(L, a=FAKE, lda=64, sa=FAKE, m=4, b=FAKE, ldb=64, sb=FAKE, n=8, k=64, bias=None, dt=0,
         c=FAKE, ldc=8, ws=None, nb=None):
    return L.sparq24_int8_gemm(a, lda, sa, m, b, ldb, sb, n, k, bias, dt, c, ldc, ws, nb, None)


def valid(st):
    """A valid call: it runs, or reports that there is no device here."""
    return st == DEVICE


@pytest.fixture()
def no_gpu():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")


def test_int8_gemm_refusals(L):
    assert gemm(L, m=-1) == INVALID and gemm(L, k=-16) == INVALID and gemm(L, dt=3) == INVALID
    assert gemm(L, k=24) == SHAPE and gemm(L, k=131072, lda=131072, ldb=131072) == SHAPE
    assert gemm(L, lda=48) == UNSUPPORTED and gemm(L, ldc=7) == UNSUPPORTED
    assert gemm(L, lda=72) == ALIGN and gemm(L, ldb=65) == ALIGN
    for name in ("a", "b", "sa", "sb", "c"):
        assert gemm(L, **{name: None}) == INVALID, name
    for name in ("a", "b", "c"):
        assert gemm(L, **{name: FAKE + 8}) == ALIGN, name
    assert gemm(L, sa=FAKE + 2) == ALIGN and gemm(L, bias=FAKE + 1) == ALIGN
    assert gemm(L, m=1 << 32) == UNSUPPORTED and gemm(L, m=2 ** 31 - 1, n=2 ** 31 - 1, ldc=2 ** 31) == UNSUPPORTED
    n = ctypes.c_size_t(5)
    assert gemm(L, nb=ctypes.byref(n)) == OK                      # size query
    assert gemm(L, m=0, a=None) == OK and gemm(L, n=0, b=None) == OK


def test_int8_gemm_accepts(L, no_gpu):
    assert valid(gemm(L)) and valid(gemm(L, k=0, a=None, b=None)) and valid(gemm(L, m=1, lda=3))
    assert valid(gemm(L, lda=80, ldb=96, ldc=11, bias=FAKE + 4, dt=1))
    assert valid(gemm(L, k=131056, lda=131056, ldb=131056))


def cache(**kw):
    d = dict(k=FAKE, k_scale=FAKE, v=FAKE, v_scale=FAKE, fmt=B.Q_INT, blocks=9, heads=2, tokens=32, dim=64)
    d.update(kw)
    return B.CKvCache(*(d[f] for f, _ in B.CKvCache._fields_))


def seqs(**kw):
    d = dict(block_table=FAKE, max_blocks=4, table_stride=4, seq_lens=FAKE, cu_tokens=None, seqs=3, total=6)
    d.update(kw)
    return B.CKvSeqs(*(d[f] for f, _ in B.CKvSeqs._fields_))


def rows(heads=2, dim=64, total=6, dtype=B.BF16, ts=None, hs=None, data=FAKE, ks=1):
    return B.CTensor(data, dtype, total, heads, dim, heads * dim if ts is None else ts,
                     dim if hs is None else hs, ks)


def append(L, c=None, s=None, k=None, v=None):
    R = ctypes.byref
    return L.sparq24_kv_append(R(c or cache()), R(s or seqs()), R(k or rows()), R(v or rows()), None)


def attend(L, c=None, s=None, q=None, scale=0.125, causal=1, window=0, out=FAKE, lse=None, ws=FAKE, nb=1 << 40):
    n = ctypes.c_size_t(nb) if isinstance(nb, int) else nb
    R = ctypes.byref
    return L.sparq24_kv_attention(R(c or cache()), R(s or seqs()), R(q or rows(heads=6)), scale, causal,
                                  window, out, lse, ws, n, None)


@pytest.mark.parametrize("call", [append, attend])
def test_cache_refusals(L, call):
    assert call(L, c=cache(fmt=9)) == INVALID and call(L, c=cache(fmt=B.Q_MXFP4)) == UNSUPPORTED
    for t in (0, 8, 24, 512):
        assert call(L, c=cache(tokens=t)) == SHAPE, t
    for d in (0, 32, 80, 320):
        assert call(L, c=cache(dim=d)) == SHAPE, d
    assert call(L, c=cache(blocks=0)) == SHAPE and call(L, c=cache(heads=0)) == SHAPE
    assert call(L, c=cache(blocks=-1)) == INVALID and call(L, c=cache(blocks=1 << 31)) == UNSUPPORTED
    for p in ("k", "k_scale", "v", "v_scale"):
        assert call(L, c=cache(**{p: None})) == INVALID, p
        assert call(L, c=cache(**{p: FAKE + 2})) == ALIGN, p
    assert call(L, s=seqs(seqs=-1)) == INVALID and call(L, s=seqs(total=-1)) == INVALID
    assert call(L, s=seqs(max_blocks=-1)) == INVALID
    assert call(L, s=seqs(table_stride=3)) == UNSUPPORTED
    assert call(L, s=seqs(seqs=4)) == SHAPE                       # 6 rows over 4 sequences
    assert call(L, s=seqs(seq_lens=None)) == INVALID and call(L, s=seqs(block_table=None)) == INVALID
    assert call(L, s=seqs(cu_tokens=FAKE + 1)) == ALIGN


def test_append_refusals(L):
    assert append(L, k=rows(total=5)) == SHAPE and append(L, v=rows(dim=128)) == SHAPE
    assert append(L, k=rows(heads=3), v=rows(heads=3)) == SHAPE
    assert append(L, k=rows(dtype=B.F16)) == UNSUPPORTED          # types of k and v differ
    assert append(L, k=rows(dtype=5)) == INVALID and append(L, k=rows(ks=2)) == UNSUPPORTED
    assert append(L, k=rows(ts=132)) == ALIGN and append(L, v=rows(hs=65)) == ALIGN
    assert append(L, k=rows(data=None)) == INVALID and append(L, v=rows(data=FAKE + 8)) == ALIGN
    e = dict(total=0)
    assert append(L, s=seqs(total=0), k=rows(data=None, **e), v=rows(data=None, **e)) == OK
    e = dict(total=0, data=None)
    assert append(L, s=seqs(seqs=0, total=0, seq_lens=None, block_table=None), k=rows(**e), v=rows(**e)) == OK


def test_attention_refusals_and_workspace(L):
    assert attend(L, q=rows(heads=3)) == SHAPE                    # 3 query heads on 2 kv heads
    assert attend(L, q=rows(heads=6, dtype=B.F32)) == UNSUPPORTED
    assert attend(L, q=rows(heads=6, dtype=9)) == INVALID
    for s in (0.0, -1.0, math.inf, math.nan):
        assert attend(L, scale=s) == INVALID, s
    assert attend(L, causal=2) == INVALID and attend(L, window=-1) == INVALID
    assert attend(L, causal=0, window=5) == INVALID
    assert attend(L, out=None) == INVALID and attend(L, out=FAKE + 4) == ALIGN and attend(L, lse=FAKE + 2) == ALIGN
    assert attend(L, q=rows(heads=6, data=None)) == INVALID
    big = seqs(max_blocks=64, table_stride=64)
    n = ctypes.c_size_t(0)
    assert attend(L, s=big, out=None, ws=None, nb=n) == OK
    assert n.value > 0
    assert attend(L, s=big, nb=n.value - 1) == WORKSPACE and attend(L, s=big, nb=None) == WORKSPACE
    assert attend(L, s=big, ws=FAKE + 8) == ALIGN
    # 1024 tokens at most: no split, no workspace
    assert attend(L, s=seqs(max_blocks=8, table_stride=8), out=None, ws=None, nb=n) == OK
    assert n.value == 0
    # the work list of more than 128 sequences
    many = dict(cu_tokens=FAKE, total=129)
    assert attend(L, s=seqs(seqs=129, **many), q=rows(heads=6, total=129), out=None, ws=None, nb=n) == OK
    assert n.value > 0
    assert attend(L, s=seqs(seqs=128, **many), q=rows(heads=6, total=129), out=None, ws=None, nb=n) == OK
    assert n.value == 0
    # more workgroups than a grid has
    most = dict(seqs=2 ** 24, total=2 ** 24)
    assert attend(L, s=seqs(**most), q=rows(heads=6, total=2 ** 24)) == UNSUPPORTED
    assert append(L, s=seqs(**most), k=rows(total=2 ** 24), v=rows(total=2 ** 24)) == UNSUPPORTED
    assert attend(L, s=seqs(total=0), q=rows(heads=6, total=0, data=None), out=None) == OK
    assert attend(L, s=seqs(total=2 ** 28, seqs=2 ** 20), q=rows(heads=64, total=2 ** 28)) == UNSUPPORTED


def test_valid_calls_reach_the_device(L, no_gpu):
    assert valid(append(L)) and valid(attend(L)) and valid(attend(L, causal=0)) and valid(attend(L, window=7))
    assert valid(append(L, s=seqs(max_blocks=0, block_table=None)))
    assert valid(append(L, s=seqs(cu_tokens=FAKE, seqs=5), k=rows(ts=1024, hs=128), v=rows(dtype=B.BF16)))
    assert valid(append(L, c=cache(fmt=B.Q_FP8, tokens=256, dim=256), k=rows(dim=256, dtype=B.F32),
                        v=rows(dim=256, dtype=B.F32)))


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    i8 = torch.zeros(4, 32, dtype=torch.int8)
    f = torch.zeros(4)
    with pytest.raises(ValueError, match="GPU"):
        B.int8_gemm(i8, f, i8, f)
    c = B.kv_cache(3, 2, 64, 16, device="cpu")
    assert c.k.shape == (3, 2, 16, 64) and c.v.shape == (3, 2, 64, 16)
    x = torch.zeros(2, 1, 2, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        B.kv_append(c, x, x, table, lens)
    with pytest.raises(ValueError, match="GPU"):
        B.kv_attention(x, c, table, lens)
    with pytest.raises(ValueError, match="int"):
        B.kv_cache(3, 2, 64, 16, q=("int", 4), device="cpu")
    # checks come before the device, so all refusals show without one
    def attend(q=x, cache=c, table=table, lens=lens, cu=None, **kw):
        B.kv_attention(q, cache, table, lens, cu, **kw)

    for bad, what in ((c._replace(v=c.k), "match"), (c._replace(k_scale=c.k_scale[:2]), "k_scale"),
                      (c._replace(k=c.k[:, :, ::2]), "match"), (c._replace(v_scale=c.v_scale.double()), "v_scale"),
                      (c._replace(k=c.k.transpose(0, 1).contiguous().transpose(0, 1)), "contiguous"),
                      (c._replace(k=c.k[0]), "blocks")):
        with pytest.raises(ValueError, match=what):
            attend(cache=bad)
        with pytest.raises(ValueError, match=what):
            B.kv_append(bad, x, x, table, lens)
    with pytest.raises(TypeError, match="e4m3"):
        attend(cache=c._replace(k=c.k.float(), v=c.v.float()))
    with pytest.raises(TypeError, match="KVCache"):
        attend(cache=c.k)
    for kw, what in (({"table": table.long()}, "block_table"), ({"table": table[:, ::2]}, "block_table"),
                     ({"lens": lens.long()}, "seq_lens"), ({"lens": lens[:1]}, "seq_lens"),
                     ({"q": x[:, 0], "cu": lens}, "cu_tokens"), ({"q": x, "cu": lens}, "cu_tokens"),
                     ({"q": x[:, 0]}, "n, heads"), ({"q": x[:1]}, "n, heads"),
                     ({"q": torch.zeros(2, 5, 2, 64)[:, :2]}, "evenly"),
                     ({"q": torch.zeros(2, 1, 64, 2).transpose(2, 3)}, "contiguous"),
                     ({"out": x[:1]}, "out"), ({"out": x.float()}, "out"), ({"lse": x[..., 0]}, "lse"),
                     ({"workspace": torch.zeros(8, 2)[:, :1]}, "workspace")):
        with pytest.raises(ValueError, match=what):
            attend(**kw)
    for kw in ({"q": x.double()}, {"q": None}, {"lens": [1, 1]}, {"scale": "1"}, {"window": 1.5}):
        with pytest.raises(TypeError):
            attend(**kw)
    with pytest.raises(ValueError, match="match"):
        B.kv_append(c, x, x.half(), table, lens)
    for args, what in (((i8, f[:3], i8, f), "scale_a"), ((i8, f, i8, f.double()), "scale_b"),
                       ((i8, f, i8[:, :16], f), "multiply"), ((i8[:, ::2], f, i8[:, ::2], f), "contiguous"),
                       ((i8.t().contiguous().t(), f, i8, f), "contiguous"),
                       ((torch.zeros(2, 3, 32, dtype=torch.int8)[:, :2], f, i8, f), "evenly"),
                       ((i8, f, i8, f, f[:2]), "bias"), ((i8, f, i8, f, None, torch.float32, f), "out")):
        with pytest.raises(ValueError, match=what):
            B.int8_gemm(*args)
    for args in ((i8.float(), f, i8, f), (i8, f, i8.float(), f), (i8, f, i8, f, None, torch.float64),
                 (i8, f, i8, f, None, "fp32")):
        with pytest.raises(TypeError):
            B.int8_gemm(*args)
