"""CPU pins of the oracles of the serving operators around 4-bit data (norm, MXFP4
product, MXFP4 cache), and the host-side refusals of their C entry points and calls."""
import ctypes
import math

import numpy as np
import pytest

import oracle as O
import oracle.serving as V8
import oracle.serving4 as V

B = pytest.importorskip("pruning_quantization_amd.binding")

FAKE = 0x7F0000000000          # 16-byte aligned, never dereferenced on the host
OK, INVALID, UNSUPPORTED, SHAPE, ALIGN, WORKSPACE, DEVICE = 0, 1, 2, 3, 4, 5, 6


# --- oracles ---------------------------------------------------------------


def test_norm_by_hand():
    # mean square (9 + 16 + 30 * 0) / 32 with eps chosen so that the root is 1
    x = np.zeros((1, 32), np.float32)
    x[0, :2] = 3, 4
    eps = 1 - 25 / 32
    w = np.ones(32, np.float32)
    w[1] = 2
    y, total = V.rmsnorm(x, "f32", w, eps)
    assert y[0, :3].tolist() == [3.0, 8.0, 0.0] and total is None
    codes, scales, _ = V.rmsnorm_quantize(x, "f32", w, eps, O.QSpec("mxfp4"))
    assert scales.tolist() == [[127 + 1]] and codes[0, 0] == 0x63          # 1.5 and 4, times 2
    codes, scales, _ = V.rmsnorm_quantize(x, "f32", w, eps, O.QSpec("int", 8))
    assert scales[0] == np.float32(8 / 127) and codes[0, :2].tolist() == [48, 127]


def test_norm_of_the_rounded_sum():
    # 256 + 1.5 in bf16: half way between 256 and 258 is 257; 257.5 rounds up
    x = np.full((1, 8), 0x4380, np.uint16)                                 # 256
    r = np.full((1, 8), 0x3FC0, np.uint16)                                 # 1.5
    y, total = V.rmsnorm(x, "bf16", np.ones(8, np.float32), 0.0, r)
    assert (O.decode_input(total, "bf16") == 258).all() and (y == 1).all()
    half = V.round_to(np.float32([257.0, 259.0, -257.0, 2.0 ** -134]), "bf16")
    assert O.decode_input(half[None], "bf16")[0].tolist() == [256.0, 260.0, -256.0, 0.0]


def test_product_by_hand():
    a = np.zeros((1, 32), np.uint8)
    b = np.zeros((2, 32), np.uint8)
    a[0, 0], a[0, 16] = 0x51, 0x02                    # 0.5, 3 and (second group) 1
    b[0, 0], b[0, 16] = 0xF2, 0x07                    # 1, -6 and 6
    b[1, 0] = 0x22
    sa, sb = np.uint8([[127, 130]]), np.uint8([[128, 127], [0, 255]])
    y, size = V.mxfp4_gemm(a, sa, b, sb, np.float32([1, 0]))
    assert y[0, 0] == (0.5 - 18) * 2 + 6 * 8 + 1 and size[0, 0] == 18.5 * 2 + 48
    assert np.isnan(y[0, 1])


def test_append_by_hand():
    cache = (np.full((2, 1, 16, 32), 9, np.uint8), np.full((2, 1, 2, 16), 7, np.uint8)) * 2
    x = np.zeros((1, 1, 64), np.float32)
    x[0, 0, :4] = 6, -3, np.nan, 0.25
    x[0, 0, 32:35] = 1e3, np.inf, -np.inf
    k, ks, v, vs = V.kv_append(cache, x, x, np.array([[1]]), [4], [0, 1])
    assert ks[1, 0, :, 3].tolist() == [127, 127 + 9 - 2] and (ks[1, 0, :, 2] == 7).all() and (ks[0] == 7).all()
    assert k[1, 0, 3, :2].tolist() == [0xD7, 0x00]                          # 6, -3; 0, a half rounds to even
    assert k[1, 0, 3, 16:18].tolist() == [0x77, 0x0F]                       # 1000 / 128 = 7.8 saturates, as the infinities do
    assert np.array_equal(k, v) and (k[1, 0, 4] == 9).all()


def test_attention_agrees_with_the_8_bit_oracle():
    # the same stored values in both forms: codes in halves are INT8 codes of scale 1/2
    rng = np.random.default_rng(1)
    blocks, kv, T, D = 4, 2, 16, 64
    codes = [rng.integers(0, 256, (blocks, kv, T, D // 2)).astype(np.uint8) for _ in range(2)]
    ones = np.full((blocks, kv, D // 32, T), 127, np.uint8)
    vals = [V.mxfp4_values(c, ones.transpose(0, 1, 3, 2)) for c in codes]
    i8 = [np.rint(2 * x).astype(np.int8) for x in vals]
    sc = np.full((blocks, kv), 0.5, np.float32)
    table, lens, cu = np.array([[3, 1], [0, -1]]), [25, 9], [0, 3, 5]
    q = rng.standard_normal((5, 4, D))
    for kw in ({}, {"window": 7}, {"causal": False}):
        a = V.kv_attention(q, (codes[0], ones, codes[1], ones), table, lens, cu, 0.125, **kw)
        b = V8.kv_attention(q, (i8[0], sc, i8[1].transpose(0, 1, 3, 2), sc), table, lens, cu, "int8", 0.125, **kw)
        for x, y in zip(a, b):
            assert np.allclose(x, y, rtol=1e-12, atol=1e-12)


# --- refusals on the host ---------------------------------------------------


@pytest.fixture(scope="module")
def L():
    try:
        return B.lib()
    except ImportError as e:
        pytest.skip(str(e))


@pytest.fixture()
def no_gpu():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")


def gemm(L, a=FAKE, lda=32, sa=FAKE, m=4, b=FAKE, ldb=32, sb=FAKE, n=8, k=64, bias=None, dt=0, c=FAKE, ldc=8,
         ws=None, nb=None):
    return L.sparq24_mxfp4_gemm(a, lda, sa, m, b, ldb, sb, n, k, bias, dt, c, ldc, ws, nb, None)


def test_product_refusals(L):
    assert gemm(L, m=-1) == INVALID and gemm(L, k=-32) == INVALID and gemm(L, dt=3) == INVALID
    assert gemm(L, k=48) == SHAPE and gemm(L, k=131104, lda=65552, ldb=65552) == SHAPE
    assert gemm(L, lda=16) == UNSUPPORTED and gemm(L, ldc=7) == UNSUPPORTED
    assert gemm(L, lda=40) == ALIGN and gemm(L, ldb=33) == ALIGN
    for name in ("a", "b", "sa", "sb", "c"):
        assert gemm(L, **{name: None}) == INVALID, name
    for name in ("a", "b", "c"):
        assert gemm(L, **{name: FAKE + 8}) == ALIGN, name
    assert gemm(L, bias=FAKE + 1) == ALIGN
    assert gemm(L, m=1 << 32) == UNSUPPORTED and gemm(L, m=2 ** 31 - 1, n=2 ** 31 - 1, ldc=2 ** 31) == UNSUPPORTED
    assert gemm(L, nb=ctypes.byref(ctypes.c_size_t(5))) == OK                      # size query
    assert gemm(L, m=0, a=None) == OK and gemm(L, n=0, b=None) == OK


def test_product_accepts(L, no_gpu):
    assert gemm(L) == gemm(L, k=0, a=None, b=None, sa=None, sb=None) == gemm(L, m=1, lda=3) == DEVICE
    assert gemm(L, lda=48, ldb=64, ldc=11, bias=FAKE + 4, dt=1, sa=FAKE + 1, sb=FAKE + 3) == DEVICE
    assert gemm(L, k=131072, lda=65536, ldb=65536) == DEVICE


def rows(dtype=B.BF16, batch=1, rows=4, k=64, bs=None, rs=None, ks=1, data=FAKE):
    rs = k if rs is None else rs
    return B.CTensor(data, dtype, batch, rows, k, rows * rs if bs is None else bs, rs, ks)


def norm(L, x=None, res=None, w=FAKE, wd=B.F32, eps=1e-6, fmt=B.Q_FP8, bits=0, codes=FAKE, scales=FAKE, total=None):
    q = B.CQSpec(fmt, bits, None)
    ref = lambda t: ctypes.byref(t) if t is not None else None  # noqa: E731
    return L.sparq24_rmsnorm_quantize(ref(x or rows()), ref(res), w, wd, eps, ctypes.byref(q), codes, scales,
                                      ref(total), None)


def test_norm_refusals(L):
    assert norm(L, x=rows(k=12)) == SHAPE and norm(L, x=rows(k=48), fmt=B.Q_MXFP4) == SHAPE
    assert norm(L, x=rows(k=32768 + 8)) == SHAPE and norm(L, x=rows(dtype=4)) == INVALID
    assert norm(L, x=rows(rs=1, ks=4)) == UNSUPPORTED                               # transposed
    assert norm(L, x=rows(rs=68)) == ALIGN and norm(L, x=rows(data=FAKE + 8)) == ALIGN
    assert norm(L, x=rows(data=None)) == INVALID
    assert norm(L, wd=5) == INVALID and norm(L, wd=B.F16) == UNSUPPORTED
    for eps in (-1e-6, math.inf, math.nan):
        assert norm(L, eps=eps) == INVALID
    for fmt, bits, want in ((B.Q_NONE, 0, UNSUPPORTED), (B.Q_NVFP4, 0, UNSUPPORTED), (B.Q_INT, 9, UNSUPPORTED),
                            (B.Q_INT, 1, UNSUPPORTED), (7, 0, INVALID)):
        assert norm(L, fmt=fmt, bits=bits) == want, fmt
    for name in ("w", "codes", "scales"):
        assert norm(L, **{name: None}) == INVALID and norm(L, **{name: FAKE + 4}) == ALIGN, name
    assert norm(L, res=rows()) == INVALID and norm(L, total=rows()) == INVALID      # both or neither
    assert norm(L, res=rows(rows=5), total=rows()) == SHAPE and norm(L, res=rows(), total=rows(k=72)) == SHAPE
    assert norm(L, res=rows(dtype=B.F16), total=rows()) == UNSUPPORTED
    assert norm(L, res=rows(), total=rows(data=None)) == INVALID
    assert norm(L, x=rows(rows=0), w=None, codes=None) == OK


def test_norm_accepts(L, no_gpu):
    assert norm(L) == norm(L, wd=B.BF16) == norm(L, fmt=B.Q_INT, bits=2) == norm(L, fmt=B.Q_MXFP4) == DEVICE
    assert norm(L, res=rows(rs=128), total=rows(rs=72)) == norm(L, x=rows(k=32768), eps=0.0) == DEVICE


def cache(**kw):
    d = dict(k=FAKE, k_scale=FAKE, v=FAKE, v_scale=FAKE, blocks=9, heads=2, tokens=32, dim=64)
    d.update(kw)
    return B.CKvCacheMx(*(d[f] for f, _ in B.CKvCacheMx._fields_))


def seqs(**kw):
    d = dict(block_table=FAKE, max_blocks=4, table_stride=4, seq_lens=FAKE, cu_tokens=None, seqs=3, total=6)
    d.update(kw)
    return B.CKvSeqs(*(d[f] for f, _ in B.CKvSeqs._fields_))


def tokens(heads=2, dim=64, total=6, dtype=B.BF16, ts=None, hs=None, data=FAKE, ks=1):
    return B.CTensor(data, dtype, total, heads, dim, heads * dim if ts is None else ts, dim if hs is None else hs, ks)


def append(L, c=None, s=None, k=None, v=None):
    R = ctypes.byref
    return L.sparq24_kv_append_mxfp4(R(c or cache()), R(s or seqs()), R(k or tokens()), R(v or tokens()), None)


def attend(L, c=None, s=None, q=None, scale=0.125, causal=1, window=0, out=FAKE, lse=None, ws=FAKE, nb=1 << 40):
    n = ctypes.c_size_t(nb) if isinstance(nb, int) else nb
    R = ctypes.byref
    return L.sparq24_kv_attention_mxfp4(R(c or cache()), R(s or seqs()), R(q or tokens(heads=6)), scale, causal,
                                        window, out, lse, ws, n, None)


@pytest.mark.parametrize("call", [append, attend])
def test_cache_refusals(L, call):
    for t in (0, 8, 24, 512):
        assert call(L, c=cache(tokens=t)) == SHAPE, t
    for d in (0, 32, 80, 320):
        assert call(L, c=cache(dim=d)) == SHAPE, d
    assert call(L, c=cache(blocks=0)) == SHAPE and call(L, c=cache(heads=0)) == SHAPE
    assert call(L, c=cache(blocks=-1)) == INVALID and call(L, c=cache(blocks=1 << 31)) == UNSUPPORTED
    for p in ("k", "k_scale", "v", "v_scale"):
        assert call(L, c=cache(**{p: None})) == INVALID, p
        assert call(L, c=cache(**{p: FAKE + 4})) == ALIGN, p
    assert call(L, s=seqs(seqs=-1)) == INVALID and call(L, s=seqs(total=-1)) == INVALID
    assert call(L, s=seqs(table_stride=3)) == UNSUPPORTED
    assert call(L, s=seqs(seqs=4)) == SHAPE                       # 6 rows over 4 sequences
    assert call(L, s=seqs(seq_lens=None)) == INVALID and call(L, s=seqs(block_table=None)) == INVALID
    assert call(L, s=seqs(cu_tokens=FAKE + 1)) == ALIGN


def test_append_refusals(L):
    assert append(L, k=tokens(total=5)) == SHAPE and append(L, v=tokens(dim=128)) == SHAPE
    assert append(L, k=tokens(heads=3), v=tokens(heads=3)) == SHAPE
    assert append(L, k=tokens(dtype=B.F16)) == UNSUPPORTED          # types of k and v differ
    assert append(L, k=tokens(ts=132)) == ALIGN and append(L, v=tokens(data=FAKE + 8)) == ALIGN
    assert append(L, k=tokens(data=None)) == INVALID
    e = dict(total=0, data=None)
    assert append(L, s=seqs(total=0), k=tokens(**e), v=tokens(**e)) == OK
    assert append(L, s=seqs(seqs=1, total=2 ** 31 - 1), c=cache(heads=64, dim=256), k=tokens(64, 256, 2 ** 31 - 1),
                  v=tokens(64, 256, 2 ** 31 - 1)) == UNSUPPORTED    # more workgroups than a grid has


def test_attention_refusals_and_workspace(L):
    assert attend(L, q=tokens(heads=3)) == SHAPE                    # 3 query heads on 2 kv heads
    assert attend(L, q=tokens(heads=6, dtype=B.F32)) == UNSUPPORTED
    for s in (0.0, -1.0, math.inf, math.nan):
        assert attend(L, scale=s) == INVALID, s
    assert attend(L, causal=2) == INVALID and attend(L, window=-1) == INVALID
    assert attend(L, causal=0, window=5) == INVALID
    assert attend(L, out=None) == INVALID and attend(L, out=FAKE + 4) == ALIGN and attend(L, lse=FAKE + 2) == ALIGN
    big = seqs(max_blocks=64, table_stride=64)
    n = ctypes.c_size_t(0)
    assert attend(L, s=big, out=None, ws=None, nb=n) == OK
    assert n.value > 0
    assert attend(L, s=big, nb=n.value - 1) == WORKSPACE and attend(L, s=big, nb=None) == WORKSPACE
    assert attend(L, s=big, ws=FAKE + 8) == ALIGN
    assert attend(L, s=seqs(max_blocks=8, table_stride=8), out=None, ws=None, nb=n) == OK
    assert n.value == 0                                             # 1024 tokens at most: no split
    most = dict(seqs=2 ** 24, total=2 ** 24)
    assert attend(L, s=seqs(**most), q=tokens(heads=6, total=2 ** 24)) == UNSUPPORTED
    assert attend(L, s=seqs(total=0), q=tokens(heads=6, total=0, data=None), out=None) == OK


def test_valid_calls_reach_the_device(L, no_gpu):
    assert append(L) == attend(L) == attend(L, causal=0) == attend(L, window=7) == DEVICE
    assert append(L, s=seqs(max_blocks=0, block_table=None)) == DEVICE
    assert append(L, c=cache(tokens=256, dim=256), k=tokens(dim=256, dtype=B.F32),
                  v=tokens(dim=256, dtype=B.F32)) == DEVICE


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    u8 = torch.zeros(4, 32, dtype=torch.uint8)
    s = torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        B.mxfp4_gemm(u8, s, u8, s)
    for args, what in (((u8, s[:3], u8, s), "scale_a"), ((u8, s, u8, s.float()), "scale_b"),
                       ((u8, s, u8[:, :16], s), "multiply"), ((u8[:, :24], s, u8[:, :24], s), "groups"),
                       ((u8[:, ::2], s, u8[:, ::2], s), "contiguous"), ((u8, s, u8, s, s), "bias"),
                       ((u8, s, u8, s, None, torch.float32, torch.zeros(4)), "out")):
        with pytest.raises(ValueError, match=what):
            B.mxfp4_gemm(*args)
    for args in ((u8.char(), s, u8, s), (u8, s, u8.float(), s), (u8, s, u8, s, None, torch.float64)):
        with pytest.raises(TypeError):
            B.mxfp4_gemm(*args)

    x, w = torch.zeros(2, 3, 64, dtype=torch.bfloat16), torch.ones(64)
    with pytest.raises(ValueError, match="GPU"):
        B.rmsnorm_quantize(x, w, "fp8", residual=x)
    for args, kw, what in (((x, w[:32], "fp8"), {}, "weight"), ((x, w[None], "fp8"), {}, "weight"),
                           ((x, w, "fp8"), {"residual": x[:1]}, "residual"),
                           ((x, w, "fp8"), {"residual": x.float()}, "residual"),
                           ((x, w, "fp8"), {"residual_out": x}, "residual"),
                           ((x, w, "fp8"), {"residual": x, "residual_out": x[:, :1]}, "residual_out"),
                           ((x[..., ::2], w[:32], "fp8"), {}, "contiguous"),
                           ((x[..., :40], w[:40], "mxfp4"), {}, "32"),
                           ((x, w, "fp8"), {"out": (x, w)}, "codes"),
                           ((x, w, ("int", 8)), {"out": (x.to(torch.int8), w[:3])}, "scales"),
                           ((torch.zeros(4, 3, 2, 64)[:, :2], w, "fp8"), {}, "evenly")):
        with pytest.raises(ValueError, match=what):
            B.rmsnorm_quantize(*args, **kw)
    for args in ((x.double(), w, "fp8"), (x, w.double(), "fp8"), (x, None, "fp8"), (None, w, "fp8")):
        with pytest.raises(TypeError):
            B.rmsnorm_quantize(*args)
    with pytest.raises(KeyError):
        B.rmsnorm_quantize(x, w, "int8")

    c = B.kv_cache(3, 2, 64, 16, "mxfp4", device="cpu")
    assert c.k.shape == c.v.shape == (3, 2, 16, 32) and c.k_scale.shape == c.v_scale.shape == (3, 2, 2, 16)
    x = torch.zeros(2, 1, 2, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        B.kv_append(c, x, x, table, lens)
    with pytest.raises(ValueError, match="GPU"):
        B.kv_attention(x, c, table, lens)
    for bad, what in ((c._replace(v=c.v[:, :, :8]), "match"), (c._replace(k_scale=c.k_scale[:2]), "k_scale"),
                      (c._replace(v_scale=c.v_scale.float()), "v_scale"),
                      (c._replace(k=c.k.transpose(0, 1).contiguous().transpose(0, 1)), "contiguous")):
        with pytest.raises(ValueError, match=what):
            B.kv_attention(x, bad, table, lens)
    with pytest.raises(TypeError):
        B.kv_attention(x, c._replace(k=c.k.char(), v=c.v.char()), table, lens)
    with pytest.raises(ValueError, match="v_scale"):                 # fp32 K scales: an 8-bit cache
        e8 = B.kv_cache(3, 2, 64, 16, "fp8", device="cpu")
        B.kv_attention(x, e8._replace(v_scale=c.v_scale), table, lens)
