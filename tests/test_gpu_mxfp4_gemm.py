"""GPU parity of the MXFP4 product against the oracle in 64 bits.

A product of two codes is a multiple of 1/4 of at most 36, so a group's 32 are exact in
fp32; the groups and the parts of K that different waves take are added in fp32, in some
order: at most K / 32 + 8 roundings, each of at most 2^-23 (truncation) of sum |a b|.
Then the bias (2^-24) and half a step of the output's type."""
import numpy as np
import pytest

import oracle as O
import oracle.serving4 as V

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU, skipped there
    pytest.skip("no GPU", allow_module_level=True)

import pruning_quantization_amd as S  # noqa: E402
from gpu_util import DEV  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def operand(rng, rows, k, low=120, high=134):
    return (rng.integers(0, 256, (rows, k // 2)).astype(np.uint8),
            rng.integers(low, high, (rows, k // 32)).astype(np.uint8))


def dev(*xs):
    return [torch.from_numpy(np.ascontiguousarray(x)).to(DEV) for x in xs]


def check(got, a, sa, b, sb, bias, dtype):
    want, size = V.mxfp4_gemm(a, sa, b, sb, bias)
    k = a.shape[1] * 2
    tol = (size * (k / 32 + 8) * 2.0 ** -23 + (0 if bias is None else np.abs(bias) * 2.0 ** -24)
           + np.abs(want) * (torch.finfo(DT[dtype]).eps / 2 + 2.0 ** -23) + torch.finfo(DT[dtype]).tiny)
    got = got.cpu().double().numpy()
    assert got.shape == want.shape
    # what lies half a step past the type's largest number (fp16: 65504 + 16) rounds to infinity
    edge = float(torch.finfo(DT[dtype]).max) * (1 + torch.finfo(DT[dtype]).eps / 4)
    far = np.abs(want) - tol > edge
    assert (got[far] == np.sign(want[far]) * np.inf).all()
    with np.errstate(invalid="ignore"):
        ok = far | (np.abs(got - want) <= tol) | ((np.abs(want) + tol >= edge) & np.isinf(got))
    assert ok.all(), f"{(~ok).sum()} of {ok.size} outside; worst {np.nanmax(np.abs(got - want) / tol):.3g}"


# one row to several tiles, ragged in every direction; K under one slab of 256, at whole
# slabs and with every rest (32 .. 224)
@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 33, 48, 64, 65, 100, 129, 257])
@pytest.mark.parametrize("n,k", [(1, 32), (17, 64), (64, 256), (70, 288), (130, 2080), (257, 480)])
def test_shapes(m, n, k):
    rng = np.random.default_rng(m * 1000 + n)
    a, sa = operand(rng, m, k)
    b, sb = operand(rng, n, k)
    bias = rng.standard_normal(n).astype(np.float32) if m % 2 else None
    dtype = ("f32", "bf16", "f16")[(m + n) % 3]
    da, dsa, db, dsb = dev(a, sa, b, sb)
    got = S.mxfp4_gemm(da, dsa, db, dsb, bias=None if bias is None else dev(bias)[0], dtype=DT[dtype])
    assert got.dtype == DT[dtype]
    check(got, a, sa, b, sb, bias, dtype)


@pytest.mark.parametrize("rest", range(0, 256, 32))
@pytest.mark.parametrize("m,n", [(3, 40), (200, 300)])
def test_every_rest_of_k(m, n, rest):
    rng = np.random.default_rng(rest)
    k = 1024 + rest
    a, sa = operand(rng, m, k)
    b, sb = operand(rng, n, k)
    check(S.mxfp4_gemm(*dev(a, sa, b, sb)), a, sa, b, sb, None, "f32")


# the tiles: whole and ragged ones of each size, K below and at a slab, odd numbers of slabs
# and of the groups in which exponents are read
@pytest.mark.parametrize("m,n,k,dtype", [
    (4096, 4096, 512, "bf16"), (4000, 4200, 544, "f32"), (3841, 4097, 768, "f16"), (4096, 4352, 1312, "f32"),
    (4096, 4096, 480, "bf16"), (2048, 4096, 512, "bf16"), (2000, 4100, 832, "f32"), (1030, 4090, 1056, "f16"),
    (1024, 2048, 256, "f32"), (600, 1500, 96, "f32"), (5000, 4111, 1024, "bf16"), (4100, 4100, 928, "f32")])
def test_tiles(m, n, k, dtype):
    rng = np.random.default_rng(m + n)
    a, sa = operand(rng, m, k, 122, 128)
    b, sb = operand(rng, n, k, 122, 128)
    bias = rng.standard_normal(n).astype(np.float32)
    da, dsa, db, dsb, dbias = dev(a, sa, b, sb, bias)
    check(S.mxfp4_gemm(da, dsa, db, dsb, bias=dbias, dtype=DT[dtype]), a, sa, b, sb, bias, dtype)


# more of the largest tiles than CUs, K in whole groups of exponents: a workgroup goes from
# tile to tile (three times over the ragged edges; one, three groups of K)
@pytest.mark.parametrize("m,n,k,dtype", [(300, 66000, 512, "f16"), (4097, 5000, 1536, "f32"), (66000, 257, 1024, "bf16")])
def test_tiles_in_turn(m, n, k, dtype):
    rng = np.random.default_rng(m + n)
    a, sa = operand(rng, m, k, 122, 128)
    b, sb = operand(rng, n, k, 122, 128)
    bias = rng.standard_normal(n).astype(np.float32)
    da, dsa, db, dsb, dbias = dev(a, sa, b, sb, bias)
    check(S.mxfp4_gemm(da, dsa, db, dsb, bias=dbias, dtype=DT[dtype]), a, sa, b, sb, bias, dtype)


def test_quantized_operands_and_leading_dims():
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.standard_normal((2, 9, 512)).astype(np.float32)).to(DEV).bfloat16()
    w = torch.from_numpy(rng.standard_normal((48, 512)).astype(np.float32)).to(DEV).bfloat16()
    (a, sa), (b, sb) = S.quantize(x, "mxfp4"), S.quantize(w, "mxfp4")
    got = S.mxfp4_gemm(a, sa, b, sb)
    assert got.shape == (2, 9, 48)
    flat = [t.cpu().numpy().reshape(-1, t.shape[-1]) for t in (a, sa, b, sb)]
    check(got.flatten(0, 1), *flat, None, "f32")


@pytest.mark.parametrize("m,n", [(5, 33), (70, 200), (300, 520)])
def test_strided_rows_and_output(m, n):
    rng = np.random.default_rng(m)
    k = 320
    a, sa = operand(rng, m, k + 64)
    b, sb = operand(rng, n, k + 32)
    da, db = dev(a, b)
    dsa, dsb = dev(sa[:, :k // 32], sb[:, :k // 32])
    out = torch.full((m, n + 3), 7.0, device=DEV)
    got = S.mxfp4_gemm(da[:, :k // 2], dsa, db[:, :k // 2], dsb, out=out[:, :n])
    assert got.data_ptr() == out.data_ptr() and (out[:, n:] == 7).all()
    check(got, a[:, :k // 2], sa[:, :k // 32], b[:, :k // 2], sb[:, :k // 32], None, "f32")
    # an output that begins at any element
    wide = torch.full((m + 1, n + 5), 7.0, dtype=torch.bfloat16, device=DEV)
    view = wide.as_strided((m, n), (n + 5, 1), 8)
    S.mxfp4_gemm(da[:, :k // 2], dsa, db[:, :k // 2], dsb, out=view)
    check(view, a[:, :k // 2], sa[:, :k // 32], b[:, :k // 2], sb[:, :k // 32], None, "bf16")


@pytest.mark.parametrize("m,n", [(4, 20), (300, 300)])
def test_scales_at_the_ends_of_the_range(m, n):
    rng = np.random.default_rng(m)
    k = 512
    a, sa = operand(rng, m, k, 0, 255)
    b, sb = operand(rng, n, k)
    sb = (254 - sa[:1].astype(int) + rng.integers(-3, 4, sb.shape)).clip(0, 254).astype(np.uint8)
    a[:, :], sa[:] = a[:1], sa[:1]                      # every product near 1
    check(S.mxfp4_gemm(*dev(a, sa, b, sb)), a, sa, b, sb, None, "f32")
    sa[:], sb[:] = 254, 254                             # past fp32
    got = S.mxfp4_gemm(*dev(a, sa, b, sb)).cpu().numpy()
    want, _ = V.mxfp4_gemm(a, sa, b, sb)
    assert (np.isinf(got) | np.isnan(got) | (want == 0)).all()


@pytest.mark.parametrize("m,n,k", [(3, 40, 96), (3, 40, 1024), (150, 290, 544), (520, 530, 512), (4096, 4096, 1056)])
def test_nan_scales_reach_their_row_and_column(m, n, k):
    rng = np.random.default_rng(k)
    a, sa = operand(rng, m, k)
    b, sb = operand(rng, n, k)
    want = S.mxfp4_gemm(*dev(a, sa, b, sb))
    a[1, :16] = 0
    sa[1, 0], sa[m - 1, -1], sb[n - 2, 1] = 255, 255, 255
    got = S.mxfp4_gemm(*dev(a, sa, b, sb))
    hit = torch.zeros(m, n, dtype=torch.bool, device=DEV)
    hit[1], hit[m - 1], hit[:, n - 2] = True, True, True
    assert got[hit].isnan().all() and torch.equal(got[~hit], want[~hit])


def test_signed_zeros_and_no_reduction():
    z = torch.zeros(4, 0, dtype=torch.uint8, device=DEV)
    w = torch.zeros(7, 0, dtype=torch.uint8, device=DEV)
    bias = torch.arange(7, dtype=torch.float32, device=DEV)
    assert torch.equal(S.mxfp4_gemm(z, z, w, w, bias=bias), bias.expand(4, 7))
    assert torch.equal(S.mxfp4_gemm(z, z, w, w), torch.zeros(4, 7, device=DEV))
    assert S.mxfp4_gemm(z[:0], z[:0], w, w).shape == (0, 7)
    a = torch.full((3, 64), 0x88, dtype=torch.uint8, device=DEV)          # -0 everywhere
    s = torch.full((3, 4), 127, dtype=torch.uint8, device=DEV)
    assert torch.equal(S.mxfp4_gemm(a, s, a, s), torch.zeros(3, 3, device=DEV))


def test_repeats_give_the_same_bits():
    rng = np.random.default_rng(6)
    for m, n, k in ((1, 512, 4096), (60, 300, 2080), (400, 700, 1056), (4096, 4096, 2048)):
        ops = dev(*operand(rng, m, k), *operand(rng, n, k))
        first = S.mxfp4_gemm(*ops)
        assert all(torch.equal(first, S.mxfp4_gemm(*ops)) for _ in range(3))


def test_refusals():
    c, s = torch.zeros(4, 32, dtype=torch.uint8, device=DEV), torch.zeros(4, 2, dtype=torch.uint8, device=DEV)
    for bad in (lambda: S.mxfp4_gemm(c, s[:, :1], c, s), lambda: S.mxfp4_gemm(c, s, c.cpu(), s),
                lambda: S.mxfp4_gemm(c, s, c, s, out=torch.empty(4, 5, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    wide = torch.zeros(4, 40, dtype=torch.uint8, device=DEV)
    with pytest.raises(S.Sparq24Error):                                   # rows 40 bytes apart
        S.mxfp4_gemm(wide[:, :32], s, c, s)


def test_offsets_past_32_bits():
    # operand, and rows 8 MiB apart (where the tiles' 32-bit offsets end)
    rng = np.random.default_rng(41)
    m, n, k = 70000, 40, 131072
    b, sb = operand(rng, n, k)
    tail, stail = operand(rng, 5, k)
    a = torch.zeros(m, k // 2, dtype=torch.uint8, device=DEV)
    sa = torch.full((m, k // 32), 127, dtype=torch.uint8, device=DEV)
    a[-5:], sa[-5:] = dev(tail, stail)
    db, dsb = dev(b, sb)
    got = S.mxfp4_gemm(a, sa, db, dsb)
    assert not got[:-5].any()
    check(got[-5:], tail, stail, b, sb, None, "f32")
    rows = a.view(-1).as_strided((37, k // 2), (1 << 23, 1))
    few, sfew = operand(rng, 37, k)
    rows.copy_(dev(few)[0])
    check(S.mxfp4_gemm(rows, dev(sfew)[0], db, dsb), few, sfew, b, sb, None, "f32")
    check(S.mxfp4_gemm(db, dsb, rows, dev(sfew)[0]), b, sb, few, sfew, None, "f32")


def test_an_output_past_32_bits():
    rng = np.random.default_rng(42)
    m, n, k = 40000, 70000, 32
    a, sa = operand(rng, m, k)
    b, sb = operand(rng, n, k)
    got = S.mxfp4_gemm(*dev(a, sa, b, sb), dtype=torch.bfloat16)
    for at in (slice(0, 3), slice(m - 3, m)):
        check(got[at], a[at], sa[at], b, sb, None, "bf16")


def test_streams_at_once_and_a_captured_product():
    # few rows, tiles, tiles in turn: on two side streams at once, then replayed on new operands
    rng = np.random.default_rng(43)
    ops = [dev(*operand(rng, m, k, 122, 128), *operand(rng, n, k, 122, 128))
           for m, n, k in ((48, 4000, 1056), (700, 900, 512), (300, 66000, 512))]
    want = [S.mxfp4_gemm(*o) for o in ops]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(3):
        for s, out in zip(streams, got):
            with torch.cuda.stream(s):
                out.append([S.mxfp4_gemm(*o) for o in ops])
    torch.cuda.synchronize()
    for outs in got:
        assert all(torch.equal(w, y) for ys in outs for w, y in zip(want, ys))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ys = [S.mxfp4_gemm(*o) for o in ops]
    for step in range(3):
        for o in ops:
            o[0].copy_(o[0].roll(step + 1, 0))
        eager = [S.mxfp4_gemm(*o) for o in ops]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, e) for y, e in zip(ys, eager))
