"""Refusals of the 4-bit serving calls that hold on the host."""
import ctypes
import random

import pytest

import pruning_quantization_amd as S
import pruning_quantization_amd.binding as B

torch = pytest.importorskip("torch")


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


# scales whose bytes are as many as needed, but do not lie as the codes' rows
@pytest.mark.parametrize("codes,scales", [
    ((4, 32), (2, 4)), ((4, 32), (8,)), ((4, 32), (1, 8)), ((4, 32), (4, 2, 1)), ((4, 32), (2, 2, 2)),
    ((2, 3, 32), (3, 2, 2)), ((2, 3, 32), (2, 2, 3)), ((2, 3, 32), (2, 6)), ((2, 3, 32), (12,)),
    ((32,), (1, 1, 2)), ((32,), (2, 1)), ((4, 0), (0,)), ((0, 32), (0, 3))])
def test_product_scales_that_do_not_lie_as_their_codes(codes, scales):
    w, ws = u8(5, codes[-1]), u8(5, codes[-1] // 16)
    with pytest.raises(ValueError, match="scale_a must be"):
        S.mxfp4_gemm(u8(*codes), u8(*scales), w, ws)
    if len(codes) == 2:
        with pytest.raises(ValueError, match="scale_b must be"):
            S.mxfp4_gemm(w, ws, u8(*codes), u8(*scales))


@pytest.mark.parametrize("codes,scales", [
    ((4, 32), (4, 2)), ((2, 3, 32), (2, 3, 2)), ((2, 3, 32), (6, 2)), ((32,), (2,)), ((32,), (1, 2)),
    ((1, 32), (1, 2)), ((0, 32), (0, 2)), ((4, 0), (4, 0)), ((2, 0, 32), (2, 0, 2))])
def test_product_scales_that_do(codes, scales):
    w, ws = u8(5, codes[-1]), u8(5, codes[-1] // 16)
    with pytest.raises(ValueError, match="on a GPU"):
        S.mxfp4_gemm(u8(*codes), u8(*scales), w, ws)


# --- the norm at the C interface ---------------------------------------------

FAKE = 0x7F0000000000
OK, INVALID, UNSUPPORTED, SHAPE, ALIGN, WORKSPACE, DEVICE = 0, 1, 2, 3, 4, 5, 6


def rows(dtype=B.BF16, batch=1, rows=4, k=64, bs=None, rs=None, data=FAKE):
    rs = k if rs is None else rs
    return B.CTensor(data, dtype, batch, rows, k, rows * rs if bs is None else bs, rs, 1)


def norm(x, res=None, total=None, fmt=B.Q_FP8):
    ref = lambda t: ctypes.byref(t) if t is not None else None  # noqa: E731
    q = B.CQSpec(fmt, 0, None)
    return B.lib().sparq24_rmsnorm_quantize(ref(x), ref(res), FAKE, B.F32, 1e-6, ctypes.byref(q), FAKE, FAKE,
                                            ref(total), None)


@pytest.fixture()
def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")


def test_norm_of_many_batches(no_gpu):
    heads = dict(batch=70000, rows=4, bs=640)          # heads of a fused projection, token by token
    assert norm(rows(**heads)) == DEVICE
    assert norm(rows(**heads), rows(batch=70000), rows(**heads)) == DEVICE
    assert norm(rows(batch=70000, rows=1, bs=640)) == DEVICE
    assert norm(rows(batch=1 << 30, rows=4, bs=640)) == UNSUPPORTED


# --- the product's grid --------------------------------------------------------


def gemm(m, n, k, lda=None, ldb=None):
    return B.lib().sparq24_mxfp4_gemm(FAKE, lda or k // 2, FAKE, m, FAKE, ldb or k // 2, FAKE, n, k, None, 0, FAKE, n,
                                      None, None, None)


def test_product_that_no_grid_holds():
    # four threads a column in tiles, eight in the streaming kernel of rows far apart, 2^32 - 1 in a grid
    assert gemm(1, 2 ** 31 - 1, 32) == gemm(2 ** 31 - 1, 1, 32) == UNSUPPORTED
    assert gemm(1, 2 ** 30 + 1, 64) == gemm(2, 2 ** 29 + 1, 64, lda=1 << 23) == UNSUPPORTED


def test_product_that_a_grid_holds(no_gpu):
    most = 2 ** 28
    for m, n in ((1, most), (most, 1), (31, most), (64, most), (most, 17), (65, (1 << 34) // 65), (1 << 17, 1 << 17)):
        for kw in ({}, {"lda": 1 << 23}, {"ldb": 1 << 23}):
            for k in (32, 512, 1056):
                assert gemm(m, n, k, **kw) == DEVICE, (m, n, kw, k)


# --- a sum that meets the norm's inputs ------------------------------------------


def test_sum_that_meets_its_inputs():
    far = FAKE + (1 << 40)
    for dtype, es in ((B.BF16, 2), (B.F32, 4)):
        r = lambda at, **kw: rows(dtype=dtype, data=at, **kw)  # noqa: E731,B023
        for kw in ({}, {"rs": 160}, {"batch": 3, "rs": 160, "bs": 1024}, {"batch": 3, "rows": 1, "bs": 640},
                   {"rows": 1}):
            for d in (16, 64 * es - 16, -16, 16 - 64 * es):
                assert norm(r(FAKE, **kw), r(far, **kw), r(FAKE + d, **kw)) == UNSUPPORTED, (kw, d)
                assert norm(r(far, **kw), r(FAKE, **kw), r(FAKE + d, **kw)) == UNSUPPORTED, (kw, d)
        strided = {"batch": 3, "rs": 160, "bs": 1024}
        for d in (160, -320, 1024, 1024 - 160, 2048 + 3 * 160 + 32, -1024 - 48):      # whole rows and batches on
            assert norm(r(FAKE, **strided), r(far, **strided), r(FAKE + d * es, **strided)) == UNSUPPORTED, d
        assert norm(r(FAKE), r(far), r(FAKE + 64 * es)) == UNSUPPORTED                # dense rows, one on


def test_sum_beside_its_inputs(no_gpu):
    far = FAKE + (1 << 40)
    for dtype, es in ((B.BF16, 2), (B.F32, 4)):
        r = lambda at, **kw: rows(dtype=dtype, data=at, **kw)  # noqa: E731,B023
        strided = {"batch": 3, "rs": 160, "bs": 1024}
        # the same rows; columns beside them, behind the last row, in between batches
        for d in (0, 64, 96, -64, -96, 640, 608, 1024 - 64, 2048 + 4 * 160, -2048 - 640, 1 << 30):
            assert norm(r(FAKE, **strided), r(far, **strided), r(FAKE + d * es, **strided)) == DEVICE, d
            assert norm(r(far, **strided), r(FAKE, **strided), r(FAKE + d * es, **strided)) == DEVICE, d
        assert norm(r(FAKE), r(far), r(FAKE + 256 * es)) == norm(r(FAKE), r(FAKE), r(FAKE)) == DEVICE
        assert norm(r(FAKE, rs=128), r(far, rs=128), r(FAKE + 64 * es, rs=128)) == DEVICE


def test_sum_at_any_place(no_gpu):
    rng = random.Random(5)
    for _ in range(400):
        g = dict(k=rng.choice((8, 16, 40)), batch=rng.randint(1, 4), rows=rng.randint(1, 4))
        g["rs"] = g["k"] + 8 * rng.randint(0, 4)
        g["bs"] = (g["rows"] - 1) * g["rs"] + g["k"] + 8 * rng.randint(0, 12)
        d = 8 * rng.randint(-60, 60)
        at = {b * g["bs"] + r * g["rs"] for b in range(g["batch"]) for r in range(g["rows"])}
        meet = d != 0 and any(abs(y + d - x) < g["k"] for x in at for y in at)
        got = norm(rows(**g), rows(**{**g, "data": FAKE + (1 << 40)}), rows(**{**g, "data": FAKE + 2 * d}))
        assert got == (UNSUPPORTED if meet else DEVICE), (g, d)
