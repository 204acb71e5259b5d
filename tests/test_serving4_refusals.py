"""Refusals of the 4-bit serving calls that hold on the host."""
import ctypes

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
