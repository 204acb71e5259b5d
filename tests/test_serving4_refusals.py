"""Refusals of the 4-bit serving calls that hold on the host."""
import pytest

import pruning_quantization_amd as S

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
