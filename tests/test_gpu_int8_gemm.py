"""GPU parity of the INT8 product: integer sums are exact, so every output must
equal the oracle's fp32 steps bit for bit (then one rounding to the output
type)."""
import numpy as np
import pytest

import oracle as O
import oracle.serving as V

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU, skipped there
    pytest.skip("no GPU", allow_module_level=True)

import pruning_quantization_amd as S  # noqa: E402
import workloads as W  # noqa: E402
from gpu_util import DEV, to_dev  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def operands(seed, m, n, k):
    rng = np.random.default_rng(seed)
    a = rng.integers(-128, 128, (m, k)).astype(np.int8)
    b = rng.integers(-128, 128, (n, k)).astype(np.int8)
    return (a, (rng.random(m) + 0.1).astype(np.float32) * 1e-2, b,
            (rng.random(n) + 0.1).astype(np.float32) * 1e-3, rng.standard_normal(n).astype(np.float32))


def dev(*xs):
    return [None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(DEV) for x in xs]


def same(got, want32, dtype):
    want = torch.from_numpy(want32).to(DT[dtype])
    got = got.cpu().reshape(want.shape)
    assert got.dtype == want.dtype
    bad = (got != want) & ~(got.isnan() & want.isnan())
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outputs differ"


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,n,k,bias", [
    (1, 1, 16, False), (1, 64, 4096, True), (16, 16, 64, False), (17, 33, 80, True), (2, 129, 2064, False),
    (31, 31, 48, True), (32, 4096, 128, False), (33, 65, 1040, True), (48, 200, 4096, True), (64, 63, 272, False),
    (65, 64, 256, True), (127, 129, 144, False), (128, 256, 512, True), (200, 1031, 2064, True),
    (256, 256, 128, False), (257, 255, 384, True), (513, 777, 1024, False), (300, 2, 4112, True),
    (1000, 530, 64, False), (3, 20000, 96, True)])
def test_parity(m, n, k, bias, dtype):
    a, sa, b, sb, bi = operands(m * 7 + n + k, m, n, k)
    bi = bi if bias else None
    da, dsa, db, dsb, dbi = dev(a, sa, b, sb, bi)
    same(S.int8_gemm(da, dsa, db, dsb, bias=dbi, dtype=DT[dtype]), V.int8_gemm(a, sa, b, sb, bi), dtype)


@pytest.mark.parametrize("m", [1, 20, 64, 70, 300])
def test_extreme_codes_and_depth(m):
    # the largest sums: every product (-128)^2, and the deepest K
    k, n = 131056, 17
    a, b = np.full((m, k), -128, np.int8), np.full((n, k), -128, np.int8)
    b[1::2] = 127
    sa, sb = np.ones(m, np.float32), np.ones(n, np.float32)
    same(S.int8_gemm(*dev(a, sa, b, sb)), V.int8_gemm(a, sa, b, sb), "f32")


@pytest.mark.parametrize("m", [1, 40, 100, 400])
def test_strided_rows_and_out(m):
    n, k = 150, 112
    a, sa, b, sb, bi = operands(m, m, n, k)
    da, dsa, db, dsb, dbi = dev(a, sa, b, sb, bi)
    wa = torch.full((m, k + 32), 77, dtype=torch.int8, device=DEV)
    wb = torch.full((n, k + 48), 77, dtype=torch.int8, device=DEV)
    wa[:, :k], wb[:, :k] = da, db
    wide = torch.full((m, n + 9), 5.0, device=DEV)
    S.int8_gemm(wa[:, :k], dsa, wb[:, :k], dsb, bias=dbi, out=wide[:, :n])
    same(wide[:, :n].contiguous(), V.int8_gemm(a, sa, b, sb, bi), "f32")
    assert (wide[:, n:] == 5.0).all(), "wrote outside its columns"


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m", [3, 60, 300])
def test_out_rows_at_any_element(m, dtype):
    # rows of the output that begin at odd elements, in both kernels
    n, k = 1100, 96
    a, sa, b, sb, bi = operands(m + 1, m, n, k)
    wide = torch.full((m, n + 7), 5.0, dtype=DT[dtype], device=DEV)
    da, dsa, db, dsb, dbi = dev(a, sa, b, sb, bi)
    S.int8_gemm(da, dsa, db, dsb, bias=dbi, out=wide[:, :n])
    same(wide[:, :n].contiguous(), V.int8_gemm(a, sa, b, sb, bi), dtype)
    assert (wide[:, n:] == 5.0).all(), "wrote outside its columns"


def test_leading_dims_empty_and_zero_depth():
    a, sa, b, sb, bi = operands(3, 30, 20, 64)
    da, dsa, db, dsb, dbi = dev(a, sa, b, sb, bi)
    y = S.int8_gemm(da.view(2, 3, 5, 64), dsa.view(2, 3, 5), db, dsb, dtype=torch.bfloat16)
    assert y.shape == (2, 3, 5, 20)
    same(y, V.int8_gemm(a, sa, b, sb), "bf16")
    assert S.int8_gemm(da[:0], dsa[:0], db, dsb).shape == (0, 20)
    assert S.int8_gemm(da, dsa, db[:0], dsb[:0]).shape == (30, 0)
    for m in (1, 30):
        z = S.int8_gemm(da[:m, :0], dsa[:m], db[:, :0], dsb, bias=dbi)
        assert torch.equal(z, dbi.expand(m, 20))


def test_row_steps_of_views():
    # the step between rows is that of whichever leading dim has more than one entry
    a, sa, b, sb, _ = operands(4, 30, 20, 64)
    da, dsa, db, dsb = dev(a, sa, b, sb)
    want = V.int8_gemm(a, sa, b, sb)
    x = da.view(5, 6, 64)
    last = torch.from_numpy(want).view(5, 6, 20)[:, -1:]
    scale = dsa.view(5, 6)[:, -1].contiguous()
    got = S.int8_gemm(x[:, -1:], scale, db, dsb)                  # the last row of each sequence
    assert got.shape == (5, 1, 20) and torch.equal(got.cpu(), last)
    out = torch.full((5, 6, 20), 7.0, device=DEV)
    S.int8_gemm(x[:, -1:], scale, db, dsb, out=out[:, -1:])
    assert torch.equal(out[:, -1:].cpu(), last) and (out[:, :-1] == 7.0).all()
    got = S.int8_gemm(x[2, 3], dsa[15:16], db, dsb)                # one row, no leading dim
    assert got.shape == (20,) and torch.equal(got.cpu(), torch.from_numpy(want[15]))
    one = da[7:8].as_strided((1, 64), (3, 1))                      # one row: its stride says nothing
    same(S.int8_gemm(one, dsa[7:8], db, dsb), want[7:8], "f32")
    same(S.int8_gemm(da, dsa, db[3:4].as_strided((1, 64), (5, 1)), dsb[3:4]), want[:, 3:4], "f32")
    with pytest.raises(S.Sparq24Error):                            # one row's codes for all rows
        S.int8_gemm(da[:1].expand(30, 64), dsa, db, dsb)
    with pytest.raises(ValueError, match="evenly"):
        S.int8_gemm(x[:, 1:3], dsa[:10], db, dsb)


def test_nonfinite_scales_stay_in_their_row():
    for m in (5, 90):
        a, sa, b, sb, _ = operands(m, m, 40, 128)
        sa[1], sa[3], sb[2] = np.nan, np.inf, np.inf
        same(S.int8_gemm(*dev(a, sa, b, sb)), V.int8_gemm(a, sa, b, sb), "f32")


def test_after_quantize():
    # the INT8 side end to end: codes and scales of quantize(), its product here
    rng = np.random.default_rng(9)
    x, w = W.to_bf16_bits(rng.standard_normal((70, 512))), W.to_bf16_bits(rng.standard_normal((96, 512)) * 0.05)
    ca, sa = S.quantize(to_dev(x, "bf16"), ("int", 8))
    cb, sb = S.quantize(to_dev(w, "bf16"), ("int", 8))
    wa, wsa = O.quantize_rows(x, "bf16", O.QSpec("int", 8))
    wb, wsb = O.quantize_rows(w, "bf16", O.QSpec("int", 8))
    same(S.int8_gemm(ca, sa, cb, sb), V.int8_gemm(wa, wsa, wb, wsb), "f32")


def test_refusals():
    a, sa, b, sb, bi = dev(*operands(1, 8, 8, 64))
    with pytest.raises(TypeError):
        S.int8_gemm(a.view(torch.uint8), sa, b, sb)
    with pytest.raises(TypeError):
        S.int8_gemm(a, sa, b, sb, dtype=torch.float64)
    for bad in (lambda: S.int8_gemm(a, sa[:7], b, sb), lambda: S.int8_gemm(a, sa, b[:, :48], sb),
                lambda: S.int8_gemm(a, sa, b, sb.half()), lambda: S.int8_gemm(a, sa, b, sb, bias=bi[:3]),
                lambda: S.int8_gemm(a, sa, b, sb, out=torch.empty(8, 9, device=DEV)),
                lambda: S.int8_gemm(a.T, sa, b, sb), lambda: S.int8_gemm(a, sa.cpu(), b, sb)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(S.Sparq24Error):
        S.int8_gemm(a[:, :24], sa, b[:, :24], sb)
