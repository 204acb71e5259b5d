"""The MXFP4 product's kernels for many rows, each at shapes that reach it: ragged edges,
every rest of K behind odd and even counts of slabs, padded rows, scales that are no
numbers or lie at the ends of the range.  Bounds: test_gpu_mxfp4_gemm.py."""
import numpy as np
import pytest

import oracle.serving4 as V

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU, skipped there
    pytest.skip("no GPU", allow_module_level=True)

import pruning_quantization_amd as S  # noqa: E402
from gpu_util import DEV  # noqa: E402
from test_gpu_mxfp4_gemm import DT, check, dev, operand  # noqa: E402

CUS = torch.cuda.get_device_properties(0).multi_processor_count


def kernel_of(m, n, k):
    """The kernel that a product of evenly spaced rows gets, by the library's rule."""
    def tiles(a, b):
        return -(-m // a) * -(-n // b)
    if min(-(-tiles(16 * i, 16 * j) // CUS) * (i + j) for i in (1, 2, 4) for j in (1, 2, 4)) <= 8:
        return "stream"
    if tiles(256, 256) >= CUS and k >= 512:
        return "wide" if k % 512 else "chained"
    if tiles(256, 128) >= CUS:
        return "256x128"
    return "128x128" if tiles(64, 64) > 4 * CUS else "64x64"


SHAPES = {"64x64": (1100, 1900), "128x128": (1500, 4000), "256x128": (2100, 4300), "wide": (4000, 4200),
          "chained": (4090, 4230)}


def reach(name, m, n, k):
    if CUS != 256:
        pytest.skip("the shapes are those of 256 CUs")
    assert kernel_of(m, n, k) == name


def product(rng, m, n, k, dtype="f32", bias=True, low=122, high=128):
    """Operands in padded rows, the product into a padded output, and both checked."""
    a, sa = operand(rng, m, k, low, high)
    b, sb = operand(rng, n, k, low, high)
    y = rng.standard_normal(n).astype(np.float32) if bias else None
    da, db = (torch.zeros(r, k // 2 + p, dtype=torch.uint8, device=DEV) for r, p in ((m, 48), (n, 80)))
    da[:, :k // 2], db[:, :k // 2] = dev(a, b)
    out = torch.full((m, n + 3), 7.0, dtype=DT[dtype], device=DEV)
    got = S.mxfp4_gemm(da[:, :k // 2], dev(sa)[0], db[:, :k // 2], dev(sb)[0], bias=dev(y)[0] if bias else None,
                       out=out[:, :n])
    check(got, a, sa, b, sb, y, dtype)
    assert (out[:, n:] == 7).all()


CASES = [(name, 256 * (slabs + rest % 3) + 32 * rest) for name, slabs in
         (("64x64", 1), ("128x128", 2), ("256x128", 1), ("wide", 2)) for rest in range(8)
         if name != "wide" or (256 * (slabs + rest % 3) + 32 * rest) % 512]
CASES += [("64x64", 224), ("128x128", 32), ("256x128", 160), ("chained", 512), ("chained", 1024), ("chained", 1536)]


@pytest.mark.parametrize("name,k", CASES)
def test_every_rest_of_k_in_padded_rows(name, k):
    m, n = SHAPES[name]
    reach(name, m, n, k)
    product(np.random.default_rng(k), m, n, k, ("f32", "bf16", "f16")[k // 32 % 3], bias=k // 32 % 2 == 0)


# few rows on more outputs than the streaming kernel takes
@pytest.mark.parametrize("name,m,n,k", [("64x64", 1, 28700, 544), ("64x64", 48, 16500, 4096), ("256x128", 8, 57345, 1056),
                                        ("256x128", 1, 128300, 480), ("wide", 3, 128300, 544),
                                        ("chained", 48, 128256, 512), ("chained", 1, 66001, 1024)])
def test_few_rows_on_many_outputs(name, m, n, k):
    reach(name, m, n, k)
    product(np.random.default_rng(n), m, n, k, "bf16" if m > 1 else "f32")


@pytest.mark.parametrize("name,k", [("64x64", 544), ("128x128", 1024), ("256x128", 800), ("wide", 1056),
                                    ("wide", 768), ("chained", 1024)])
def test_nan_scales_reach_their_row_and_column(name, k):
    m, n = SHAPES[name]
    reach(name, m, n, k)
    rng = np.random.default_rng(k)
    a, sa = operand(rng, m, k)
    b, sb = operand(rng, n, k)
    want = S.mxfp4_gemm(*dev(a, sa, b, sb))
    a[1, :16] = 0                                          # zeros of a NaN group count, too
    b[0, -16:] = 0
    groups = k // 32
    rows = {1: 0, m // 2: groups // 2, m - 1: groups - 1}  # one of the first, a middle and the last group
    cols = {0: groups - 1, n // 2 + 1: groups // 2 - 1, n - 1: 0}
    hit = torch.zeros(m, n, dtype=torch.bool, device=DEV)
    for r, g in rows.items():
        sa[r, g], hit[r] = 255, True
    for c, g in cols.items():
        sb[c, g], hit[:, c] = 255, True
    got = S.mxfp4_gemm(*dev(a, sa, b, sb))
    assert got[hit].isnan().all() and torch.equal(got[~hit], want[~hit])


@pytest.mark.parametrize("name,k", [("64x64", 544), ("128x128", 512), ("256x128", 800), ("wide", 1056), ("chained", 1024)])
def test_scales_at_the_ends_of_the_range(name, k):
    m, n = SHAPES[name]
    reach(name, m, n, k)
    rng = np.random.default_rng(k + 1)
    a, sa = operand(rng, m, k, 0, 255)
    b, sb = operand(rng, n, k)
    sa[:] = sa[:1]
    sb = (254 - sa[:1].astype(int) + rng.integers(-3, 4, sb.shape)).clip(0, 254).astype(np.uint8)
    check(S.mxfp4_gemm(*dev(a, sa, b, sb)), a, sa, b, sb, None, "f32")   # every product near 1
    sa[:], sb[:] = 254, 254                                              # past fp32
    got = S.mxfp4_gemm(*dev(a, sa, b, sb)).cpu().numpy()
    want, _ = V.mxfp4_gemm(a, sa, b, sb)
    assert (np.isinf(got) | np.isnan(got) | (want == 0)).all()


def test_tiles_on_streams_at_once_and_captured():
    rng = np.random.default_rng(9)
    ks = {"64x64": 544, "128x128": 512, "256x128": 288, "wide": 800, "chained": 512}
    ops = []
    for name, (m, n) in SHAPES.items():
        reach(name, m, n, ks[name])
        ops.append(dev(*operand(rng, m, ks[name], 122, 128), *operand(rng, n, ks[name], 122, 128)))
    want = [S.mxfp4_gemm(*o) for o in ops]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append([S.mxfp4_gemm(*o) for o in ops])
    torch.cuda.synchronize()
    assert all(torch.equal(w, y) for ys in got for w, y in zip(want, ys))
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
