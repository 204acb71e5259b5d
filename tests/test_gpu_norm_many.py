"""The norm of very many rows, against itself on the same rows in parts: a row's codes
depend on that row alone."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU, skipped there
    pytest.skip("no GPU", allow_module_level=True)

import pruning_quantization_amd as S  # noqa: E402
from gpu_util import DEV  # noqa: E402

Q = ["mxfp4", "fp8", ("int", 8)]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


# heads of a fused projection: batches that do not lie back to back, more than 65535 of them
@pytest.mark.parametrize("heads", [1, 3])
@pytest.mark.parametrize("q", Q, ids=str)
def test_heads_of_many_tokens(q, heads):
    tokens, dim = 70001, 64
    x = torch.randn(tokens, heads + 2, dim, device=DEV).half()
    res = torch.randn(tokens, heads, dim, device=DEV).half()
    w = torch.randn(dim, device=DEV)
    into = torch.full_like(x, 7.0)
    part = x[:, 1:1 + heads]
    got = S.rmsnorm_quantize(part, w, q, residual=res, residual_out=into[:, 1:1 + heads])
    want = S.rmsnorm_quantize(part.contiguous(), w, q, residual=res)
    assert same(want, got)
    assert (into[:, 0] == 7).all() and (into[:, 1 + heads:] == 7).all()


# a grid holds 2^32 - 1 threads along x, a row takes 64 of them (2^26 rows), past 1024 elements 256 (2^24)
@pytest.mark.parametrize("rows,k,q", [((1 << 26) + 5, 8, "fp8"), ((1 << 26) + 1, 32, "mxfp4"),
                                      (3 * (1 << 26) + 7, 8, ("int", 8)), ((1 << 24) + 3, 1056, "mxfp4")], ids=str)
def test_more_workgroups_than_a_grid_has_along_x(rows, k, q):
    x = torch.randn(1 << 16, k, device=DEV).bfloat16()
    x = x.repeat(-(-rows // (1 << 16)), 1)[:rows]
    x[-1], x[1 << 24] = 3.0, 5.0
    w = torch.randn(k, device=DEV)
    codes, scales = S.rmsnorm_quantize(x, w, q)
    step = 1 << 22                                     # whole copies of the 65536 rows
    first = S.rmsnorm_quantize(x[:step], w, q)
    for at in range(0, rows, step):
        end = min(at + step, rows)
        if at == 1 << 24 or end == rows:
            want = S.rmsnorm_quantize(x[at:end], w, q)
        else:
            want = first
        assert torch.equal(codes[at:end].view(torch.uint8), want[0].view(torch.uint8)), at
        assert torch.equal(scales[at:end].view(torch.uint8), want[1].view(torch.uint8)), at
