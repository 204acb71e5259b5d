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
