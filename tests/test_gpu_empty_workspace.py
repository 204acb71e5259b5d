"""An empty workspace tensor has a null address, which the C calls take for a
query of the size: a call with one runs where it needs none and is refused
where it needs one, with the outputs as they were."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU, skipped there
    pytest.skip("no GPU", allow_module_level=True)

import pruning_quantization_amd as S  # noqa: E402
from gpu_util import DEV  # noqa: E402


def test_empty_workspace():
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = torch.randn(64, 512, generator=g, device=DEV, dtype=torch.bfloat16)
    empty = torch.empty(0, dtype=torch.uint8, device=DEV)
    rotated = torch.full_like(x, 7.0)
    S.hadamard(x, 64, out=rotated, workspace=empty)          # needs none
    assert torch.equal(rotated, S.hadamard(x, 64))
    codes, scales = S.quantize(x, "fp8", workspace=empty)
    want = S.quantize(x, "fp8")
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])
    for call, shape in ((lambda o: S.predict_R(x, ["fp8"], [("int", 8)], out=o, workspace=empty), (1, 1, 5)),
                        (lambda o: S.operator_error(x, x, [("2:4", "fp8")], out=o, workspace=empty), (64, 2))):
        out = torch.full(shape, 7.0, dtype=torch.float64, device=DEV)
        with pytest.raises(S.Sparq24Error, match="workspace"):
            call(out)
        assert (out == 7).all()
    norms = torch.full((512,), 7.0, device=DEV)
    with pytest.raises(S.Sparq24Error, match="workspace"):
        S.col_l2norm(x, out=norms, workspace=empty)
    assert (norms == 7).all()
