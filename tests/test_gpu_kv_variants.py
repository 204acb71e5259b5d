"""Every variant of the attention kernels (head dim, blocks below and from 64 tokens
on, code type, whole and split sequences; prompt rows, few rows and the join in
one call) against the oracle in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU, skipped there
    pytest.skip("no GPU", allow_module_level=True)

import pruning_quantization_amd as S  # noqa: E402
from kv_check import check_attention  # noqa: E402
from test_gpu_kv import Pool, offsets, stored  # noqa: E402

HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.mark.parametrize("kw", [{}, {"window": 37}, {"causal": False}], ids=str)
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("tokens", [16, 32, 64, 256])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_every_variant(dim, tokens, fmt, wide, kw):
    # a prompt, chunks behind a context, single tokens, nothing; three heads to a kv head
    lens, news = [130, 1400 if wide else 400, 77, 9, 64, 300, 1], [130, 90, 1, 0, 64, 2, 1]
    dtype = "bf16" if (dim + tokens) // 64 % 2 else "f16"
    p = Pool(dim + tokens, lens, 2, dim, tokens, fmt, wide=wide)
    cu, dcu = offsets(news)
    q, q64 = stored(p.rng.standard_normal((cu[-1], 6, dim)), dtype)
    out, lse = S.kv_attention(q, p.dev(), *p.args(), cu_tokens=dcu, return_lse=True, **kw)
    # log2 of scales, scores and references below 2^4
    check_attention(out, lse, p.ref, p.table, lens, cu, q64, fmt, dim ** -0.5, HALF[dtype], bits=4, **kw)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("tokens", [16, 64])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("n", [1, 5, 43])
def test_every_variant_same_count(n, dim, tokens, fmt, wide):
    lens = [n, n + 1, n + 63, n + (1300 if wide else 200), 64]
    if n > 1:
        lens[-1] = 2 * n
    p = Pool(n + dim, lens, 1, dim, tokens, fmt, wide=wide)
    q, q64 = stored(p.rng.standard_normal((5, n, 3, dim)), "bf16")
    out, lse = S.kv_attention(q, p.dev(), *p.args(), return_lse=True)
    check_attention(out, lse, p.ref, p.table, lens, np.arange(6) * n, q64.reshape(5 * n, 3, dim), fmt, dim ** -0.5,
                    HALF["bf16"], bits=4)
