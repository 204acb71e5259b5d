"""Calls of the cache that the documentation allows and no other test makes: the
output over the queries, sequences that share blocks, lengths past their table,
captured appends to the largest blocks."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU, skipped there
    pytest.skip("no GPU", allow_module_level=True)

import oracle.serving as V  # noqa: E402
import pruning_quantization_amd as S  # noqa: E402
from gpu_util import DEV  # noqa: E402
from kv_check import check_attention  # noqa: E402
from test_gpu_kv import Pool, offsets, stored, unchanged  # noqa: E402


@pytest.mark.parametrize("nan", [False, True])
@pytest.mark.parametrize("wide", [False, True])
def test_output_over_the_queries(wide, nan):
    # a query row is read by the workgroups of its own kv head only, before its output is stored; with NaN codes too
    lens, news = [150, 1300 if wide else 200, 40, 90], [90, 33, 1, 2]
    p = Pool(9, lens, 2, 64, 16, "fp8", wide=wide)
    if nan:
        for b, n in enumerate(lens):
            p.ref[2][p.table[b, (n - 1) // 16], :, 5, (n - 1) % 16] = 0x7F
    cu, dcu = offsets(news)
    q, _ = stored(p.rng.standard_normal((cu[-1], 6, 64)), "bf16")
    want = S.kv_attention(q, p.dev(), *p.args(), cu_tokens=dcu)
    assert want.isnan().any() == nan
    got = S.kv_attention(q, p.dev(), *p.args(), cu_tokens=dcu, out=q)
    assert got.data_ptr() == q.data_ptr()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("n", [1, 30])
def test_sequences_that_share_blocks(n):
    # a common prefix of three blocks, read by all; each appends to a block of its own
    lens = [48 + n, 48 + n, 48 + n]
    p = Pool(n, lens, 2, 64, 16, "int8")
    p.table[1:, :3] = p.table[0, :3]
    k, k64 = stored(p.rng.standard_normal((3, n, 2, 64)) * 2, "bf16")
    v, v64 = stored(p.rng.standard_normal((3, n, 2, 64)), "bf16")
    cu = np.arange(4) * n
    cache = p.dev()
    S.kv_append(cache, k, v, *p.args())
    ref = V.kv_append(p.ref, k64.reshape(-1, 2, 64), v64.reshape(-1, 2, 64), p.table, lens, cu, "int8")
    unchanged(cache, ref)
    q, q64 = stored(p.rng.standard_normal((3, n, 4, 64)), "bf16")
    out, lse = S.kv_attention(q, cache, *p.args(), return_lse=True)
    check_attention(out, lse, ref, p.table, lens, cu, q64.reshape(-1, 4, 64), "int8", 0.125, 2.0 ** -8, bits=4)


@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("tokens", [16, 64])
def test_lengths_past_the_table(tokens, n, window):
    # positions past a table hold no token; a window may lie behind it altogether
    width = 128 // tokens
    p = Pool(n + tokens, [128, 128, 100], 1, 64, tokens, "int8", width=width)
    p.lens = [150, 1000, 100]
    q, q64 = stored(p.rng.standard_normal((3, n, 3, 64)), "bf16")
    out, lse = S.kv_attention(q, p.dev(), *p.args(), return_lse=True, window=window)
    check_attention(out, lse, p.ref, p.table, p.lens, np.arange(4) * n, q64.reshape(-1, 3, 64), "int8", 0.125,
                    2.0 ** -8, bits=4, window=window)
    if window:
        assert not out[1].any() and torch.isneginf(lse[1]).all()


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_captured_append_to_the_largest_blocks(fmt):
    # more than 64 KiB of LDS a workgroup, asked for while a stream is captured
    tokens, dim = 256, 256
    p = Pool(3, [300, 700], 1, dim, tokens, fmt)
    k, k64 = stored(p.rng.standard_normal((2, 290, 1, dim)), "bf16")
    cache, args = p.dev(), p.args()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        S.kv_append(cache, k, k, *args)
    unchanged(cache, p.ref)
    for step in range(3):
        for t, x in zip(cache, p.dev()):
            t.copy_(x)
        k.mul_(-1.5)
        rows = k.double().cpu().numpy().reshape(-1, 1, dim)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        unchanged(cache, V.kv_append(p.ref, rows, rows, p.table, p.lens, [0, 290, 580], fmt))
