"""Attention over the MXFP4 cache: V and the softmax weights in the second product.

They enter it in fp16 for queries of either type, so a weight is off by 2^-11 of itself,
and below fp16's 2^-14, where the largest stands at 2^8 or more, by 2^-25: 2^-33 of the
largest |V| a token.  With bf16 queries it is bf16, 2^-8, where a V scale of a seen token lies
outside 2^-23 .. 2^8.  The other terms of a bound are those of test_gpu_kv4.py: with P =
sum_t p_t |V_t| / sum_t p_t, a score's error twice (numerator and sum), the fp32 sums over
the tokens, and half a step of the output."""
import numpy as np
import pytest

import oracle.serving4 as V

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU, skipped there
    pytest.skip("no GPU", allow_module_level=True)

import pruning_quantization_amd as S  # noqa: E402
from gpu_util import DEV  # noqa: E402
from test_gpu_kv4 import DT, Pool, offsets, stored  # noqa: E402

# new tokens per sequence of the few-rows kernel with one and two row tiles a wave, and of the prompt kernel;
# query heads per kv head
KERNELS = {"few": (1, 3), "two row tiles": (5, 5), "prompt": (70, 2)}


def check(p, n, group, dtype, weight, scale=None, lens=None, **kw):
    """The attention of the last n tokens of each sequence within bounds for weights off by `weight`."""
    scale = np.float32(scale or p.dim ** -0.5)
    q, q64 = stored(p.rng.standard_normal((len(p.lens) * n, p.kv * group, p.dim)), dtype)
    cu, dcu = offsets([n] * len(p.lens))
    got = S.kv_attention(q.view(len(p.lens), n, p.kv * group, p.dim), p.dev(), *p.args(), scale=float(scale), **kw)
    assert torch.equal(got.flatten(0, 1), S.kv_attention(q, p.dev(), *p.args(), cu_tokens=dcu, scale=float(scale), **kw))
    out, _, spread, reach = V.kv_attention(q64, p.ref, p.table, p.lens, cu, float(scale), **kw)
    seen = max(max(p.lens), 1)
    vmax = 6 * 2.0 ** (float(p.ref[3][p.ref[3] < 255].max()) - 127)
    ds = (p.dim + 8) * 2.0 ** -24 * reach + 2.0 ** -18
    tol = (spread * (weight + 2 * ds[..., None] + 2 * min(seen, kw.get("window", seen)) * 2.0 ** -23)
           + (seen * 2.0 ** -33 * vmax if weight < 2.0 ** -10 else 0)
           + np.abs(out) * torch.finfo(DT[dtype]).eps / 2 + 2.0 ** -24)
    got = got.cpu().to(torch.float64).numpy().reshape(out.shape)
    ok = np.abs(got - out) <= tol
    assert ok.all(), f"{(~ok).sum()} of {ok.size} outside; worst {np.nanmax(np.abs(got - out) / tol):.3g}"


def lengths(n):
    return [max(n, 2) + i for i in (0, 5, 62, 300, 1100)]


@pytest.mark.parametrize("dim,tokens", [(64, 16), (64, 64), (128, 32), (128, 128), (192, 16), (192, 64), (256, 32), (256, 64)])
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_weights_of_two_tokens_whose_values_cancel(dtype, kernel, dim, tokens):
    # V is +1 and -1 in turn: out is the difference of two weights over their sum
    n, group = KERNELS[kernel]
    p = Pool(dim + n, lengths(n), 2, dim, tokens)
    odd = (np.arange(tokens) % 2).reshape(1, 1, tokens, 1)
    p.ref = (p.ref[0], p.ref[1] - 3, np.broadcast_to(np.where(odd, 0xAA, 0x22), p.ref[2].shape).astype(np.uint8),
             np.full_like(p.ref[3], 127))
    check(p, n, group, dtype, 2.0 ** -11, window=2)


@pytest.mark.parametrize("dim,tokens", [(64, 16), (128, 64), (192, 32), (256, 64)])
@pytest.mark.parametrize("kernel", KERNELS)
def test_scales_that_no_one_sees_change_nothing(kernel, dim, tokens):
    # V scales outside of fp16 behind the sequences, before the windows and of groups of zeros
    n, group = KERNELS[kernel]
    p = Pool(dim + n, lengths(n), 2, dim, tokens)
    k, ks, v, vs = (x.copy() for x in p.ref)
    far = p.rng.choice([0, 60, 103, 136, 200, 252, 254, 255], vs.shape).astype(np.uint8)
    hidden = np.ones((v.shape[0], tokens), bool)
    for b, length in enumerate(p.lens):
        for t in range(max(0, length - n - 9), length):
            hidden[p.table[b, t // tokens], t % tokens] = False
    hide = hidden[:, None, None, :]
    zero = p.rng.random(vs.shape) < 0.2                    # groups of zeros, with any scale but NaN
    vs = np.where(hide, far, np.where(zero, np.minimum(far, 252), vs)).astype(np.uint8)
    v = np.where(np.repeat(zero.transpose(0, 1, 3, 2), 16, -1) & ~hidden[:, None, :, None], 0x80, v).astype(np.uint8)
    p.ref = (k, ks, v & 0x80 | np.where(v == 0x80, 0, v), vs)
    want = S.kv_attention(torch.ones(len(p.lens), n, 2 * group, dim, dtype=torch.bfloat16, device=DEV), p.dev(), *p.args(),
                          window=10)
    assert not want.isnan().any()
    clean = p.ref
    q, q64 = stored(p.rng.standard_normal((len(p.lens) * n, 2 * group, dim)), "bf16")
    cu, _ = offsets([n] * len(p.lens))
    got = S.kv_attention(q.view(len(p.lens), n, 2 * group, dim), p.dev(), *p.args(), window=10)
    tame = (k, ks, clean[2], np.where(hide | zero, 124, vs).astype(np.uint8))
    same = S.kv_attention(q.view(len(p.lens), n, 2 * group, dim), p.dev(tame), *p.args(), window=10)
    assert torch.equal(got, same)


@pytest.mark.parametrize("dim,tokens", [(64, 16), (64, 64), (128, 32), (128, 64), (192, 16), (192, 128), (256, 32), (256, 64)])
@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("where", ["first", "middle", "last", "here and there", "everywhere"])
def test_scales_outside_of_fp16(where, kernel, dim, tokens):
    # one token or many with V scales of 2^-127 to 2^90 in some of their groups, among others
    n, group = KERNELS[kernel]
    p = Pool(dim + n, lengths(n), 2, dim, tokens)
    vs = p.ref[3]
    for b, length in enumerate(p.lens):
        at = {"first": [0], "middle": [length // 2], "last": [length - 1], "everywhere": range(length),
              "here and there": np.flatnonzero(p.rng.random(length) < 0.02)}[where]
        for t in at:
            g = p.rng.integers(0, dim // 32)
            vs[p.table[b, t // tokens], :, g, t % tokens] = p.rng.choice([0, 1, 40, 103, 136, 137, 140, 141, 150, 217])
    check(p, n, group, "bf16", 2.0 ** -8)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_scales_at_the_ends_of_fp16(dim, kernel):
    # 2^-23 and 2^8, the smallest and largest codes: exact
    n, group = KERNELS[kernel]
    for low in (104, 135):
        p = Pool(dim + n, lengths(n), 2, dim, 32)
        p.ref[3][:] = low
        p.ref[2][:] = p.rng.choice([0x11, 0x77, 0x17, 0x91, 0xF7], p.ref[2].shape)
        check(p, n, group, "bf16", 2.0 ** -11)
        p = Pool(dim + n, lengths(n), 2, dim, 64)
        p.ref[3][:] = p.rng.integers(104, 136, p.ref[3].shape)
        check(p, n, group, "bf16", 2.0 ** -11)


@pytest.mark.parametrize("kernel", KERNELS)
def test_nan_scales_among_scales_outside_of_fp16(kernel):
    # a NaN scale makes the rows that see it NaN and no others, on both sides of the change to bf16
    n, group = KERNELS[kernel]
    lens = [max(n, 2) + i for i in (150, 400)]
    p = Pool(n, lens, 2, 128, 64)
    for b, length in enumerate(lens):
        for t, e in ((70, 200), (length - 3, 10)):
            p.ref[3][p.table[b, t // 64], :, 1, t % 64] = e
    q, _ = stored(p.rng.standard_normal((2, n, 2 * group, 128)), "bf16")
    want = S.kv_attention(q, p.dev(), *p.args())
    assert not want.isnan().any()
    for t in (30, 100, lens[0] - 1):
        ref = tuple(x.copy() for x in p.ref)
        ref[3][p.table[0, t // 64], 1, 2, t % 64] = 255
        got = S.kv_attention(q, p.dev(ref), *p.args())
        sees = torch.arange(lens[0] - n, lens[0], device=DEV) >= t
        assert got[0, sees, group:].isnan().all()
        assert torch.equal(got[0, ~sees], want[0, ~sees]) and torch.equal(got[0, :, :group], want[0, :, :group])
        assert torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype,most", [("bf16", 252), ("f16", 140)])
@pytest.mark.parametrize("kernel", KERNELS)
def test_scales_above_the_types_range_count_as_its_largest(kernel, dtype, most):
    n, group = KERNELS[kernel]
    p = Pool(n, lengths(n), 2, 128, 32)
    k, ks, v, vs = p.ref
    high = p.rng.random(ks.shape) < 0.3
    ks = np.where(high, p.rng.integers(most, 255, ks.shape), most - 3).astype(np.uint8)
    q = p.rng.standard_normal((len(p.lens), n, 2 * group, 128)) * 2.0 ** (124 - most)
    q, _ = stored(np.where(np.abs(q) < 2.0 ** -24, 0, q) if dtype == "f16" else q, dtype)
    got = S.kv_attention(q, p.dev((k, ks, v, vs)), *p.args())
    assert got.isfinite().all() and got.any()
    assert torch.equal(got, S.kv_attention(q, p.dev((k, np.minimum(ks, most), v, vs)), *p.args()))
    vs = np.where(high, p.rng.integers(most, 255, vs.shape), vs).astype(np.uint8)
    got = S.kv_attention(q, p.dev((k, ks, v, vs)), *p.args())
    want = S.kv_attention(q, p.dev((k, ks, v, np.minimum(vs, most))), *p.args())
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))     # infinities and NaN alike
