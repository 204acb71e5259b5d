"""Bounds of cache attention's outputs, for tests of the kernels against the
oracle in 64 bits; P = sum_t p_t |V_t| / sum_t p_t, all errors relative to it
unless said otherwise:

* a score is off by the fp32 sum of D exact products and by its fp32 scaling:
  (D + 8) 2^-24 of scale * sum_d |q_d K_td|;
* its exponent, in units of log2, holds the score, log2 of a block's V scale and
  the reference, each below 2^b, with three roundings and an instruction of one
  unit in the last place: 2.5 2^(b - 23), so 2^(b - 22) of the weight (ln 2 < 1);
* a weight is rounded to fp16, 2^-11; below 2^-14, where the largest stands at
  2^8 at least, by 2^-25: 2^-33 of the largest |V| for each token;
* the fp32 sums over the tokens: len * 2^-23, in numerator and sum;
* the output's rounding: half a step of its type, and 2^-24 absolute (of fp16's
  subnormals).
An error of the weights counts twice, in the numerator and in the sum."""
import numpy as np

import oracle.serving as V


def bounds(ref, lens, fmt, dim, spread, reach, out, half_step, bits=3, n=None):
    """(bound of an output, bound of a log-sum's own part): see above; ``bits`` is b."""
    n = n or max(max(lens), 1)
    vmax = float(ref[3].max()) * (127 if fmt == "int8" else 448)
    ds = (dim + 8) * 2.0 ** -24 * reach + 2.0 ** (bits - 22)
    tol = (spread * (2.0 ** -11 + 2 * ds[..., None] + 2 * n * 2.0 ** -23) + n * 2.0 ** -33 * vmax
           + np.abs(out) * half_step + 2.0 ** -24)
    return tol, ds + n * 2.0 ** -23


def check_attention(got, lse, ref, table, lens, cu, q64, fmt, scale, half_step, bits=3, **kw):
    """Outputs and log-sums (tensors) of a call against the oracle; NaN fails."""
    out, want, spread, reach = V.kv_attention(q64, ref, table, lens, cu, fmt, scale, **kw)
    tol, own = bounds(ref, lens, fmt, q64.shape[-1], spread, reach, out, half_step, bits)
    got = got.cpu().double().numpy().reshape(out.shape)
    ok = np.abs(got - out) <= tol
    assert ok.all(), f"{(~ok).sum()} of {ok.size} outputs outside; worst {np.nanmax(np.abs(got - out) / tol):.3g}"
    if lse is not None:
        l64 = lse.cpu().double().numpy().reshape(want.shape)
        none = np.isneginf(want)
        assert np.array_equal(none, np.isneginf(l64))
        with np.errstate(invalid="ignore"):
            ok = np.abs(l64 - want) <= own + 2.0 ** -21 * np.abs(want)
        assert ok[~none].all(), f"{(~ok[~none]).sum()} log-sums outside"
