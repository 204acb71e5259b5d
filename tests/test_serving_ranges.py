"""CPU pins of the serving oracle and the entry points at the ends of their ranges."""
import ctypes

import numpy as np
import pytest

import oracle.serving as V

B = pytest.importorskip("pruning_quantization_amd.binding")


def test_append_of_infinities_by_hand():
    # a block of one kept and two new tokens: the infinities are no maximum (254 is) and saturate
    cache = (np.full((1, 1, 16, 64), 5, np.int8), np.full((1, 1), 1.0, np.float32),
             np.full((1, 1, 64, 16), 5, np.int8), np.full((1, 1), 1.0, np.float32))
    x = np.zeros((2, 1, 64), np.float32)
    x[0, 0, :4] = (np.inf, -np.inf, np.nan, 254.0)
    x[1, 0, 0] = -20.0
    k, ks, v, vs = V.kv_append(cache, x, x, np.array([[0]], np.int32), [3], [0, 2], "int8")
    assert ks[0, 0] == 2.0 and vs[0, 0] == 2.0
    assert k[0, 0, :4, :4].tolist() == [[2, 2, 2, 2], [127, -127, 0, 127], [-10, 0, 0, 0], [5, 5, 5, 5]]
    assert v[0, 0, :4, 1].tolist() == [127, -127, 0, 127]
    # nothing finite: the kept codes stay, by their scale the infinities saturate
    x[:] = np.inf
    k, ks, _, _ = V.kv_append(cache, x, x, np.array([[0]], np.int32), [3], [0, 2], "int8")
    assert ks[0, 0] == 1.0 and (k[0, 0, 0] == 5).all() and (k[0, 0, 1:3] == 127).all()
    # a block of infinities alone has no scale to count them in
    k, ks, _, _ = V.kv_append(cache, x, x, np.array([[0]], np.int32), [2], [0, 2], "fp8")
    assert ks[0, 0] == 0.0 and not k[0, 0, :2].any()


def test_int8_gemm_of_no_codes_takes_any_strides():
    # K = 0 reads no code: the strides of torch.empty(30, 0) are (1, 1)
    fake, c = 0x7F0000000000, ctypes.c_size_t(0)
    try:
        L = B.lib()
    except ImportError as e:
        pytest.skip(str(e))
    for lda, ldb in ((0, 0), (1, 1), (64, 3)):
        st = L.sparq24_int8_gemm(None, lda, fake, 30, None, ldb, fake, 20, 0, None, 0, fake, 20, None,
                                 ctypes.byref(c), None)
        assert st == 0, (lda, ldb)
