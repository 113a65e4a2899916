"""Host-side checks of the 8-bit product's calls; no GPU is used."""
import ctypes

import numpy as np

import ternary_weight_a8_b200 as tb


def test_refusals_come_before_any_pointer():
    L = tb.lib()
    raw = lambda N, K, M, xt, yt: L.bitlinear_forward_i8(None, None, N, K, None, xt, M, None, yt, None, None, 0, None)
    codes = lambda N, K, M, yt: L.bitlinear_forward_i8_quantized(None, None, N, K, None, None, M, None, yt, None, None, 0,
                                                                 None)
    assert raw(8, 64, 1, 7, 0) == tb.BL_ERR_INVALID_ARG
    assert raw(8, 64, 1, 0, 7) == tb.BL_ERR_INVALID_ARG and codes(8, 64, 1, 7) == tb.BL_ERR_INVALID_ARG
    for call in (lambda N, K, M: raw(N, K, M, 0, 0), lambda N, K, M: codes(N, K, M, 0)):
        assert call(0, 64, 1) == tb.BL_ERR_UNSUPPORTED_SHAPE
        assert call((1 << 24) + 1, 64, 1) == tb.BL_ERR_UNSUPPORTED_SHAPE
        assert call(8, 32, 1) == tb.BL_ERR_UNSUPPORTED_SHAPE and call(8, 100, 1) == tb.BL_ERR_UNSUPPORTED_SHAPE
        assert call(8, 131072, 1) == tb.BL_ERR_UNSUPPORTED_SHAPE and "131008" in tb.last_error()
        assert call(8, 64, -1) == tb.BL_ERR_INVALID_ARG
        assert call(8, 64, 0) == tb.BL_OK
        assert call(8, 64, 1) == tb.BL_ERR_INVALID_ARG and "wq is NULL" in tb.last_error()
        assert L.bitlinear_set_path(tb.PATH_GEMV) == tb.BL_OK
        try:
            assert call(8, 64, 33) == tb.BL_ERR_UNSUPPORTED_SHAPE and "GEMV" in tb.last_error()
        finally:
            assert L.bitlinear_set_path(tb.PATH_AUTO) == tb.BL_OK


def test_workspace_holds_the_codes():
    for M, K in ((1, 64), (47, 2560), (2048, 8640)):
        pitch = (K + 127) // 128 * 128
        up = lambda v: (v + 255) // 256 * 256
        assert tb.i8_workspace_bytes(M, 12345, K) == 256 + up(M * pitch) + 2 * up(4 * M)


def test_largest_sums_fit_int32():
    assert 128 * 128 * 131008 < 2 ** 31 <= 128 * 128 * 131072


def test_five_roundings_bound_the_output():
    """fp32(acc) * ((1 / s) * (1 / ws)) is within 5 * 2^-24 (1 + 2^-20) of acc / (s ws)."""
    rng = np.random.RandomState(0)
    acc = rng.randint(-(2 ** 31), 2 ** 31, 200000)
    s, ws = (np.exp(rng.uniform(-10, 10, 200000)).astype(np.float32) for _ in range(2))
    y = acc.astype(np.float32) * ((np.float32(1) / s) * (np.float32(1) / ws))
    real = acc / (s.astype(np.float64) * ws.astype(np.float64))
    assert (np.abs(y - real) <= 5 * 2.0 ** -24 * (1 + 2.0 ** -20) * np.abs(real)).all()
