"""Host-side checks of the residual norm's calls and of its gradient's formula; no GPU is used."""
import ctypes

import numpy as np
import pytest

import ternary_weight_a8_b200 as tb


def test_refusals_come_before_any_pointer():
    L = tb.lib()
    vp, f = ctypes.c_void_p, ctypes.c_float
    fwd = lambda dt, M, K, eps: L.bitlinear_add_rmsnorm_quant(None, None, dt, M, K, None, f(eps), None, None, None, None,
                                                              None, None)
    assert fwd(7, 1, 64, 1e-6) == tb.BL_ERR_INVALID_ARG
    assert fwd(0, -1, 64, 1e-6) == tb.BL_ERR_INVALID_ARG
    assert fwd(0, 1, 96, 1e-6) == tb.BL_ERR_UNSUPPORTED_SHAPE
    assert fwd(0, 1, 0, 1e-6) == tb.BL_ERR_UNSUPPORTED_SHAPE
    for eps in (-1.0, float("inf"), float("nan")):
        assert fwd(0, 1, 64, eps) == tb.BL_ERR_INVALID_ARG
    assert fwd(0, 1, 64, 1e-6) == tb.BL_ERR_INVALID_ARG and "x is NULL" in tb.last_error()
    assert fwd(0, 0, 64, 1e-6) == tb.BL_OK
    back = lambda zt, dt, M, K, eps, gain, dgain: L.bitlinear_add_rmsnorm_backward(
        None, zt, None, dt, M, K, gain, f(eps), None, None, dgain, None, 0, None)
    assert back(7, 0, 1, 64, 1e-6, None, None) == tb.BL_ERR_INVALID_ARG
    assert back(0, 7, 1, 64, 1e-6, None, None) == tb.BL_ERR_INVALID_ARG
    assert back(0, 0, -1, 64, 1e-6, None, None) == tb.BL_ERR_INVALID_ARG
    assert back(0, 0, 1, 100, 1e-6, None, None) == tb.BL_ERR_UNSUPPORTED_SHAPE
    assert back(0, 0, 1, 64, -1e-6, None, None) == tb.BL_ERR_INVALID_ARG
    assert back(0, 0, 1, 64, 1e-6, None, vp(256)) == tb.BL_ERR_INVALID_ARG and "gain" in tb.last_error()
    assert back(0, 0, 0, 64, 1e-6, None, None) == tb.BL_OK


def test_workspace_grows_with_the_tokens_up_to_the_grid():
    small = tb.add_rmsnorm_backward_workspace_bytes(1, 2560, tb.torch.bfloat16)
    assert small == 256 + 2560 * 4 + 256
    assert tb.add_rmsnorm_backward_workspace_bytes(0, 2560, tb.torch.bfloat16) == 256
    for K in (0, 1, 7, 63, 100):  # no such norm, but a size all the same
        assert tb.add_rmsnorm_backward_workspace_bytes(3, K, tb.torch.float32) >= 256
    sizes = [tb.add_rmsnorm_backward_workspace_bytes(M, 8192, tb.torch.bfloat16) for M in (1, 64, 1 << 20)]
    assert sizes[0] < sizes[1] < sizes[2] < 256 + 4 * 148 * 8192 * 4 + (4 << 20) + 256


@pytest.mark.parametrize("with_gain", [False, True])
def test_gradient_formula_against_differences(with_gain):
    """dz = r (gd - n mean(gd n)) + dz_in and dgain = sum dnorm n are the derivatives of the forward in 64 bits."""
    rng = np.random.RandomState(0)
    M, K, eps, h = 3, 64, 1e-5, 1e-6
    z, d, past = rng.randn(M, K), rng.randn(M, K), rng.randn(M, K)
    g = 1 + 0.1 * rng.randn(K) if with_gain else np.ones(K)

    def loss(z, g):
        return (d * (z / np.sqrt((z * z).mean(1, keepdims=True) + eps) * g)).sum() + (past * z).sum()
    r = 1 / np.sqrt((z * z).mean(1, keepdims=True) + eps)
    n = z * r
    dz = r * (d * g - n * (d * g * n).mean(1, keepdims=True)) + past
    dg = (d * n).sum(0)
    for _ in range(5):
        p, q = rng.randn(M, K), rng.randn(K)
        want = (loss(z + h * p, g + h * q) - loss(z - h * p, g - h * q)) / (2 * h)
        assert abs((dz * p).sum() + (dg * q).sum() - want) <= 1e-7 * (np.abs(dz * p).sum() + np.abs(dg * q).sum())
