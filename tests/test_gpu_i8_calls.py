"""The 8-bit product called as a program calls it: one call behind the other, nothing waited for in between."""
import pytest
import torch

import ternary_weight_a8_b200 as tb
from parity import activations, dev, weights
from test_gpu_i8 import _check, _codes

pytestmark = pytest.mark.gpu


# The decode kernel on raw tokens and on codes, the tensor cores' split, single and pair forms.
@pytest.mark.parametrize("M,N,K", [(1, 2560, 2560), (8, 4096, 2560), (24, 2560, 2560), (47, 2560, 2560),
                                   (128, 6912, 2560), (1024, 6912, 2560)])
def test_activations_and_scales_change_between_calls(M, N, K):
    """Calls in a row share the workspace, whose scales and codes each of them writes anew; token and channel scales far
    apart, so that one call's in another's would be seen."""
    wq, ws = tb.quant_weights_i8(dev(weights(N, K, seed=1)))
    xs = [activations(M, K, seed=20 + k, dtype="bf16")[0] * 8.0 ** k for k in range(3)]
    scales = [ws * 4.0 ** k for k in range(2)]
    want = {}
    for i, x in enumerate(xs):
        for j, s in enumerate(scales):
            want[i, j] = tb.forward_i8(wq, s, x, out_dtype=torch.float32)
            torch.cuda.synchronize()
    rows = torch.empty_like(ws)
    got = []
    for k in range(60):
        i, j = k % 3, k % 2
        torch.mul(ws, 4.0 ** j, out=rows)  # the kernel just before writes the channels' scales
        got.append((i, j, tb.forward_i8(wq, rows, xs[i], out_dtype=torch.float32)))
    for k, (i, j, y) in enumerate(got):
        assert torch.equal(y, want[i, j]), k


def test_a_wait_that_runs_out_is_seen_without_a_workspace():
    """The product's own bounded wait, with nothing to end it: the workspace and the device's word say so, eager or in a
    replayed graph; the context stays usable."""
    wq, ws = tb.quant_weights_i8(dev(weights(640, 2560, seed=1)))
    x, _ = activations(47, 2560, seed=2, dtype="bf16")
    want = tb.forward_i8(wq, ws, x)
    assert tb.i8_status() == tb.BL_OK
    buf = tb.new_workspace(256)
    tb.selftest_i8_wait_timeout(buf, 2000)
    assert tb.i8_status() == tb.BL_ERR_DEVICE_TIMEOUT and "8-bit product" in tb.last_error()
    assert tb.i8_status() == tb.BL_OK
    assert tb.device_status(buf) == tb.BL_ERR_DEVICE_TIMEOUT and tb.device_status(buf) == tb.BL_OK
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = tb.forward_i8(wq, ws, x)
        tb.selftest_i8_wait_timeout(torch.empty(256, dtype=torch.uint8, device="cuda"), 2000)
    for _ in range(2):
        with torch.cuda.stream(side):
            graph.replay()
        assert tb.i8_status(side) == tb.BL_ERR_DEVICE_TIMEOUT
        assert tb.i8_status(side) == tb.BL_OK
    assert torch.equal(y, want) and torch.equal(tb.forward_i8(wq, ws, x), want)
    assert tb.i8_status() == tb.BL_OK


# Few tokens through either kernel, sizes that automatic dispatch gives to the other one among them.
@pytest.mark.parametrize("M,N,K", [(1, 1, 64), (1, 6912, 2560), (2, 5, 192), (5, 64, 8640), (8, 128000, 64), (8, 100, 16384),
                                   (9, 1000, 640), (12, 12800, 2560), (16, 200, 16384), (16, 3200, 8640), (17, 16, 2560),
                                   (24, 515, 1024), (31, 257, 64), (32, 12800, 2560), (32, 333, 28672), (32, 2560, 6912)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_both_kernels_by_force(M, N, K, dtype):
    """Accumulators exact and outputs the documented fp32 steps, on codes and on raw tokens, whichever kernel is forced."""
    q, s = _codes(M, K, M + K)
    w, ws = _codes(N, K, N + K)
    wd, wsd, qd, sd = dev(w), dev(ws), dev(q), dev(s)
    x = activations(M, K, seed=M + K, dtype="bf16")[0].to(dtype)
    xq, xs, _ = tb.quant_act(x)
    out = {}
    for path in (tb.PATH_GEMV, tb.PATH_GEMM, tb.PATH_AUTO):
        tb.set_path(path)
        try:
            y, acc = tb.forward_i8_quantized(wd, wsd, qd, sd, out_dtype=dtype, acc_out=True)
            raw = tb.forward_i8(wd, wsd, x, out_dtype=torch.float32, acc_out=True)
        finally:
            tb.set_path(tb.PATH_AUTO)
        _check(y, acc, q, s, w, ws)
        _check(raw[0], raw[1], xq.cpu().numpy(), xs.cpu().numpy(), w, ws)
        out[path] = y
    assert torch.equal(out[tb.PATH_GEMV], out[tb.PATH_GEMM]) and torch.equal(out[tb.PATH_GEMV], out[tb.PATH_AUTO])
