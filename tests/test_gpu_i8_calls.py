"""The 8-bit product called as a program calls it: one call behind the other, nothing waited for in between."""
import pytest
import torch

import ternary_weight_a8_b200 as tb
from parity import activations, dev, weights

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
