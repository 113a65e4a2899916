"""Calls that follow one another with nothing between them, each on what the one before wrote: every result as when the
device is waited for after every call."""
import numpy as np
import pytest
import torch

import ternary_weight_a8_b200 as tb
from parity import activations, dev, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K", [(8, 192), (304, 2560), (2048, 2560)])
def test_training_step(M, K):
    """Norm and codes, the norm's gradient, and the straight-through backward of the layer in front of it, whose dy is that
    gradient: step after step, on inputs that change from step to step."""
    packed, gamma = tb.pack_weights(dev(weights(K, K, seed=1)))
    g = torch.ones(K, device="cuda")
    x = [activations(M, K, seed=20 + k, dtype="bf16")[0] * 2.0 ** k for k in range(3)]
    d = [activations(M, K, seed=30 + k, dtype="bf16")[0] * 0.1 ** k for k in range(3)]

    def step(k, wait=lambda: None):
        z, q, s, _ = tb.add_rmsnorm_quant(x[k], x[(k + 1) % 3], g)
        wait()
        dz, dg = tb.add_rmsnorm_backward(z, d[k], g, dz_in=x[k])
        wait()
        dx, dw = tb.ste_backward(packed, gamma, K, dz, q, s)
        wait()
        dn, dg2 = tb.add_rmsnorm_backward(z, dx, g)  # the layer's own norm
        wait()
        return dz, dg, dx, dw, dn, dg2, tb.ste_backward(packed, gamma, K, dn, q, s, dx=False)[1]

    want = [step(k, torch.cuda.synchronize) for k in range(3)]
    torch.cuda.synchronize()
    assert not torch.equal(want[0][2], want[1][2])
    got = [(k % 3, step(k % 3)) for k in range(24)]
    for i, (k, outs) in enumerate(got):
        for j, (a, b) in enumerate(zip(outs, want[k])):
            assert torch.equal(a, b), (i, j)
    # dx = gamma dy . t once: exact products, K sums in fp32 that may be cut instead of rounded, and the scaling
    t = torch.from_numpy(_ternary(packed.cpu().numpy(), K)).cuda().double()
    dx = float(gamma) * (want[0][0].double() @ t)
    terms = float(gamma) * (want[0][0].double().abs() @ t.abs())
    assert ((want[0][2].double() - dx).abs() <= 2.0 ** -24 * (2 * K + 4) * terms).all()


@pytest.mark.parametrize("M,K", [(8, 192), (304, 2560)])
def test_training_step_captured(M, K):
    """The same calls in one graph, replayed on inputs that change between replays."""
    packed, gamma = tb.pack_weights(dev(weights(K, K, seed=1)))
    g = torch.ones(K, device="cuda")
    ws = [tb.new_workspace(tb.ste_workspace_bytes(M, K, K)) for _ in range(2)]
    x, d = (torch.zeros((M, K), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step(wait=lambda: None):
        z, q, s, _ = tb.add_rmsnorm_quant(x, x, g)
        wait()
        dz, dg = tb.add_rmsnorm_backward(z, d, g, dz_in=x)
        wait()
        dx, dw = tb.ste_backward(packed, gamma, K, dz, q, s, workspace=ws[0])
        wait()
        dn, dg2 = tb.add_rmsnorm_backward(z, dx, g)
        wait()
        return dz, dg, dx, dw, dn, dg2, tb.ste_backward(packed, gamma, K, dn, q, s, dx=False, workspace=ws[1])[1]

    inputs = [(activations(M, K, seed=20 + k, dtype="bf16")[0], activations(M, K, seed=30 + k, dtype="bf16")[0] * 0.1 ** k)
              for k in range(3)]
    want = []
    for a, b in inputs:
        x.copy_(a)
        d.copy_(b)
        want.append([t.clone() for t in step(torch.cuda.synchronize)])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(9):
        x.copy_(inputs[i % 3][0])
        d.copy_(inputs[i % 3][1])
        graph.replay()
        for j, (a, b) in enumerate(zip(out, want[i % 3])):
            assert torch.equal(a, b), (i, j)


def _ternary(packed, K):
    """Ternary values [N][K] of packed weights (element 16 g + 4 j + b in byte b of word g, bits 2 j and 2 j + 1)."""
    words = packed.reshape(packed.shape[0], K // 16, 4)  # [N][g][b]
    t = np.stack([(words >> (2 * j)) & 3 for j in range(4)], axis=2)  # [N][g][j][b]
    return t.reshape(packed.shape[0], K).astype(np.int8) - 1


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 2560), (64, 8192), (513, 2560), (300, 4096), (40, 16384 + 64), (3, 131072 + 64)])
def test_gains_written_just_before(M, K, dtype):
    """Gains that the kernel just before the call wrote, as an optimiser's step does: every call reads the new ones."""
    x = torch.randn((M, K), generator=torch.Generator("cuda").manual_seed(K), device="cuda").to(dtype)
    sets = [torch.full((K,), 4.0 ** k, device="cuda") for k in range(3)]
    want = []
    for g in sets:
        fwd = tb.add_rmsnorm_quant(x, x, g, x_norm=True)
        torch.cuda.synchronize()
        want.append((fwd, tb.add_rmsnorm_backward(x, x, g)))
        torch.cuda.synchronize()
    g = torch.empty_like(sets[0])
    got = []
    for k in range(30):
        torch.mul(sets[k % 3], 1.0, out=g)
        got.append((tb.add_rmsnorm_quant(x, x, g, x_norm=True), tb.add_rmsnorm_backward(x, x, g)))
    for k, pair in enumerate(got):
        for a, b in zip(pair[0] + pair[1], want[k % 3][0] + want[k % 3][1]):
            assert torch.equal(a, b), k
