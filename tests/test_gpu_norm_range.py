"""The residual norm's gradient where fp32 sums leave their range, and the gain's gradient against its own depth.

The bars are those of the formula's roundings, u = 2^-24 each (44 u of the
absolute terms of dz, and DEPTH u of the projection's, which fp32 sums or 64-bit
ones both keep) and half a step of the output's type; and where values are
subnormal, half a step of those, 2^-150: of gd and of gd - n mean, r times, of
the mean, r |n| times, and of the output.
"""
import numpy as np
import pytest
import torch

import ternary_weight_a8_b200 as tb
from parity import dev
from test_gpu_norm import _back_ref, _gain

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
# One warp, one block, clusters of two to eight, read twice; for fp32 tokens.
LENGTHS = [64, 256, 4096, 8192, 12288, 40960, 66048]


def _norm(z, eps):
    z = z.astype(np.float64)
    r = 1.0 / np.sqrt((z * z).mean(1, keepdims=True) + float(np.float32(eps)))
    return r, z * r


def _rows(K, seed):
    """(z, dnorm, eps) of rows whose statistics lie in fp32's range one by one or not at all."""
    rng = np.random.RandomState(seed)
    n = lambda: rng.randn(K).astype(np.float32)
    z = n()
    return [
        (z * np.float32(1e25), n() * np.float32(1e15), 1e-6),        # z^2 and gd z above the range
        (z * np.float32(1e18), z * np.float32(1e21), 1e-6),          # gd z alone
        (z * np.float32(1e3), z * np.float32(2e34), 1e-6),           # the same with z^2 far inside
        (z / np.float32(3), z * np.float32(6e36), 0.0),              # few inputs: the sum in range, its product with r not
        (z * np.float32(1e-22), z * np.float32(1e-12), 0.0),         # z^2 below, gd z nearly
        (z * np.float32(1e-10), z * np.float32(1e-33), 0.0),         # gd z among the subnormals, dz not
        (z * np.float32(1e-10), (z + n()) * np.float32(1e-35), 0.0),
        (z * np.float32(1e-12), z * np.float32(1e-37), 0.0),         # every product rounds to nothing
        (z, np.zeros(K, np.float32), 1e-6),                          # no gradient: dz = dz_in
        (np.zeros(K, np.float32), n(), 1e-6),
        (z, n(), 1e-6),
    ]


@pytest.mark.parametrize("with_gain", [False, True])
@pytest.mark.parametrize("past", [False, True])
@pytest.mark.parametrize("K", LENGTHS)
def test_statistics_outside_of_fp32(K, past, with_gain):
    rows = _rows(K, K)
    g = _gain(K, 3) if with_gain else None
    gd = None if g is None else dev(g)
    depth = 1 + max(32, -(-K // 512)) + 1 + 5 + 16 + 21 + 3
    for eps in (1e-6, 0.0):
        some = [(z, d) for z, d, e in rows if e == eps]
        z, d = np.stack([a for a, _ in some]), np.stack([b for _, b in some])
        want0 = _back_ref(z, d, g, eps, None)[0]
        # what reaches z past the norm, of the size of the row's own gradient (a sixteenth of its largest, 1.7e38, so that
        # five standard deviations are fp32 numbers still)
        i = (np.random.RandomState(7).randn(*z.shape) * np.abs(want0).max(1, keepdims=True) / 16).astype(np.float32) \
            if past else None
        want, _, terms, dots, _ = _back_ref(z, d, g, eps, i)
        assert np.isfinite(want).all()
        dz, _ = tb.add_rmsnorm_backward(dev(z), dev(d), gd, eps=eps, dz_in=None if i is None else dev(i))
        got = dz.cpu().numpy().astype(np.float64)
        r, n = _norm(z, eps)
        bar = U * (44 * terms + depth * dots) + U * (1 + 2.0 ** -8) * np.abs(want) + 2.0 ** -150 * (r * (2 + np.abs(n)) + 1)
        bad = ~(np.abs(got - want) <= bar)
        assert not bad.any(), (eps, sorted(set(np.argwhere(bad)[:, 0].tolist())))


@pytest.mark.parametrize("M,K,dtype", [(2, 2560, torch.bfloat16), (9, 8640, torch.bfloat16), (7, 16448, torch.bfloat16),
                                       (40, 192, torch.bfloat16), (5, 28672, torch.bfloat16)])
def test_statistics_outside_of_fp32_in_bf16(M, K, dtype):
    """Rows of 1e25 and gradients of 1e15, and rows without a gradient, among ordinary ones."""
    rng = np.random.RandomState(K)
    z, d = (torch.from_numpy(rng.randn(M, K).astype(np.float32)) for _ in range(2))
    z[0], d[0] = z[0] * 1e25, d[0] * 1e15
    d[1] = 0
    z, d = z.to(dtype), d.to(dtype)
    want, _, terms, dots, _ = _back_ref(z.float().numpy(), d.float().numpy(), None, 1e-6, None)
    dz, _ = tb.add_rmsnorm_backward(z.cuda(), d.cuda(), None, eps=1e-6)
    depth = 1 + max(32, -(-K // 512)) + 1 + 5 + 16 + 21 + 3
    bar = U * (44 * terms + depth * dots) + 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -8) + 2.0 ** -133
    err = np.abs(dz.float().cpu().numpy().astype(np.float64) - want)
    assert (err <= bar).all() and not dz[1].any()


@pytest.mark.parametrize("M,K,dtype", [(1, 64, torch.bfloat16), (20000, 192, torch.bfloat16), (3001, 2560, torch.bfloat16),
                                       (777, 3200, torch.float32), (2500, 8192, torch.float32), (700, 28672, torch.bfloat16),
                                       (700, 40960, torch.float32), (300, 65536, torch.float32),
                                       (300, 65536 + 64, torch.float32)])
def test_gain_gradient_against_its_own_depth(M, K, dtype):
    """A term dnorm n is off by 23 u at most (r, n and the fused step); then it passes the chain over a group's tokens, at
    most ceil(M / rows) of them, up to 8 groups of a block, and of the closing kernel a thread's ceil(rows / 128) rows,
    two shuffles and 32 warps.  The rows of partial sums are counted in the workspace, where no sum is a NaN."""
    gen = torch.Generator("cuda").manual_seed(M)
    z, d = (torch.randn((M, K), device="cuda", generator=gen).to(dtype) for _ in range(2))
    g = dev(_gain(K, K))
    need = tb.add_rmsnorm_backward_workspace_bytes(M, K, dtype)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    _, dgain = tb.add_rmsnorm_backward(z, d, g, eps=1e-5, workspace=ws)
    part = ws[256:256 + (need - 256) // (4 * K) * 4 * K].view(torch.int32).view(-1, K)
    rows = int((part != -1).all(1).sum())
    assert 1 <= rows <= M
    zd, dd = z.double(), d.double()
    n = zd / ((zd * zd).mean(1, keepdim=True) + float(np.float32(1e-5))).sqrt()
    depth = 23 + -(-M // rows) + 8 + -(-rows // 128) + 2 + 32
    bar = U * depth * (dd * n).abs().sum(0)
    err = (dgain.double() - (dd * n).sum(0)).abs()
    assert (err <= bar).all(), (rows, float((err / bar).max()))
