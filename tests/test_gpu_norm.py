"""The residual sum with its norm and codes, and the gradient of both, on the GPU.

Forward: z against the fp32 sum rounded to the activation type, the rest
against the oracle's RMSNorm and quantisation of z, all bit for bit, and
against ``rmsnorm_quant`` on z.

Backward, against the formula in 64 bits.  The bar counts the kernel's fp32
roundings, u = 2^-24 each, on the absolute terms of the formula.  With
n = z r and D = (r / K) sum |gd z|:
  * r: a square passes the thread's chain (its product fused, at most 16 terms
    a half), the join of two halves, a tree of 5 steps, at most 4 warps in
    turn and another tree of 5, so the sum is off by 31 u, the mean with eps
    by 33 u, and r by half of that and 2 units in the last place (4 u) of
    rsqrtf: R = 20.5 u (where K is longer still, squares are summed in 64
    bits);
  * r gd: R, gd, the two fused steps, 23.5 u; r n mean: R twice, n, the two
    fused steps, 44 u; dz_in: 1 u.  So at most 44 u of
    |r gd| + |r n mean| + |dz_in|;
  * mean: a term of the dot product passes its own rounding, the thread's
    chain (at most 32 terms when held in registers, K / 512 otherwise), the
    join of two halves, 5 shuffles, 4 + 5 more or 16 warps, then R and the
    roundings of the products with r and 1 / K and of 1 / K: DEPTH u of D,
    times |r n|;
  * the last rounding to the output type: eps / 2 of |dz|.
dgain: a term dnorm n has R, n and the fused step, at most 23 u, then the
chain over a group's tokens (at most ceil(M / 64): there are at least 64
groups, or one token each), the 148 partial rows that a warp of the closing
kernel takes at most and its 32 warps.
"""
import threading

import numpy as np
import pytest
import torch

import oracle
import synth
import ternary_weight_a8_b200 as tb
from parity import dev, f32_bits

U = 2.0 ** -24


def _act(M, K, seed, dtype, scale=1.0):
    """Activations as (device tensor, exact fp32 values)."""
    xf = synth.activations_f32(M, K, seed=seed) * np.float32(scale)
    t = torch.from_numpy(xf).to(dtype)
    return t.cuda(), t.float().numpy()


def _gain(K, seed):
    return (1.0 + 0.1 * synth.activations_f32(1, K, seed=seed)[0]).astype(np.float32)


def _round(a, dtype):
    return torch.from_numpy(a).to(dtype).float().numpy()


DT = {"bf16": torch.bfloat16, "f32": torch.float32}

FORWARD = [
    (1, 64, "bf16", True, 1e-6), (1, 2560, "bf16", True, 1e-6), (3, 64, "f32", False, 1e-5), (16, 8192, "bf16", True, 1e-6),
    (7, 3200, "f32", True, 1e-6), (33, 8640, "f32", False, 1e-6), (5, 192, "bf16", True, 0.0), (2048, 2560, "bf16", True, 1e-5),
    (3000, 64, "bf16", True, 1e-6), (2500, 320, "f32", True, 1e-6), (2, 32768, "bf16", True, 1e-6),
    (2, 16384, "bf16", True, 1e-6), (2, 8192, "f32", True, 1e-6),              # the longest held in registers
    (3, 16384 + 64, "bf16", True, 1e-6), (2, 8192 + 64, "f32", False, 1e-6),   # held in shared memory
    (2, 114688, "bf16", True, 1e-6), (2, 57344, "f32", True, 1e-6),            # the longest held there
    (3, 114688 + 64, "bf16", True, 1e-6), (2, 57344 + 64, "f32", False, 1e-6),  # z is read back
    (1100, 8192, "bf16", False, 1e-6),
]


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,dtype,with_gain,eps", FORWARD)
def test_forward_parity(M, K, dtype, with_gain, eps):
    dt = DT[dtype]
    x, xf = _act(M, K, M + K, dt)
    res, rf = _act(M, K, M + K + 1, dt, 3.0)
    g = _gain(K, K) if with_gain else None
    z_ref = _round(xf + rf, dt)
    v_ref, q_ref, s_ref, r_ref = oracle.rmsnorm_quant(z_ref, g, eps, dtype == "bf16")
    gd = None if g is None else dev(g)
    z, v, q, s, r = tb.add_rmsnorm_quant(x, res, gd, eps=eps, x_norm=True)
    assert np.array_equal(f32_bits(z.float().cpu().numpy()), f32_bits(z_ref))
    assert np.array_equal(f32_bits(v.float().cpu().numpy()), f32_bits(v_ref))
    assert np.array_equal(q.cpu().numpy(), q_ref)
    assert np.array_equal(f32_bits(s.cpu().numpy()), f32_bits(s_ref))
    assert np.array_equal(r.cpu().numpy(), r_ref)
    # the framework's own norm on z, and the sum in place of either input
    q2, s2, r2 = tb.rmsnorm_quant(z, gd, eps=eps)
    assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(r, r2)
    for which in (0, 1):
        a, b = x.clone(), res.clone()
        z3, q3, s3, _ = tb.add_rmsnorm_quant(a, b, gd, eps=eps, z=(a, b)[which])
        assert z3 is (a, b)[which] and torch.equal(z3, z) and torch.equal(q3, q) and torch.equal(s3, s)
        assert torch.equal((a, b)[1 - which], (x, res)[1 - which])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K,eps", [(256, 1e-6), (256, 0.0), (40960, 1e-6), (131072, 1e-6)])
def test_forward_degenerate_tokens(dtype, K, eps):
    """Zero, one-hot, cancelling, huge and tiny tokens, and tokens with infinities and NaN: whatever rmsnorm_quant
    makes of z, and the other tokens untouched by them."""
    dt = DT[dtype]
    x = torch.randn((10, K), generator=torch.Generator().manual_seed(K)).to(dt)
    res = torch.randn((10, K), generator=torch.Generator().manual_seed(K + 1)).to(dt)
    x[0], res[0] = 0, 0
    x[1], res[1] = 0, 0
    x[1, 17] = -3.0
    res[2] = -x[2]
    x[3] *= 1e18
    x[4], res[4] = x[4] * 1e-30, res[4] * 1e-30
    x[5, 3] = float("inf")
    x[6, 5] = float("nan")
    x[7, 5], res[7, 5] = float("inf"), float("-inf")
    x[9], res[9] = x[9] * 1e-39, res[9] * 1e-39  # subnormal
    x, res = x.cuda(), res.cuda()
    g = dev(_gain(K, 3))
    z, v, q, s, r = tb.add_rmsnorm_quant(x, res, g, eps=eps, x_norm=True)
    zr = (x.float() + res.float()).to(dt)
    assert torch.equal(torch.nan_to_num(z.float(), nan=7.0), torch.nan_to_num(zr.float(), nan=7.0))
    v2, q2, s2, r2 = tb.rmsnorm_quant(z, g, eps=eps, x_norm=True)
    assert torch.equal(q, q2) and torch.equal(r, r2)
    assert torch.equal(torch.nan_to_num(s, nan=-1.0), torch.nan_to_num(s2, nan=-1.0))
    assert torch.equal(torch.nan_to_num(v.float(), nan=7.0), torch.nan_to_num(v2.float(), nan=7.0))
    assert not q[0].any() and not q[2].any()  # zero, or NaN (0 / 0 without an eps), is code 0


def _back_ref(z, d, g, eps, dz_in):
    """dz and dgain in 64 bits, and the sums of absolute terms that the bars scale."""
    z, d = z.astype(np.float64), d.astype(np.float64)
    K = z.shape[1]
    r = 1.0 / np.sqrt((z * z).mean(1, keepdims=True) + float(np.float32(eps)))
    n = z * r
    gd = d if g is None else d * g.astype(np.float64)
    mean = (gd * n).mean(1, keepdims=True)
    past = 0.0 if dz_in is None else dz_in.astype(np.float64)
    dz = r * (gd - n * mean) + past
    terms = np.abs(r * gd) + np.abs(r * n * mean) + np.abs(past)
    dots = np.abs(r * n) * (np.abs(gd * z).sum(1, keepdims=True) * r / K)
    return dz, (d * n).sum(0), terms, dots, np.abs(d * n).sum(0)


BACKWARD = [
    (1, 64, "bf16", "bf16", True, True), (1, 2560, "f32", "f32", True, False), (5, 192, "bf16", "f32", True, True),
    (3, 320, "f32", "bf16", False, True), (2049, 64, "bf16", "bf16", True, False), (777, 3200, "f32", "f32", True, True),
    (1500, 2560, "bf16", "f32", True, True), (700, 8192, "bf16", "bf16", True, True), (300, 8192, "f32", "f32", True, True),
    (64, 16384, "bf16", "bf16", True, True), (9, 8640, "bf16", "bf16", False, False),
    (70, 16384 + 64, "bf16", "f32", True, True), (33, 8192 + 64, "f32", "bf16", True, False),
    (300, 8640, "bf16", "f32", True, True), (500, 8640, "f32", "f32", True, True), (40, 32768, "f32", "f32", False, False),
    (7, 65536, "f32", "bf16", True, True), (5, 131072, "bf16", "f32", True, True),  # the largest cluster
    (70, 65536 + 64, "f32", "f32", True, True), (3, 131072 + 64, "bf16", "bf16", True, False),  # read twice
    (2, 28672, "bf16", "bf16", False, True), (20, 12288, "bf16", "f32", True, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,dtype,grad,with_gain,past", BACKWARD)
def test_backward_parity(M, K, dtype, grad, with_gain, past):
    dt, gt, eps = DT[dtype], DT[grad], 1e-5
    z, zf = _act(M, K, M + K, dt, 3.0)
    d, df = _act(M, K, M + K + 1, gt, 0.01)
    i, inf = _act(M, K, M + K + 2, dt, 0.02) if past else (None, None)
    g = _gain(K, K) if with_gain else None
    gdev = None if g is None else dev(g)
    dz, dgain = tb.add_rmsnorm_backward(z, d, gdev, eps=eps, dz_in=i)
    want, wg, terms, dots, tg = _back_ref(zf, df, g, eps, inf)
    depth = 1 + max(32, -(-K // 512)) + 1 + 5 + 16 + 21 + 3
    bar = U * (44 * terms + depth * dots) + torch.finfo(dt).eps / 2 * np.abs(want) * (1 + 2.0 ** -8)
    err = np.abs(dz.float().cpu().numpy().astype(np.float64) - want)
    assert (err <= bar).all(), (err / bar).max()
    if g is None:
        assert dgain is None
    else:
        bar = U * (23 + -(-M // 64) + 148 + 32) * tg
        err = np.abs(dgain.cpu().numpy().astype(np.float64) - wg)
        assert (err <= bar).all(), (err / bar).max()
    # again, in place of dz_in, and without the gain's gradient: the same
    if past:
        j = i.clone()
        dz2, dg2 = tb.add_rmsnorm_backward(z, d, gdev, eps=eps, dz_in=j, dz=j, dgain=False)
        assert dz2 is j and dg2 is None and torch.equal(dz2, dz)
    dz3, dg3 = tb.add_rmsnorm_backward(z, d, gdev, eps=eps, dz_in=i)
    assert torch.equal(dz3, dz) and (dgain is None or torch.equal(dg3, dgain))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(20000, 192), (9000, 512), (5000, 1024), (3100, 2048), (3001, 2560), (2500, 8192), (1300, 8640),
                                 (1300, 16384), (700, 28672), (700, 40960)])
def test_many_tokens(M, K, dtype):
    """Several waves of tokens: the codes of rmsnorm_quant, in place too, and gradients as in calls of few tokens."""
    dt = DT[dtype]
    gen = torch.Generator("cuda").manual_seed(M)
    x, res, d = (torch.randn((M, K), device="cuda", generator=gen).to(dt) for _ in range(3))
    g = dev(_gain(K, K))
    z, q, s, r = tb.add_rmsnorm_quant(x, res, g)
    assert torch.equal(z, (x.float() + res.float()).to(dt))
    q2, s2, r2 = tb.rmsnorm_quant(z, g)
    assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(r, r2)
    dz, dgain = tb.add_rmsnorm_backward(z, d, g, dz_in=x)
    for at in (0, M // 3, M - 70):
        part, _ = tb.add_rmsnorm_backward(z[at:at + 70], d[at:at + 70], g, dz_in=x[at:at + 70])
        assert torch.equal(part, dz[at:at + 70])
    zd, dd = z.double(), d.double()
    n = zd / ((zd * zd).mean(1, keepdim=True) + float(np.float32(1e-6))).sqrt()
    bar = U * (23 + -(-M // 64) + 148 + 32) * (dd * n).abs().sum(0)
    assert ((dgain - (dd * n).sum(0)).abs() <= bar).all()
    kept = x.clone()
    z3, q3, s3, _ = tb.add_rmsnorm_quant(x, res, g, z=x)
    assert z3 is x and torch.equal(z3, z) and torch.equal(q3, q) and torch.equal(s3, s)
    dz3, _ = tb.add_rmsnorm_backward(z, d, g, dz_in=kept, dz=kept)
    assert dz3 is kept and torch.equal(kept, dz)


@pytest.mark.gpu
def test_backward_against_differences():
    """Directional derivatives of L = <d, norm(z)> + <dz_in, z> by central differences in 64 bits."""
    M, K, eps = 6, 640, 1e-5
    z, zf = _act(M, K, 1, torch.float32)
    d, df = _act(M, K, 2, torch.float32)
    i, inf = _act(M, K, 3, torch.float32)
    g = _gain(K, 4)
    dz, dgain = tb.add_rmsnorm_backward(z, d, dev(g), eps=eps, dz_in=i)
    e = float(np.float32(eps))

    def loss(zz, gg):
        return float((df * (zz / np.sqrt((zz * zz).mean(1, keepdims=True) + e) * gg)).sum() + (inf * zz).sum())

    z0, g0 = zf.astype(np.float64), g.astype(np.float64)
    rng = np.random.RandomState(5)
    h = 1e-5
    for _ in range(4):
        p, q = rng.randn(M, K), rng.randn(K)
        want = (loss(z0 + h * p, g0 + h * q) - loss(z0 - h * p, g0 - h * q)) / (2 * h)
        a, b = dz.cpu().numpy().astype(np.float64) * p, dgain.cpu().numpy().astype(np.float64) * q
        # the differences: h^2 of the third derivative (1e-10 of the terms) and 2^-52 / h of the loss
        assert abs(a.sum() + b.sum() - want) <= 1e-6 * (np.abs(a).sum() + np.abs(b).sum())


@pytest.mark.gpu
@pytest.mark.parametrize("K", [256, 4096, 12288, 40960, 66048])
def test_backward_of_large_and_zero_rows(K):
    """Rows far out of range for r^3 in fp32, and zero rows (r = 1 / sqrt(eps)), in every form of the kernel."""
    M = 4
    z, _ = _act(M, K, 7, torch.float32)
    z[0] *= 1e25  # squares beyond fp32
    z[1] *= 1e-22
    z[2] = 0
    d, df = _act(M, K, 8, torch.float32)
    want, *_ = _back_ref(z.cpu().numpy(), df, None, 1e-6, None)
    dz, _ = tb.add_rmsnorm_backward(z, d, None, eps=1e-6)
    got = dz.cpu().numpy().astype(np.float64)
    scale = np.abs(want).max(1, keepdims=True)
    assert np.isfinite(got).all() and (np.abs(got - want) <= 1e-5 * scale).all()


@pytest.mark.gpu
def test_c_call_without_sums_gain_or_normalised_output():
    M, K = 5, 320
    x, _ = _act(M, K, 1, torch.float32)
    want = tb.add_rmsnorm_quant(x, x)
    z, q, s = torch.empty_like(x), torch.empty((M, K), dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    rc = tb.lib().bitlinear_add_rmsnorm_quant(x.data_ptr(), x.data_ptr(), tb.BL_F32, M, K, None, 1e-6, z.data_ptr(), None,
                                              q.data_ptr(), s.data_ptr(), None, torch.cuda.current_stream().cuda_stream)
    assert rc == tb.BL_OK
    assert torch.equal(z, want[0]) and torch.equal(q, want[1]) and torch.equal(s, want[2])


@pytest.mark.gpu
def test_empty_batch():
    x = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    z, q, s, r = tb.add_rmsnorm_quant(x, x)
    assert z.shape == (0, 128) and s.shape == (0,)
    g = torch.ones(128, device="cuda")
    dz, dg = tb.add_rmsnorm_backward(x, x, g, dgain=torch.full((128,), 3.0, device="cuda"))
    assert dz.shape == (0, 128) and not dg.any()


@pytest.mark.gpu
def test_no_writes_outside_outputs():
    pad, canary = 4096, 0x5A
    for M, K, dt in ((3, 192, torch.bfloat16), (5, 40960, torch.bfloat16), (1, 64, torch.float32), (2, 65536, torch.float32)):
        x, _ = _act(M, K, 1, dt)
        d, _ = _act(M, K, 2, dt)
        g = torch.ones(K, device="cuda")

        def out(n, t):
            size = torch.empty((), dtype=t).element_size() * n
            buf = torch.full((2 * pad + size,), canary, dtype=torch.uint8, device="cuda")
            return buf, buf[pad:pad + size].view(t)
        bufs = [out(M * K, dt), out(M * K, dt), out(M * K, torch.int8), out(M, torch.float32), out(M, torch.int32),
                out(M * K, dt), out(K, torch.float32)]
        o = [b[1] for b in bufs]
        tb.add_rmsnorm_quant(x, x, g, z=o[0].view(M, K), x_norm=o[1].view(M, K), xq=o[2].view(M, K), scale=o[3], rowsum=o[4])
        need = tb.add_rmsnorm_backward_workspace_bytes(M, K, dt)
        wbuf = torch.full((need + pad,), canary, dtype=torch.uint8, device="cuda")
        tb.add_rmsnorm_backward(x, d, g, dz=o[5].view(M, K), dgain=o[6], workspace=wbuf[:need])
        torch.cuda.synchronize()
        for buf, _ in bufs:
            assert (buf[:pad] == canary).all() and (buf[-pad:] == canary).all()
        assert (wbuf[need:] == canary).all() and (wbuf[:256] == canary).all()


@pytest.mark.gpu
def test_streams_threads_and_graphs():
    """Another stream, host threads on one stream, and two captured graphs replayed side by side: the same results."""
    M, K = 513, 2560
    g = dev(_gain(K, 1))
    sets = []
    for k in range(3):
        z, _ = _act(M, K, 20 + k, torch.bfloat16, 2.0)
        d, _ = _act(M, K, 30 + k, torch.bfloat16)
        sets.append((z, d, tb.add_rmsnorm_backward(z, d, g), tb.add_rmsnorm_quant(z, d, g)))
    torch.cuda.synchronize()

    def same(got, k):
        return all(torch.equal(a, b) for a, b in zip(got[0], sets[k][2])) and \
            all(torch.equal(a, b) for a, b in zip(got[1], sets[k][3]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (tb.add_rmsnorm_backward(sets[0][0], sets[0][1], g, stream=side),
           tb.add_rmsnorm_quant(sets[0][0], sets[0][1], g, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    assert same(got, 0)

    bad = []

    def work(k):
        with torch.cuda.stream(side):
            for _ in range(20):
                got = (tb.add_rmsnorm_backward(sets[k][0], sets[k][1], g), tb.add_rmsnorm_quant(sets[k][0], sets[k][1], g))
                side.synchronize()
                if not same(got, k):
                    bad.append(k)
    threads = [threading.Thread(target=work, args=(k,)) for k in (0, 1)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad

    graphs = []
    for k in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = (tb.add_rmsnorm_backward(sets[k][0], sets[k][1], g), tb.add_rmsnorm_quant(sets[k][0], sets[k][1], g))
        graphs.append((graph, got))
    other = torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(side):
            graphs[0][0].replay()
        with torch.cuda.stream(other):
            graphs[1][0].replay()
    torch.cuda.synchronize()
    assert same(graphs[0][1], 0) and same(graphs[1][1], 1)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """More than 2^31 values: the last tokens as a call of their own gives them, the first ones too."""
    M, K = 262144 + 5, 8192
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    for i in range(0, M, 65536):
        x[i:i + 65536] = torch.randn((min(65536, M - i), K), device="cuda")
    g = dev(_gain(K, 1))
    z, q, s, r = tb.add_rmsnorm_quant(x, x, g)
    dz, dg = tb.add_rmsnorm_backward(z, x, g, dz_in=x)
    assert torch.isfinite(dg).all()
    for at in (slice(0, 7), slice(131068, 131077), slice(M - 7, M)):
        part = x[at].contiguous()
        z2, q2, s2, r2 = tb.add_rmsnorm_quant(part, part, g)
        assert torch.equal(z[at], z2) and torch.equal(q[at], q2) and torch.equal(s[at], s2) and torch.equal(r[at], r2)
        assert torch.equal(dz[at], tb.add_rmsnorm_backward(z2, part, g, dz_in=part, dgain=False)[0])


@pytest.mark.gpu
def test_refusals():
    x = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")
    f = torch.zeros((4, 128), device="cuda")
    g = torch.ones(128, device="cuda")
    for bad in (lambda: tb.add_rmsnorm_quant(x, f), lambda: tb.add_rmsnorm_quant(x, x[:3]),
                lambda: tb.add_rmsnorm_quant(x, x.cpu()), lambda: tb.add_rmsnorm_quant(x.cpu(), x),
                lambda: tb.add_rmsnorm_quant(x.half(), x.half()), lambda: tb.add_rmsnorm_quant(x, x, g.bfloat16()),
                lambda: tb.add_rmsnorm_quant(x, x, g[:64]), lambda: tb.add_rmsnorm_quant(x.t(), x.t()),
                lambda: tb.add_rmsnorm_quant(x, x, xq=torch.empty((4, 64), dtype=torch.int8, device="cuda")),
                lambda: tb.add_rmsnorm_backward(x, x, g, dz_in=f), lambda: tb.add_rmsnorm_backward(x, x[:2], g),
                lambda: tb.add_rmsnorm_backward(x, x.half(), g), lambda: tb.add_rmsnorm_backward(x, x, g, dz=f)):
        with pytest.raises(ValueError):
            bad()
    wide = torch.zeros(4 * 128 + 64, dtype=torch.bfloat16, device="cuda")
    a, b = wide[:512].view(4, 128), wide[8:520].view(4, 128)
    for bad, code in ((lambda: tb.add_rmsnorm_quant(x[:, :96].contiguous(), x[:, :96].contiguous()), tb.BL_ERR_UNSUPPORTED_SHAPE),
                      (lambda: tb.add_rmsnorm_quant(x, x, eps=-1.0), tb.BL_ERR_INVALID_ARG),
                      (lambda: tb.add_rmsnorm_quant(x, x, eps=float("nan")), tb.BL_ERR_INVALID_ARG),
                      (lambda: tb.add_rmsnorm_quant(a, x, z=b), tb.BL_ERR_INVALID_ARG),
                      (lambda: tb.add_rmsnorm_quant(a, x, x_norm=a), tb.BL_ERR_INVALID_ARG),
                      (lambda: tb.add_rmsnorm_quant(wide[1:513].view(4, 128), x), tb.BL_ERR_MISALIGNED),
                      (lambda: tb.add_rmsnorm_backward(a, x, g, dz=a), tb.BL_ERR_INVALID_ARG),
                      (lambda: tb.add_rmsnorm_backward(x, x, None, dgain=torch.empty(128, device="cuda")), tb.BL_ERR_INVALID_ARG),
                      (lambda: tb.add_rmsnorm_backward(x, x, g, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")),
                       tb.BL_ERR_WORKSPACE_TOO_SMALL)):
        with pytest.raises(tb.BitLinearError) as e:
            bad()
        assert e.value.code == code
