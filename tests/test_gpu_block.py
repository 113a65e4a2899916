"""The residual norm, the 8-bit product and the ternary products run together, as a model runs them.

Serving: the blocks' inputs are summed, normalised and quantised once and the
codes feed ternary BitLinears and, after the last block, the 8-bit head; each
step is decided bit for bit by the oracle from the step before it.  Training:
a norm and a BitLinear there and back.
"""
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import oracle
import synth
import ternary_weight_a8_b200 as tb
from conftest import ROOT
from parity import activations, dev, f32_bits, weights

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _gain(K, seed):
    return (1.0 + 0.1 * synth.activations_f32(1, K, seed=seed)[0]).astype(np.float32)


@pytest.mark.parametrize("M", [1, 5, 40, 300])
def test_blocks_and_head(M):
    K, V, eps = 640, 1003, 1e-6
    Ws = [oracle.pack_weights(weights(K, K, seed=50 + i)) for i in range(2)]
    gains = [_gain(K, 60 + i) for i in range(3)]
    wq_ref, ws_ref, _ = oracle.quant_act(weights(V, K, seed=70))
    packed = [dev(p) for p, _, _ in Ws]
    gammas = [dev(np.array([g], np.float32)) for _, g, _ in Ws]
    gd = [dev(g) for g in gains]
    wq, ws = tb.quant_weights_i8(dev(weights(V, K, seed=70)))
    x0, _ = activations(M, K, seed=80, dtype="bf16")
    r0, _ = activations(M, K, seed=81, dtype="bf16")

    def model():
        x, z, steps = x0, r0.clone(), []
        for i in range(3):
            before = z.clone()
            z, q, s, r = tb.add_rmsnorm_quant(x, z, gd[i], eps=eps, z=z)  # the residual stream, in place
            if i < 2:
                y = tb.forward_quantized(packed[i], gammas[i], q, s, r)
            else:
                y = tb.forward_i8_quantized(wq, ws, q, s, out_dtype=torch.float32)
            steps.append((x, before, z.clone(), q, s, r, y))
            x = y
        return steps

    steps = model()
    for i, (x, before, z, q, s, r, y) in enumerate(steps):
        z_ref = (x.float() + before.float()).bfloat16()
        assert torch.equal(z, z_ref)
        _, q_ref, s_ref, r_ref = oracle.rmsnorm_quant(z.float().cpu().numpy(), gains[i], eps, True)
        assert np.array_equal(q.cpu().numpy(), q_ref) and np.array_equal(r.cpu().numpy(), r_ref)
        assert np.array_equal(f32_bits(s.cpu().numpy()), f32_bits(s_ref))
        if i < 2:
            acc = oracle.accumulate(q_ref, Ws[i][2])
            want = oracle.dequant(acc, Ws[i][1], s_ref)
            # two roundings in fp32 and one to bf16
            assert (np.abs(y.float().cpu().numpy() - want) <= (2.0 ** -8 + 4 * U) * np.abs(want)).all()
        else:
            acc = (q_ref.astype(np.int64) @ wq_ref.astype(np.int64).T).astype(np.int32)
            f = (np.float32(1) / s_ref)[:, None] * (np.float32(1) / ws_ref)[None, :]
            assert np.array_equal(f32_bits(y.cpu().numpy()), f32_bits(acc.astype(np.float32) * f))
    # captured and replayed on new inputs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = model()
    logits = steps[-1][-1].clone()
    x0.mul_(0.5)
    graph.replay()
    changed = captured[-1][-1].clone()
    x0.mul_(2.0)
    graph.replay()
    assert torch.equal(captured[-1][-1], logits) and not torch.equal(changed, logits)


@pytest.mark.parametrize("M,K,N", [(8, 128, 64), (304, 2560, 640)])
def test_norm_and_layer_backward(M, K, N):
    """y = BitLinear(norm(x + residual)): dz through ste_backward's dx and the norm's gradient, against the formulas in
    64 bits on the codes that the forward made."""
    eps = 1e-5
    W = weights(N, K, seed=1)
    packed_ref, gamma_ref, T = oracle.pack_weights(W)
    packed, gamma = tb.pack_weights(dev(W))
    g = _gain(K, 2)
    x, _ = activations(M, K, seed=3, dtype="bf16")
    res, _ = activations(M, K, seed=4, dtype="bf16")
    z, q, s, r = tb.add_rmsnorm_quant(x, res, dev(g), eps=eps)
    rng = np.random.RandomState(5)
    dy = torch.from_numpy(rng.randn(M, N).astype(np.float32)).cuda().bfloat16()
    past = torch.from_numpy(rng.randn(M, K).astype(np.float32)).cuda().bfloat16()
    dn, _ = tb.ste_backward(packed, gamma, K, dy, q, s, dx_dtype=torch.float32, dw=False)
    dz, dgain = tb.add_rmsnorm_backward(z, dn, dev(g), eps=eps, dz_in=past)
    d64 = float(gamma_ref) * (dy.float().cpu().numpy().astype(np.float64) @ T.astype(np.float64))
    z64, g64 = z.float().cpu().numpy().astype(np.float64), g.astype(np.float64)
    rr = 1 / np.sqrt((z64 * z64).mean(1, keepdims=True) + float(np.float32(eps)))
    n = z64 * rr
    gd = d64 * g64
    want = rr * (gd - n * (gd * n).mean(1, keepdims=True)) + past.float().cpu().numpy()
    # The layer's gradient is off by N roundings of its terms at most; the norm's own error is far below that.
    terms = float(gamma_ref) * (np.abs(dy.float().cpu().numpy()).astype(np.float64) @ np.abs(T).astype(np.float64)) * np.abs(g64)
    off = U * (N + 200) * rr * (terms + np.abs(n) * (terms * np.abs(n)).mean(1, keepdims=True))
    bar = off + (2.0 ** -8 + 60 * U) * np.abs(want) + 60 * U * np.abs(past.float().cpu().numpy())
    assert (np.abs(dz.float().cpu().numpy() - want) <= bar).all()
    wg = (d64 * n).sum(0)
    assert (np.abs(dgain.cpu().numpy() - wg) <= U * (N + M + 300) * (terms / np.abs(g64) * np.abs(n)).sum(0)).all()


def test_all_calls_at_once_on_two_streams():
    """Two host threads, each on a stream of its own, every operator in every form at the same time."""
    sets = []
    for k in range(2):
        gen = torch.Generator(device="cuda").manual_seed(k)
        rnd = lambda *shape: torch.randn(shape, generator=gen, device="cuda")
        g = rnd(2560) * 0.1 + 1
        wide = rnd(40960) * 0.1 + 1
        wq, ws = tb.quant_weights_i8(rnd(6912, 2560))
        x = {m: rnd(m, 2560).bfloat16() for m in (1, 12, 47, 129, 700)}
        long = rnd(9, 40960)

        def calls(x=x, g=g, wide=wide, wq=wq, ws=ws, long=long):
            out = []
            for v in x.values():
                out.append(tb.forward_i8(wq, ws, v))
                z, q, s, r = tb.add_rmsnorm_quant(v, v, g)
                out += [z, q, s, r, tb.forward_i8_quantized(wq, ws, q, s, out_dtype=torch.float32)]
                out += tb.add_rmsnorm_backward(z, v, g, dz_in=v)
            out += tb.add_rmsnorm_backward(long, long, wide)
            out += tb.add_rmsnorm_quant(long, long, wide)
            return out
        sets.append((calls, calls()))
    torch.cuda.synchronize()
    bad = []

    def work(k):
        calls, want = sets[k]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(15):
                got = calls()
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want)):
                    bad.append(k)
    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad


def test_first_calls_inside_a_capture():
    """A process whose first calls are captured: nothing in them needs a call before."""
    code = """
import torch, ternary_weight_a8_b200 as tb
x = torch.randn((40, 2560), device="cuda").bfloat16()
g = torch.ones(2560, device="cuda")
W = torch.randint(-127, 128, (300, 2560), dtype=torch.int8, device="cuda")
ws = torch.ones(300, device="cuda")
big = torch.randint(-127, 128, (9000, 2560), dtype=torch.int8, device="cuda")
bws = torch.ones(9000, device="cuda")
xx = torch.randn((300, 2560), device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    z, q, s, r = tb.add_rmsnorm_quant(x, x, g)
    y = tb.forward_i8_quantized(W, ws, q, s)
    y1 = tb.forward_i8(W, ws, x[:1])
    y2 = tb.forward_i8(big, bws, xx)
    d = tb.add_rmsnorm_backward(x, x, g, dz_in=x)
graph.replay()
torch.cuda.synchronize()
e = tb.add_rmsnorm_quant(x, x, g)
assert torch.equal(e[1], q) and torch.equal(tb.forward_i8_quantized(W, ws, q, s), y)
assert torch.equal(tb.forward_i8(W, ws, x[:1]), y1) and torch.equal(tb.forward_i8(big, bws, xx), y2)
f = tb.add_rmsnorm_backward(x, x, g, dz_in=x)
assert torch.equal(f[0], d[0]) and torch.equal(f[1], d[1])
print("same")
"""
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=240)
    assert out.returncode == 0 and out.stdout.strip() == "same", out.stderr[-2000:]
