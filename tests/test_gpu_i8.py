"""The 8-bit product with a scale for each token and each output channel, on the GPU.

Accumulators against 64-bit products of the codes, which are exact, bit for
bit.  Outputs bit for bit against the documented fp32 steps
fp32(acc) * ((1 / s) * (1 / ws)), done by numpy, and within the bar of their
roundings of the exact acc / (s ws): both reciprocals, their product, the
accumulator's conversion and the last product are half a step each, 5 * 2^-24
(1 + 2^-20), and for bf16 one more of 2^-8.
"""
import threading

import numpy as np
import pytest
import torch

import oracle
import ternary_weight_a8_b200 as tb
from parity import activations, dev, f32_bits, weights

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _codes(rows, K, seed, full=True):
    rng = np.random.RandomState(seed)
    q = rng.randint(-128 if full else -127, 128, size=(rows, K)).astype(np.int8)
    s = np.exp(rng.uniform(-3, 8, size=rows)).astype(np.float32)
    return q, s


def _exact_acc(q, w):
    return (q.astype(np.float64) @ w.astype(np.float64).T).astype(np.int64)


def _want(acc, s, ws, dtype):
    f = (np.float32(1) / s)[:, None] * (np.float32(1) / ws)[None, :]
    y = acc.astype(np.int32).astype(np.float32) * f
    return torch.from_numpy(y).to(dtype).float().numpy()


def _check(y, acc, q, s, w, ws):
    acc_ref = _exact_acc(q, w)
    assert np.array_equal(acc.cpu().numpy(), acc_ref)
    got = y.float().cpu().numpy()
    assert np.array_equal(f32_bits(got), f32_bits(_want(acc_ref, s, ws, y.dtype)))
    real = acc_ref / (s.astype(np.float64)[:, None] * ws.astype(np.float64)[None, :])
    rel = 5 * U * (1 + 2.0 ** -20) + (2.0 ** -8 if y.dtype == torch.bfloat16 else 0.0)
    assert (np.abs(got - real) <= rel * np.abs(real)).all()


SHAPES = [  # M, N, K
    (1, 1, 64), (1, 17, 64), (2, 5, 192), (1, 6912, 2560), (3, 333, 320), (7, 64, 8640), (8, 100, 128), (9, 1000, 640),
    (16, 3200, 8640), (17, 16, 2560), (24, 515, 1024), (31, 257, 64), (32, 2560, 6912),
    (33, 1, 64), (33, 130, 192), (47, 6912, 2560), (64, 63, 8640), (100, 2561, 320), (128, 64, 28672), (128, 10240, 512),
    (129, 70, 128), (129, 2560, 2560), (200, 20000, 192), (255, 333, 1024), (256, 4096, 64), (300, 7001, 448),
    (513, 515, 2560), (700, 6912, 320), (1025, 9472, 256),
]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_parity(M, N, K, dtype):
    q, s = _codes(M, K, M + K)
    w, ws = _codes(N, K, N + K)
    wd, wsd, qd, sd = dev(w), dev(ws), dev(q), dev(s)
    y, acc = tb.forward_i8_quantized(wd, wsd, qd, sd, out_dtype=dtype, acc_out=True)
    _check(y, acc, q, s, w, ws)
    assert torch.equal(tb.forward_i8_quantized(wd, wsd, qd, sd, out_dtype=dtype), y)
    if M <= 32:  # the other kernel
        tb.set_path(tb.PATH_GEMM)
        try:
            y2, acc2 = tb.forward_i8_quantized(wd, wsd, qd, sd, out_dtype=dtype, acc_out=True)
            y3 = tb.forward_i8_quantized(wd, wsd, qd, sd, out_dtype=dtype)
        finally:
            tb.set_path(tb.PATH_AUTO)
        assert torch.equal(acc2, acc) and torch.equal(y2, y) and torch.equal(y3, y)


# 64-byte chunks of a row, which 8 warps share in batches: none for some warps,
# one each, shares of unequal length, whole batches and batches cut short.
@pytest.mark.parametrize("chunks", [1, 7, 8, 9, 16, 17, 24, 39, 40, 41, 63, 64, 65, 81, 135])
def test_decode_batches_and_grids(chunks):
    K = 64 * chunks
    gen = torch.Generator("cuda").manual_seed(chunks)
    w = torch.randint(-128, 128, (38001, K), dtype=torch.int8, device="cuda", generator=gen)
    ws = torch.rand(38001, device="cuda", generator=gen) + 0.5
    for M in (1, 8, 16, 31):
        q = torch.randint(-128, 128, (M, K), dtype=torch.int8, device="cuda", generator=gen)
        s = torch.rand(M, device="cuda", generator=gen) + 0.5
        x = torch.randn(M, K, device="cuda", generator=gen)
        full = (q.double() @ w.double().T).to(torch.int32)  # exact
        xq, xs, _ = tb.quant_act(x)
        raw = (xq.double() @ w.double().T).to(torch.int32)
        # One to five and sixteen blocks of 16 rows per SM, the last one cut.
        for N in (2361, 4733, 7101, 9470, 11800, 38001):
            y, acc = tb.forward_i8_quantized(w[:N], ws[:N], q, s, out_dtype=torch.float32, acc_out=True)
            assert torch.equal(acc, full[:, :N]), (M, N)
            f = torch.ones_like(s).div(s)[:, None] * torch.ones_like(ws[:N]).div(ws[:N])
            assert torch.equal(y, full[:, :N].float() * f), (M, N)
            acc = tb.forward_i8(w[:N], ws[:N], x, acc_out=True)[1]
            assert torch.equal(acc, raw[:, :N]), (M, N)


@pytest.mark.parametrize("M", [1, 2, 3, 5, 8, 32, 40, 300])
@pytest.mark.parametrize("K", [64, 2048, 2560, 8640, 16384, 16448])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantises_activations(M, K, dtype):
    """forward_i8 = quant_act, then the product on its codes; the weights through quant_weights_i8."""
    N = 210
    W = weights(N, K, seed=K)
    x, xf = activations(M, K, seed=M + K, dtype=dtype)
    wq_ref, ws_ref, _ = oracle.quant_act(W)
    q_ref, s_ref, _ = oracle.quant_act(xf)
    wq, ws = tb.quant_weights_i8(dev(W))
    assert np.array_equal(wq.cpu().numpy(), wq_ref) and np.array_equal(f32_bits(ws.cpu().numpy()), f32_bits(ws_ref))
    y, acc = tb.forward_i8(wq, ws, x, out_dtype=torch.float32, acc_out=True)
    _check(y, acc, q_ref, s_ref, wq_ref, ws_ref)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(8, 64), (6, 512), (3, 1024), (7, 960), (4, 2048), (3, 320),  # quantised by the product's blocks
                                 (9, 192), (9, 8640), (700, 320), (2500, 64), (3, 16448), (3, 40960)])
def test_codes_of_any_activations(M, K, dtype):
    """The call's own codes are quant_act's: zero, tiny and huge tokens, tokens with infinities and NaN, lengths of every
    form of the kernel; seen through the identity's rows as weights."""
    x = torch.randn((M, K), generator=torch.Generator().manual_seed(K)).to(dtype)
    x[0] = 0
    x[1] *= 1e20
    x[2, 3] = float("inf")
    if M > 5:
        x[3] *= 1e-30
        x[4, 5] = float("nan")
        x[5, 6], x[5, 7] = float("-inf"), float("nan")
    x = x.cuda()
    q, s, _ = tb.quant_act(x)
    rows = torch.arange(0, K, max(1, K // 500), device="cuda")
    eye = torch.zeros((rows.numel(), K), dtype=torch.int8, device="cuda")
    eye[torch.arange(rows.numel(), device="cuda"), rows] = 1
    ones = torch.ones(rows.numel(), device="cuda")
    y, acc = tb.forward_i8(eye, ones, x, out_dtype=torch.float32, acc_out=True)
    y2, acc2 = tb.forward_i8_quantized(eye, ones, q, s, out_dtype=torch.float32, acc_out=True)
    assert torch.equal(acc, q[:, rows].int()) and torch.equal(acc2, acc)
    assert torch.equal(torch.nan_to_num(y, nan=7.0), torch.nan_to_num(y2, nan=7.0))


@pytest.mark.parametrize("M", [1, 40])
def test_extreme_sums(M):
    """The longest sums of the largest codes: -128 * -128 * K stays inside int32."""
    K, N = 131008, 3
    q = np.full((M, K), -128, np.int8)
    w = np.full((N, K), -128, np.int8)
    w[1] = 127
    s, ws = np.full(M, 2.0, np.float32), np.full(N, 4.0, np.float32)
    y, acc = tb.forward_i8_quantized(dev(w), dev(ws), dev(q), dev(s), out_dtype=torch.float32, acc_out=True)
    _check(y, acc, q, s, w, ws)
    big = torch.zeros((1, 131072), dtype=torch.int8, device="cuda")
    with pytest.raises(tb.BitLinearError) as e:
        tb.forward_i8_quantized(big, dev(ws[:1]), big, dev(s[:1]))
    assert e.value.code == tb.BL_ERR_UNSUPPORTED_SHAPE


@pytest.mark.parametrize("M", [2, 50])
def test_zero_tokens_and_channels(M):
    """A zero token or channel gives zeros; its scale is 127 / 1e-5."""
    W = weights(70, 256, seed=1)
    W[3] = 0
    x, xf = activations(M, 256, seed=2, dtype="f32")
    x[1] = 0
    wq, ws = tb.quant_weights_i8(dev(W))
    y = tb.forward_i8(wq, ws, x, out_dtype=torch.float32)
    assert not y[1].any() and not y[:, 3].any() and torch.isfinite(y).all() and y[0].any()
    assert tb.forward_i8(wq, ws, x[:0]).shape == (0, 70)


@pytest.mark.parametrize("M,N,K", [(1, 333, 320), (20, 64, 128), (40, 100, 8640), (150, 4001, 192), (300, 9000, 128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_no_writes_outside_outputs(M, N, K, dtype):
    pad, canary = 4096, 0x5A
    q, s = _codes(M, K, 1)
    w, ws = _codes(N, K, 2)
    size = M * N * (2 if dtype == torch.bfloat16 else 4)
    ybuf = torch.full((2 * pad + size,), canary, dtype=torch.uint8, device="cuda")
    abuf = torch.full((2 * pad + M * N * 4,), canary, dtype=torch.uint8, device="cuda")
    wbuf = torch.full((256 + pad,), canary, dtype=torch.uint8, device="cuda")
    wbuf[:256] = 0
    y, acc = ybuf[pad:pad + size].view(dtype).view(M, N), abuf[pad:pad + M * N * 4].view(torch.int32).view(M, N)
    tb.forward_i8_quantized(dev(w), dev(ws), dev(q), dev(s), y=y, acc_out=acc, workspace=wbuf[:256])
    _check(y, acc, q, s, w, ws)
    for buf in (ybuf[:pad], ybuf[-pad:], abuf[:pad], abuf[-pad:], wbuf[256:]):
        assert (buf == canary).all()
    assert tb.device_status(wbuf[:256]) == tb.BL_OK


@pytest.mark.parametrize("M", [1, 48, 512])
def test_weights_written_just_before(M):
    """Weights that the kernel just before the call wrote: every call sees them whole."""
    N, K = 4096, 2560
    x, _ = activations(M, K, seed=1, dtype="bf16")
    xq, s, _ = tb.quant_act(x)
    sets = [dev(weights(N, K, seed=10 + i)) for i in range(2)]
    want = []
    for W in sets:
        wq, ws = tb.quant_weights_i8(W)
        torch.cuda.synchronize()
        want.append(tb.forward_i8_quantized(wq, ws, xq, s))
    torch.cuda.synchronize()
    wq, ws = torch.empty((N, K), dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    got = []
    for i in range(30):
        tb.quant_weights_i8(sets[i % 2], wq, ws)
        got.append((tb.forward_i8_quantized if i % 4 < 2 else tb.forward_i8)(wq, ws, *((xq, s) if i % 4 < 2 else (x,))))
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 2]), i


@pytest.mark.parametrize("M", [3, 40, 300])
def test_streams_threads_and_graphs(M):
    N, K = 3001, 2560
    wq, ws = tb.quant_weights_i8(dev(weights(N, K, seed=1)))
    xs = [activations(M, K, seed=20 + k, dtype="bf16")[0] for k in range(2)]
    want = [tb.forward_i8(wq, ws, x) for x in xs]
    torch.cuda.synchronize()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = tb.forward_i8(wq, ws, xs[0], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want[0])
    bad = []

    def work(k):
        with torch.cuda.stream(side):
            for _ in range(20):
                y = tb.forward_i8(wq, ws, xs[k])
                side.synchronize()
                if not torch.equal(y, want[k]):
                    bad.append(k)
    threads = [threading.Thread(target=work, args=(k,)) for k in (0, 1)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad
    graphs = []
    for k in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = tb.forward_i8(wq, ws, xs[k])
        graphs.append((graph, y))
    for _ in range(10):
        with torch.cuda.stream(side):
            graphs[0][0].replay()
        with torch.cuda.stream(other):
            graphs[1][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], want[0]) and torch.equal(graphs[1][1], want[1])


@pytest.mark.parametrize("M", [2, 12, 40, 300])
def test_weight_offsets_past_32_bits(M):
    """Weights of more than 2^31 bytes: the first, middle and last channels as calls of their own give them."""
    N, K = 262144 + 37, 8192
    w = torch.empty((N, K), dtype=torch.int8, device="cuda")
    for i in range(0, N, 65536):
        w[i:i + 65536] = torch.randint(-127, 128, (min(65536, N - i), K), dtype=torch.int8, device="cuda")
    ws = torch.rand(N, device="cuda") + 0.5
    q, s = _codes(M, K, 5)
    qd, sd = dev(q), dev(s)
    y = tb.forward_i8_quantized(w, ws, qd, sd, out_dtype=torch.float32)
    for at in (slice(0, 50), slice(131060, 131090), slice(N - 70, N)):
        assert torch.equal(y[:, at], tb.forward_i8_quantized(w[at].contiguous(), ws[at], qd, sd, out_dtype=torch.float32))


@pytest.mark.parametrize("N,dtype", [(65536, torch.bfloat16), (65529, torch.float32)])
def test_output_offsets_past_32_bits(N, dtype):
    """More than 2^31 outputs, in boxes and row by row: the first, middle and last tokens."""
    M, K = 32768 + 41, 64
    w, ws = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda"), torch.rand(N, device="cuda") + 0.5
    q = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda")
    s = torch.rand(M, device="cuda") + 0.5
    y = tb.forward_i8_quantized(w, ws, q, s, out_dtype=dtype)
    for at in (slice(0, 9), slice(16380, 16390), slice(M - 60, M)):
        assert torch.equal(y[at], tb.forward_i8_quantized(w, ws, q[at].contiguous(), s[at].contiguous(), out_dtype=dtype))


def test_refusals():
    w, ws = torch.zeros((64, 128), dtype=torch.int8, device="cuda"), torch.ones(64, device="cuda")
    q, s = torch.zeros((4, 128), dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda")
    x = torch.zeros((4, 128), device="cuda")
    for bad in (lambda: tb.forward_i8(w, ws, x[:, :64].contiguous()), lambda: tb.forward_i8(w.float(), ws, x),
                lambda: tb.forward_i8(w, ws[:3], x), lambda: tb.forward_i8(w, ws.double(), x),
                lambda: tb.forward_i8(w, ws, x.half()), lambda: tb.forward_i8(w, ws, x, out_dtype=torch.float16),
                lambda: tb.forward_i8(w.cpu(), ws, x), lambda: tb.forward_i8(w, ws, x.cpu()),
                lambda: tb.forward_i8(w.t(), ws, x), lambda: tb.forward_i8(w, ws, x, y=torch.empty((4, 65), device="cuda")),
                lambda: tb.forward_i8_quantized(w, ws, x, s), lambda: tb.forward_i8_quantized(w, ws, q, s[:2]),
                lambda: tb.forward_i8_quantized(w, ws, q, s, acc_out=torch.empty((4, 64), device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    odd = torch.zeros((4, 96), dtype=torch.int8, device="cuda")
    many = torch.zeros((33, 128), dtype=torch.int8, device="cuda")
    buf = torch.zeros(4 * 128 + 64, dtype=torch.int8, device="cuda")
    for bad, code in ((lambda: tb.forward_i8_quantized(odd, torch.ones(4, device="cuda"), odd, s), tb.BL_ERR_UNSUPPORTED_SHAPE),
                      (lambda: tb.forward_i8(w, ws, x, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")),
                       tb.BL_ERR_WORKSPACE_TOO_SMALL),
                      (lambda: tb.forward_i8_quantized(w, ws, buf[1:513].view(4, 128), s), tb.BL_ERR_MISALIGNED),
                      (lambda: tb.forward_i8_quantized(w, ws, q, s, y=w.view(-1)[:1024].view(torch.float32).view(4, 64)),
                       tb.BL_ERR_INVALID_ARG)):
        with pytest.raises(tb.BitLinearError) as e:
            bad()
        assert e.value.code == code
    tb.set_path(tb.PATH_GEMV)
    try:
        with pytest.raises(tb.BitLinearError) as e:
            tb.forward_i8_quantized(w, ws, many, torch.ones(33, device="cuda"))
        assert e.value.code == tb.BL_ERR_UNSUPPORTED_SHAPE
    finally:
        tb.set_path(tb.PATH_AUTO)
