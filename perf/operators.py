"""What is measured of the 8-bit operators around the ternary layers: the cases, their plain forms and their 64-bit values.

Three operators of a block whose products run on 8-bit activations:

  norm       z = x + residual, stored; v = RMSNorm(z) * gain, stored precision; the 8-bit codes of v with a scale and a
             code sum for each token (``add_rmsnorm_quant``);
  norm_back  the gradient of that norm and sum for training through latent weights: dz from the gradient of v and the
             gradient that reaches z past the norm, and the gradient of the gain (``add_rmsnorm_backward``);
  product    y = x . W^T in 8-bit integers with a scale for each token and each output channel, for the layers that
             are not ternary (``forward_i8``, and ``forward_i8_quantized`` on codes that a norm wrote).

``own`` chooses between the plain forms (elementary torch operations) and the framework's calls on the same state.
"""
import random

import numpy as np
import torch

own = False

EPS = 1e-5
ACT_EPS = 1e-5  # the smallest absolute maximum that a token's scale divides by

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _tb():
    import ternary_weight_a8_b200 as tb
    return tb


# ----------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # One decoded token of the 2560-wide model: the call's own latency.
        {"name": "norm_1x2560", "op": "norm", "M": 1, "K": 2560, "dtype": "bf16", "gain": True},
        # Sixteen sequences decoded together at the 8192-wide model.
        {"name": "norm_16x8192", "op": "norm", "M": 16, "K": 8192, "dtype": "bf16", "gain": True},
        # A prompt of 2048 tokens at the 2560-wide model.
        {"name": "norm_2048x2560", "op": "norm", "M": 2048, "K": 2560, "dtype": "bf16", "gain": True},
        # The sub-layer norm in front of the down layer, fp32 activations, a ragged prompt, no gain.
        {"name": "norm_1021x8640_f32", "op": "norm", "M": 1021, "K": 8640, "dtype": "f32", "gain": False},
        # A training step's tokens at the 8192-wide model, there and back.
        {"name": "norm_8192x8192", "op": "norm", "M": 8192, "K": 8192, "dtype": "bf16", "gain": True},
        {"name": "norm_back_8192x8192", "op": "norm_back", "M": 8192, "K": 8192, "dtype": "bf16", "grad": "bf16",
         "gain": True, "past": True},
        # A small training batch of ragged length at the 3200-wide model, fp32 gradients as the layers' backward gives
        # them, nothing past the norm (the first block).
        {"name": "norm_back_777x3200_f32", "op": "norm_back", "M": 777, "K": 3200, "dtype": "f32", "grad": "f32",
         "gain": True, "past": False},
        # One token through a vocabulary's 128000 output channels: the weights' stream.
        {"name": "product_1x2560x128000", "op": "product", "M": 1, "K": 2560, "N": 128000, "x": "bf16", "y": "f32"},
        # Eight tokens through the short, wide layer of the 3200-wide model, on codes that the norm before it wrote.
        {"name": "product_8x8640x3200_codes", "op": "product", "M": 8, "K": 8640, "N": 3200, "x": "codes", "y": "bf16"},
        # A ragged batch of 47 tokens, more than one token tile of the decode form holds.
        {"name": "product_47x2560x6912", "op": "product", "M": 47, "K": 2560, "N": 6912, "x": "bf16", "y": "bf16"},
        # A prompt of 2048 tokens at the 2560-wide model.
        {"name": "product_2048x2560x6912", "op": "product", "M": 2048, "K": 2560, "N": 6912, "x": "bf16", "y": "bf16"},
        # The same at the 8192-wide model's feed-forward width: the tensor cores' rate.
        {"name": "product_2048x8192x28672", "op": "product", "M": 2048, "K": 8192, "N": 28672, "x": "bf16", "y": "bf16"},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng: random.Random):
    """A case of the same ranges: any token count and output width, inputs in multiples of 64."""
    op = rng.choice(["norm", "norm_back", "product", "product"])
    K = 64 * _log_uniform(rng, 1, 448)
    if op == "product":
        N = min(_log_uniform(rng, 1, 131072), 327_680_000 // K)
        M = _log_uniform(rng, 1, 4096)
        M = max(1, min(M, 2048 * 8192 * 28672 // (N * K), 2048 * 28672 // N))
        return {"op": op, "M": M, "K": K, "N": N, "x": rng.choice(["bf16", "f32", "codes"]), "y": rng.choice(["bf16", "f32"])}
    M = min(_log_uniform(rng, 1, 16384), 8192 * 8192 // (2 * K))
    case = {"op": op, "M": M, "K": K, "dtype": rng.choice(["bf16", "f32"]), "gain": rng.random() < 0.75}
    if op == "norm_back":
        case["grad"] = rng.choice(["bf16", "f32"])
        case["past"] = rng.random() < 0.75
    return case


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------

def _activations(M, K, dtype, gen, spread=1.0):
    """N(0, spread) with one channel in a hundred twenty times larger, as a trained model's activations have."""
    x = torch.randn((M, K), generator=gen, device="cuda") * spread
    n = max(1, K // 100)
    x[:, torch.randperm(K, generator=gen, device="cuda")[:n]] *= 20.0
    return x.to(dtype)


def _codes(v):
    """The per-token codes and scale of v (fp32): s = 127 / max(|v|), q = rint(v * s)."""
    amax = v.abs().amax(dim=-1).clamp_min(ACT_EPS)
    s = torch.full_like(amax, 127.0) / amax  # one 32-bit division (a number over a tensor would be a reciprocal's product)
    return torch.round(v * s[:, None]).clamp_(-128, 127).to(torch.int8), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    M, K = case["M"], case["K"]
    s = {"case": case}
    if case["op"] == "product":
        W = torch.randn((case["N"], K), generator=gen, device="cuda") * 0.02
        s["wq"], s["wscale"] = _codes(W)
        if case["x"] == "codes":
            s["xq"], s["scale"] = _codes(_activations(M, K, torch.bfloat16, gen).float())
        else:
            s["x"] = _activations(M, K, _DTYPES[case["x"]], gen)
        return s
    dt = _DTYPES[case["dtype"]]
    s["gain"] = 1.0 + 0.1 * torch.randn(K, generator=gen, device="cuda") if case["gain"] else None
    if case["op"] == "norm":
        s["x"] = _activations(M, K, dt, gen)
        s["residual"] = _activations(M, K, dt, gen, 4.0)
    else:
        s["z"] = _activations(M, K, dt, gen, 4.0)
        s["dnorm"] = (torch.randn((M, K), generator=gen, device="cuda") * 1e-2).to(_DTYPES[case["grad"]])
        s["dz_in"] = (torch.randn((M, K), generator=gen, device="cuda") * 1e-2).to(dt) if case["past"] else None
    return s


# ----------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    tb = _tb()
    c = s["case"]
    if c["op"] == "norm":
        z, xq, scale, rowsum = tb.add_rmsnorm_quant(s["x"], s["residual"], s["gain"], eps=EPS)
        return {"z": z, "v": xq / scale[:, None], "scale": scale, "rowsum": rowsum}
    if c["op"] == "norm_back":
        dz, dgain = tb.add_rmsnorm_backward(s["z"], s["dnorm"], s["gain"], eps=EPS, dz_in=s["dz_in"])
        return {"dz": dz} if dgain is None else {"dz": dz, "dgain": dgain}
    if c["x"] == "codes":
        return tb.forward_i8_quantized(s["wq"], s["wscale"], s["xq"], s["scale"], out_dtype=_DTYPES[c["y"]])
    return tb.forward_i8(s["wq"], s["wscale"], s["x"], out_dtype=_DTYPES[c["y"]])


def _rstd(z):
    """1 / sqrt(mean z^2 + eps) of each row: summed in 64 bits (v and its codes are decided from it), rounded once."""
    ms = z.double().square().mean(dim=-1)
    return (1.0 / torch.sqrt(ms + float(np.float32(EPS)))).float()


def _plain(s):
    c = s["case"]
    if c["op"] == "norm":
        z = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
        v = z.float() * _rstd(z)[:, None]
        if s["gain"] is not None:
            v = v * s["gain"]
        q, scale = _codes(v.to(z.dtype).float())
        return {"z": z, "v": q / scale[:, None], "scale": scale, "rowsum": q.sum(dim=-1, dtype=torch.int32)}
    if c["op"] == "norm_back":
        z, dv = s["z"].float(), s["dnorm"].float()
        n = z * _rstd(z)[:, None]
        g = dv if s["gain"] is None else dv * s["gain"]
        dz = (g - n * (g * n).mean(dim=-1, keepdim=True)) * _rstd(z)[:, None]
        if s["dz_in"] is not None:
            dz = dz + s["dz_in"].float()
        out = {"dz": dz.to(s["z"].dtype)}
        if s["gain"] is not None:
            out["dgain"] = (dv * n).sum(dim=0)
        return out
    q, scale = (s["xq"], s["scale"]) if c["x"] == "codes" else _codes(s["x"].float())
    y = (q.float() @ s["wq"].float().t()) / scale[:, None] / s["wscale"]
    return y.to(_DTYPES[c["y"]])


# ----------------------------------------------------------------------------
# What one pass cannot do without
# ----------------------------------------------------------------------------

_BYTES = {"bf16": 2, "f32": 4, "codes": 1}


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "product":
        N = case["N"]
        x = _BYTES[case["x"]] * M * K + (4 * M if case["x"] == "codes" else 0)
        return {"bytes": N * K + 4 * N + x + _BYTES[case["y"]] * M * N, "flops": 2 * M * N * K}
    e = _BYTES[case["dtype"]]
    gain = 4 * K if case["gain"] else 0
    if case["op"] == "norm":
        # x and the residual in, z and the codes out, scale and code sum of each token.
        return {"bytes": M * K * (3 * e + 1) + gain + 8 * M, "flops": 8 * M * K}
    # z, the gradient of v and the gradient past the norm in; dz and the gain's gradient out.
    return {"bytes": M * K * ((3 if case["past"] else 2) * e + _BYTES[case["grad"]]) + 2 * gain, "flops": 10 * M * K}


# ----------------------------------------------------------------------------
# The definitions in 64 bits
# ----------------------------------------------------------------------------

def _f32(a):
    """Rounds 64-bit values to 32 bits where the definition does (a product of two 32-bit values is exact in 64)."""
    return a.to(torch.float32).to(torch.float64)


def _exact_codes(v):
    """Codes and scale of 64-bit copies of stored values: a 32-bit quotient, 32-bit products, ties to even."""
    amax = torch.clamp(torch.max(torch.abs(v), dim=1).values, min=float(np.float32(ACT_EPS)))
    s = _f32(127.0 / amax)
    return torch.round(_f32(v * s.unsqueeze(1))).clamp(-128.0, 127.0), s


def exact(case, seed):
    st = prepare(case, seed)
    M, K = case["M"], case["K"]
    f64 = torch.float64
    if case["op"] == "product":
        if case["x"] == "codes":
            q, sx = st["xq"].to(f64), st["scale"].to(f64)
        else:
            q, sx = _exact_codes(st["x"].to(f64))
        y = torch.empty((M, case["N"]), dtype=f64, device="cuda")
        rows = max(1, (1 << 28) // K)  # a quarter of a gigavalue of weights at a time
        for n in range(0, case["N"], rows):
            w = st["wq"][n:n + rows].to(f64) / st["wscale"][n:n + rows].to(f64).unsqueeze(1)
            y[:, n:n + rows] = torch.matmul(q / sx.unsqueeze(1), w.t())
        return y
    eps = float(np.float32(EPS))
    gain = st["gain"].to(f64) if st["gain"] is not None else torch.ones(K, dtype=f64, device="cuda")
    if case["op"] == "norm":
        z = (st["x"].to(f64) + st["residual"].to(f64))
        z = _f32(z).to(st["x"].dtype).to(f64)
        r = _f32(torch.rsqrt(torch.sum(z * z, dim=1) / K + eps))
        v = _f32(_f32(z * r.unsqueeze(1)) * gain).to(st["x"].dtype).to(f64)
        q, s = _exact_codes(v)
        return {"z": z, "v": q / s.unsqueeze(1), "scale": s, "rowsum": torch.sum(q, dim=1).to(torch.int32)}
    z, dv = st["z"].to(f64), st["dnorm"].to(f64)
    r = torch.rsqrt(torch.sum(z * z, dim=1) / K + eps)
    dn = dv * gain
    dot = torch.sum(dn * z, dim=1)
    dz = dn * r.unsqueeze(1) - z * (dot * r ** 3 / K).unsqueeze(1)
    if st["dz_in"] is not None:
        dz += st["dz_in"].to(f64)
    out = {"dz": dz}
    if st["gain"] is not None:
        out["dgain"] = torch.sum(dv * z * r.unsqueeze(1), dim=0)
    return out
