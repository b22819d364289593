"""Cases of the W8A8 layer's operators around and including its matrix product.

Three operators, each with its plain form in elementary torch operations:

* ``norm``: residual addition, root-mean-square norm, optional Hadamard
  rotation and int8 quantization with one scale per token
  (``w8a8_add_rmsnorm_quantize``);
* ``silu``: SiLU(gate) * up with the same rotation and quantization
  (``w8a8_silu_mul_quantize``);
* ``matmul``: the int8 product with a scale per token and per output channel
  (``w8a8_matmul``).

Codes are returned as the values they stand for (code times scale, in bf16),
beside the scales themselves.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one decoded token through a block's input norm
        dict(name="norm_decode", op="norm", M=1, K=4096, dtype="bf16", group=0, residual=True, pad=0),
        # the tokens of one image and its text, rotated for layers whose weights are rotated
        dict(name="norm_rotated", op="norm", M=4608, K=4096, dtype="bf16", group=128, residual=True, pad=0),
        # odd width and token count, no alignment of the rows, no residual yet (first block)
        dict(name="norm_ragged", op="norm", M=517, K=2777, dtype="fp16", group=0, residual=False, pad=0),
        # a long prefill of a wide model
        dict(name="norm_prefill", op="norm", M=16384, K=8192, dtype="bf16", group=0, residual=True, pad=0),
        # a decoded batch between the two products of a gated MLP
        dict(name="silu_decode", op="silu", M=8, K=14336, dtype="bf16", group=0),
        # the tokens of one image at the MLP width, rotated
        dict(name="silu_rotated", op="silu", M=4608, K=12288, dtype="bf16", group=128),
        # fp32 activations of an odd width: the second half starts off every alignment
        dict(name="silu_ragged", op="silu", M=1021, K=5461, dtype="fp32", group=0),
        # one decoded token through a square projection
        dict(name="matmul_decode", op="matmul", M=1, N=4096, K=4096, out="bf16", bias=False, group=0),
        # a decoded batch through gate and up laid side by side
        dict(name="matmul_batch", op="matmul", M=16, N=28672, K=4096, out="bf16", bias=False, group=0),
        # a short prompt through the MLP's down projection, rotated codes
        dict(name="matmul_prompt", op="matmul", M=256, N=4096, K=12288, out="bf16", bias=True, group=128),
        # odd sizes in every direction, unrounded output
        dict(name="matmul_ragged", op="matmul", M=333, N=1013, K=2995, out="fp32", bias=True, group=0),
        # a long prefill of a wide model
        dict(name="matmul_prefill", op="matmul", M=8192, N=24576, K=8192, out="bf16", bias=False, group=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "silu", "matmul"])
    if op == "matmul":
        M, N, K = _log(rng, 1, 8192), _log(rng, 8, 28672), _log(rng, 16, 16384)
        while M * N * K > 8192 * 24576 * 8192:
            M = max(1, M // 2)
        return dict(op=op, M=M, N=N, K=K, out=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    bias=rng.random() < 0.5, group=rng.choice([0, 64, 128]))
    most = 16384 * 8192
    M, K = _log(rng, 1, 16384), _log(rng, 32, 32768 if op == "silu" else 16384)
    group = rng.choice([0, 0, 64, 128])
    if group:
        K = max(128, K // 128 * 128)
    while M * K * (1 if op == "norm" else 2) > most:
        M = max(1, M // 2)
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if dtype == "fp32":
        M = max(1, M // 2)
    if op == "silu":
        return dict(op=op, M=M, K=K, dtype=dtype, group=group)
    return dict(op=op, M=M, K=K, dtype=dtype, group=group, residual=rng.random() < 0.7,
                pad=rng.choice([0, 0, 8, 24, 5]))


def _rows(K, per=16):
    return (K + per - 1) // per * per


def _channels(n, gen, dev):
    """Per-channel magnitudes of activations: one in a hundred is 5 to 15 times the rest."""
    u = torch.rand(n, generator=gen, device=dev)
    big = 5 + 10 * torch.rand(n, generator=gen, device=dev)
    return torch.where(u < 0.01, big, torch.ones_like(big))


def _codes(rows, K, gen, dev):
    """int8 codes [rows, K] as a quantizer leaves them, rows 16-byte aligned."""
    c = torch.empty((rows, _rows(K)), dtype=torch.int8, device=dev)
    step = max(1, (1 << 27) // c.shape[1])
    for i in range(0, rows, step):
        x = torch.randn(c[i:i + step].shape, generator=gen, device=dev)
        c[i:i + step] = x.mul_(34).round_().clamp_(-127, 127).to(torch.int8)
    return c[:, :K]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed) & 0x7FFFFFFF)
    M, K = case["M"], case["K"]
    st = dict(case)
    if case["op"] == "matmul":
        N = case["N"]
        st["A"] = _codes(M, K, gen, dev)
        st["B"] = _codes(N, K, gen, dev)
        st["a_scale"] = 0.01 + 0.05 * torch.rand(M, generator=gen, device=dev)
        st["b_scale"] = 0.0002 + 0.0006 * torch.rand(N, generator=gen, device=dev)
        dt = DTYPES[case["out"]]
        st["bias_v"] = torch.randn(N, generator=gen, device=dev).mul_(0.1).to(dt) if case["bias"] else None
        st["Y"] = torch.empty((M, N), dtype=dt, device=dev)
        return st
    dt = DTYPES[case["dtype"]]
    if case["op"] == "silu":
        # gate and up as one product leaves them: the halves of [M, 2 K]
        both = torch.randn((M, 2 * K), generator=gen, device=dev)
        both *= _channels(2 * K, gen, dev)
        both = both.to(dt)
        st["gate"], st["up"] = both[:, :K], both[:, K:]
    else:
        X = torch.randn((M, K + case["pad"]), generator=gen, device=dev)
        X *= _channels(K + case["pad"], gen, dev)
        live = torch.arange(M, device=dev)[:, None] % 97 != 96     # every 97th row is padding, all zeros
        X *= live
        st["X"] = X.to(dt)[:, :K]
        st["R"] = None
        st["H"] = None
        if case["residual"]:
            R = torch.randn((M, K), generator=gen, device=dev).mul_(2.0)
            st["R"] = (R * live).to(dt)
            st["H"] = torch.empty((M, K), dtype=dt, device=dev)
        st["gamma"] = (1 + 0.1 * torch.randn(K, generator=gen, device=dev)).to(dt)
    st["Xq"] = torch.empty((M, _rows(K)), dtype=torch.int8, device=dev)[:, :K]
    st["x_scale"] = torch.empty((M,), dtype=torch.float32, device=dev)
    st["values"] = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
    return st


def _hadamard(g, dtype, dev):
    i = torch.arange(g, device=dev)
    bits = i[:, None] & i[None, :]
    odd = torch.zeros_like(bits)
    odd = odd ^ bits ^ (bits >> 1) ^ (bits >> 2) ^ (bits >> 3) ^ (bits >> 4) ^ (bits >> 5) ^ (bits >> 6)
    return (1 - 2 * (odd & 1)).to(dtype)


def _quantized(y, group):
    """Plain rotation and quantization of fp32 rows: (values of the codes in bf16, scales)."""
    M, K = y.shape
    if group:
        y = (y.view(M, K // group, group) @ _hadamard(group, y.dtype, y.device)).view(M, K)
    s = y.abs().amax(dim=1) / 127
    q = torch.where(s[:, None] > 0, torch.round(y / s[:, None]), torch.zeros_like(y)).clamp(-127, 127)
    return (q * s[:, None]).to(torch.bfloat16), s


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op == "matmul":
        # the codes' sums pass 2^24: fp64 holds them exactly
        acc = state["A"].double() @ state["B"].double().t()
        inv_g = 1.0 / state["group"] if state["group"] else 1.0
        y = acc.float() * state["a_scale"][:, None] * state["b_scale"][None, :] * inv_g
        if state["bias_v"] is not None:
            y = y + state["bias_v"].float()
        return {"Y": y.to(DTYPES[state["out"]])}
    if op == "silu":
        a = state["gate"].float()
        y = a / (1 + torch.exp(-a)) * state["up"].float()
        v, s = _quantized(y, state["group"])
        return {"values": v, "scale": s}
    h = state["X"].float()
    out = {}
    if state["R"] is not None:
        h = h + state["R"].float()
        out["sum"] = h.to(state["X"].dtype)
    y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * state["gamma"].float()
    out["values"], out["scale"] = _quantized(y, state["group"])
    return out


def _run_own(state):
    import w4a4_int4_quantized_b200 as w4

    op = state["op"]
    if op == "matmul":
        return {"Y": w4.w8a8_matmul(state["A"], state["a_scale"], state["B"], state["b_scale"], group=state["group"],
                                    bias=state["bias_v"], Y=state["Y"])}
    if op == "silu":
        q, s = w4.w8a8_silu_mul_quantize(state["gate"], state["up"], state["group"], Xq=state["Xq"],
                                         x_scale=state["x_scale"])
        return {"values": torch.mul(q, s[:, None], out=state["values"]), "scale": s}
    q, s, h = w4.w8a8_add_rmsnorm_quantize(state["X"], state["gamma"], EPS, state["group"], residual=state["R"],
                                           H=state["H"], Xq=state["Xq"], x_scale=state["x_scale"])
    out = {"values": torch.mul(q, s[:, None], out=state["values"]), "scale": s}
    if h is not None:
        out["sum"] = h
    return out


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "matmul":
        N = case["N"]
        e = DTYPES[case["out"]].itemsize
        return {"bytes": M * K + N * K + 4 * (M + N) + M * N * e + (N * e if case["bias"] else 0),
                "flops": 2 * M * N * K}
    e = DTYPES[case["dtype"]].itemsize
    turn = {0: 0, 64: 6, 128: 7}[case["group"]]
    if case["op"] == "silu":
        return {"bytes": 2 * M * K * e + M * K + 4 * M, "flops": M * K * (9 + turn)}
    reads_writes = 3 if case["residual"] else 1
    return {"bytes": M * K * (reads_writes * e + 1) + K * e + 4 * M, "flops": M * K * (9 + turn)}


def _exact_codes(y, group):
    """64-bit rotation (butterflies) and quantization: (values, scales)."""
    M, K = y.shape
    if group:
        h = 1
        while h < group:
            p = y.reshape(M, K // (2 * h), 2, h)
            y = torch.stack((p[:, :, 0] + p[:, :, 1], p[:, :, 0] - p[:, :, 1]), dim=2).reshape(M, K)
            h *= 2
    s = y.abs().max(dim=1).values / 127.0
    q = torch.round(y / s.clamp_min(1e-300)[:, None])
    return q * s[:, None], s


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "matmul":
        N, g = case["N"], case["group"] or 1
        Y = torch.empty((case["M"], N), dtype=torch.float64, device=st["A"].device)
        A = st["A"].double() * (st["a_scale"].double() / g)[:, None]
        for n in range(0, N, 4096):     # the scales applied to the operands, a block of channels at a time
            B = st["B"][n:n + 4096].double() * st["b_scale"][n:n + 4096].double()[:, None]
            Y[:, n:n + 4096] = torch.einsum("mk,nk->mn", A, B)
            if st["bias_v"] is not None:
                Y[:, n:n + 4096] += st["bias_v"][n:n + 4096].double()
        return {"Y": Y}
    if case["op"] == "silu":
        a, b = st["gate"].double(), st["up"].double()
        v, s = _exact_codes(a * torch.sigmoid(a) * b, case["group"])
        return {"values": v, "scale": s}
    h = st["X"].double()
    out = {}
    if st["R"] is not None:
        h = st["R"].double() + h
        out["sum"] = h
    rms = (torch.linalg.vector_norm(h, dim=1) ** 2 / case["K"] + EPS).sqrt()
    out["values"], out["scale"] = _exact_codes(h / rms[:, None] * st["gamma"].double(), case["group"])
    return out
