"""The int8 product with token and channel scales (w8a8_matmul) against the
same formula in 64 bits, and the run of the operators around it.

Tolerance, with u = 2^-24 and h = half a step of the output type relative to
the value: the product p = acc sx sw / g carries the conversion and two
multiplications (3 u; 1/g is a power of two), the bias one addition (u of the
sum), the store h (and half of the smallest fp16 step):
|Y - Y64| <= 3 u |p| + (u + h (1 + 2^-7)) |Y64| + tiny; h's factor covers the
store's rounding acting on a value already off by the other terms."""
from __future__ import annotations

import numpy as np
import pytest

import w4a4_int4_quantized_b200 as w4

from test_row_quantize import EPS, _data, _dt, _f64, _rows, check_codes, norm64, silu64, silu_c

U = 2.0 ** -24
OK, INVALID, SHAPE, MISALIGNED = 0, 1, 2, 3


# ------------------------------------------------------------------ refusals, no GPU
@pytest.fixture(scope="module")
def lib():
    from w4a4_int4_quantized_b200 import build
    build.build()
    return w4.load_library()


def test_refusals(lib):
    f = lib.w8a8_matmul
    names = ["Xq", "ldx", "sx", "Wq", "ldw", "sw", "M", "N", "K", "group", "bias", "dtype", "Y", "ldy", "st"]
    good = dict(zip(names, [0x10000, 64, 0x20000, 0x30000, 64, 0x40000, 4, 24, 50, 0, 0x50000, 0, 0x60000, 24, None]))

    def call(**kw):
        return f(*[{**good, **kw}[n] for n in names])

    for missing in ("Xq", "sx", "Wq", "sw", "Y"):
        assert call(**{missing: None}) == INVALID
    for dtype in (-1, 3):
        assert call(dtype=dtype) == INVALID
    for kw in (dict(M=-1), dict(N=0), dict(K=0), dict(K=131072, ldx=131072, ldw=131072), dict(group=1), dict(group=32),
               dict(ldx=48), dict(ldx=72), dict(ldw=48), dict(ldw=65), dict(ldy=23)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(Xq=0x10008), dict(Wq=0x30001), dict(sx=0x20002), dict(sw=0x40001), dict(bias=0x50001),
               dict(Y=0x60001), dict(Y=0x60002, dtype=2), dict(bias=0x50002, dtype=2)):
        assert call(**kw) == MISALIGNED, kw
    assert call(M=0, Xq=None, Y=None) == OK


# ------------------------------------------------------------------ GPU
gpu = pytest.mark.gpu


def _codes(rows, K, seed, pad=0, full=False):
    """int8 codes as a CUDA matrix with rows 16-byte aligned, `pad` more bytes apart."""
    import torch
    rng = np.random.default_rng(seed)
    ld = (K + 15) // 16 * 16 + pad
    buf = torch.full((rows, ld), 77, dtype=torch.int8, device="cuda")      # bytes past K must not count
    c = np.full((rows, K), -128, np.int8) if full else rng.integers(-128, 128, (rows, K)).astype(np.int8)
    buf[:, :K] = torch.from_numpy(c)
    return buf[:, :K]


def _case(M, N, K, seed, dtype, bias, pad=0, full=False):
    import torch
    rng = np.random.default_rng(seed)
    sx = torch.from_numpy((0.01 + 0.05 * rng.random(M)).astype(np.float32)).cuda()
    sw = torch.from_numpy((0.0002 + 0.0006 * rng.random(N)).astype(np.float32)).cuda()
    v = torch.from_numpy(rng.standard_normal(N)).to(_dt(dtype)).cuda() if bias else None
    return _codes(M, K, seed + 1, pad, full), sx, _codes(N, K, seed + 2, pad, full), sw, v


def check_product(Y, Xq, sx, Wq, sw, g, v):
    import torch
    acc = (Xq.double() @ Wq.double().t()).cpu().numpy()       # exact: below 2^31
    p = acc * _f64(sx)[:, None] * _f64(sw)[None, :] / (g or 1)
    y = p + (0.0 if v is None else _f64(v)[None, :])
    h = torch.finfo(Y.dtype).eps / 2
    tiny = 2.0 ** -25 if Y.dtype == torch.float16 else 0.0
    bound = 3 * U * np.abs(p) + (U + h * (1 + 2.0 ** -7)) * np.abs(y) + tiny
    off = np.abs(_f64(Y) - y)
    assert np.all(off <= bound), (float(np.max(off - bound)), np.argwhere(off > bound)[:5].tolist())


SHAPES = [
    # M, N, K, group
    (1, 1, 1, 0), (1, 16, 64, 64), (1, 17, 16, 0), (3, 40, 65, 0), (1, 4096, 4096, 128), (2, 100, 1000, 0),
    (8, 33, 511, 0), (9, 1000, 640, 64), (16, 257, 2047, 0), (17, 64, 128, 0), (31, 1001, 130, 0), (32, 520, 4100, 0),
    (33, 7, 100, 0), (33, 256, 512, 0), (64, 129, 1025, 0), (65, 1024, 4096, 128), (100, 3000, 1000, 0),
    (128, 512, 127, 0), (129, 1280, 2048, 0), (255, 255, 255, 0), (256, 2048, 1536, 64), (257, 333, 900, 0),
    (300, 4104, 512, 0), (333, 1013, 2995, 0), (512, 5000, 384, 0), (1000, 1000, 1000, 0), (1025, 4352, 256, 128),
    (2050, 2049, 130, 0), (5000, 24, 777, 0), (40, 20000, 264, 0), (700, 9000, 48, 0),
]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,N,K,group", SHAPES)
def test_product(M, N, K, group, dtype):
    import torch
    Xq, sx, Wq, sw, v = _case(M, N, K, M + N + K, dtype, (M + N + K) % 2, pad=16 * (K % 3))
    ldy = N + (N % 3)
    buf = torch.full((M + 1, ldy), 5.0, dtype=_dt(dtype), device="cuda")
    Y = buf[:M, :N]
    out = w4.w8a8_matmul(Xq, sx, Wq, sw, group, v, Y=Y)
    torch.cuda.synchronize()
    assert out is Y
    check_product(Y, Xq, sx, Wq, sw, group, v)
    assert (buf[M] == 5).all() and (buf[:, N:] == 5).all()


FEW_SHAPES = [                                               # on both sides of the few-token forms' limits
    (1, 7200, 100, 0), (5, 14500, 333, 128), (8, 21500, 2000, 0), (7, 200, 8192, 0), (7, 200, 8193, 0), (2, 22600, 2048, 0),
    (9, 4736, 65, 0), (9, 4737, 65, 0), (13, 4700, 1000, 64), (16, 300, 8192, 0), (16, 300, 8208, 0), (12, 17, 30, 0),
    (3, 500, 16384, 0), (3, 500, 16385, 0), (32, 500, 4096, 0), (32, 500, 4097, 0),
    (17, 4736, 50, 0), (25, 4737, 500, 0), (31, 1000, 2047, 0), (32, 1000, 2049, 0), (32, 15, 2048, 128), (20, 9, 1, 0),
]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K,group", FEW_SHAPES)
def test_few_tokens(M, N, K, group, dtype):
    test_product(M, N, K, group, dtype)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("N,K", [(5304, 109), (5294, 110), (5299, 109), (5295, 109), (5303, 1000), (5296, 1000)])
def test_many_tiles_by_alignment(N, K, dtype):
    """Several tiles per pair of SMs; rows of Y at 16, 4 and 2 bytes, and ends inside a store."""
    test_product(2550, N, K, 64, dtype)


@gpu
@pytest.mark.parametrize("M", [2, 30, 80, 300])
def test_longest_sums_of_the_lowest_code(M):
    import torch
    Xq, sx, Wq, sw, _ = _case(M, 40, 131071, 3, "fp32", False, full=True)
    Y = w4.w8a8_matmul(Xq, sx, Wq, sw, dtype=torch.float32)
    torch.cuda.synchronize()
    check_product(Y, Xq, sx, Wq, sw, 0, None)


@gpu
@pytest.mark.parametrize("M,N,K", [(1, 256, 512), (20, 256, 512), (64, 256, 1024), (256, 520, 1024), (1000, 2048, 512)])
def test_equal_to_the_layers_product(M, N, K):
    import torch
    Xq, sx, Wq, sw, v = _case(M, N, K, 9, "bf16", True)
    want = w4.w8a8_gemm(Xq, sx, Wq, sw, 128, v)
    got = w4.w8a8_matmul(Xq, sx, Wq, sw, 128, v)
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@gpu
@pytest.mark.parametrize("M", [4, 40, 600])
def test_non_finite_scales_stay_in_their_rows(M):
    import torch
    Xq, sx, Wq, sw, v = _case(M, 300, 256, 11, "bf16", True)
    clean = w4.w8a8_matmul(Xq, sx, Wq, sw, 0, v).clone()
    sx[1] = float("nan")
    sx[2] = 0.0
    Y = w4.w8a8_matmul(Xq, sx, Wq, sw, 0, v)
    torch.cuda.synchronize()
    assert torch.isnan(Y[1]).all() and torch.equal(Y[2], v)
    keep = [m for m in range(M) if m not in (1, 2)]
    assert torch.equal(Y[keep], clean[keep])


@gpu
@pytest.mark.parametrize("M", [1, 12, 40, 300])
def test_rows_far_apart(M):
    """Offsets past 2^31 bytes in the codes and past 2^31 elements in Y."""
    import torch
    N, K = 24, 100
    Xq, sx, Wq, sw, _ = _case(M, N, K, 13, "bf16", False)
    far = (1 << 31) // min(M, 20) // 16 * 16 + 16
    bufw = torch.empty(((N - 1) * (1 << 27) + 128,), dtype=torch.int8, device="cuda")
    W2 = bufw.as_strided((N, K), (1 << 27, 1))
    W2.copy_(Wq)
    bufx = torch.empty(((M - 1) * far + 128,), dtype=torch.int8, device="cuda")
    X2 = bufx.as_strided((M, K), (far, 1)) if M > 1 else Xq
    if M > 1:
        X2.copy_(Xq)
    bufy = torch.empty(((M - 1) * far + N,), dtype=torch.bfloat16, device="cuda")
    Y2 = bufy.as_strided((M, N), (far, 1))
    w4.w8a8_matmul(X2, sx, W2, sw, Y=Y2)
    Y = w4.w8a8_matmul(Xq, sx, Wq, sw)
    torch.cuda.synchronize()
    assert torch.equal(Y, Y2)


@gpu
def test_no_rows_and_binding_refusals():
    import torch
    Xq, sx, Wq, sw, v = _case(4, 64, 128, 1, "bf16", True)
    Y = w4.w8a8_matmul(Xq[:0], sx[:0], Wq, sw, 0, v)
    assert Y.shape == (0, 64)
    bad = [dict(x_scale=sx[:3]), dict(w_scale=sw[:8]), dict(bias=v.float()), dict(Y=torch.empty(4, 63, device="cuda")),
           dict(Wq=Wq[:, :64]), dict(Xq=Xq.cpu()), dict(Wq=Wq.cpu()), dict(Xq=Xq.to(torch.uint8)), dict(group=3),
           dict(dtype=torch.float64), dict(Y=torch.empty(64, 4, device="cuda", dtype=torch.bfloat16).t()),
           dict(Wq=torch.zeros(64, 129, dtype=torch.int8, device="cuda")[:, :128])]
    for kw in bad:
        with pytest.raises(w4.W4A4Error):
            w4.w8a8_matmul(**{**dict(Xq=Xq, x_scale=sx, Wq=Wq, w_scale=sw, bias=v), **kw})


@gpu
@pytest.mark.parametrize("M,N,K", [(5, 512, 768), (40, 512, 2048), (700, 2304, 640)])
def test_two_streams_and_a_graph(M, N, K):
    """Two streams at once, and a captured call replayed on new codes."""
    import torch
    Xq, sx, Wq, sw, v = _case(M, N, K, 17, "bf16", True)
    X2 = _codes(M, K, 99)
    want, want2 = (w4.w8a8_matmul(x, sx, Wq, sw, 0, v) for x in (Xq, X2))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        got.append((w4.w8a8_matmul(Xq, sx, Wq, sw, 0, v, stream=a), want))
        got.append((w4.w8a8_matmul(X2, sx, Wq, sw, 0, v, stream=b), want2))
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in got)
    Y = torch.empty_like(want)
    codes = Xq.clone(memory_format=torch.contiguous_format)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=a):
        w4.w8a8_matmul(codes, sx, Wq, sw, 0, v, Y=Y)
    for x, w in ((X2, want2), (Xq, want)):
        codes.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, w)
    del graph


@gpu
@pytest.mark.parametrize("M,D,F,group,dtype", [(1, 256, 640, 0, "bf16"), (7, 1000, 1500, 0, "fp16"),
                                               (70, 512, 1408, 64, "bf16"), (600, 1024, 2816, 128, "bf16")])
def test_gated_mlp(M, D, F, group, dtype):
    """A gated MLP as a block runs it: norm -> gate | up -> SiLU * up -> down,
    every step checked against 64 bits on the step's own inputs."""
    import torch
    dt = _dt(dtype)
    rng = np.random.default_rng(5)
    X, R = _rows(_data(M, D, 41), dt), _rows(_data(M, D, 42), dt)
    gamma = _rows(1 + 0.1 * _data(1, D, 43), dt)[0]

    def weights(n, k):
        W = torch.from_numpy(rng.standard_normal((n, k)) * 0.05)
        if group:
            i = np.arange(group)
            H = torch.from_numpy(1.0 - 2.0 * np.array([[bin(a & b).count("1") & 1 for b in i] for a in i]))
            W = (W.reshape(n, k // group, group) @ H).reshape(n, k)
        s = W.abs().amax(dim=1) / 127
        q = torch.zeros((n, (k + 15) // 16 * 16), dtype=torch.int8)
        q[:, :k] = torch.round(W / s[:, None]).to(torch.int8)
        return q.cuda()[:, :k], s.float().cuda()

    Wgu, sgu = weights(2 * F, D)
    Wd, sd = weights(D, F)
    q, s, h = w4.w8a8_add_rmsnorm_quantize(X, gamma, EPS, group, residual=R)
    gu = w4.w8a8_matmul(q, s, Wgu, sgu, group, dtype=dt)
    q2, s2 = w4.w8a8_silu_mul_quantize(gu[:, :F], gu[:, F:], group)
    Y = w4.w8a8_matmul(q2, s2, Wd, sd, group, dtype=dt)
    torch.cuda.synchronize()
    _, y = norm64(_f64(X), _f64(R), _f64(gamma), EPS)
    check_codes(y, group, 21, _f64(q), _f64(s))
    check_product(gu, q, s, Wgu, sgu, group, None)
    check_codes(silu64(_f64(gu[:, :F]), _f64(gu[:, F:])), group, silu_c(_f64(gu[:, :F])), _f64(q2), _f64(s2))
    check_product(Y, q2, s2, Wd, sd, group, None)


_FIRST_CALL = """
import sys
import torch
import w4a4_int4_quantized_b200 as w4
M, D, F = (int(v) for v in sys.argv[1:4])
g = torch.Generator(device="cuda").manual_seed(3)
X = torch.randn((M, D), generator=g, device="cuda").to(torch.bfloat16)
W = torch.randint(-127, 128, (2 * F, D), generator=g, device="cuda", dtype=torch.int8)
sw = torch.rand(2 * F, generator=g, device="cuda") * 0.001
q, s = torch.empty((M, D), dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
q2, s2 = torch.empty((M, F), dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
Y = torch.empty((M, 2 * F), dtype=torch.bfloat16, device="cuda")

def block():
    w4.w8a8_add_rmsnorm_quantize(X, None, 1e-6, Xq=q, x_scale=s)
    w4.w8a8_matmul(q, s, W, sw, Y=Y)
    w4.w8a8_silu_mul_quantize(Y[:, :F], Y[:, F:], Xq=q2, x_scale=s2)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    block()                      # the process's first call of each kernel
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (q, s, Y, q2, s2)]
block()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (q, s, Y, q2, s2)))
assert w4.w4a4_get_device_error() == 0
print("same")
"""


@gpu
@pytest.mark.parametrize("M,D,F", [(2, 512, 640), (40, 1024, 640), (300, 1024, 640), (2000, 4096, 2560)])
def test_first_calls_of_a_process_inside_a_capture(M, D, F):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST_CALL, str(M), str(D), str(F)], cwd=root, capture_output=True,
                       text=True, timeout=120)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


@gpu
def test_host_threads_on_their_own_streams():
    """Calls of all three operators from several host threads at once."""
    import concurrent.futures as cf

    import torch
    cases = []
    for M, D, F in ((1, 1024, 512), (20, 1024, 1536), (200, 768, 1024), (500, 2048, 512)):
        X = _rows(_data(M, D, M), torch.bfloat16)
        Wq, sw = _codes(2 * F, D, M + 1), torch.rand(2 * F, device="cuda") * 1e-3
        cases.append((X, Wq, sw, F))

    def run(case, stream):
        X, Wq, sw, F = case
        q, s, _ = w4.w8a8_add_rmsnorm_quantize(X, None, EPS, stream=stream)
        Y = w4.w8a8_matmul(q, s, Wq, sw, stream=stream)
        return (q, s, Y, *w4.w8a8_silu_mul_quantize(Y[:, :F], Y[:, F:], stream=stream))

    want = [run(c, torch.cuda.current_stream()) for c in cases]
    torch.cuda.synchronize()

    def worker(i):
        st = torch.cuda.Stream()
        got = [run(cases[(i + k) % 4], st) for k in range(40)]
        st.synchronize()
        return all(torch.equal(a, b) for k in range(40) for a, b in zip(got[k], want[(i + k) % 4]))

    with cf.ThreadPoolExecutor(4) as ex:
        assert all(ex.map(worker, range(4)))


@gpu
def test_large_output_and_many_tiles():
    """An output of more than 2^31 elements: its first, last and middle rows."""
    import torch
    M, N, K = 66000, 33000, 64
    Xq, sx, Wq, sw, v = _case(M, N, K, 23, "bf16", True)
    Y = w4.w8a8_matmul(Xq, sx, Wq, sw, 0, v)
    torch.cuda.synchronize()
    for rows in (slice(0, 40), slice(32990, 33030), slice(M - 40, M)):
        check_product(Y[rows], Xq[rows], sx[rows], Wq, sw, 0, v)


_WAITING = r"""
#include <unistd.h>
static volatile int go = 0;
extern "C" void let_go() { go = 1; }
extern "C" int entry() {                  // stands in for an entry point whose launch waits
  for (int i = 0; i < 3000 && !go; ++i) usleep(1000);
  const int seen = go;
  go = 0;
  return seen ? 0 : 5;
}
"""

_LOCK = """
import ctypes, sys, threading, time
import torch
import w4a4_int4_quantized_b200 as w4
lib = ctypes.CDLL(sys.argv[1])
w4._bind_calls()
at = ctypes.cast(lib.entry, ctypes.c_void_p).value
w4._calls.bind(at, at, at)
x = torch.zeros((2, 64), device="cuda")
q, s = torch.zeros((2, 64), dtype=torch.int8, device="cuda"), torch.zeros(2, device="cuda")
for call in (lambda: w4.w8a8_add_rmsnorm_quantize(x, None, 1e-6), lambda: w4.w8a8_silu_mul_quantize(x, x),
             lambda: w4.w8a8_matmul(q, s, q, s)):
    def other():
        time.sleep(0.1)
        lib.let_go()
    t = threading.Thread(target=other)
    t.start()
    call()                                # raises where the other thread could not run
    t.join()
print("ran")
"""


@gpu
def test_other_host_threads_run_while_a_call_waits(tmp_path):
    """A call lets the interpreter lock go: what its launch waits for may need it.  The library's
    entry points are replaced by a host function that waits; nothing is launched."""
    import os
    import subprocess
    import sys
    src, lib = tmp_path / "entry.cpp", tmp_path / "entry.so"
    src.write_text(_WAITING)
    subprocess.run(["g++", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _LOCK, str(lib)], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "ran" in r.stdout, r.stderr[-2000:]


# ------------------------------------------------------------------ every form of the product
EVERY_FORM = [
    # kernel, tokens or columns per tile, slices of K, M, N, K: what w8a8_plan_matmul gives on 148 SMs
    (0, 8, 1, 1, 48, 64), (0, 8, 1, 1, 65, 71), (0, 16, 1, 9, 48, 64), (0, 16, 1, 9, 67, 75), (0, 32, 1, 17, 48, 64),
    (0, 32, 1, 17, 69, 65),
    (1, 16, 1, 10, 4824, 64), (1, 16, 1, 13, 4939, 67), (1, 16, 2, 15, 5784, 960), (1, 16, 2, 11, 5713, 933),
    (1, 16, 4, 11, 4824, 1024), (1, 16, 4, 15, 5141, 909), (1, 16, 8, 10, 48, 9344), (1, 16, 8, 13, 65, 8293),
    (1, 32, 1, 18, 4776, 64), (1, 32, 1, 23, 5507, 67), (1, 32, 2, 23, 4776, 960), (1, 32, 2, 23, 4777, 905),
    (1, 32, 4, 30, 4896, 1408), (1, 32, 4, 19, 5143, 1381), (1, 32, 8, 23, 48, 4160), (1, 32, 8, 23, 65, 4147),
    (1, 64, 1, 36, 48, 64), (1, 64, 1, 35, 69, 71), (1, 64, 2, 39, 48, 832), (1, 64, 2, 35, 81, 673),
    (1, 64, 4, 35, 48, 960), (1, 64, 4, 35, 65, 925), (1, 64, 8, 36, 48, 1984), (1, 64, 8, 45, 67, 1931),
    (1, 128, 1, 77, 18960, 64), (1, 128, 1, 69, 19327, 69), (1, 128, 2, 66, 9600, 3008), (1, 128, 2, 67, 10505, 2695),
    (1, 128, 4, 75, 4512, 6080), (1, 128, 4, 69, 5655, 4503), (1, 128, 8, 72, 2400, 8384), (1, 128, 8, 1057, 149, 11321),
    (2, 128, 1, 194, 19632, 64), (2, 128, 1, 199, 19573, 69), (2, 128, 2, 2188, 264, 3136), (2, 128, 2, 2147, 273, 3089),
    (2, 128, 3, 1547, 264, 2240), (2, 128, 3, 2763, 131, 2243), (2, 128, 4, 1547, 144, 4160), (2, 128, 4, 1569, 131, 4119),
    (2, 256, 1, 258, 16296, 64), (2, 256, 1, 265, 15177, 71), (2, 256, 2, 332, 3312, 2752), (2, 256, 2, 545, 2057, 2763),
    (2, 256, 3, 72, 5112, 3648), (2, 256, 3, 2103, 265, 3405), (2, 256, 4, 784, 648, 2880), (2, 256, 4, 2925, 133, 3351),
]


def test_every_form_has_its_cases(lib):
    """The cases take the forms that they are listed under, an even and a ragged one each, and no size takes
    a form that is not among them."""
    rng = np.random.default_rng(8)
    kinds = {(0, w, 1) for w in (8, 16, 32)} | {(1, w, s) for w in (16, 32, 64, 128) for s in (1, 2, 4, 8)} | \
        {(2, w, s) for w in (128, 256) for s in (1, 2, 3, 4)}
    assert {(*c[:3], c[5] % 2) for c in EVERY_FORM} == {(*k, odd) for k in kinds for odd in (0, 1)}
    for *form, M, N, K in EVERY_FORM:
        for dtype in ("bf16", "fp16", "fp32"):
            assert w4.w8a8_plan_matmul(M, N, K, dtype) == tuple(form), (M, N, K, dtype)
    for _ in range(5000):
        M, N, K = np.exp(rng.uniform(0, np.log([9000, 30000, 131071]))).astype(int)
        assert w4.w8a8_plan_matmul(int(M), int(N), int(K), "fp32") in kinds


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("kernel,width,split,M,N,K", EVERY_FORM)
def test_every_form(kernel, width, split, M, N, K, dtype):
    """With and without a bias, rows of Y on and off the alignment of a wide store."""
    import torch
    for bias, pad, offset in ((True, -N % 8, 0), (False, 3, 1), (True, 2, 2)):
        Xq, sx, Wq, sw, v = _case(M, N, K, M + N + K + offset, dtype, bias)
        ldy = N + pad
        buf = torch.full(((M + 1) * ldy + offset,), 5.0, dtype=_dt(dtype), device="cuda")
        Y = buf[offset:].as_strided((M, N), (ldy, 1))
        w4.w8a8_matmul(Xq, sx, Wq, sw, 64, v, Y=Y)
        torch.cuda.synchronize()
        check_product(Y, Xq, sx, Wq, sw, 64, v)
        Y.fill_(5.0)
        assert (buf == 5.0).all()                     # nothing between the rows, before or behind them


@gpu
@pytest.mark.parametrize("M,N,K", [(256, 4096, 12288), (512, 4096, 4096), (256, 2048, 16384), (509, 4001, 4111)])
def test_split_products_of_ordinary_size(M, N, K):
    test_product(M, N, K, 128, "bf16")


def test_plan_refusals(lib):
    import ctypes
    f = lib.w8a8_plan_matmul
    cl, out = (ctypes.c_int * 6)(148, 71, 33, 33, 22, 15), (ctypes.c_int * 3)()
    assert f(4, 64, 64, 64, 64, 0, 148, cl, out) == OK
    assert f(4, 64, 64, 64, 64, 0, 148, cl, None) == INVALID and f(4, 64, 64, 64, 64, 3, 148, cl, out) == INVALID
    for bad in ((0, 64, 64, 64, 64), (4, 0, 64, 64, 64), (4, 64, 0, 64, 64), (4, 64, 131072, 131072, 131072),
                (4, 64, 64, 48, 64), (4, 64, 64, 64, 72)):
        assert f(*bad, 0, 148, cl, out) == SHAPE, bad
    assert f(4, 64, 64, 64, 64, 0, 1, cl, out) == SHAPE


@gpu
def test_each_refusal_of_the_binding_has_its_status():
    """One argument at a time is wrong, and the call is refused for it."""
    import torch
    Xq, sx, Wq, sw, v = _case(4, 64, 128, 1, "bf16", True)
    good = dict(Xq=Xq, x_scale=sx, Wq=Wq, w_scale=sw, bias=v)
    Y = torch.full((5, 80), 3.0, dtype=torch.bfloat16, device="cuda")
    bad = [(SHAPE, dict(Y=Y[:4, :63])), (SHAPE, dict(Y=Y[:4, :65])), (SHAPE, dict(Y=Y[:3, :64])), (SHAPE, dict(Y=Y[0, :64])),
           (SHAPE, dict(Y=Y[:4, 0:64:2])), (SHAPE, dict(Y=Y[:1, :64].expand(4, 64))), (INVALID, dict(Y=Y[:4, :64].float())),
           (INVALID, dict(Y=Y[:4, :64].cpu())), (INVALID, dict(Y=Y[:4, :64], dtype=torch.float16)),
           (INVALID, dict(bias=None, dtype=torch.float64)), (INVALID, dict(bias=None, Y=Y[:4, :64].double())),
           (INVALID, dict(bias=v.float())), (INVALID, dict(bias=v.cpu())), (SHAPE, dict(bias=v[:63])),
           (SHAPE, dict(bias=v[None])), (SHAPE, dict(bias=torch.cat([v, v])[::2])),
           (SHAPE, dict(x_scale=sx[:3])), (INVALID, dict(x_scale=sx.double())), (SHAPE, dict(w_scale=sw[:8])),
           (INVALID, dict(w_scale=sw.half())), (SHAPE, dict(Wq=Wq[:, :64])), (INVALID, dict(Wq=Wq.cpu())),
           (INVALID, dict(Wq=Wq.view(torch.uint8))), (INVALID, dict(Xq=Xq.view(torch.uint8))), (SHAPE, dict(group=3)),
           (SHAPE, dict(group=-64)), (SHAPE, dict(Wq=torch.zeros(64, 136, dtype=torch.int8, device="cuda")[:, :128])),
           (MISALIGNED, dict(Xq=torch.zeros(4, 160, dtype=torch.int8, device="cuda")[:, 8:136]))]
    for status, kw in bad:
        with pytest.raises(w4.W4A4Error) as e:
            w4.w8a8_matmul(**{**good, **kw})
        assert e.value.status == status, (kw.keys(), e.value)
    with pytest.raises(w4.W4A4Error) as e:
        w4.w8a8_matmul(Xq.cpu(), sx, Wq, sw)
    assert e.value.status == 6
    torch.cuda.synchronize()
    assert (Y == 3.0).all()
