"""Residual + RMS norm + int8 (w8a8_add_rmsnorm_quantize) and SiLU * up + int8
(w8a8_silu_mul_quantize) against the same formulas in 64 bits.

Tolerances, with u = 2^-24 (half a step of fp32, relative):
  norm  y carries h's own rounding (1 u), the sum of squares (a chain of at
        most 16 fused adds in a thread, 1 add, 10 adds across the row, 2 u
        from h: 29 u), its product with 1 / K and eps (3 u), halved by the
        square root, whose Newton step leaves 1.5 u, the products with gamma
        and with the factor (1 u each): at most 21 u of |y|.
  silu  t = 2^(-a log2 e): the exponent's two roundings put 1.5 |a| u into t and
        ex2.approx 4 u, of which t / (1 + t) reaches y: for a >= 0 at most 2 u +
        0.5 u, for a < 0 all of it; 1 + t (1 u), rcp.approx 1 ulp (2 u), two
        products (2 u): at most 9 u + 1.5 max(0, -a) u of |y|.  Below a = -87
        four powers e^(a / 4) take the place of t: 1.22 |a| u from their exponents,
        16 u of their own and 11 u of the rest, under the same sum.
  rotation  a sum of g values in log2 g roundings: at most (c + log2 g) u of
        the group's sum of |y|.
With D the largest such error of a row, the scale is off by at most
D / 127 + u s, and y / s by at most 2 * 127 D / max|y| + 4 * 127 u (1 / s
2 u at most, s and the factor 1 u each), so a code is within half a step plus
that of the 64-bit quotient."""
from __future__ import annotations

import numpy as np
import pytest

import w4a4_int4_quantized_b200 as w4

U = 2.0 ** -24
EPS = float(np.float32(1e-6))


# ------------------------------------------------------------------ oracle
def hadamard(y, g):
    M, K = y.shape
    i = np.arange(g)
    H = 1.0 - 2.0 * (np.array([[bin(a & b).count("1") & 1 for b in i] for a in i]))
    return (y.reshape(M, K // g, g) @ H).reshape(M, K)


def norm64(x, r, gamma, eps):
    h = x + (0.0 if r is None else r)
    y = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    return h, y if gamma is None else y * gamma


def silu64(a, b):
    return a / (1.0 + np.exp(-a)) * b


def silu_c(a):
    return 9 + 1.5 * np.maximum(0.0, -a)


def check_codes(y, g, c, q, s):
    """Codes q and scales s of the 64-bit rows y, c u of relative error in y (a
    number, or one for each element)."""
    M, K = y.shape
    mag = np.abs(y)
    if g:
        D = U * ((c + np.log2(g)) * mag).reshape(M, K // g, g).sum(axis=2).max(axis=1)
        y = hadamard(y, g)
    else:
        D = U * (c * mag).max(axis=1)
    amax = np.abs(y).max(axis=1)
    s64 = amax / 127.0
    assert np.all(np.abs(s - s64) <= D / 127.0 + U * s64 + 2.0 ** -149)
    for m in range(M):
        if amax[m] == 0.0:
            assert s[m] == 0.0 and not np.any(q[m])
            continue
        slack = 2 * 127 * D[m] / amax[m] + 4 * 127 * U
        off = np.abs(q[m] - y[m] / s64[m])
        assert off.max() <= 0.5 + slack, (m, off.max(), slack)
    assert np.abs(q.astype(np.int64)).max() <= 127


def test_oracle_catches_planted_mistakes():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 256))
    _, y = norm64(x, None, None, EPS)
    for g in (0, 64):
        z = hadamard(y, g) if g else y
        s = np.abs(z).max(axis=1) / 127
        q = np.rint(z / s[:, None])
        check_codes(y, g, 21, q, s)
        with pytest.raises(AssertionError):
            check_codes(y, g, 21, q + (np.arange(256) == 7), s)
        with pytest.raises(AssertionError):
            check_codes(y, g, 21, q, s * (1 + 1e-4))
        with pytest.raises(AssertionError):
            check_codes(y * 1.01, g, 21, q, s)


# ------------------------------------------------------------------ refusals, no GPU
OK, INVALID, SHAPE, MISALIGNED = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from w4a4_int4_quantized_b200 import build
    build.build()
    return w4.load_library()


def test_norm_refusals(lib):
    f = lib.w8a8_add_rmsnorm_quantize
    names = ["X", "ldx", "r", "ldr", "gamma", "eps", "M", "K", "group", "dtype", "H", "ldh", "Xq", "ldq", "s", "st"]
    good = dict(zip(names, [0x10000, 256, 0x20000, 256, 0x30000, 1e-6, 4, 256, 64, 0, 0x40000, 256, 0x50000, 256,
                            0x60000, None]))

    def call(**kw):
        return f(*[{**good, **kw}[n] for n in names])

    for missing in ("X", "Xq", "s"):
        assert call(**{missing: None}) == INVALID
    for eps in (0.0, -1e-6, float("nan"), float("inf"), 1e-37):
        assert call(eps=eps) == INVALID
    for dtype in (-1, 3):
        assert call(dtype=dtype) == INVALID
    for kw in (dict(M=-1), dict(K=0), dict(K=32832, ldx=40000, ldr=40000, ldh=40000, ldq=40000), dict(group=32),
               dict(group=128, K=192), dict(ldx=255), dict(ldr=255), dict(ldh=255), dict(ldq=248), dict(ldq=264),
               dict(K=-8)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(X=0x10001), dict(r=0x20001), dict(gamma=0x30001), dict(H=0x40001), dict(Xq=0x50008),
               dict(s=0x60002), dict(X=0x10002, dtype=2)):
        assert call(**kw) == MISALIGNED, kw
    assert call(M=0, X=None, Xq=None, s=None) == OK      # nothing to do
    assert call(M=0, K=0) == SHAPE


def test_silu_refusals(lib):
    f = lib.w8a8_silu_mul_quantize
    names = ["gate", "ldg", "up", "ldu", "M", "K", "group", "dtype", "Xq", "ldq", "s", "st"]
    good = dict(zip(names, [0x10000, 512, 0x10200, 512, 4, 256, 0, 0, 0x50000, 256, 0x60000, None]))

    def call(**kw):
        return f(*[{**good, **kw}[n] for n in names])

    for missing in ("gate", "up", "Xq", "s"):
        assert call(**{missing: None}) == INVALID
    assert call(dtype=7) == INVALID
    for kw in (dict(M=-1), dict(K=0), dict(K=32769, ldg=40000, ldu=40000, ldq=40000), dict(group=96),
               dict(group=64, K=100), dict(ldg=255), dict(ldu=255), dict(ldq=240), dict(ldq=257)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(gate=0x10001), dict(up=0x10201), dict(Xq=0x50004), dict(s=0x60001)):
        assert call(**kw) == MISALIGNED, kw
    assert call(M=0, gate=None, up=None, Xq=None, s=None) == OK


def test_binding_refuses_host_tensors():
    import torch
    x = torch.zeros(2, 64)
    with pytest.raises(w4.W4A4Error):
        w4.w8a8_add_rmsnorm_quantize(x, None, 1e-6)
    with pytest.raises(w4.W4A4Error):
        w4.w8a8_silu_mul_quantize(x, x)


# ------------------------------------------------------------------ GPU
gpu = pytest.mark.gpu
TYPES = ["bf16", "fp16", "fp32"]


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def _rows(x, dtype, pad=0, offset=0):
    """x as a CUDA tensor whose rows are `pad` elements apart beyond their
    width and start `offset` elements into their buffer."""
    import torch
    M, K = x.shape
    buf = torch.full((offset + M * (K + pad),), 7.0, dtype=dtype, device="cuda")
    view = buf.as_strided((M, K), (K + pad, 1), offset)
    view.copy_(torch.from_numpy(x).to(dtype))
    return view


def _f64(t):
    return t.detach().double().cpu().numpy()


def _data(M, K, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)) * scale
    x[:, :: max(1, K // 3)] *= 12.0
    return x


SHAPES = [
    # M, K, group, pad, offset
    (1, 1, 0, 0, 0), (3, 7, 0, 0, 0), (2, 8, 0, 0, 0), (5, 31, 0, 3, 1), (4, 64, 64, 0, 0), (9, 128, 128, 0, 0),
    (6, 192, 64, 8, 8), (5, 256, 128, 0, 0), (7, 257, 0, 0, 0), (13, 640, 128, 5, 3), (3, 1000, 0, 0, 0),
    (2, 1031, 0, 0, 1), (700, 264, 0, 0, 0), (601, 384, 64, 1, 0), (333, 1024, 128, 0, 0), (320, 2304, 0, 24, 0),
    (1, 4096, 128, 0, 0), (310, 4096, 0, 0, 0), (2, 8192, 64, 0, 0), (300, 8200, 0, 0, 0), (299, 16384, 128, 0, 0),
    (700, 9, 0, 0, 0), (900, 13, 0, 0, 1), (640, 8, 0, 1, 0), (701, 257, 0, 0, 0), (400, 1031, 0, 3, 1),
    (350, 2777, 0, 0, 0), (333, 8191, 0, 0, 0), (320, 5461, 0, 1, 5), (500, 128, 128, 1, 1), (1500, 300, 0, 2, 3),
    (2000, 1029, 0, 0, 0), (600, 12289, 0, 0, 0), (400, 264, 0, 1, 0), (400, 4100, 0, 0, 7),
    (1, 20001, 0, 0, 0), (3, 32768, 128, 0, 0), (300, 32768, 0, 0, 0), (301, 32767, 0, 0, 0),
]


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,group,pad,offset", SHAPES)
def test_norm(M, K, group, pad, offset, dtype):
    import torch
    dt = _dt(dtype)
    X = _rows(_data(M, K, 1), dt, pad, offset)
    R = _rows(_data(M, K, 2, 2.0), dt, K % 4, offset) if (M + K) % 3 else None
    gamma = _rows(1 + 0.1 * _data(1, K, 3), dt, 0, offset)[0] if K % 5 else None
    if M > 4:
        X[3] = 0                       # a padding row
        if R is not None:
            R[3] = 0
    ldq = (K + 15) // 16 * 16 + 16
    buf = torch.full((M + 1, ldq), 99, dtype=torch.int8, device="cuda")
    H, hbuf = None, None
    if R is not None:                  # rows of H at an offset and a stride of their own
        ldh = K + (M % 5)
        hbuf = torch.full((M * ldh + 9,), 5.0, dtype=dt, device="cuda")
        H = hbuf.as_strided((M, K), (ldh, 1), M % 7)
    q, s, h = w4.w8a8_add_rmsnorm_quantize(X, gamma, EPS, group, residual=R, H=H, Xq=buf[:M, :K])
    torch.cuda.synchronize()
    h64, y64 = norm64(_f64(X), None if R is None else _f64(R), None if gamma is None else _f64(gamma), EPS)
    check_codes(y64, group, 21, _f64(q), _f64(s))
    assert (buf[M] == 99).all() and (buf[:, K:] == 99).all()      # nothing past the rows or the width
    if R is None:
        assert h is None
    else:
        half = torch.finfo(dt).eps / 2
        tiny = 2.0 ** -25 if dtype == "fp16" else 0.0             # half a step below fp16's normal range
        rest = hbuf.clone()
        rest.as_strided((M, K), (ldh, 1), M % 7).fill_(5.0)
        assert (rest == 5.0).all()                                # nothing between the rows or around them
        assert np.all(np.abs(_f64(h) - h64) <= (half + 2 * U) * np.abs(h64) + tiny)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,group,pad,offset", SHAPES)
def test_silu(M, K, group, pad, offset, dtype):
    import torch
    dt = _dt(dtype)
    # the halves of one product: the second starts K (+ pad) elements in
    both = _rows(_data(M, 2 * K + pad, 4), dt, 0, offset)
    gate, up = both[:, :K], both[:, K + pad:]
    if M > 4:
        up[3] = 0
    q, s = w4.w8a8_silu_mul_quantize(gate, up, group)
    torch.cuda.synchronize()
    check_codes(silu64(_f64(gate), _f64(up)), group, silu_c(_f64(gate)), _f64(q), _f64(s))


FORMS = [                                            # M, K, group, pad, offset: the ways rows are read and worked on
    (300, 1537, 0, 3, 1), (1500, 1537, 0, 1, 0), (300, 12289, 0, 0, 1), (310, 20003, 0, 5, 2), (2000, 300, 0, 3, 1),
    (900, 40, 0, 1, 1), (5000, 1000, 0, 0, 0), (3000, 1152, 128, 8, 0), (3000, 1152, 128, 5, 0), (600, 640, 64, 3, 1),
    (2, 9001, 0, 7, 3), (1, 2001, 0, 0, 5), (2, 5, 0, 0, 1), (400, 7, 0, 0, 1), (299, 4160, 64, 1, 0),
]


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,group,pad,offset", FORMS)
def test_forms(M, K, group, pad, offset, dtype):
    test_norm(M, K, group, pad, offset, dtype)
    test_silu(M, K, group, pad, offset, dtype)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [40, 1027, 4096])
def test_non_finite_rows(K, dtype):
    import torch
    dt = _dt(dtype)
    x = _data(8, K, 5)
    X = _rows(x, dt)
    X[1, K // 2] = float("inf")
    X[2, 0] = float("-inf")
    X[3, K - 1] = float("nan")
    X[4] = float("nan")
    X[5] = 0
    X[6] = torch.finfo(dt).min
    for q, s, _ in [w4.w8a8_add_rmsnorm_quantize(X, None, EPS),
                    (*w4.w8a8_silu_mul_quantize(X, torch.ones_like(X)), None),
                    (*w4.w8a8_silu_mul_quantize(torch.ones_like(X), X), None)]:
        s, q = s.cpu(), q.cpu()
        for m in (1, 2, 3, 4):
            assert torch.isnan(s[m]) and not q[m].any()
        assert s[5] == 0 and not q[5].any()
        for m in (0, 7):
            assert torch.isfinite(s[m]) and q[m].abs().max() == 127
    # rows of the type's lowest value: the norm is -1 everywhere
    q, s, _ = w4.w8a8_add_rmsnorm_quantize(X, None, EPS)
    assert (q[6] == -127).all() and abs(float(s[6]) * 127 - 1) < 40 * U


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("big", [1e18, 1e25, 1e38])
@pytest.mark.parametrize("K", [24, 5000])
def test_squares_past_fp32(K, big, dtype):
    import torch
    x = _data(3, K, 6)
    x[1] *= big / np.abs(x[1]).max()
    X = _rows(x, _dt(dtype))
    q, s, _ = w4.w8a8_add_rmsnorm_quantize(X, None, EPS)
    torch.cuda.synchronize()
    check_codes(norm64(_f64(X), None, None, EPS)[1], 0, 21, _f64(q), _f64(s))


@gpu
@pytest.mark.parametrize("small", [1e-3, 1e-20, 1e-30])
def test_small_values(small):
    import torch
    X = _rows(_data(3, 700, 6) * small, torch.float32)
    one = torch.ones_like(X)
    q, s, _ = w4.w8a8_add_rmsnorm_quantize(X, None, 1e-30)
    check_codes(norm64(_f64(X), None, None, float(np.float32(1e-30)))[1], 0, 21, _f64(q), _f64(s))
    q, s = w4.w8a8_silu_mul_quantize(X, one)
    check_codes(silu64(_f64(X), _f64(one)), 0, silu_c(_f64(X)), _f64(q), _f64(s))
    q, s = w4.w8a8_silu_mul_quantize(one, X)
    check_codes(silu64(_f64(one), _f64(X)), 0, silu_c(_f64(one)), _f64(q), _f64(s))


@gpu
@pytest.mark.parametrize("M", [3, 400])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_extreme_gates(M, dtype):
    """Finite gates to either end of the type: no row turns into NaN, strongly
    negative ones count as 0 and the rest keeps its values."""
    import torch
    dt = _dt(dtype)
    K = 512
    gate, up = _rows(_data(M, K, 50), dt), _rows(_data(M, K, 51), dt)
    gate[:, 3] = torch.finfo(dt).min
    gate[:, 5], gate[:, 6], gate[:, 7] = -90.0, -1000.0, -85.0
    gate[1], up[1] = torch.finfo(dt).min, 1.0
    gate[2], up[2] = torch.finfo(dt).max, 1.0
    q, s = w4.w8a8_silu_mul_quantize(gate, up)
    assert s[1] == 0 and not q[1].any()
    assert (q[2] == 127).all() and abs(float(s[2]) * 127 / torch.finfo(dt).max - 1) < 20 * U
    a = _f64(gate)
    with np.errstate(over="ignore"):
        y = np.where(a < -87.0, 0.0, silu64(np.maximum(a, -87.0), _f64(up)))
    keep = [m for m in range(M) if m not in (1, 2)]
    check_codes(y[keep], 0, silu_c(np.maximum(a, -87.0))[keep], _f64(q)[keep], _f64(s)[keep])


@gpu
@pytest.mark.parametrize("K", [512, 4096, 5120, 12288])
def test_many_rows_of_unlike_size(K):
    """Neighbouring rows a million apart in size: a maximum taken from another
    row would show."""
    import torch
    M = 3000
    x = _data(M, K, 60)
    x *= 10.0 ** np.random.default_rng(61).integers(-3, 4, M)[:, None]
    X = _rows(x, torch.bfloat16)
    one = torch.ones_like(X)
    for _ in range(3):
        q, s = w4.w8a8_silu_mul_quantize(one, X)
        q2, s2, _ = w4.w8a8_add_rmsnorm_quantize(X, None, EPS)
        check_codes(silu64(_f64(one), _f64(X)), 0, silu_c(_f64(one)), _f64(q), _f64(s))
        check_codes(norm64(_f64(X), None, None, EPS)[1], 0, 21, _f64(q2), _f64(s2))


@gpu
@pytest.mark.parametrize("M", [4, 400])
@pytest.mark.parametrize("group", [0, 128])
def test_weights_of_extreme_size(M, group):
    """Weights whose product with h leaves fp32's range although y does not, and
    ones that make every y tiny."""
    import torch
    K = 1024
    X = _rows(_data(M, K, 70, 1e6), torch.float32)
    for size in (1e33, 1e-33, 1e-36):
        gamma = torch.full((K,), size, device="cuda")
        q, s, _ = w4.w8a8_add_rmsnorm_quantize(X, gamma, EPS, group)
        torch.cuda.synchronize()
        check_codes(norm64(_f64(X), None, _f64(gamma), EPS)[1], group, 21, _f64(q), _f64(s))


@gpu
@pytest.mark.parametrize("M,K", [(300, 1537), (500, 5001), (300, 12289), (4, 30001)])
def test_sum_in_place_off_the_alignment(M, K):
    for _ in range(3):
        test_sum_in_place_of_an_input(M, K)


@gpu
@pytest.mark.parametrize("M,K", [(40, 63), (40, 2048), (1000, 63), (1000, 2048), (2000, 1025)])
def test_sum_in_place_of_an_input(M, K):
    import torch
    for which in ("X", "residual"):
        X, R = _rows(_data(M, K, 7), torch.bfloat16), _rows(_data(M, K, 8), torch.bfloat16)
        q, s, h = w4.w8a8_add_rmsnorm_quantize(X.clone(), None, EPS, residual=R.clone())
        into = X if which == "X" else R
        q2, s2, h2 = w4.w8a8_add_rmsnorm_quantize(X, None, EPS, residual=R, H=into)
        torch.cuda.synchronize()
        assert h2 is into and torch.equal(h2, h) and torch.equal(q2, q) and torch.equal(s2, s)


@gpu
def test_rows_far_apart():
    """Offsets past 2^31 elements."""
    import torch
    K, ld = 4096, (1 << 30) + 8
    buf = torch.empty((3 * ld + K,), dtype=torch.bfloat16, device="cuda")
    X = buf.as_strided((4, K), (ld, 1))
    x = _data(4, K, 9)
    X.copy_(torch.from_numpy(x).to(torch.bfloat16))
    near = X.contiguous()
    q, s, _ = w4.w8a8_add_rmsnorm_quantize(X, None, EPS, 128)
    q2, s2, _ = w4.w8a8_add_rmsnorm_quantize(near, None, EPS, 128)
    g, t = w4.w8a8_silu_mul_quantize(X, X)
    g2, t2 = w4.w8a8_silu_mul_quantize(near, near)
    torch.cuda.synchronize()
    assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(g, g2) and torch.equal(t, t2)


@gpu
def test_no_rows():
    import torch
    X = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    q, s, h = w4.w8a8_add_rmsnorm_quantize(X, None, EPS, residual=X)
    assert q.shape == (0, 128) and s.shape == (0,) and h.shape == (0, 128)
    q, s = w4.w8a8_silu_mul_quantize(X, X)
    assert q.shape == (0, 128) and s.shape == (0,)


@gpu
def test_binding_refusals():
    import torch
    X = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")
    bad = [dict(residual=X.float()), dict(residual=X[:3]), dict(gamma=X[0, :64]), dict(gamma=X[0].cpu()),
           dict(residual=torch.zeros((128, 4), dtype=torch.bfloat16, device="cuda").t()),
           dict(Xq=torch.zeros((4, 136), dtype=torch.int8, device="cuda")[:, :128]),
           dict(Xq=torch.zeros((4, 128), dtype=torch.uint8, device="cuda")),
           dict(x_scale=torch.zeros((5,), device="cuda")), dict(group=48), dict(eps=0.0), dict(H=X.half())]
    for kw in bad:
        with pytest.raises(w4.W4A4Error):
            w4.w8a8_add_rmsnorm_quantize(**{**dict(X=X, gamma=None, eps=EPS), **kw})
    with pytest.raises(w4.W4A4Error):
        w4.w8a8_add_rmsnorm_quantize(X.double(), None, EPS)
    with pytest.raises(w4.W4A4Error):
        w4.w8a8_silu_mul_quantize(X, X[:, ::2])


@gpu
@pytest.mark.parametrize("K,group", [(4096, 128), (1001, 0)])
def test_captured_and_replayed(K, group):
    import torch
    M = 70
    X, R, G = (_rows(_data(M, K, k), torch.bfloat16) for k in (10, 11, 12))
    side = torch.cuda.Stream()
    q0 = torch.empty((M, (K + 15) // 16 * 16), dtype=torch.int8, device="cuda")[:, :K]
    q1 = torch.empty((M, (K + 15) // 16 * 16), dtype=torch.int8, device="cuda")[:, :K]
    s0, s1, H = torch.empty(M, device="cuda"), torch.empty(M, device="cuda"), torch.empty_like(X)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        w4.w8a8_add_rmsnorm_quantize(X, None, EPS, group, residual=R, H=H, Xq=q0, x_scale=s0)
        w4.w8a8_silu_mul_quantize(H, G, group, Xq=q1, x_scale=s1)
    for seed in (20, 21):
        X.copy_(torch.from_numpy(_data(M, K, seed)).to(X.dtype))
        graph.replay()
        torch.cuda.synchronize()
        a = w4.w8a8_add_rmsnorm_quantize(X, None, EPS, group, residual=R)
        b = w4.w8a8_silu_mul_quantize(a[2], G, group)
        torch.cuda.synchronize()
        assert torch.equal(q0, a[0]) and torch.equal(s0, a[1]) and torch.equal(H, a[2])
        assert torch.equal(q1, b[0]) and torch.equal(s1, b[1])
    del graph


@gpu
def test_on_another_stream():
    """Outputs allocated for a given stream are that stream's, and the call is
    ordered behind what the stream was doing."""
    import torch
    side = torch.cuda.Stream()
    want = w4.w8a8_add_rmsnorm_quantize(_rows(_data(64, 2048, 30), torch.bfloat16), None, EPS)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        X = torch.zeros((64, 2048), dtype=torch.bfloat16, device="cuda")
        for _ in range(20):
            X.mul_(1.0)
        X.copy_(_rows(_data(64, 2048, 30), torch.bfloat16))
    q, s, _ = w4.w8a8_add_rmsnorm_quantize(X, None, EPS, stream=side)
    side.synchronize()
    assert torch.equal(q, want[0]) and torch.equal(s, want[1])


@gpu
def test_repeated_calls_are_bit_equal():
    import torch
    X, R = _rows(_data(600, 5120, 31), torch.bfloat16), _rows(_data(600, 5120, 32), torch.bfloat16)
    first = w4.w8a8_add_rmsnorm_quantize(X, None, EPS, 128, residual=R)
    for _ in range(5):
        again = w4.w8a8_add_rmsnorm_quantize(X, None, EPS, 128, residual=R)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@gpu
@pytest.mark.parametrize("M,K", [(2000, 384), (40, 4093)])
def test_codes_next_to_a_half(M, K):
    """Rows y = 32 up (SiLU(32) = 32 in fp32: 1 + e^-32 rounds to 1) whose values lie one to
    three fp32 steps on either side of (k + 1/2) s.  The product y (1 / s) is rounded to an
    integer without an intermediate rounding, and 1 / s is off by 1.01 u of itself, so every
    quotient farther than that from its half has one code only."""
    import torch
    rng = np.random.default_rng(90)
    m = (1.0 + rng.random(M)).astype(np.float32)
    s = (m / np.float32(127.0)).astype(np.float32)
    half = (rng.integers(0, 126, (M, K)) + 0.5) * s.astype(np.float64)[:, None]
    y = half.astype(np.float32)
    y = y.view(np.int32) + rng.integers(-3, 4, (M, K)).astype(np.int32)
    y = y.view(np.float32) * np.where(rng.random((M, K)) < 0.5, -1, 1).astype(np.float32)
    y[:, K // 2] = m
    up = torch.from_numpy(y / np.float32(32.0)).cuda()
    q, got = w4.w8a8_silu_mul_quantize(torch.full_like(up, 32.0), up)
    torch.cuda.synchronize()
    assert np.array_equal(got.cpu().numpy(), s)
    r = y.astype(np.float64) / s.astype(np.float64)[:, None]
    apart = np.abs(np.abs(r) - np.floor(np.abs(r)) - 0.5) > 1.01 * U * np.abs(r)
    assert 0.5 < apart.mean() < 1.0
    assert np.array_equal(q.cpu().numpy()[apart], np.rint(r)[apart].astype(np.int8))


@gpu
@pytest.mark.parametrize("M,K,pad", [(40, 64, 0), (300, 1000, 0), (300, 1001, 1), (4000, 3200, 0), (1500, 6001, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_large_values_behind_strongly_negative_gates(M, K, pad, dtype):
    """silu(-100) = -3.7e-42 leaves fp32's normal range, times 1e38 it does not: each row has gates
    around one of -80 to -170 and values up to the type's largest."""
    import torch
    dt = _dt(dtype)
    rng = np.random.default_rng(91)
    base = rng.uniform(-170.0, -80.0, (M, 1))
    gate = _rows(base + rng.uniform(-4.0, 4.0, (M, K)), dt, pad)
    up = _rows(rng.choice([-1.0, 1.0], (M, K)) * np.exp(rng.uniform(80.0, 88.0, (M, K))), dt, pad)
    gate[:, 1], up[:, 1] = torch.finfo(dt).min, 1.0
    q, s = w4.w8a8_silu_mul_quantize(gate, up)
    torch.cuda.synchronize()
    a, b = _f64(gate), _f64(up)
    with np.errstate(over="ignore"):
        y, c = silu64(a, b), silu_c(np.maximum(a, -200.0))
    y[:, 1] = 0.0
    assert (np.abs(y).max(axis=1) > 2.0 ** -126).all()
    check_codes(y, 0, c, _f64(q), _f64(s))


@pytest.mark.parametrize("group", [1 << 32, (1 << 32) + 64, -(1 << 32), -1, 1 << 31])
def test_marshalling_refuses_a_group_that_is_no_int(lib, group):
    """Before anything else is looked at: the low 32 bits of these are groups that the library takes."""
    import torch
    w4._bind_calls()
    x, q, s = torch.zeros(2, 64), torch.zeros((2, 64), dtype=torch.int8), torch.zeros(2)
    c = w4._calls
    assert c.add_rmsnorm_quantize(x, None, EPS, group, None, None, q, s, 0) == SHAPE
    assert c.silu_mul_quantize(x, x, group, q, s, 0) == SHAPE
    assert c.matmul(q, s, q, s, group, None, x, 0) == SHAPE
    assert c.silu_mul_quantize(x, x, 64, q, s, 0) == INVALID      # host tensors
    with pytest.raises(TypeError):
        c.silu_mul_quantize(x, x, 64.0, q, s, 0)


@gpu
@pytest.mark.parametrize("group", [1 << 32, (1 << 32) + 64])
def test_a_group_past_32_bits_is_refused(group):
    import torch
    X = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")
    q, s = torch.zeros((4, 128), dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda")
    for call in (lambda: w4.w8a8_add_rmsnorm_quantize(X, None, EPS, group), lambda: w4.w8a8_silu_mul_quantize(X, X, group),
                 lambda: w4.w8a8_matmul(q, s, q, s, group)):
        with pytest.raises(w4.W4A4Error) as e:
            call()
        assert e.value.status == SHAPE


@gpu
def test_each_refusal_of_the_binding_has_its_status():
    """One argument at a time is wrong, and the call is refused for it."""
    import torch
    X = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")
    code = torch.zeros((5, 160), dtype=torch.int8, device="cuda")
    s = torch.zeros(5, device="cuda")
    common = [(SHAPE, dict(Xq=code[:3, :128])), (SHAPE, dict(Xq=code[:4, :127])), (MISALIGNED, dict(Xq=code[:4, 8:136])),
              (SHAPE, dict(Xq=torch.zeros((4, 136), dtype=torch.int8, device="cuda")[:, :128])),
              (INVALID, dict(Xq=code[:4, :128].view(torch.uint8))), (INVALID, dict(Xq=code[:4, :128].cpu())),
              (SHAPE, dict(x_scale=s)), (INVALID, dict(x_scale=s[:4].double())),
              (SHAPE, dict(x_scale=torch.zeros(8, device="cuda")[::2])), (SHAPE, dict(group=48)), (SHAPE, dict(group=-64))]
    norm = [(SHAPE, dict(gamma=X[0, :64])), (INVALID, dict(gamma=X[0].float())), (INVALID, dict(gamma=X[0].cpu())),
            (SHAPE, dict(residual=X[:3])), (INVALID, dict(residual=X.float())), (SHAPE, dict(H=X[:, :64])),
            (INVALID, dict(H=X.half())), (SHAPE, dict(H=X[:1].expand(4, 128))), (INVALID, dict(eps=0.0)),
            (INVALID, dict(eps=float("nan"))), (INVALID, dict(X=X.double())),
            (SHAPE, dict(X=torch.zeros((128, 4), dtype=torch.bfloat16, device="cuda").t()))]
    for status, kw in common + norm:
        with pytest.raises(w4.W4A4Error) as e:
            w4.w8a8_add_rmsnorm_quantize(**{**dict(X=X, gamma=None, eps=EPS), **kw})
        assert e.value.status == status, (kw.keys(), e.value)
    for status, kw in common + [(SHAPE, dict(up=X[:3])), (INVALID, dict(up=X.half())), (INVALID, dict(up=X.cpu())),
                                (SHAPE, dict(up=torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")[:, ::2])),
                                (SHAPE, dict(gate=X[:1].expand(4, 128)))]:
        with pytest.raises(w4.W4A4Error) as e:
            w4.w8a8_silu_mul_quantize(**{**dict(gate=X, up=X), **kw})
        assert e.value.status == status, (kw.keys(), e.value)
    torch.cuda.synchronize()
    assert not code.any() and not s.any()


@gpu
@pytest.mark.parametrize("M,K,group", [(7, 128, 64), (400, 1024, 128), (3000, 3200, 128)])
def test_strongly_negative_gates_in_fp16_and_rotated(M, K, group):
    """Rows whose gates all lie below -87: y is some 1e-35, its scale under 2^-100."""
    import torch
    rng = np.random.default_rng(92)
    base = rng.uniform(-96.0, -92.0, (M, 1))
    gate = _rows(base + rng.uniform(-4.0, 4.0, (M, K)), torch.float16)
    up = _rows(rng.choice([-1.0, 1.0], (M, K)) * rng.uniform(2e4, 6.5e4, (M, K)), torch.float16)
    q, s = w4.w8a8_silu_mul_quantize(gate, up, group)
    torch.cuda.synchronize()
    a, b = _f64(gate), _f64(up)
    check_codes(silu64(a, b), group, silu_c(a), _f64(q), _f64(s))
