"""Every form in which the norm and the gated activation are launched (direct
or through a ring in shared memory, by alignment, chunks per thread and threads
per row), several rounds of rows each, against the formulas in 64 bits.  The
tolerances are those of test_row_quantize; the formulas run on the device."""
from __future__ import annotations

import numpy as np
import pytest

import w4a4_int4_quantized_b200 as w4

from test_row_quantize import EPS, INVALID, OK, SHAPE, U, _dt, hadamard, lib  # noqa: F401

gpu = pytest.mark.gpu

# form of w8a8_plan_rows on 148 SMs, chunks per thread, most threads of the kernel, M, K
DIRECT = [
    (0, 1, 128, 5, 8), (0, 1, 1024, 5, 264), (0, 2, 128, 2505, 264), (0, 2, 1024, 5, 8200), (0, 4, 128, 1205, 832),
    (0, 4, 1024, 5, 16392), (1, 1, 1024, 5, 257), (1, 2, 1024, 5, 8193), (1, 4, 1024, 5, 16385), (2, 1, 128, 5, 1),
    (2, 2, 128, 2505, 257),
]
RING_16 = [
    (3, 1, 384, 70000, 256), (3, 2, 384, 40000, 512), (3, 2, 1024, 785, 12800), (3, 4, 384, 1955, 6144),
    (3, 4, 1024, 637, 17408), (4, 1, 384, 70000, 240), (4, 2, 384, 40000, 424), (4, 2, 1024, 785, 12296),
    (4, 4, 384, 1911, 6152), (4, 4, 1024, 637, 16392), (5, 2, 1024, 785, 12289), (5, 4, 1024, 637, 16385),
]
RING_32 = [
    (3, 1, 384, 40000, 256), (3, 1, 1024, 785, 6400), (3, 2, 384, 1955, 4608), (3, 2, 1024, 637, 8192),
    (4, 1, 384, 40000, 216), (4, 1, 1024, 785, 6152), (4, 2, 384, 1467, 3560), (4, 2, 1024, 637, 7688),
    (4, 4, 384, 1955, 3080), (5, 1, 1024, 785, 6145), (5, 2, 1024, 637, 7681),
]
# (gated, bytes of an element) -> cases with two inputs, and of a norm without a residual
CASES = {
    (0, 2): DIRECT + RING_16 + [(5, 1, 384, 200000, 193), (5, 2, 384, 100000, 401), (5, 4, 384, 977, 12270),
                                (3, 4, 384, 4608, 4096), (4, 4, 384, 4608, 4104), (3, 4, 384, 16384, 1024),
                                (4, 4, 384, 20000, 1000), (5, 4, 384, 13340, 5222)],
    (1, 2): DIRECT + RING_16 + [(5, 1, 384, 40000, 193), (5, 2, 384, 20000, 401), (5, 4, 384, 1955, 6121)],
    (0, 4): DIRECT + RING_32 + [(5, 1, 384, 100000, 201), (5, 2, 384, 977, 6134), (5, 4, 384, 6000, 3495)],
    (1, 4): DIRECT + RING_32 + [(5, 1, 384, 20000, 201), (5, 2, 384, 1955, 3066), (5, 4, 384, 1955, 3073)],
}
ALONE = {
    2: [(3, 4, 384, 8200, 6144), (5, 4, 384, 16384, 5003)],
    4: [(3, 4, 384, 20000, 1024), (3, 4, 1024, 637, 17408), (4, 4, 1024, 637, 16392), (5, 4, 1024, 637, 16385),
        (5, 4, 384, 16384, 5003)],
}
NAMES = {2: ("bf16", "fp16"), 4: ("fp32",)}


def kind(plan):
    form, vpt, threads = plan[:3]
    return form, vpt, (128 if threads == 32 else 1024) if form < 3 else 384 if threads <= 384 else 1024


def aligned(form):
    return form in (0, 3, 4)


def test_every_form_has_its_cases(lib):
    """The cases take the forms that they are listed under, and no size takes a form that is not among them."""
    listed = {key: {c[:3] for c in cases} for key, cases in CASES.items()}
    for (gated, size), cases in CASES.items():
        for dtype in NAMES[size]:
            for form, vpt, most, M, K in cases:
                assert kind(w4.w8a8_plan_rows(gated, M, K, dtype, aligned=aligned(form))) == (form, vpt, most), (M, K)
    for size, cases in ALONE.items():
        listed[0, size] |= {c[:3] for c in cases}
        for form, vpt, most, M, K in cases:
            plan = w4.w8a8_plan_rows(0, M, K, NAMES[size][0], residual=False, aligned=aligned(form))
            assert kind(plan) == (form, vpt, most), (M, K)
    widths = sorted({*range(1, 1100, 3), *range(8, 32769, 136), *range(256, 32769, 256), *range(257, 32769, 509), 32767, 32768})
    for K in widths:
        for M in (1, 297, 700, 1500, 3000, 9000, 70000, 2 ** 31 - 1):
            for (gated, size), forms in listed.items():
                for residual in ((True,) if gated else (False, True)):
                    for al in ((False, True) if K % 8 == 0 else (False,)):
                        assert kind(w4.w8a8_plan_rows(gated, M, K, NAMES[size][0], residual, al)) in forms, (M, K)


def test_plan_refusals(lib):
    import ctypes
    f, out = lib.w8a8_plan_rows, (ctypes.c_int * 5)()
    assert f(0, 1, 1, 4, 64, 0, 148, out) == OK
    assert f(0, 1, 1, 4, 64, 0, 148, None) == INVALID and f(0, 1, 1, 4, 64, 3, 148, out) == INVALID
    for M, K, sms in ((0, 64, 148), (-1, 64, 148), (4, 0, 148), (4, 32769, 148), (4, 64, 0)):
        assert f(0, 1, 1, M, K, 0, sms, out) == SHAPE


def check(y, g, c, q, s):
    """check_codes of test_row_quantize on tensors: codes q and scales s of the 64-bit rows y, c u of
    relative error in y."""
    import torch
    M, K = y.shape
    q, s, mag = q.double(), s.double(), y.abs()
    if g:
        D = U * ((c + np.log2(g)) * mag).view(M, K // g, g).sum(dim=2).amax(dim=1)
        y = (y.view(M, K // g, g) @ torch.from_numpy(hadamard(np.eye(g), g)).to(y.device)).view(M, K)
    else:
        D = U * (c * mag).amax(dim=1)
    amax = y.abs().amax(dim=1)
    s64 = amax / 127.0
    assert ((s - s64).abs() <= D / 127.0 + U * s64 + 2.0 ** -149).all()
    some = amax > 0
    assert not q[~some].any() and not s[~some].any()
    off = (q - y / s64[:, None]).abs().amax(dim=1) - 2 * 127 * D / amax - 4 * 127 * U
    assert (off[some] <= 0.5).all(), float(off[some].max())
    assert q.abs().max() <= 127


@pytest.mark.parametrize("g", [0, 64])
def test_check_catches_planted_mistakes(g):
    import torch
    rng = np.random.default_rng(1)
    y = torch.from_numpy(rng.standard_normal((5, 256)))
    y[3] = 0
    z = torch.from_numpy(hadamard(y.numpy(), g)) if g else y
    s = z.abs().amax(dim=1) / 127
    q = torch.where(s[:, None] > 0, torch.round(z / s[:, None]), torch.zeros_like(z))
    check(y, g, 21, q, s)
    one = torch.zeros_like(q)
    one[1, 7] = 1
    empty = torch.zeros_like(q)
    empty[3, 200] = 1
    for bad in ((y, q + one, s), (y, q + empty, s), (y, q, s * (1 + 1e-4)), (y * 1.01, q, s), (y, q, s.roll(1))):
        with pytest.raises(AssertionError):
            check(bad[0], g, 21, bad[1], bad[2])


def data(M, K, dtype, seed, scale=1.0):
    """Rows of unlike size, a channel in a few larger than the rest, one row of zeros."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((M, K), generator=gen, device="cuda") * scale
    x[:, :: max(1, K // 3)] *= 12.0
    x *= 10.0 ** torch.randint(-2, 2, (M, 1), generator=gen, device="cuda")
    x[M // 2] = 0
    return x.to(dtype)


def place(x, offset):
    """A copy of x with rows one after the other from `offset` elements on, and its buffer."""
    import torch
    buf = torch.full((x.numel() + 2 * offset,), 7.0, dtype=x.dtype, device="cuda")
    view = buf[offset:offset + x.numel()].view(x.shape)
    view.copy_(x)
    return view, buf


def untouched(buf, offset):
    return not offset or bool((buf[:offset] == 7.0).all() and (buf[-offset:] == 7.0).all())


def parametrised(table):
    return [(dtype, *c) for size in (2, 4) for dtype in NAMES[size] for c in table[size]]


@gpu
@pytest.mark.parametrize("dtype,form,vpt,most,M,K", parametrised({2: CASES[0, 2], 4: CASES[0, 4]}))
def test_norm(dtype, form, vpt, most, M, K):
    """With a residual and weights; the sum beside its inputs, then in place of either."""
    import torch
    dt, off = _dt(dtype), 0 if aligned(form) else 1
    x, r, w = data(M, K, dt, 1), data(M, K, dt, 2, 2.0), (1 + 0.1 * data(1, K, torch.float32, 3)[0]).to(dt)
    h64 = x.double() + r.double()
    y64 = h64 / (h64.square().mean(dim=1, keepdim=True) + EPS).sqrt() * w.double()
    X, R, gamma = place(x, off)[0], place(r, off)[0], place(w[None], off)[0][0]
    H, hbuf = place(torch.zeros_like(x), off)
    tiny = 2.0 ** -25 if dtype == "fp16" else 0.0
    for group in (0, 128) if K % 128 == 0 else (0,):
        q, s, h = w4.w8a8_add_rmsnorm_quantize(X, gamma, EPS, group, residual=R, H=H)
        check(y64, group, 21, q, s)
        assert h is H and untouched(hbuf, off)
        assert ((h.double() - h64).abs() <= (torch.finfo(dt).eps / 2 + 2 * U) * h64.abs() + tiny).all()
        assert torch.equal(X, x) and torch.equal(R, r)
        for which in (0, 1):
            both = [place(x, off), place(r, off)]
            into, buf = both[which]
            q2, s2, h2 = w4.w8a8_add_rmsnorm_quantize(both[0][0], gamma, EPS, group, residual=both[1][0], H=into)
            assert h2 is into and torch.equal(h2, h) and torch.equal(q2, q) and torch.equal(s2, s)
            assert untouched(buf, off)


@gpu
@pytest.mark.parametrize("dtype,form,vpt,most,M,K", parametrised(ALONE))
def test_norm_without_a_residual(dtype, form, vpt, most, M, K):
    import torch
    dt, off = _dt(dtype), 0 if aligned(form) else 1
    x = data(M, K, dt, 4)
    y64 = x.double() / (x.double().square().mean(dim=1, keepdim=True) + EPS).sqrt()
    X, _ = place(x, off)
    for group in (0, 64) if K % 64 == 0 else (0,):
        q, s, h = w4.w8a8_add_rmsnorm_quantize(X, None, EPS, group)
        check(y64, group, 21, q, s)
        assert h is None and torch.equal(X, x)


@gpu
@pytest.mark.parametrize("dtype,form,vpt,most,M,K", parametrised({2: CASES[1, 2], 4: CASES[1, 4]}))
def test_silu(dtype, form, vpt, most, M, K):
    import torch
    dt, off = _dt(dtype), 0 if aligned(form) else 1
    a, b = data(M, K, dt, 5, 0.5), data(M, K, dt, 6)
    y64 = a.double() / (1.0 + torch.exp(-a.double())) * b.double()
    c = 9 + 1.5 * (-a.double()).clamp_min(0.0)
    gate, up = place(a, off)[0], place(b, off)[0]
    for group in (0, 128) if K % 128 == 0 else (0,):
        q, s = w4.w8a8_silu_mul_quantize(gate, up, group)
        check(y64, group, c, q, s)
