"""Matrix product with bias, activation and residual, and its gradient,
against a plain implementation in 64 bits at sizes around every tile edge and
path (few rows, CTA pairs at each tile width, one launch for two products),
with odd strides, and the entry points' refusals.

Tolerances, derived from the arithmetic.  A sum of K products is accumulated
in fp32 in steps of 16: its error is at most (K / 16 + 16) 2^-23 of the sum of
the products' sizes.  An activation's slope is below 1.2 and its own error
below 2^-19 of its argument's size; each bf16 result adds one rounding (2^-8 of
the value bounds it).  The gradient's products have dz as a bf16 operand, one
more rounding (bf16 keeps 8 bits, so at most 2^-8) of each dz: at most 2^-8 of
the sum of sizes, and in the 2-norm, where independent roundings add in
squares, the two roundings of 2^-9 / sqrt(3) * 1.5 relative each stay below
4e-3.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import workloads as wl

FAKE = ctypes.c_void_p(0x10000)
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def mat(seed, rows, cols, sigma, pad=0, dtype=torch.bfloat16):
    """(CUDA view, float64 CPU copy) of normal draws in a buffer `pad` wider."""
    x = torch.from_numpy(wl.normal_matrix(seed, rows, cols + pad, sigma, dtype="f32"))
    t = x.to(dtype).cuda()[:, :cols]
    return t, t.double().cpu()


def act64(z, act):
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z * (z > 0), (z > 0).double()
    if act == "silu":
        q = 1 / (1 + torch.exp(-z))
        return z * q, q * (1 + z * (1 - q))
    if act == "gelu":
        c = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    a = math.sqrt(2 / math.pi)
    t = torch.tanh(a * (z + 0.044715 * z ** 3))
    return z * (1 + t) / 2, (1 + t) / 2 + z * (1 - t * t) / 2 * a * (1 + 3 * 0.044715 * z * z)


def check(got, exp, tol, what):
    got = got.double().cpu()
    assert got.shape == exp.shape
    assert torch.isfinite(got).all(), what
    err = (got - exp).abs() - tol
    assert (err <= 0).all(), (what, float(err.max()), int(err.argmax()))


def sum_tol(k, sizes):
    return (k / 16 + 16) * 2.0 ** -23 * sizes


# (M, N, K): few rows, tile edges, odd sizes, several waves of tiles
SHAPES = [(1, 1, 8), (1, 128, 64), (1, 4096, 4096), (3, 130, 72), (16, 257, 640), (17, 300, 136),
          (33, 1000, 520), (64, 127, 2048), (65, 513, 64), (100, 2100, 1032), (128, 129, 4096),
          (129, 64, 64), (129, 200, 72), (200, 1531, 1160), (256, 256, 128), (257, 257, 264),
          (300, 5000, 256), (1000, 2050, 200), (2111, 3333, 104), (9, 40000, 16),
          # single tokens: every CTA width, and the rows that go to the tensor cores
          (1, 3000, 264), (1, 5000, 1032), (1, 77, 9000), (2, 301, 5000), (2, 2500, 4104),
          (3, 4099, 2048), (3, 20, 8), (4, 1000, 640), (4, 3000, 4096), (4, 513, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear_matches_64_bits(sga_lib, shape):
    M, N, K = shape
    i = SHAPES.index(shape)
    act = ACTS[i % 5]
    pad = (0, 8, 64)[i % 3]
    x, x64 = mat(i + 1, M, K, 1.0, pad)
    w, w64 = mat(i + 101, N, K, K ** -0.5, (0, 16)[i % 2])
    bias = res = pre = None
    z64 = x64 @ w64.T
    size = x64.abs() @ w64.abs().T
    if i % 3 != 1:
        b, b64 = mat(i + 201, 1, N, 0.7, 0, (torch.float32, torch.bfloat16)[i % 2])
        bias = b[0].contiguous()
        z64 = z64 + b64
        size = size + b64.abs()
    y64, _ = act64(z64, act)
    if i % 2 == 0:
        res, r64 = mat(i + 301, M, N, 1.0, (0, 1, 8)[i % 3])
        y64 = y64 + r64
    if i % 4 < 2:
        pre = torch.full((M, N + 3), 9.0, dtype=torch.bfloat16, device="cuda")[:, :N]
    buf = torch.full((M, N + (0, 1, 2)[i % 3]), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, :N]
    sga_lib.sga_linear(x, w, out, bias, ACTS.index(act), res, pre)
    tol = 1.2 * sum_tol(K, size) + 2.0 ** -19 * z64.abs()
    check(out, y64, tol + 2.0 ** -8 * y64.abs() + 1e-30, "out")
    if pre is not None:
        check(pre, z64, tol + 2.0 ** -8 * z64.abs() + 1e-30, "preact")
    assert (buf[:, N:] == 7.0).all()
    assert sga_lib.sga_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("M", [5, 300])
@pytest.mark.parametrize("act", ACTS)
def test_activations_over_their_range(sga_lib, M, act):
    """x . I: the pre-activation is exact, so the activation itself is tested,
    far into both tails; and the residual is read in place."""
    K = 64
    x = torch.linspace(-30, 30, M * K).reshape(M, K).to(torch.bfloat16).cuda()
    x[0, :4] = torch.tensor([0.0, -0.0, 1e30, -1e30])
    eye = torch.eye(K, dtype=torch.bfloat16, device="cuda")
    z64 = x.double().cpu()
    y64, _ = act64(z64, act)
    y64 = torch.where(z64 < -1e3, 0.0 if act != "none" else z64, y64)
    y64 = torch.where(z64 > 1e3, z64, y64)
    out = torch.full((M, K), 3.0, dtype=torch.bfloat16, device="cuda")
    sga_lib.sga_linear(x, eye, out, act=ACTS.index(act))
    check(out, y64, 2.0 ** -19 * z64.abs().clamp(max=100) + 2.0 ** -8 * y64.abs() + 1e-30, act)
    acc = torch.full((M, K), 3.0, dtype=torch.bfloat16, device="cuda")
    sga_lib.sga_linear(x, eye, acc, act=ACTS.index(act), residual=acc)
    y64 = y64 + 3.0
    check(acc, y64, 2.0 ** -19 * z64.abs().clamp(max=100) + 2.0 ** -8 * y64.abs() + 1e-30, act)


def tail_exponent(z, act):
    """u of the e^-u that an activation's left tail falls with."""
    if act == "gelu":
        return z * z / 2
    if act == "gelu_tanh":
        return 2 * math.sqrt(2 / math.pi) * (z.abs() + 0.044715 * z.abs() ** 3)
    return z.abs()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [2, 40, 300, 3000])
@pytest.mark.parametrize("act", ACTS)
def test_activation_tails_relative_to_their_values(sga_lib, M, act):
    """x . I from -12 to 12, where the values fall to 1e-32, and the derivatives
    (dz . I of an upstream gradient of ones).  Relative to the value, or to the
    sizes of a derivative's terms: the tails fall as e^-u, whose exponent takes at
    most eight roundings (u 2^-21), 32 ulps for the rest (2^-19), and one rounding
    to bf16; 1e-36 for what is flushed below the normal numbers of fp32."""
    K = 64
    x = torch.linspace(-12, 12, M * K).reshape(M, K).to(torch.bfloat16).cuda()
    eye = torch.eye(K, dtype=torch.bfloat16, device="cuda")
    z = x.double().cpu()
    y64, d64 = act64(z, act)
    if act == "gelu_tanh":       # (1 + tanh u) / 2 = 1 / (1 + e^-2u), which does not cancel
        u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        q = torch.sigmoid(2 * u)
        y64 = z * q
        d64 = q + 2 * y64 * torch.sigmoid(-2 * u) * math.sqrt(2 / math.pi) * (
            1 + 3 * 0.044715 * z * z)
    rel = 2.0 ** -19 + tail_exponent(z, act) * 2.0 ** -21
    out = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    sga_lib.sga_linear(x, eye, out, act=ACTS.index(act))
    check(out, y64, (2.0 ** -8 + rel) * y64.abs() + 1e-36, act)
    ws = torch.empty(sga_lib.sga_linear_grad_workspace(M, K, K), dtype=torch.uint8, device="cuda")
    sga_lib.sga_linear_grad(torch.ones_like(out), x, eye, ws, ACTS.index(act),
                            None if act == "none" else x, grad_x=out)
    # d = y / z + (d - y / z): the value's factor and z times that factor's slope
    factor = torch.where(z == 0, 0.5, y64 / torch.where(z == 0, 1.0, z))
    check(out, d64, 2.0 ** -8 * d64.abs() + rel * (factor.abs() + (d64 - factor).abs()) + 1e-36,
          act + " derivative")


@pytest.mark.gpu
@pytest.mark.parametrize("M", [4, 200])
def test_runs_are_identical_on_any_stream_and_in_a_graph(sga_lib, M):
    N, K = 1000, 2048
    x, _ = mat(1, M, K, 1.0)
    w, _ = mat(2, N, K, K ** -0.5)
    g, _ = mat(3, M, N, 1.0)
    z, _ = mat(4, M, N, 1.0)
    ws = torch.empty(sga_lib.sga_linear_grad_workspace(M, N, K), dtype=torch.uint8, device="cuda")
    outs = [torch.empty((M, N), dtype=torch.bfloat16, device="cuda"),
            torch.empty((M, K), dtype=torch.bfloat16, device="cuda"),
            torch.empty((N, K), dtype=torch.bfloat16, device="cuda"),
            torch.empty(N, device="cuda")]

    def step():
        sga_lib.sga_linear(x, w, outs[0], act=2)
        sga_lib.sga_linear_grad(g, x, w, ws, 2, z, outs[1], outs[2], outs[3])

    step()
    torch.cuda.synchronize()
    first = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for o in outs:
            o.fill_(1.0)
        step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, outs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for o in outs:
        o.fill_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))


GRAD_SHAPES = [(1, 1, 8), (1, 128, 64), (2, 300, 72), (16, 1000, 1032), (60, 77, 200),
               (128, 520, 640), (129, 129, 136), (130, 1001, 264), (257, 600, 1000),
               (777, 1001, 336), (1030, 2048, 72), (64, 4096, 2048)]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", GRAD_SHAPES, ids=str)
def test_gradient_matches_64_bits(sga_lib, shape):
    M, N, K = shape
    i = GRAD_SHAPES.index(shape)
    act = ACTS[i % 5]
    x, x64 = mat(i + 1, M, K, 1.0, (0, 8)[i % 2])
    w, w64 = mat(i + 101, N, K, K ** -0.5, (0, 24)[i % 2])
    g, g64 = mat(i + 201, M, N, 1.0, (0, 1, 8)[i % 3])
    z, z64 = mat(i + 301, M, N, 1.5, (0, 5)[i % 2])
    dz = g64 * act64(z64, act)[1] if act != "none" else g64
    ws = torch.full((sga_lib.sga_linear_grad_workspace(M, N, K),), 255, dtype=torch.uint8,
                    device="cuda")
    gx = torch.full((M, K + i % 3), 5.0, dtype=torch.bfloat16, device="cuda")[:, :K]
    gw = torch.full((N, K + i % 2), 5.0, dtype=torch.bfloat16, device="cuda")[:, :K]
    gb = torch.full((N,), 5.0, dtype=(torch.float32, torch.bfloat16)[i % 2], device="cuda")
    sga_lib.sga_linear_grad(g, x, w, ws, ACTS.index(act), None if act == "none" else z, gx, gw, gb)
    round_dz = 2.0 ** -8 + 2.0 ** -18
    for got, exp, size, k, name in (
            (gx, dz @ w64, dz.abs() @ w64.abs(), N, "grad_x"),
            (gw, dz.T @ x64, dz.abs().T @ x64.abs(), M, "grad_weight")):
        check(got, exp, sum_tol(k, size) + round_dz * size + 2.0 ** -8 * exp.abs() + 1e-30, name)
        if got.numel() >= 1000:
            rel = (got.double().cpu() - exp).norm() / exp.norm()
            assert rel < 4e-3, (name, float(rel))
    exp = dz.sum(0)
    tol = (M * 2.0 ** -24 + 2.0 ** -18) * (g64.abs() * 1.2).sum(0) + 1e-30
    if gb.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * exp.abs()
    check(gb, exp, tol, "grad_bias")
    assert sga_lib.sga_device_error() == 0
    # each output alone gives the same
    one = [torch.empty_like(gx), torch.empty_like(gw), torch.empty_like(gb)]
    for n in range(3):
        out = [o if j == n else None for j, o in enumerate(one)]
        sga_lib.sga_linear_grad(g, x, w, ws, ACTS.index(act), None if act == "none" else z, *out)
    assert torch.equal(one[0], gx) and torch.equal(one[1], gw) and torch.equal(one[2], gb)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
def test_gradient_against_differences(sga_lib, act):
    """Central differences, in 64 bits, of the formula of the forward pass:
    truncation h^2 / 6 times a third derivative below 4 of the sizes."""
    M, N, K, h = 6, 10, 16, 1e-3
    x, x64 = mat(1, M, K, 1.0)
    w, w64 = mat(2, N, K, K ** -0.5)
    g, g64 = mat(3, M, N, 1.0)
    b, b64 = mat(4, 1, N, 1.0, 0, torch.float32)
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    pre = torch.empty_like(out)
    sga_lib.sga_linear(x, w, out, b[0].contiguous(), ACTS.index(act), None, pre)
    ws = torch.empty(sga_lib.sga_linear_grad_workspace(M, N, K), dtype=torch.uint8, device="cuda")
    gx, gw = torch.empty_like(x), torch.empty_like(w)
    gb = torch.empty(N, device="cuda")
    sga_lib.sga_linear_grad(g, x, w, ws, ACTS.index(act), pre, gx, gw, gb)
    z0 = pre.double().cpu()        # the saved (rounded) pre-activation is the point

    def loss(dx, dw, db):
        z = z0 + dx @ w64.T + x64 @ dw.T + dx @ dw.T + db
        return float((g64 * act64(z, act)[0]).sum())

    def diff(shape, place):
        d = torch.zeros(shape, dtype=torch.float64)
        out = torch.zeros(shape, dtype=torch.float64)
        for j in range(d.numel()):
            vals = []
            for s in (h, -h):
                d.view(-1)[j] = s
                vals.append(loss(*place(d)))
            d.view(-1)[j] = 0.0
            out.view(-1)[j] = (vals[0] - vals[1]) / (2 * h)
        return out

    zx, zw, zb = torch.zeros(M, K).double(), torch.zeros(N, K).double(), torch.zeros(N).double()
    for got, exp, size in (
            (gx, diff((M, K), lambda d: (d, zw, zb)), g64.abs() @ w64.abs()),
            (gw, diff((N, K), lambda d: (zx, d, zb)), g64.abs().T @ x64.abs()),
            (gb, diff((N,), lambda d: (zx, zw, d)), g64.abs().sum(0))):
        check(got, exp, 1.2 * size * 2.0 ** -9 + 2.0 ** -8 * exp.abs() + 1e-4 * (1 + size), act)


@pytest.mark.gpu
def test_no_rows(sga_lib):
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((40, 64), dtype=torch.bfloat16, device="cuda")
    y = torch.empty((0, 40), dtype=torch.bfloat16, device="cuda")
    sga_lib.sga_linear(x, w, y)
    buf = torch.ones((40, 72), dtype=torch.bfloat16, device="cuda")
    gb = torch.ones(40, device="cuda")
    sga_lib.sga_linear_grad(y, x, w, torch.empty(0, dtype=torch.uint8, device="cuda"),
                            grad_weight=buf[:, :64], grad_bias=gb)
    assert (buf[:, :64] == 0).all() and (buf[:, 64:] == 1).all() and (gb == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [0, 3])
def test_relu_cuts_off_infinities(sga_lib, pad):
    """Where relu gave 0 nothing comes back, whatever the upstream gradient is."""
    M, N, K = 40, 72, 64
    x, x64 = mat(21, M, K, 1.0)
    w, w64 = mat(22, N, K, 1.0)
    z, z64 = mat(23, M, N, 1.0, pad)
    g, g64 = mat(24, M, N, 1.0, pad)
    z[3, 5] = 0.0
    z64 = z.double().cpu()
    bad = torch.tensor([float("inf"), float("-inf"), float("nan")], dtype=torch.bfloat16).cuda()
    g.copy_(torch.where(z > 0, g, bad[torch.arange(M * N, device="cuda").reshape(M, N) % 3]))
    dz64 = torch.where(z64 > 0, g64, 0.0)
    gx, gw = torch.empty_like(x), torch.empty_like(w)
    gb = torch.empty(N, device="cuda")
    ws = torch.empty(sga_lib.sga_linear_grad_workspace(M, N, K), dtype=torch.uint8, device="cuda")
    sga_lib.sga_linear_grad(g, x, w, ws, ACTS.index("relu"), z, gx, gw, gb)
    check(gx, dz64 @ w64, sum_tol(N, dz64.abs() @ w64.abs()) + 2.0 ** -8 * (dz64 @ w64).abs(), "x")
    check(gw, dz64.T @ x64, sum_tol(M, dz64.abs().T @ x64.abs()) + 2.0 ** -8 * (dz64.T @ x64).abs(),
          "w")
    check(gb, dz64.sum(0), sum_tol(M, dz64.abs().sum(0)), "b")


# few rows: each number of parts of the sum, either ring, and around the numbers of
# clusters that the GPU holds at once
SPLIT_SHAPES = [(5, 1000, 8192), (20, 2000, 4104), (40, 1900, 5128), (40, 2100, 5128),
                (96, 1920, 5128), (100, 2060, 5128), (96, 4608, 2056), (90, 4700, 2056),
                (70, 9500, 1032), (70, 9700, 1032), (250, 1024, 5128)]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SPLIT_SHAPES, ids=str)
def test_split_sums_match_64_bits(sga_lib, shape):
    M, N, K = shape
    i = SPLIT_SHAPES.index(shape)
    act = ACTS[i % 5]
    x, x64 = mat(i + 401, M, K, 1.0)
    w, w64 = mat(i + 501, N, K, K ** -0.5)
    b, b64 = mat(i + 601, 1, N, 0.7, 0, torch.float32)
    res, r64 = mat(i + 701, M, N, 1.0, i % 4)
    out, pre = torch.empty_like(res), torch.empty_like(res)
    sga_lib.sga_linear(x, w, out, b[0].contiguous(), ACTS.index(act), res, pre)
    z64 = x64 @ w64.T + b64
    y64 = act64(z64, act)[0] + r64
    tol = 1.2 * sum_tol(K, x64.abs() @ w64.abs().T + b64.abs()) + 2.0 ** -19 * z64.abs()
    check(out, y64, tol + 2.0 ** -8 * y64.abs() + 1e-30, "out")
    check(pre, z64, tol + 2.0 ** -8 * z64.abs() + 1e-30, "preact")
    assert sga_lib.sga_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 40, 300])
def test_row_offsets_past_32_bits(sga_lib, M):
    """Every matrix with rows so far apart that the last ones lie more than 2^32
    elements on: the same results as from packed rows."""
    N, K = 200, 136
    ld = ((1 << 32) // (M - 1) // 8 + 33) * 8
    buf = torch.empty((M - 1) * ld + 2048, dtype=torch.bfloat16, device="cuda")

    def far(cols, at):
        return torch.as_strided(buf, (M, cols), (ld, 1), at)

    x, _ = mat(31, M, K, 1.0)
    w, _ = mat(32, N, K, 1.0)
    r, _ = mat(33, M, N, 1.0)
    act = ACTS.index("silu")
    out, z = torch.empty_like(r), torch.empty_like(r)
    sga_lib.sga_linear(x, w, out, None, act, r, z)
    fx, fr, fz, fout = far(K, 0), far(N, 256), far(N, 512), far(N, 768)
    fx.copy_(x)
    fr.copy_(r)
    sga_lib.sga_linear(fx, w, fout, None, act, fr, fz)
    assert torch.equal(fout, out) and torch.equal(fz, z)
    ws = torch.empty(sga_lib.sga_linear_grad_workspace(M, N, K), dtype=torch.uint8, device="cuda")
    gx, gw, gb = torch.empty_like(x), torch.empty_like(w), torch.empty(N, device="cuda")
    sga_lib.sga_linear_grad(r, x, w, ws, act, z, gx, gw, gb)
    fgx, fgw, fgb = far(K, 1024), torch.empty_like(w), torch.empty_like(gb)
    sga_lib.sga_linear_grad(fr, fx, w, ws, act, fz, fgx, fgw, fgb)
    assert torch.equal(fgx, gx) and torch.equal(fgw, gw) and torch.equal(fgb, gb)
    assert sga_lib.sga_device_error() == 0


# ----------------------------------------------------------------- refusals


def test_linear_validation(sga_lib):
    f = sga_lib.lib().sga_linear

    def call(**kw):
        a = dict(dict(x=FAKE, M=4, K=64, ldx=64, w=FAKE, N=10, ldw=64, b=FAKE, bd=0, act=0,
                      r=FAKE, ldr=10, z=FAKE, ldp=10, y=FAKE, ldo=10), **kw)
        return f(a["x"], a["M"], a["K"], a["ldx"], a["w"], a["N"], a["ldw"], a["b"], a["bd"],
                 a["act"], a["r"], a["ldr"], a["z"], a["ldp"], a["y"], a["ldo"], None)

    assert call(M=-1) == -2 and call(M=(1 << 20) + 1) == -2
    assert call(N=0) == -2 and call(N=(1 << 24) + 1) == -2
    assert call(K=0) == -2 and call(K=60, ldx=64) == -2
    assert call(ldx=56) == -2 and call(ldx=68) == -2 and call(ldw=56) == -2
    assert call(ldo=9) == -2 and call(ldr=9) == -2 and call(ldp=9) == -2
    assert call(act=5) == -11 and call(act=-1) == -11
    assert call(bd=3) == -5
    assert call(x=None) == -1 and call(w=None) == -1 and call(y=None) == -1
    off8, off1, off2 = (ctypes.c_void_p(0x10000 + o) for o in (8, 1, 2))
    assert call(x=off8) == -6 and call(w=off8) == -6
    assert call(r=off1) == -6 and call(z=off1) == -6 and call(y=off1) == -6
    assert call(b=off2) == -6 and call(b=off1, bd=1) == -6
    assert call(M=0, x=None) == 0


def test_linear_grad_validation(sga_lib):
    L = sga_lib.lib()
    ws = L.sga_linear_grad_workspace(4, 10, 64)
    assert ws > 0 and L.sga_linear_grad_workspace(0, 10, 64) == 0
    f = L.sga_linear_grad

    def call(**kw):
        a = dict(dict(g=FAKE, M=4, N=10, ldg=10, z=FAKE, ldp=10, act=2, x=FAKE, K=64, ldx=64,
                      w=FAKE, ldw=64, gx=FAKE, ldgx=64, gw=FAKE, ldgw=64, gb=FAKE, bd=1, ws=FAKE,
                      n=ws), **kw)
        return f(a["g"], a["M"], a["N"], a["ldg"], a["z"], a["ldp"], a["act"], a["x"], a["K"],
                 a["ldx"], a["w"], a["ldw"], a["gx"], a["ldgx"], a["gw"], a["ldgw"], a["gb"],
                 a["bd"], a["ws"], a["n"], None)

    assert call(M=-1) == -2 and call(N=0) == -2 and call(K=4) == -2 and call(ldg=9) == -2
    assert call(ldp=9) == -2 and call(ldgx=63) == -2 and call(ldgw=63) == -2
    assert call(act=7) == -11 and call(bd=2) == -5
    for name in ("g", "x", "w", "ws", "z"):
        assert call(**{name: None}) == -1, name
    off8, off1 = ctypes.c_void_p(0x10008), ctypes.c_void_p(0x10001)
    for name in ("x", "w", "ws"):
        assert call(**{name: off8}) == -6, name
    for name in ("g", "z", "gx", "gw", "gb"):
        assert call(**{name: off1}) == -6, name
    assert call(n=ws - 1) == -7
    assert call(M=0, gw=None, gb=None) == 0


def test_binding_refuses_wrong_tensors(sga_lib):
    b = torch.bfloat16
    x, w, y = torch.zeros(3, 64, dtype=b), torch.zeros(5, 64, dtype=b), torch.zeros(3, 5, dtype=b)
    with pytest.raises(ValueError):
        sga_lib.sga_linear(x.float(), w, y)
    with pytest.raises(ValueError):
        sga_lib.sga_linear(x, w[:, :32], y)
    with pytest.raises(ValueError):
        sga_lib.sga_linear(x, w, y[:, :4])
    with pytest.raises(ValueError):
        sga_lib.sga_linear(x, w, y.float())
    with pytest.raises(ValueError):
        sga_lib.sga_linear(x, w, y, bias=torch.zeros(4))
    with pytest.raises(ValueError):
        sga_lib.sga_linear(x, w, y, residual=y.t())
    with pytest.raises(ValueError):
        sga_lib.sga_linear_grad(y, x, w, torch.zeros(1), grad_x=w)
    with pytest.raises(ValueError):
        sga_lib.sga_linear_grad(y, x, w, torch.zeros(1), preact=x)


def test_binding_refuses_host_tensors(sga_lib):
    b = torch.bfloat16
    x, w, y = torch.zeros(3, 64, dtype=b), torch.zeros(5, 64, dtype=b), torch.zeros(3, 5, dtype=b)
    with pytest.raises(ValueError, match="CUDA"):
        sga_lib.sga_linear(x, w, y)
    with pytest.raises(ValueError, match="CUDA"):
        sga_lib.sga_linear_grad(y, x, w, torch.zeros(40), grad_x=torch.zeros(3, 64, dtype=b))


def test_binding_refuses_tensors_of_another_device(sga_lib, monkeypatch):
    class Tensor:
        is_cuda = True

        def __init__(self, device):
            self.device = device

        def get_device(self):
            return self.device

    monkeypatch.setattr(sga_lib, "_current_device", lambda: 1)
    sga_lib._on_gpu(None, Tensor(1), None, Tensor(1))
    for other in (0, 2):
        with pytest.raises(ValueError, match="current"):
            sga_lib._on_gpu(Tensor(1), None, Tensor(other))


@pytest.mark.gpu
def test_calls_refuse_tensors_of_another_device(sga_lib, monkeypatch):
    """Their kernels run on the current device's stream: nothing is launched."""
    b = torch.bfloat16
    x, w, y = (torch.zeros(s, dtype=b, device="cuda") for s in ((3, 64), (5, 64), (3, 5)))
    f, t = torch.zeros(3, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    parts = torch.zeros(1, 3, 4, device="cuda")
    ws = torch.zeros(64, dtype=torch.uint8, device="cuda")
    monkeypatch.setattr(sga_lib, "_current_device", lambda: 1)
    for call in (lambda: sga_lib.sga_linear(x, w, y),
                 lambda: sga_lib.sga_linear_grad(y, x, w, ws, grad_x=x.clone()),
                 lambda: sga_lib.sga_token_logprobs(y, 5, t, f),
                 lambda: sga_lib.sga_local_logprobs(y, 0, 5, 5, t, parts[0]),
                 lambda: sga_lib.sga_logprob_reduce(parts, None, 1, t, f),
                 lambda: sga_lib.sga_token_logprobs_grad(y, 0, 5, t, f, f, f, y.clone())):
        with pytest.raises(ValueError, match="current"):
            call()
