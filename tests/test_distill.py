"""Distillation from a teacher's top logits, forward and backward, against the
definition in 64 bits (its gradient by automatic differentiation), at the sizes,
masks and alignments where the kernels change path, and the refusals.

Tolerances, by counting roundings: a term 2^t, t = (x - max) log2(e) / T, is off by
5 ln2 2^-24 |t| + 2^-22 of itself; weighted by the terms themselves, |t| is at most
some 40 on average (log2 of the largest vocabulary, and spread), and the sums of
n terms have at most n / 256 + 64 additions along any path: 256 threads or more add
up two halves each (rows of up to 72 KB 128, of up to 48 KB 64 threads: at most n / 128
+ 16 there, which is less up to n = 12288, and from there to the 24576 ids of such a
row at most 48 roundings of 2^-24 more, if all went the same way).  So lse and lse_rest
are within

    tol(n) = (5 ln2 40 + 4 + n / 256 + 64) 2^-24

of the exact ones, plus half a step of what they are rounded to (2^-24 of their
size).  The loss holds lse once with the list's weight (at most 1) and lse_rest -
lse with the rest's; the teacher's own numbers are in 64 bits, with logarithms to
2^-25: 3 tol(n), and its own rounding.  A gradient's parts are s_j and p_r e^(y_j - lse_rest), each off
by the error of its exponent (that of its sum; of t, 5 ln2 2^-24 |t|; of y = x / T,
2^-23 |y|; of the rounded sums, 2^-23 of theirs) and a few products; the output
rounding is half a step.
"""
import ctypes
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

NEG = float("-inf")
FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10002)
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
GUARD = -77.0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def guarded(rows, cols, pad, offset, dtype):
    ld = cols + pad
    buf = torch.full((offset + (rows + 1) * ld + 8,), GUARD, dtype=dtype, device="cuda")
    return buf, buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]


def check_guard(buf, rows, cols, pad, offset):
    seen = torch.ones(buf.numel(), dtype=torch.bool, device="cuda")
    seen[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = False
    assert (buf[seen] == GUARD).all(), "written outside of the rows"


def tol_sum(n):
    return (5 * math.log(2.0) * 40 + 4 + n / 256 + 64) * 2.0 ** -24


# ------------------------------------------------------------ plain, 64 bits


def plain(x, org, ids, z, tlse, temp, g):
    """The definition by torch in 64 bits, row by row: (loss, lse, lse_rest, grad,
    size), `size` the sum of a gradient's parts."""
    rows, width = x.shape
    f64 = dict(dtype=torch.float64, device=x.device)
    loss, lse, rest = (torch.zeros(rows, **f64) for _ in range(3))
    grad, size = torch.zeros((rows, width), **f64), torch.zeros((rows, width), **f64)
    for r in range(rows):
        xr = x[r, :org].double().requires_grad_()
        y = xr / temp
        entry = (ids[r] >= 0) & (ids[r] < org)
        e = ids[r][entry].long()
        zt = z[r][entry].double() / temp
        off = torch.ones(org, dtype=torch.bool, device=x.device)
        off[e] = False
        a, b = torch.logsumexp(y, 0), torch.logsumexp(y[off], 0) if off.any() else y.new_tensor(NEG)
        bad = bool(torch.isnan(y).any() or (y == math.inf).any())
        if bad:
            a = b = y.new_tensor(math.nan)
        lse[r], rest[r] = a.detach(), b.detach()
        if len(e) == 0 or (tlse is None and bool((zt == NEG).all())):
            continue
        logp = zt - (torch.logsumexp(zt, 0) if tlse is None else tlse[r].double())
        p = torch.exp(logp)
        pr = max(0.0, 1.0 - float(p.sum())) if tlse is not None else 0.0
        if float(b.detach()) == NEG:
            pr = 0.0
        if bad:
            loss[r], grad[r, :org] = math.nan, math.nan
            continue
        some = p > 0
        if float(a.detach()) == NEG:
            loss[r] = math.inf if some.any() else 0.0
            continue
        live = some & (y[e].detach() > NEG)
        l = (p[live] * (logp[live] - (y[e[live]] - a))).sum()
        # (a listed logit of -inf: its term's gradient is p (s_j - [j listed]) all the same)
        l = l + (p[some & ~live] * a).sum()
        if pr > 0:
            l = l + pr * (math.log(pr) - (b - a))
        l.backward()
        loss[r] = math.inf if (some & ~live).any() else l.detach()
        up = 1.0 if g is None else float(g[r])
        d = torch.nan_to_num(xr.grad)
        d.scatter_add_(0, e[some & ~live], -p[some & ~live] / temp)
        grad[r, :org] = d * up
        s = torch.exp(y.detach() - a.detach())
        size[r, :org] = s * float(p.sum() + pr)
        if pr > 0:
            size[r, :org] += torch.where(off, pr * torch.exp(y.detach() - b.detach()), 0.0)
        size[r, :org].scatter_add_(0, e, p * 2.0 ** -3)
        size[r] *= abs(up) / temp
    return loss, lse, rest, grad, size


def near(got, exp, tol, what):
    got, tol = got.double(), torch.as_tensor(tol, dtype=torch.float64, device=got.device)
    same = (got == exp) | (torch.isnan(got) & torch.isnan(exp))
    bad = ~(same | ((got - exp).abs() <= tol))
    assert not bad.any(), (what, bad.nonzero()[:4].tolist(), got[bad][:4].tolist(),
                           exp[bad][:4].tolist())


def check_sums(got, exp, n, what):
    near(got, exp, tol_sum(n) + 2.0 ** -24 * torch.nan_to_num(exp, 0, 0, 0).abs(), what)


def grad_tol(x, org, temp, exp, size, lse, dtype):
    y = torch.zeros_like(exp)
    y[:, :org] = torch.nan_to_num(x[:, :org].double() / temp, 0, 0, 0).abs()
    l = torch.nan_to_num(lse, 0, 0, 0).abs()[:, None]
    rel = 2 * tol_sum(org) + (5 * math.log(2.0) + 2) * 2.0 ** -24 * (y + l) + 2.0 ** -23 * l
    return size * rel + exp.nan_to_num(0, 0, 0).abs() * torch.finfo(dtype).eps / 2 + 1e-38


def check_all(x, org, lists, temp, g, got, dtype):
    loss, lse, rest, grad, size = plain(x, org, *lists, temp, g)
    check_sums(got["lse"], lse, org, "lse")
    check_sums(got["rest"], rest, org, "lse_rest")
    near(got["loss"], loss, 3 * tol_sum(org) + 2.0 ** -23 * loss.nan_to_num(0, 0, 0).abs(), "loss")
    if "grad" in got:
        near(got["grad"], grad, grad_tol(x, org, temp, grad, size, lse, dtype), "grad")
        assert (got["grad"][:, org:] == 0).all()


# ------------------------------------------------------------------- inputs


def make(seed, rows, vocab, org, dtype, k, rest, temp, pad, offset):
    g = gen(seed)
    xbuf, x = guarded(rows, vocab, pad, offset, DT[dtype])
    x.normal_(0.0, 3.0, generator=g)
    ids = torch.randint(0, org, (rows, k), generator=g, device="cuda")     # repeats among them
    z = torch.randn((rows, k), generator=g, device="cuda") * 3.0 + 10.0
    at = torch.gather(x, 1, ids)
    x.scatter_(1, ids, (at.float() + 0.6 * z).to(x.dtype))
    lowest = torch.finfo(x.dtype).min
    if rows > 3:
        x[1, ::3] = NEG                       # masked, listed ids among them
        x[2] = NEG                            # nothing left
        x[3, :org // 2] = lowest
    if rows > 6:
        ids[4, k // 2:] = -1
        ids[5] = -1                           # no teacher
        x[5, 0] = math.nan
        x[6, org // 2] = math.nan
    if rows > 10:
        x[7, org - 1] = math.inf
        z[8, 0] = NEG
        x[9] = NEG                            # only listed ids are left
        x[9].scatter_(0, ids[9], z[9].to(x.dtype))
        ids[10, 0] = org                      # padding: no entry
        ids[10, -1] = -5
    if rows > 12:
        ids[11] = ids[11, 0].clone()          # the same id k times
        x[12] += 200.0
    if rows > 14:
        x[14] = -1e4                          # a rest that only a low value masks
        x[14].scatter_(0, ids[14], z[14].to(x.dtype))
    ids = ids.to(torch.int32)
    tlse = None
    if rest:
        tlse = torch.logsumexp(z / temp, 1) + 0.2 * torch.rand(rows, generator=g, device="cuda")
        if rows > 13:
            tlse[13] -= 0.5                   # the list's sum is above 1
    up = torch.randn(rows, generator=g, device="cuda")
    return xbuf, x, (ids, z, tlse), up


CASES = [  # rows, vocab, org, dtype, k, rest, temperature, pad, offset
    (1, 1, 1, "f32", 1, True, 1.0, 0, 0), (1, 2, 2, "bf16", 1, True, 1.0, 0, 1),
    (15, 33, 30, "f32", 3, True, 1.0, 2, 3), (15, 1000, 1000, "bf16", 20, True, 1.0, 0, 0),
    (15, 4099, 4090, "bf16", 32, True, 0.5, 1, 1), (15, 4099, 4099, "f32", 64, False, 2.0, 0, 1),
    (333, 5003, 5000, "bf16", 5, True, 1.0, 0, 0), (15, 50257, 50257, "f32", 128, True, 1.0, 1, 0),
    (2, 152064, 151936, "bf16", 20, True, 1.0, 0, 0),
    (40, 152064, 151936, "bf16", 20, False, 1.5, 8, 0),
    (16, 202048, 202048, "f32", 32, True, 1.0, 0, 0),
    # longer than the shared memory of a cluster
    (15, 900001, 900001, "bf16", 20, True, 1.0, 0, 0), (15, 480003, 480000, "f32", 5, True, 1.0, 1, 1),
    (900, 300, 290, "bf16", 8, True, 1.0, 1, 0),
    # several such rows per cluster, and short rows longer than a small ring
    (60, 900001, 900001, "bf16", 20, True, 1.0, 0, 0), (900, 24001, 24000, "bf16", 20, True, 1.0, 0, 0),
    (900, 12001, 12001, "f32", 40, False, 1.0, 1, 1), (900, 17001, 17000, "bf16", 40, True, 1.0, 0, 0),
    (900, 33001, 33001, "bf16", 20, True, 1.0, 1, 1),
]


def run_forward(sga_lib, x, org, lists, temp, up, with_grad, out_grad=None, stream=None):
    rows = x.size(0)
    ids, z, tlse = lists
    got = {n: torch.full((rows,), GUARD, device="cuda") for n in ("loss", "lse", "rest")}
    sga_lib.sga_distill(x, org, ids, z, got["loss"], teacher_lse=tlse, temperature=temp,
                        out_lse=got["lse"], out_lse_rest=got["rest"],
                        grad_loss=up if with_grad else None, out_grad=out_grad, stream=stream)
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_loss_and_gradient_match_64_bits(sga_lib, case):
    rows, vocab, org, dtype, k, rest, temp, pad, offset = case
    xbuf, x, lists, up = make(rows + vocab, rows, vocab, org, dtype, k, rest, temp, pad, offset)
    before = xbuf.clone()
    alone = run_forward(sga_lib, x, org, lists, temp, up, False)
    check_all(x, org, lists, temp, up, alone, DT[dtype])
    for opad, ooff in ((pad, offset), (3, 1)):
        gbuf, grad = guarded(rows, vocab, opad, ooff, DT[dtype])
        got = run_forward(sga_lib, x, org, lists, temp, up, True, grad)
        got["grad"] = grad
        check_all(x, org, lists, temp, up, got, DT[dtype])
        check_guard(gbuf, rows, vocab, opad, ooff)
        # the separate backward call
        bbuf, back = guarded(rows, vocab, opad, ooff, DT[dtype])
        sga_lib.sga_distill_grad(x, org, lists[0], lists[1], got["lse"], got["rest"], back,
                                 teacher_lse=lists[2], temperature=temp, grad_loss=up)
        check_guard(bbuf, rows, vocab, opad, ooff)
        got["grad"] = back
        check_all(x, org, lists, temp, up, got, DT[dtype])
    assert torch.equal(xbuf.view(torch.int16), before.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,vocab,dtype", [(20, 5000, "bf16"), (20, 50257, "f32"),
                                              (3, 480003, "f32"), (3, 900001, "bf16")])
def test_the_gradient_may_take_the_logits_place(sga_lib, rows, vocab, dtype):
    org, temp = vocab - 2, 1.0
    _, x, lists, up = make(7, rows, vocab, org, dtype, 20, True, temp, 1, 1)
    a, b = x.clone(), x.clone()
    x = x.clone()      # laid out like them: at other alignments sums have another order
    grad = torch.empty_like(x)
    got = run_forward(sga_lib, x, org, lists, temp, up, True, grad)
    here = run_forward(sga_lib, a, org, lists, temp, up, True, a)
    for name in got:
        assert torch.equal(got[name].nan_to_num(9.0), here[name].nan_to_num(9.0)), name
    assert torch.equal(grad.nan_to_num(9.0), a.nan_to_num(9.0))
    sga_lib.sga_distill_grad(x, org, lists[0], lists[1], got["lse"], got["rest"], grad,
                             teacher_lse=lists[2], temperature=temp, grad_loss=up)
    sga_lib.sga_distill_grad(b, org, lists[0], lists[1], got["lse"], got["rest"], b,
                             teacher_lse=lists[2], temperature=temp, grad_loss=up)
    assert torch.equal(grad.nan_to_num(9.0), b.nan_to_num(9.0))


@pytest.mark.gpu
def test_a_rest_of_little_probability(sga_lib):
    """Student and teacher agree on the list but for 1e-7 of the probability: the
    rest's terms keep their relative accuracy, as no difference of sums would."""
    rows, vocab, k = 4, 30000, 4
    x = torch.full((rows, vocab), -16.0, device="cuda")
    x += 0.5 * torch.randn((rows, vocab), generator=gen(4), device="cuda")
    ids = torch.tensor([[5, 800, 20000, 29999]] * rows, dtype=torch.int32, device="cuda")
    x[:, ids[0].long()] = torch.tensor([10.0, 9.0, 8.0, 7.0], device="cuda")
    z = torch.tensor([[10.0, 9.0, 8.0, 7.0]] * rows, device="cuda")
    tlse = torch.logsumexp(z.double(), 1).float() + 2.0 ** -20
    got = run_forward(sga_lib, x, vocab, (ids, z, tlse), 1.0, None, False)
    check_all(x, vocab, (ids, z, tlse), 1.0, None, got, torch.float32)
    share = torch.exp(got["rest"].double() - got["lse"].double())
    off = torch.ones(vocab, dtype=torch.bool, device="cuda")
    off[ids[0].long()] = False
    exact = torch.softmax(x.double(), 1)[:, off].sum(1)
    # both sums' errors and the rounding of two numbers of size up to 11
    assert ((share / exact - 1).abs() <= 2 * tol_sum(vocab) + 2 * 11 * 2.0 ** -24).all()


@pytest.mark.gpu
def test_gradient_against_differences(sga_lib):
    """Central differences of the kernel's own loss with h = 2^-6: their error is
    at most h^2 / 6 of a third derivative (below 1 for log-sum-exps) = 4.1e-5, and
    the losses' rounding, 2 (2^-24 of some 4) / 2h = 1.6e-5; the losses' errors are
    common to both sides but for the terms that move: 2^-21 / 2h = 1.5e-5."""
    vocab, k, temp, h = 40, 6, 1.3, 2.0 ** -6
    g = gen(5)
    x0 = torch.randn((1, vocab), generator=g, device="cuda")
    ids = torch.tensor([[3, 17, 17, 39, -1, 0]], dtype=torch.int32, device="cuda")
    z = torch.randn((1, k), generator=g, device="cuda")
    tlse = torch.logsumexp(z / temp, 1) + 0.4
    grad = torch.empty_like(x0)
    run_forward(sga_lib, x0, vocab, (ids, z, tlse), temp, None, False, grad)
    x = x0.repeat(2 * vocab, 1)
    j = torch.arange(vocab, device="cuda")
    x[2 * j, j] += h
    x[2 * j + 1, j] -= h
    lists = [t.repeat(2 * vocab, *([1] * (t.dim() - 1))) for t in (ids, z, tlse)]
    loss = run_forward(sga_lib, x, vocab, lists, temp, None, False)["loss"].double()
    step = (x[2 * j, j].double() - x[2 * j + 1, j].double())
    diff = (loss[0::2] - loss[1::2]) / step
    assert ((diff - grad[0].double()).abs() <= 8e-5).all(), (diff - grad[0]).abs().max()


@pytest.mark.gpu
def test_a_teachers_list_of_the_library(sga_lib):
    """The target's top log probabilities, as sga_token_logprobs gives them, are a
    teacher with teacher_lse 0; a student equal to it has no loss and no gradient."""
    rows, vocab, k = 9, 20000, 16
    x = torch.empty((rows, vocab), device="cuda").normal_(0.0, 3.0, generator=gen(6))
    ids = torch.empty((rows, k), dtype=torch.int32, device="cuda")
    lp, zero = torch.empty((rows, k), device="cuda"), torch.zeros(rows, device="cuda")
    sga_lib.sga_token_logprobs(x, vocab, None, None, None, None, ids, lp)
    grad = torch.empty_like(x)
    got = run_forward(sga_lib, x, vocab, (ids, lp, zero), 1.0, None, False, grad)
    assert (got["loss"].abs() <= 4 * tol_sum(vocab) + 1e-5).all()   # 1e-5: the listed lp's own error
    assert (grad.abs() <= 4 * tol_sum(vocab) + 2e-5).all()
    got = run_forward(sga_lib, x + torch.randn(x.shape, generator=gen(7), device="cuda"), vocab,
                      (ids, lp, zero), 1.0, None, False)
    assert (got["loss"] > 0.01).all()


@pytest.mark.gpu
def test_every_output_is_optional(sga_lib):
    _, x, lists, up = make(3, 14, 3000, 3000, "bf16", 9, True, 1.0, 0, 0)
    ids, z, tlse = lists
    full = run_forward(sga_lib, x, 3000, lists, 1.0, up, True, torch.empty_like(x))
    for name, key in (("out_loss", "loss"), ("out_lse", "lse"), ("out_lse_rest", "rest")):
        one = torch.full((14,), GUARD, device="cuda")
        sga_lib.sga_distill(x, 3000, ids, z, teacher_lse=tlse, **{name: one})
        assert torch.equal(one.nan_to_num(9.0), full[key].nan_to_num(9.0))
    grad, ref = torch.empty_like(x), torch.empty_like(x)
    sga_lib.sga_distill(x, 3000, ids, z, teacher_lse=tlse, out_grad=grad)     # grad_loss 1
    sga_lib.sga_distill(x, 3000, ids, z, teacher_lse=tlse, out_grad=ref,
                        grad_loss=torch.ones(14, device="cuda"))
    assert torch.equal(grad.nan_to_num(9.0), ref.nan_to_num(9.0))
    sga_lib.sga_distill(x, 3000, ids, z)                                     # nothing asked for
    # a list by itself needs no lse_rest
    sga_lib.sga_distill_grad(x, 3000, ids, z, full["lse"], None, grad)
    sga_lib.sga_distill_grad(x, 3000, ids, z, full["lse"], full["rest"], ref)
    assert torch.equal(grad.nan_to_num(9.0), ref.nan_to_num(9.0))


@pytest.mark.gpu
def test_rows_past_32_bits(sga_lib):
    stride = (1 << 31) // 3 + 5
    buf = torch.empty(3 * stride + 4096, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (4, 4000), (stride, 1))
    x.normal_(0.0, 3.0, generator=gen(8))
    gbuf = torch.empty(3 * stride + 4096, dtype=torch.bfloat16, device="cuda")
    grad = torch.as_strided(gbuf, (4, 4000), (stride, 1))
    ids = torch.randint(0, 4000, (4, 5), generator=gen(9), device="cuda").to(torch.int32)
    z = torch.randn((4, 5), generator=gen(10), device="cuda")
    got = run_forward(sga_lib, x, 4000, (ids, z, None), 1.0, None, False, grad)
    got["grad"] = grad
    check_all(x, 4000, (ids, z, None), 1.0, None, got, torch.bfloat16)
    sga_lib.sga_distill_grad(x, 4000, ids, z, got["lse"], None, grad)
    check_all(x, 4000, (ids, z, None), 1.0, None, got, torch.bfloat16)


@pytest.mark.gpu
def test_own_stream_and_graph_replay(sga_lib):
    rows, vocab, k = 20, 9001, 12
    _, x, lists, up = make(11, rows, vocab, vocab, "bf16", k, True, 1.0, 0, 0)
    ids, z, tlse = lists
    grad, back = torch.empty_like(x), torch.empty_like(x)
    got = {n: torch.empty(rows, device="cuda") for n in ("loss", "lse", "rest")}

    def step():
        sga_lib.sga_distill(x, vocab, ids, z, got["loss"], teacher_lse=tlse, out_lse=got["lse"],
                            out_lse_rest=got["rest"], grad_loss=up, out_grad=grad)
        sga_lib.sga_distill_grad(x, vocab, ids, z, got["lse"], got["rest"], back,
                                 teacher_lse=tlse, grad_loss=up)

    def check():
        for t in (grad, back):
            check_all(x, vocab, lists, 1.0, up, dict(got, grad=t), torch.bfloat16)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for seed in (12, 13):
        _, x2, lists2, up2 = make(seed, rows, vocab, vocab, "bf16", k, True, 1.0, 0, 0)
        for a, b in zip((x, ids, z, tlse, up), (x2, *lists2, up2)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        check()


@pytest.mark.gpu
@pytest.mark.parametrize("temp", [1e-6, 1e-2, 50.0, 1e6])
@pytest.mark.parametrize("rest", [False, True])
def test_temperatures_far_from_one(sga_lib, temp, rest):
    """Logits of the temperature's size, so that the softmax is one of spread 3.
    The row is drawn before it is scaled, in fp32: an exponent of size |y| is then
    off by the roundings that grad_tol counts."""
    rows, vocab, k = 8, 5003, 12
    x = torch.randn((rows, vocab), generator=gen(21), device="cuda") * 3.0
    ids = torch.randint(0, vocab, (rows, k), generator=gen(22), device="cuda").to(torch.int32)
    z = torch.randn((rows, k), generator=gen(23), device="cuda") * 3.0
    x *= temp
    z *= temp
    tlse = torch.logsumexp(z.double() / temp, 1).float() + 0.3 if rest else None
    up = torch.randn(rows, generator=gen(24), device="cuda") * temp
    grad, back = torch.empty_like(x), torch.empty_like(x)
    temp = float(torch.tensor(temp))                 # as the call takes it
    got = run_forward(sga_lib, x, vocab, (ids, z, tlse), temp, up, True, grad)
    got["grad"] = grad
    check_all(x, vocab, (ids, z, tlse), temp, up, got, torch.float32)
    sga_lib.sga_distill_grad(x, vocab, ids, z, got["lse"], got["rest"], back, teacher_lse=tlse,
                             temperature=temp, grad_loss=up)
    got["grad"] = back
    check_all(x, vocab, (ids, z, tlse), temp, up, got, torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_largest_vocabulary(sga_lib, dtype):
    vocab, k = sga_lib.SGA_MAX_VOCAB, 128
    x = torch.empty((2, vocab), dtype=DT[dtype], device="cuda").normal_(0.0, 3.0, generator=gen(31))
    ids = torch.randint(0, vocab, (2, k), generator=gen(32), device="cuda")
    ids[:, 0], ids[:, 1] = vocab - 1, 0
    z = torch.randn((2, k), generator=gen(33), device="cuda") + 8.0
    x.scatter_(1, ids, (z + 4.0).to(x.dtype))
    lists = (ids.to(torch.int32), z, torch.logsumexp(z, 1) + 0.2)
    up = torch.randn(2, generator=gen(34), device="cuda")
    grad, back = torch.empty_like(x), torch.empty_like(x)
    got = run_forward(sga_lib, x, vocab, lists, 1.0, up, True, grad)
    got["grad"] = grad
    check_all(x, vocab, lists, 1.0, up, got, DT[dtype])
    sga_lib.sga_distill_grad(x, vocab, lists[0], z, got["lse"], got["rest"], back,
                             teacher_lse=lists[2], grad_loss=up)
    got["grad"] = back
    check_all(x, vocab, lists, 1.0, up, got, DT[dtype])


@pytest.mark.gpu
@pytest.mark.parametrize("rest", [False, True])
def test_a_draft_head_learns_from_a_targets_list(sga_lib, rest):
    """Target logits -> their best log probabilities -> the draft head's step
    (examples/draft_head.py), against automatic differentiation in 64 bits."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "draft_head.py")
    spec = importlib.util.spec_from_file_location("draft_head_distill", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    rows, hidden, vocab, org, k, g = 150, 256, 1000, 990, 16, gen(51)

    def normal(*shape, sigma):
        return torch.empty(shape, device="cuda").normal_(0.0, sigma, generator=g)

    head = example.DraftHead(normal(hidden, hidden, sigma=hidden ** -0.5).bfloat16(),
                             normal(hidden, sigma=0.3),
                             normal(vocab, hidden, sigma=2 * hidden ** -0.5).bfloat16(), rows,
                             org_vocab=org)
    x, target = normal(rows, hidden, sigma=1.0).bfloat16(), normal(rows, vocab, sigma=3.0)
    ids = torch.empty((rows, k), dtype=torch.int32, device="cuda")
    z = torch.empty((rows, k), device="cuda")
    sga_lib.sga_token_logprobs(target, org, None, None, None, None, ids, z)
    ids[::10] = -1                                # prompt rows: no teacher
    loss, gw, gb = head.distill_and_grads(x, ids, z, torch.zeros(rows, device="cuda")
                                          if rest else None)
    weight = head.weight.double().requires_grad_()
    bias = head.bias.double().requires_grad_()
    h = x.double() @ weight.T + bias
    h = x.double() + h * torch.sigmoid(h)
    y = h @ head.lm_weight.double()[:org].T
    live = (ids >= 0).any(1)
    e = ids.clamp(min=0).long()
    logp = z.double() if rest else torch.log_softmax(z.double(), 1)
    p = logp.exp()
    lse = torch.logsumexp(y, 1)
    exp = (p * (logp - torch.gather(y, 1, e) + lse[:, None])).sum(1)
    if rest:
        pr = 1.0 - p.sum(1)
        off = torch.ones_like(y, dtype=torch.bool).scatter_(1, e, False)
        exp = exp + pr * (pr.log() - torch.logsumexp(y.masked_fill(~off, NEG), 1) + lse)
    exp = torch.where(live, exp, 0.0)
    exp.mean().backward()
    # logits of size up to about 8 went through two roundings to bf16 (2^-8 of 8 each, and
    # 2^-8 of h summed over the LM head): 0.1 covers both
    assert ((loss.double() - exp).abs() <= 0.1).all()
    # h, the logits, their gradient, dh and dz are each rounded to bf16 (about 2e-3 of the
    # value in the 2-norm), the logits' rounding also moves s by up to 2^-8 * 8: below 3 %
    for got, want in ((gw, weight.grad), (gb, bias.grad)):
        rel = (got.double() - want).norm() / want.norm()
        assert rel < 0.03, float(rel)


@pytest.mark.gpu
def test_two_graphs_at_once(sga_lib):
    """Two graphs of the same calls on other data, replayed on two streams at the
    same time: each has its own results every time."""
    work = []
    for seed in (41, 42):
        rows, vocab = 40, 30011
        _, x, lists, up = make(seed, rows, vocab, vocab, "bf16", 40, True, 1.0, 0, 0)
        ids, z, tlse = lists
        out = [torch.empty(rows, device="cuda") for _ in range(3)]
        out += [torch.empty_like(x), torch.empty_like(x)]

        def step(x=x, ids=ids, z=z, tlse=tlse, up=up, out=out):
            sga_lib.sga_distill(x, vocab, ids, z, out[0], teacher_lse=tlse, out_lse=out[1],
                                out_lse_rest=out[2], grad_loss=up, out_grad=out[3])
            sga_lib.sga_distill_grad(x, vocab, ids, z, out[1], out[2], out[4], teacher_lse=tlse,
                                     grad_loss=up)

        step()
        torch.cuda.synchronize()
        want = [t.nan_to_num(9.0) for t in out]
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=stream):
            for _ in range(20):
                step()
        for t in out:
            t.fill_(GUARD)
        work.append((graph, stream, want, out, step))      # (step holds the inputs)
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, stream, *_ in work:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for _, _, want, out, _ in work:
            assert all(torch.equal(a, b.nan_to_num(9.0)) for a, b in zip(want, out))


# --------------------------------- sums that an fp32 log-sum-exp does not hold


def shifted_exp(y):
    """Softmax of each row and log2 of its terms relative to the largest one (rows
    without a finite logit: 0)."""
    top = y.max(1, keepdim=True).values
    t = torch.where(y > NEG, y - top, NEG)
    e = torch.exp(t)
    return e / e.sum(1, keepdim=True).clamp(min=1.0), torch.nan_to_num(t, 0, 0, 0) / math.log(2.0)


def formula(x, org, ids, z, tlse, temp, up):
    """(gradient, tolerance) in 64 bits by the closed form, each softmax relative to
    its own largest logit, so that no log-sum-exp has to hold a small sum beside a
    large offset.

    Tolerance: s_j and the rest's share of itself are terms 2^t over a sum.  A term is
    off by 5 ln2 2^-24 (|t| + 24) + 2^-22 of itself (its exponent counts from a logit at
    most 12 below the largest, the rest's from there to the row's another 12), where it
    is not below 2^-126 altogether; a sum, and the factors of it, by 2 tol_sum.  Where the
    saved sums are used, |lse| and |lse_rest| are at most 512 and each rounded once, and the
    difference and product with them again: 2^-22 512.  An entry's p is rounded to fp32, and
    its s_j is a term; the output's rounding is half a step."""
    y = x[:, :org].double() / temp
    rows, k = ids.shape
    entry = (ids >= 0) & (ids < org)
    at = torch.where(entry, ids, 0).long()
    zt = torch.where(entry, z.double() / temp, NEG)
    logp = zt - (torch.logsumexp(zt, 1, keepdim=True) if tlse is None else tlse.double()[:, None])
    p = torch.where(entry, torch.exp(logp), 0.0)
    on = torch.zeros_like(y).scatter_add_(1, at, p)
    off = torch.zeros_like(y).scatter_add_(1, at, entry.double()) == 0
    yr = torch.where(off, y, NEG)
    pr = (1.0 - p.sum(1)).clamp(min=0.0) if tlse is not None else torch.zeros_like(p[:, 0])
    pr = torch.where((yr > NEG).any(1) & entry.any(1), pr, 0.0)[:, None]
    total = p.sum(1, keepdim=True) + pr
    live = ((y > NEG).any(1) & entry.any(1)).double()[:, None]
    (s, t), (r, tr) = shifted_exp(y), shifted_exp(yr)
    scale = up.double()[:, None] / temp * live
    grad = scale * (total * s - on - pr * r)
    rel = 2 * tol_sum(org) + 2.0 ** -22 + 2.0 ** -22 * 512
    ln = 5 * math.log(2.0) * 2.0 ** -24
    tol = total * s * (rel + ln * (24 - t.clamp(min=-150))) + on * 2.0 ** -22
    tol = scale.abs() * (tol + pr * r * (rel + ln * (24 - tr.clamp(min=-150))) + 1e-37)
    return grad, tol + grad.abs() * torch.finfo(x.dtype).eps / 2 + 1e-38


def both_gradients(sga_lib, x, org, lists, temp, up, pad, offset):
    """The gradient of the loss's own pass, and that of the separate call from the sums
    that the pass gave, each checked for what lies around it."""
    rows, vocab = x.shape
    ids, z, tlse = lists
    gbuf, grad = guarded(rows, vocab, pad, offset, x.dtype)
    got = run_forward(sga_lib, x, org, lists, temp, up, True, grad)
    bbuf, back = guarded(rows, vocab, pad, offset, x.dtype)
    sga_lib.sga_distill_grad(x, org, ids, z, got["lse"], got["rest"], back, teacher_lse=tlse,
                             temperature=temp, grad_loss=up)
    for buf in (gbuf, bbuf):
        check_guard(buf, rows, vocab, pad, offset)
    return grad, back, got


@pytest.mark.gpu
@pytest.mark.parametrize("rows,vocab,dtype,k,pad,offset", [
    (14, 4001, "f32", 5, 1, 3), (14, 3000, "bf16", 40, 0, 0), (700, 1001, "bf16", 20, 1, 1),
    (700, 900, "f32", 70, 0, 0), (5, 200003, "bf16", 20, 0, 0), (5, 200003, "f32", 20, 1, 1),
    (470, 30011, "bf16", 12, 1, 3)], ids=str)
@pytest.mark.parametrize("temp", [0.5, 1.0, 1.5])
def test_rests_that_only_low_values_mask(sga_lib, rows, vocab, dtype, k, pad, offset, temp):
    """The rest's logits are all the same low value, or far below the listed ones: its
    log-sum-exp in fp32 holds nothing of how many there are (and overflows, for the
    lowest value of the type below T = 1)."""
    org, g = vocab - 1, gen(rows + vocab)
    _, x = guarded(rows, vocab, pad, offset, DT[dtype])
    x.normal_(0.0, 3.0, generator=g)
    ids = torch.randint(0, org, (rows, k), generator=g, device="cuda")
    z = torch.randn((rows, k), generator=g, device="cuda") * 2.0
    lowest = torch.finfo(x.dtype).min
    kinds = [None, -1e9, lowest, -700.0, -400.0, -1e4, lowest / 2, NEG, "spread", "all", None, "up"]
    for r in range(rows):
        kind = kinds[r % len(kinds)]
        own = x[r, ids[r]].clone()
        if kind == "spread":
            x[r] -= 2000.0
        elif kind == "all":                      # listed logits too: lse is lost as well
            x[r], own = lowest, torch.full_like(own, lowest)
        elif kind == "up":                       # lse lost by logits far above 0
            x[r] += 3000.0
            own = own + 3000.0
        elif kind is not None:
            x[r] = kind
        x[r, ids[r]] = own
    ids = ids.to(torch.int32)
    tlse = torch.logsumexp(z / temp, 1) + 0.3 * torch.rand(rows, generator=g, device="cuda")
    up = torch.randn(rows, generator=g, device="cuda")
    for t in (tlse, None):
        grad, back, _ = both_gradients(sga_lib, x, org, (ids, z, t), temp, up, pad, offset)
        exp, tol = formula(x, org, ids, z, t, temp, up)
        for name, got in (("grad", grad), ("back", back)):
            near(got[:, :org], exp, tol, name)
            assert (got[:, org:] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("temp", [1e-6, 1e-5, 1e-3, 0.02])
@pytest.mark.parametrize("rows,vocab", [(30, 5003), (700, 1001), (3, 150001)])
@pytest.mark.parametrize("rest", [False, True])
def test_low_temperatures_of_ordinary_logits(sga_lib, temp, rows, vocab, rest):
    """Logits of 20 to 60 that differ by some T: |lse| is up to 6e7."""
    g, k = gen(17), 12
    x = torch.randn((rows, vocab), generator=g, device="cuda") * (3.0 * temp)
    x += 20.0 + 40.0 * torch.rand((rows, 1), generator=g, device="cuda")
    ids = torch.randint(0, vocab, (rows, k), generator=g, device="cuda").to(torch.int32)
    z = torch.randn((rows, k), generator=g, device="cuda") * temp
    temp = float(torch.tensor(temp))
    tlse = (torch.logsumexp(z.double() / temp, 1) + 0.3).float() if rest else None
    up = torch.randn(rows, generator=g, device="cuda") * temp
    grad, back, _ = both_gradients(sga_lib, x, vocab, (ids, z, tlse), temp, up, 0, 0)
    exp, tol = formula(x, vocab, ids, z, tlse, temp, up)
    near(grad, exp, tol, "grad")
    near(back, exp, tol, "back")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sums_that_overflow(sga_lib, dtype):
    """Below T = 1 a finite logit's y can pass the largest fp32 number, either way."""
    rows, vocab, k, temp, g = 8, 2001, 6, 0.5, gen(19)
    x = torch.randn((rows, vocab), generator=g, device="cuda").to(DT[dtype])
    big = torch.finfo(x.dtype).max
    ids = torch.randint(0, vocab, (rows, k), generator=g, device="cuda")
    x[0, 7], x[0, 1900] = big, big           # two ids have all the probability
    x[1] = -big                              # all have the same
    x[2] = NEG
    x[3] = -big
    x[3, ids[3]] = NEG                       # the listed ones have none
    x[4] = NEG
    x[4, ids[4]] = -big                      # the listed ones have all of it
    x[5, 3] = math.nan
    x[6, 3] = math.inf
    ids = ids.to(torch.int32)
    z = torch.randn((rows, k), generator=g, device="cuda")
    tlse = torch.logsumexp(z / temp, 1) + 0.2
    up = torch.randn(rows, generator=g, device="cuda")
    for t in (tlse, None):
        grad, back, _ = both_gradients(sga_lib, x, vocab, (ids, z, t), temp, up, 3, 1)
        exp, tol = formula(x, vocab, ids, z, t, temp, up)
        exp[5:7] = math.nan
        near(grad, exp, tol.nan_to_num(0), "grad")
        near(back, exp, tol.nan_to_num(0), "back")


@pytest.mark.gpu
@pytest.mark.parametrize("rows,vocab,dtype", [(40, 3001, "bf16"), (6, 150001, "f32"),
                                              (500, 5000, "bf16")])
def test_lost_sums_in_the_logits_place(sga_lib, rows, vocab, dtype):
    """Every other row is masked by a low value; the gradient is written over the logits."""
    temp, g = 1.5, gen(23)
    _, x = guarded(rows, vocab, 1, 3, DT[dtype])
    x.normal_(0.0, 3.0, generator=g)
    ids = torch.randint(0, vocab, (rows, 9), generator=g, device="cuda")
    own = torch.gather(x, 1, ids)
    x[::2] = -1e9
    x.scatter_(1, ids, own)
    ids = ids.to(torch.int32)
    z = torch.randn((rows, 9), generator=g, device="cuda")
    tlse = torch.logsumexp(z / temp, 1) + 0.2
    up = torch.randn(rows, generator=g, device="cuda")
    exp, tol = formula(x, vocab, ids, z, tlse, temp, up)
    _, back, got = both_gradients(sga_lib, x, vocab, (ids, z, tlse), temp, up, 1, 3)
    sga_lib.sga_distill_grad(x, vocab, ids, z, got["lse"], got["rest"], x, teacher_lse=tlse,
                             temperature=temp, grad_loss=up)
    near(x, exp, tol, "in place")
    assert torch.equal(x, back)


@pytest.mark.gpu
def test_lost_sums_of_the_largest_vocabulary(sga_lib):
    vocab, temp, g = sga_lib.SGA_MAX_VOCAB, 1.5, gen(29)
    x = torch.full((2, vocab), -1e9, device="cuda")
    x[1].normal_(-4000.0, 3.0, generator=g)
    ids = torch.randint(0, vocab, (2, 100), generator=g, device="cuda")
    ids[:, 0], ids[:, 1] = vocab - 1, 0
    z = torch.randn((2, 100), generator=g, device="cuda")
    x.scatter_(1, ids, z)
    lists = (ids.to(torch.int32), z, torch.logsumexp(z / temp, 1) + 0.2)
    up = torch.randn(2, generator=g, device="cuda")
    grad, back, _ = both_gradients(sga_lib, x, vocab, lists, temp, up, 0, 0)
    exp, tol = formula(x, vocab, *lists, temp, up)
    near(grad, exp, tol, "grad")
    near(back, exp, tol, "back")


@pytest.mark.gpu
def test_a_graph_of_rows_with_and_without_lost_sums(sga_lib):
    """Which rows are summed anew is found at each replay."""
    rows, vocab, k, temp, g = 600, 9001, 10, 1.5, gen(37)
    x = torch.zeros((rows, vocab), dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros((rows, k), dtype=torch.int32, device="cuda")
    z, up = torch.zeros((rows, k), device="cuda"), torch.zeros(rows, device="cuda")
    tlse = torch.zeros(rows, device="cuda")
    loss, lse, rest = (torch.zeros(rows, device="cuda") for _ in range(3))
    back = torch.empty_like(x)

    def step():
        sga_lib.sga_distill(x, vocab, ids, z, loss, teacher_lse=tlse, temperature=temp,
                            out_lse=lse, out_lse_rest=rest)
        sga_lib.sga_distill_grad(x, vocab, ids, z, lse, rest, back, teacher_lse=tlse,
                                 temperature=temp, grad_loss=up)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for share in (0.0, 0.5, 1.0, 0.1):
        x.normal_(0.0, 3.0, generator=g)
        at = torch.randint(0, vocab, (rows, k), generator=g, device="cuda")
        own = torch.gather(x, 1, at)
        x[torch.rand(rows, generator=g, device="cuda") < share] = -1e9
        x.scatter_(1, at, own)
        ids.copy_(at)
        z.normal_(generator=g)
        tlse.copy_(torch.logsumexp(z / temp, 1) + 0.2)
        up.normal_(generator=g)
        graph.replay()
        exp, tol = formula(x, vocab, ids, z, tlse, temp, up)
        near(back, exp, tol, share)


# ------------------------------------------------------------------ refusals


@pytest.mark.parametrize("grad_call", [False, True])
def test_validation(sga_lib, grad_call):
    f = sga_lib.lib().sga_distill_grad if grad_call else sga_lib.lib().sga_distill
    ok = dict(logits=FAKE, dtype=1, rows=4, ld=10, vocab=10, org=10, ids=FAKE, z=FAKE, k=3,
              tlse=FAKE, t=1.0, a=FAKE, b=FAKE, c=FAKE, up=FAKE, grad=FAKE, ldg=10)

    def call(**kw):
        v = dict(ok, **kw)
        mid = [v["a"], v["b"]] + ([] if grad_call else [v["c"]])
        return f(v["logits"], v["dtype"], v["rows"], v["ld"], v["vocab"], v["org"], v["ids"],
                 v["z"], v["k"], v["tlse"], v["t"], *mid, v["up"], v["grad"], v["ldg"], None)

    assert call(dtype=3) == -5
    assert call(rows=-1) == -2 and call(rows=(1 << 28) + 1) == -2
    assert call(k=0) == -2 and call(k=129) == -2
    for t in (0.0, -1.0, math.nan, math.inf, 1e-7, 1e7):
        assert call(t=t) == -2, t
    assert call(vocab=0) == -3 and call(ld=9) == -3 and call(ldg=9) == -3
    assert call(org=0) == -4 and call(vocab=(1 << 24) + 1, ld=1 << 25, ldg=1 << 25) == -4
    for name in ("logits", "ids", "z"):
        assert call(**{name: None}) == -1, name
    for name in ("ids", "z", "tlse", "a", "b", "up") + (() if grad_call else ("c",)):
        assert call(**{name: ODD}) == -6, name
    assert call(dtype=0, logits=ODD) == -6 and call(dtype=0, grad=ODD) == -6
    assert call(rows=0, logits=None) == 0
    if grad_call:
        assert call(a=None) == -1 and call(grad=None) == -1 and call(b=None) == -1
    else:
        assert call(a=None, b=None, c=None, grad=None) == 0      # nothing asked for


def test_binding_says_what_is_wrong(sga_lib):
    """The specific refusal comes before that of host memory."""
    i32 = torch.int32
    ok = dict(logits=torch.zeros(2, 8), org_vocab=8, teacher_ids=torch.zeros(2, 3, dtype=i32),
              teacher_logits=torch.zeros(2, 3))
    for wrong, word in ((dict(teacher_ids=torch.zeros(2, 3, dtype=torch.int64)), "teacher_ids"),
                        (dict(teacher_ids=torch.tensor(1, dtype=i32)), "teacher_ids"),
                        (dict(teacher_logits=torch.zeros(2, 4)), "teacher_logits"),
                        (dict(teacher_lse=torch.zeros(3)), "teacher_lse"),
                        (dict(out_loss=torch.zeros(4)[::2]), "out_loss"),
                        (dict(out_grad=torch.zeros(8, 2).t()), "out_grad"), (dict(), "CUDA")):
        with pytest.raises(ValueError, match=word):
            sga_lib.sga_distill(**dict(ok, **wrong))


@pytest.mark.gpu
def test_binding_refuses_host_tensors_among_others(sga_lib):
    i32 = torch.int32

    def t(*shape, dtype=torch.float32):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    ok = dict(logits=t(2, 8), org_vocab=8, teacher_ids=t(2, 3, dtype=i32), teacher_logits=t(2, 3),
              teacher_lse=t(2), out_loss=t(2), out_grad=t(2, 8))
    sga_lib.sga_distill(**ok)
    for name in ("logits", "teacher_ids", "teacher_logits", "teacher_lse", "out_loss", "out_grad"):
        with pytest.raises(ValueError):
            sga_lib.sga_distill(**dict(ok, **{name: ok[name].cpu()}))


def test_binding_refuses_wrong_tensors(sga_lib):
    def t(*shape, dtype=torch.float32):
        return torch.zeros(shape, dtype=dtype)

    i32 = torch.int32
    ok = dict(logits=t(2, 8), org_vocab=8, teacher_ids=t(2, 3, dtype=i32), teacher_logits=t(2, 3))
    for wrong in (dict(logits=t(8)), dict(teacher_ids=t(2, 3, dtype=torch.int64)),
                  dict(teacher_ids=t(3, 3, dtype=i32)), dict(teacher_logits=t(2, 4)),
                  dict(teacher_lse=t(3)), dict(out_loss=t(3)), dict(out_lse=t(2, dtype=i32)),
                  dict(out_grad=t(2, 9)), dict(out_grad=t(2, 8, dtype=torch.bfloat16)),
                  dict(out_grad=t(8, 2).t()), dict(grad_loss=t(1)), dict()):
        with pytest.raises(ValueError):
            sga_lib.sga_distill(**dict(ok, **wrong))
    ok.update(lse=t(2), lse_rest=t(2), out_grad=t(2, 8))
    for wrong in (dict(lse=t(3)), dict(lse_rest=t(1)), dict(out_grad=t(3, 8)), dict()):
        with pytest.raises(ValueError):
            sga_lib.sga_distill_grad(**dict(ok, **wrong))


@pytest.mark.parametrize("grad_call", [False, True])
def test_lists_in_another_order_are_refused(sga_lib, grad_call):
    """A contiguous [k, rows] tensor has a list's size, but not its order; lists of rows
    in more dimensions, and flat ones, have it (and come as far as the device's check)."""
    i32 = torch.int32
    ok = dict(logits=torch.zeros(6, 8), org_vocab=8, teacher_ids=torch.zeros(6, 3, dtype=i32),
              teacher_logits=torch.zeros(6, 3))
    if grad_call:
        ok.update(lse=torch.zeros(6), lse_rest=torch.zeros(6), out_grad=torch.zeros(6, 8))
    call = sga_lib.sga_distill_grad if grad_call else sga_lib.sga_distill
    for wrong, word in ((dict(teacher_logits=torch.zeros(3, 6)), "teacher_logits"),
                        (dict(teacher_ids=torch.zeros(3, 6, dtype=i32)), "teacher_ids"),
                        (dict(teacher_logits=torch.zeros(3, 3, 2)), "teacher_logits"),
                        (dict(teacher_logits=torch.zeros(18)), "CUDA"),
                        (dict(teacher_ids=torch.zeros(2, 3, 3, dtype=i32),
                              teacher_logits=torch.zeros(2, 3, 3)), "CUDA")):
        with pytest.raises(ValueError, match=word):
            call(**dict(ok, **wrong))
