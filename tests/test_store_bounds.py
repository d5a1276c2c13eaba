"""Every call of the draft-head and log-probability operators writes its results
and nothing beside them: outputs are views into flat buffers, at assorted offsets
and row strides, whose elements before, between and after the rows have to keep
their bits, while the results are those of packed outputs, bit for bit."""
import pytest
import torch

import workloads as wl

FILL = {torch.bfloat16: -77.0, torch.float32: -77.0, torch.int32: -77}
PLACES = [(0, 0), (1, 1), (3, 2), (7, 5), (8, 3), (2, 6), (5, 7), (8, 8)]   # row padding, offset
FRONT = 128


class Framed:
    """A rows x cols view `offset` elements (and a guard) into a flat buffer."""

    def __init__(self, rows, cols, pad, offset, dtype):
        ld = cols + pad
        self.flat = torch.full((2 * FRONT + offset + rows * ld,), FILL[dtype], dtype=dtype,
                               device="cuda")
        self.at = ((rows, cols), (ld, 1), FRONT + offset)
        self.view = torch.as_strided(self.flat, *self.at)

    def check(self, packed, what):
        assert torch.equal(self.view, packed), what
        seen = self.flat.clone()
        torch.as_strided(seen, *self.at).fill_(FILL[seen.dtype])
        assert (seen == FILL[seen.dtype]).all(), what


def mat(seed, rows, cols, sigma=1.0, dtype=torch.bfloat16):
    return torch.from_numpy(wl.normal_matrix(seed, rows, cols, sigma, dtype="f32")).to(dtype).cuda()


# single tokens; few rows in 2, 4, 1 and 4 parts; CTA pairs at each tile width
FORWARD = [(1, 77, 72), (3, 130, 264), (5, 203, 64), (40, 130, 200), (20, 20001, 64),
           (100, 301, 2056), (300, 100, 64), (333, 192, 64), (1000, 1531, 200), (3000, 901, 136)]


@pytest.mark.gpu
@pytest.mark.parametrize("place", PLACES, ids=str)
@pytest.mark.parametrize("shape", FORWARD, ids=str)
def test_linear_writes_its_rows_only(sga_lib, shape, place):
    M, N, K = shape
    x, w, r = mat(1, M, K), mat(2, N, K, K ** -0.5), mat(3, M, N)
    act = sga_lib.SGA_ACT_SILU
    packed = [torch.empty_like(r), torch.empty_like(r)]
    sga_lib.sga_linear(x, w, packed[0], None, act, r, packed[1])
    pad, offset = place
    out = Framed(M, N, pad, offset, torch.bfloat16)
    pre = Framed(M, N, offset, pad, torch.bfloat16)
    sga_lib.sga_linear(x, w, out.view, None, act, r, pre.view)
    out.check(packed[0], "out")
    pre.check(packed[1], "out_preact")
    out = Framed(M, N, pad, offset, torch.bfloat16)      # the residual in place
    out.view.copy_(r)
    sga_lib.sga_linear(x, w, out.view, None, act, out.view)
    out.check(packed[0], "in place")


# both products in one launch at either tile width; grad_x as few rows (the last two)
GRADIENT = [(1, 33, 72), (40, 130, 200), (130, 200, 264), (777, 301, 136), (1030, 1100, 2056),
            (5, 9001, 520), (134, 5804, 936)]


@pytest.mark.gpu
@pytest.mark.parametrize("place", PLACES, ids=str)
@pytest.mark.parametrize("shape", GRADIENT, ids=str)
def test_linear_grad_writes_its_rows_only(sga_lib, shape, place):
    M, N, K = shape
    pad, offset = place
    act = sga_lib.SGA_ACT_GELU_TANH if offset % 2 else sga_lib.SGA_ACT_NONE
    x, w, g, z = mat(1, M, K), mat(2, N, K, K ** -0.5), mat(3, M, N), mat(4, M, N)
    z = z if act else None
    size = sga_lib.sga_linear_grad_workspace(M, N, K)
    ws = torch.empty(size + 64, dtype=torch.uint8, device="cuda").fill_(119)
    bias = torch.float32 if pad % 2 else torch.bfloat16
    packed = [torch.empty_like(x), torch.empty_like(w), torch.empty(1, N, dtype=bias, device="cuda")]
    sga_lib.sga_linear_grad(g, x, w, ws[:size], act, z, packed[0], packed[1], packed[2][0])
    gx = Framed(M, K, pad, offset, torch.bfloat16)
    gw = Framed(N, K, offset, pad, torch.bfloat16)
    gb = Framed(1, N, 0, offset, bias)
    sga_lib.sga_linear_grad(g, x, w, ws[:size], act, z, gx.view, gw.view, gb.view[0])
    gx.check(packed[0], "grad_x")
    gw.check(packed[1], "grad_weight")
    gb.check(packed[2], "grad_bias")
    assert (ws[size:] == 119).all()


# a cluster per row, persistent wide CTAs, small CTAs
LOGPROBS = [(1, 70001, 20), (3, 50, 32), (30, 9001, 5), (500, 700, 3)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", LOGPROBS, ids=str)
def test_logprobs_write_their_rows_only(sga_lib, shape, dtype):
    rows, vocab, k = shape
    x = mat(5, rows, vocab, 3.0, dtype)
    tok = (torch.arange(rows, device="cuda") % vocab).to(torch.int32)
    f32, i32 = torch.float32, torch.int32

    def outputs():
        return [Framed(1, rows, 0, 1, f32) for _ in range(3)] + [Framed(1, rows * k, 0, 3, i32),
                                                                 Framed(1, rows * k, 0, 1, f32)]

    def tensors(out):
        return [o.view[0] for o in out[:3]] + [o.view.view(rows, k) for o in out[3:]]

    packed = [torch.empty(rows, device="cuda") for _ in range(3)]
    packed += [torch.empty((rows, k), dtype=i32, device="cuda"), torch.empty((rows, k), device="cuda")]
    sga_lib.sga_token_logprobs(x, vocab, tok, *packed)
    out = outputs()
    sga_lib.sga_token_logprobs(x, vocab, tok, *tensors(out))
    for o, p in zip(out, packed):
        o.check(p.view(1, -1), "whole vocabulary")
    # two shards and their reduce
    cut = vocab // 2 + 1
    parts, tops = Framed(1, 2 * rows * 4, 0, 1, f32), Framed(1, 2 * rows * k * 2, 0, 2, i32)
    pv, tv = parts.view.view(2, rows, 4), tops.view.view(2, rows, k, 2)
    for i, (a, b) in enumerate(((0, cut), (cut, vocab))):
        sga_lib.sga_local_logprobs(x[:, a:b], a, b - a, vocab, tok, pv[i], tv[i])
    parts.check(parts.view.clone(), "parts")
    tops.check(tops.view.clone(), "lists")
    packed[:3] = [torch.empty(rows, device="cuda") for _ in range(3)]
    packed[4] = torch.empty((rows, k), device="cuda")
    ids = packed[3].clone()
    sga_lib.sga_logprob_reduce(pv, tv, 2, tok, *packed)
    out = outputs()
    sga_lib.sga_logprob_reduce(pv, tv, 2, tok, *tensors(out))
    for o, p in zip(out, packed):
        o.check(p.view(1, -1), "reduced")
    assert torch.equal(ids, packed[3])


# one vector and less, odd sizes, padding ids, several pieces of a row
LOGPROBS_GRAD = [(2, 1, 1), (3, 5, 5), (9, 64, 8), (30, 257, 250), (30, 1001, 1001),
                 (5, 33000, 32999), (3, 70003, 70000)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("place", PLACES, ids=str)
@pytest.mark.parametrize("shape", LOGPROBS_GRAD, ids=str)
def test_logprobs_grad_writes_its_rows_only(sga_lib, shape, place, dtype):
    rows, vocab, org = shape
    pad, offset = place
    x = mat(6, rows, vocab, 3.0, dtype)
    tok = (torch.arange(rows, device="cuda") % org).to(torch.int32)
    lse, ent = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    sga_lib.sga_token_logprobs(x, org, tok, None, ent, lse)
    up = torch.ones(rows, device="cuda")
    packed = torch.empty_like(x)
    sga_lib.sga_token_logprobs_grad(x, 0, org, tok, lse, ent, up, packed, grad_entropy=up)
    for logits in ((pad, offset), (0, 0), (offset, 1)):      # the logits' own places
        src = Framed(rows, vocab, *logits, dtype)
        src.view.copy_(x)
        out = Framed(rows, vocab, pad, offset, dtype)
        sga_lib.sga_token_logprobs_grad(src.view, 0, org, tok, lse, ent, up, out.view,
                                        grad_entropy=up)
        out.check(packed, "gradient")
    src = Framed(rows, vocab, pad, offset, dtype)            # in place
    src.view.copy_(x)
    sga_lib.sga_token_logprobs_grad(src.view, 0, org, tok, lse, ent, up, src.view, grad_entropy=up)
    src.check(packed, "in place")
