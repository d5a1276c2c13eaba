"""Token log probabilities, entropy, alternatives and their gradient against a
plain implementation in 64 bits, at the sizes, masks and alignments where the
kernels change path, and the entry points' refusals.

Tolerances, derived from the arithmetic: the row's sum of 2^t has at most a few
dozen roundings along any path and each term an error of a few ulp plus
|t| 2^-24, so the log-sum-exp is within 1e-5 absolute of the exact one plus the
fp32 rounding of the operands (2^-22 of their size); the entropy is a
difference of two such quantities of size at most log(vocab) each.  A gradient
term p (A + B (log p + H)) has a relative error of (|log p| + 16) 2^-22 on the
sum of its parts' sizes, and bf16 results one more rounding (2^-8 of the
value).
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import workloads as wl

NEG = float("-inf")
FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10001)
LOWEST = {"bf16": float(torch.finfo(torch.bfloat16).min), "f32": float(np.finfo(np.float32).min)}


# ------------------------------------------------------------ plain, 64 bits


def order_desc(x):
    """Ids of a row in the argmax order: NaN first, then descending, ties by id."""
    return np.array(sorted(range(len(x)), key=lambda j: (
        0 if math.isnan(x[j]) else 1, 0.0 if math.isnan(x[j]) else -x[j], j)), np.int64)


def plain_row(x, token, k):
    """x: float64 logits of the non-padding ids.  (logprob, entropy, lse, ids, logprobs)."""
    n = len(x)
    ids = order_desc(x)[:k]
    full = np.full(k, -1, np.int64)
    full[:len(ids)] = ids
    bad = np.isnan(x).any() or np.isposinf(x).any()
    m = x.max() if n else NEG
    if bad:
        lse = ent = math.nan
    elif m == NEG:
        lse, ent = NEG, 0.0
    else:
        e = np.exp(x - m)
        s = e.sum()
        lse = m + math.log(s)
        d = np.where(e > 0, x - m, 0.0)
        ent = math.log(s) - (e * d).sum() / s

    def lp(v):
        if bad:
            return math.nan
        return NEG if v == NEG else v - lse

    at = 0.0 if token < 0 else lp(x[token] if token < n else NEG)
    tops = np.array([lp(x[j] if j >= 0 else NEG) for j in full])
    return at, ent, lse, full, tops


def plain_grad_row(x, width, token, lse, ent, gl, ge, ids, gt):
    out, scale = np.zeros(width), np.zeros(width)
    if lse == NEG:
        return out, scale
    n = len(x)
    gl = 0.0 if token < 0 else gl
    a = -(gl + sum(g for j, g in zip(ids, gt) if j >= 0))
    live = x > NEG
    lp = np.where(live, x - lse, 0.0)
    p = np.where(live, np.exp(lp), 0.0)
    out[:n] = p * (a - ge * (lp + ent))
    scale[:n] = p * (abs(a) + abs(ge) * (np.abs(lp) + abs(ent))) * (np.abs(lp) + 16) * 2.0 ** -22
    for j, g in [(token, gl)] + list(zip(ids, gt)):
        if 0 <= j < n:
            out[j] += g
            scale[j] += abs(g) * 2.0 ** -22
    return out, scale


# ------------------------------------------------------------------- inputs


def make_logits(seed, rows, vocab, dtype, pad, offset, sigma=3.0):
    """(float64 view, CUDA tensor): rows of a buffer `pad` wider, `offset`
    elements into it, so rows start at assorted 16-byte misalignments."""
    flat = wl.normal_matrix(seed, 1, rows * (vocab + pad) + offset, sigma, dtype="f32")[0]
    x = flat[offset:].reshape(rows, vocab + pad).copy()
    return x, dtype


def to_cuda(x, dtype, vocab, offset):
    t = torch.from_numpy(np.ascontiguousarray(x))
    t = t.to(torch.bfloat16) if dtype == "bf16" else t
    buf = torch.zeros(t.numel() + offset, dtype=t.dtype, device="cuda")
    buf[offset:].copy_(t.reshape(-1))
    dev = buf[offset:].view(t.shape)[:, :vocab]
    return dev, dev.double().cpu().numpy()


def plant(x, dtype):
    """Special rows, as many as the matrix has room for."""
    rows, vocab = x.shape
    special = [
        lambda r: r.fill(NEG),                                   # nothing left
        lambda r: r.__setitem__(slice(0, vocab - 1), NEG),       # one id left
        lambda r: r.fill(LOWEST[dtype]),                         # all at the lowest value
        lambda r: r.__setitem__(slice(0, vocab, 2), LOWEST[dtype]),
        lambda r: r.fill(0.25),                                  # all tied
        lambda r: r.__setitem__(vocab // 2, math.nan),
        lambda r: r.__setitem__(vocab // 3, math.inf),
        lambda r: r.__iadd__(1000.0),
        lambda r: r.__isub__(30000.0),
        lambda r: r.__imul__(1e30),
        lambda r: r.__setitem__(0, 3e38),
        lambda r: r.__setitem__(vocab - 1, 80.0),                # one id takes everything
        lambda r: r.__setitem__(slice(vocab // 4, None), NEG),
        lambda r: np.round(r, out=r),                            # many ties
    ]
    for i, f in enumerate(special):
        if 2 * i + 1 < rows:
            f(x[2 * i + 1])
    return x


CASES = [  # rows, vocab, org, dtype, k, pad, offset
    (1, 1, 1, "f32", 1, 0, 0), (3, 1, 1, "bf16", 4, 0, 1), (2, 7, 5, "f32", 7, 0, 0),
    (30, 40, 40, "f32", 32, 1, 3), (30, 257, 250, "bf16", 20, 3, 5),
    (30, 1000, 1000, "bf16", 5, 0, 0), (30, 1001, 990, "f32", 20, 0, 0),
    (30, 4099, 4099, "bf16", 32, 0, 7), (4, 20000, 19990, "bf16", 20, 8, 0),
    (2, 50257, 50257, "f32", 1, 0, 0), (1, 152064, 151936, "bf16", 20, 0, 0),
    (700, 600, 600, "bf16", 0, 0, 0), (30, 8192, 8192, "f32", 3, 0, 1),
    (300, 3001, 3000, "bf16", 20, 0, 3), (300, 2000, 1999, "f32", 32, 1, 0),
]


def close(got, exp, tol):
    got, exp = np.asarray(got, np.float64), np.asarray(exp, np.float64)
    assert (np.isnan(got) == np.isnan(exp)).all(), (got, exp)
    inf = np.isinf(exp)
    assert (got[inf] == exp[inf]).all(), (got, exp)
    ok = np.isfinite(exp)
    err = np.abs(got[ok] - exp[ok]) - (tol[ok] if np.ndim(tol) else tol)
    assert (err <= 0).all(), (err.max(), got[ok][err.argmax()], exp[ok][err.argmax()])


def make_tokens(rows, org, vocab, seed):
    rng = np.random.default_rng(seed)
    t = rng.integers(0, org, rows).astype(np.int32)
    t[rng.random(rows) < 0.1] = -1
    if vocab > org and rows > 2:
        t[2] = org                       # a padding id
    return t


def check_outputs(x64, org, tokens, k, out, log_extra=0.0):
    lo, en, ls, ids, tl = (None if o is None else o.cpu().numpy() for o in out)
    for r in range(len(x64)):
        at, ent, lse, eids, elp = plain_row(x64[r, :org], int(tokens[r]), k)
        size = 0.0 if not math.isfinite(lse) else abs(lse)
        tol = 1e-5 + 2.0 ** -22 * size
        if k:
            assert (ids[r] == eids).all(), (r, ids[r], eids)
            close(tl[r], elp, 1e-5 + 2.0 ** -22 * (size + np.abs(elp)))
        close(ls[r], lse, tol)
        close(lo[r], at, tol + (2.0 ** -22 * abs(at) if math.isfinite(at) else 0.0))
        close(en[r], ent, 2e-5 * (1.0 + math.log(max(org, 2))))


def run_forward(sga, dev, org, tok, k):
    rows = dev.size(0)
    f = lambda *s: torch.full(s, 77.0, device="cuda")       # noqa: E731
    out = [f(rows), f(rows), f(rows),
           torch.full((rows, k), -77, dtype=torch.int32, device="cuda") if k else None,
           f(rows, k) if k else None]
    sga.sga_token_logprobs(dev, org, tok, *out)
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_logprobs_match_64_bits(sga_lib, case):
    rows, vocab, org, dtype, k, pad, offset = case
    x, _ = make_logits(rows + vocab, rows, vocab, dtype, pad, offset)
    plant(x[:, :vocab], dtype)
    dev, x64 = to_cuda(x, dtype, vocab, offset)
    tokens = make_tokens(rows, org, vocab, vocab)
    out = run_forward(sga_lib, dev, org, torch.from_numpy(tokens).cuda(), k)
    check_outputs(x64, org, tokens, k, out)


@pytest.mark.gpu
@pytest.mark.parametrize("offset", [0.0, -1e4, 1e5, -4.9e5, 4.9e5, 3e6])
@pytest.mark.parametrize("rows,vocab,shards", [(1, 40000, 1), (60, 40000, 1), (955, 5455, 1),
                                               (40, 5455, 3)])
def test_entropy_of_rows_far_from_zero(sga_lib, rows, vocab, shards, offset):
    """The entropy does not depend on where the logits lie.  Sixteen ulps of the
    sum of 2^t and as many of the sum of t 2^t (2e-6 each), relative to a size of
    1 + log(vocab) at most."""
    x = torch.from_numpy(wl.normal_matrix(vocab + rows, rows, vocab, 3.0, dtype="f32")).cuda()
    x += offset
    ent, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    if shards == 1:
        sga_lib.sga_token_logprobs(x, vocab, None, None, ent, lse)
    else:
        parts = torch.empty((shards, rows, 4), device="cuda")
        for s, (o, w) in enumerate(wl.even_shards(vocab, shards)):
            sga_lib.sga_local_logprobs(x[:, o:o + w], o, w, vocab, None, parts[s])
        sga_lib.sga_logprob_reduce(parts, None, shards, None, None, ent, lse)
    m = x.amax(1, keepdim=True).double()
    d = x.double() - m
    total = torch.logsumexp(d, 1, keepdim=True)
    exp = -(torch.exp(d - total) * (d - total)).sum(1)
    assert ((ent.double() - exp).abs() <= 4e-6 * (1 + math.log(vocab))).all()
    want = (m + total)[:, 0]
    assert ((lse.double() - want).abs() <= 4e-6 * (1 + math.log(vocab)) + 2.0 ** -23 * want.abs()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("shards", [1, 2, 5])
@pytest.mark.parametrize("case", [CASES[4], CASES[6], CASES[8], CASES[3]], ids=str)
def test_sharded_parts_reduce_to_the_same(sga_lib, case, shards):
    rows, vocab, org, dtype, k, pad, offset = case
    x, _ = make_logits(rows + vocab, rows, vocab, dtype, pad, offset)
    plant(x[:, :vocab], dtype)
    dev, x64 = to_cuda(x, dtype, vocab, offset)
    tokens = make_tokens(rows, org, vocab, 3)
    tok = torch.from_numpy(tokens).cuda()
    parts = torch.full((shards, rows, 4), 9.0, device="cuda")
    tops = torch.full((shards, rows, k, 2), -9, dtype=torch.int32, device="cuda")
    for s, (o, w) in enumerate(wl.even_shards(vocab, shards)):
        sga_lib.sga_local_logprobs(dev[:, o:o + w], o, w, org, tok, parts[s], tops[s])
    whole = run_forward(sga_lib, dev, org, tok, k)
    out = [torch.full_like(t, 5) for t in whole]
    sga_lib.sga_logprob_reduce(parts, tops, shards, tok, *out)
    check_outputs(x64, org, tokens, k, out)
    assert torch.equal(out[3], whole[3])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shards,k", [(70, 32), (8, 20), (40, 1), (33, 7), (300, 3)])
def test_many_shards(sga_lib, shards, k, dtype):
    """Lists shorter than k, all of whose entries may be among the best; many
    entries that reach every list's last."""
    rows, vocab, org = 19, 700, 689
    x, _ = make_logits(shards, rows, vocab, dtype, 0, 0)
    plant(x[:, :vocab], dtype)
    x[15] = np.linspace(3, -3, vocab)        # the best ids all in the first shards
    x[16] = np.linspace(-3, 3, vocab)
    dev, x64 = to_cuda(x, dtype, vocab, 0)
    tokens = make_tokens(rows, org, vocab, 3)
    tok = torch.from_numpy(tokens).cuda()
    parts = torch.full((shards, rows, 4), 9.0, device="cuda")
    tops = torch.full((shards, rows, k, 2), -9, dtype=torch.int32, device="cuda")
    for s, (o, w) in enumerate(wl.even_shards(vocab, shards)):
        sga_lib.sga_local_logprobs(dev[:, o:o + w], o, w, org, tok, parts[s], tops[s])
    whole = run_forward(sga_lib, dev, org, tok, k)
    out = [torch.full_like(t, 5) for t in whole]
    sga_lib.sga_logprob_reduce(parts, tops, shards, tok, *out)
    check_outputs(x64, org, tokens, k, out)
    assert torch.equal(out[3], whole[3])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k", [1, 5, 32])
@pytest.mark.parametrize("vocab", [20000, 70001])
def test_rows_that_are_hard_to_select_from(sga_lib, vocab, k, dtype):
    """Rising and falling rows, equal values, masks that leave fewer ids than
    top_k or none in the first thousands, NaNs among them."""
    rng = np.random.default_rng(vocab + k)
    x = rng.standard_normal((14, vocab)).astype(np.float32)
    x[0] = np.linspace(-5, 5, vocab)
    x[1] = np.linspace(5, -5, vocab)
    x[2] = 1.5
    x[3] = LOWEST[dtype]
    x[3, [7, vocab - 3]] = 2.0
    x[4] = NEG
    x[4, [vocab // 2, vocab - 1]] = [1.0, 3.0]
    x[5, :15000] = NEG
    x[6] = NEG
    x[6, 15000:15030] = 0.5
    x[7, 9000:] = NEG
    x[8] = np.round(x[8])
    x[9, ::1000] = math.nan
    x[10, -5:] = 40.0
    x[11] = NEG
    x[12, :] = np.where(rng.random(vocab) < 1e-3, x[12], NEG)
    x[13] = -0.0
    x[13, 5::11] = 0.0
    dev, x64 = to_cuda(x, dtype, vocab, 1)
    tokens = make_tokens(14, vocab, vocab, 1)
    out = run_forward(sga_lib, dev, vocab, torch.from_numpy(tokens).cuda(), k)
    check_outputs(x64, vocab, tokens, k, out)
    # many rows at once: other CTA shapes
    many = dev.repeat(60, 1)
    big = run_forward(sga_lib, many, vocab, torch.from_numpy(np.tile(tokens, 60)).cuda(), k)
    check_outputs(x64, vocab, tokens, k, [o[-14:] for o in big])
    assert sga_lib.sga_device_error() == 0


@pytest.mark.gpu
def test_a_shard_of_padding_only(sga_lib):
    x, _ = make_logits(5, 6, 300, "f32", 0, 0)
    dev, x64 = to_cuda(x, "f32", 300, 0)
    org, k = 150, 6
    tokens = np.array([0, 149, 150, 299, -1, 20], np.int32)
    tok = torch.from_numpy(tokens).cuda()
    parts = torch.empty((2, 6, 4), device="cuda")
    tops = torch.empty((2, 6, k, 2), dtype=torch.int32, device="cuda")
    for s, o in enumerate((0, 150)):
        sga_lib.sga_local_logprobs(dev[:, o:o + 150], o, 150, org, tok, parts[s], tops[s])
    out = [torch.empty(6, device="cuda") for _ in range(3)] + [
        torch.empty((6, k), dtype=torch.int32, device="cuda"), torch.empty((6, k), device="cuda")]
    sga_lib.sga_logprob_reduce(parts, tops, 2, tok, *out)
    check_outputs(x64, org, tokens, k, out)


@pytest.mark.gpu
def test_every_output_is_optional(sga_lib):
    x, _ = make_logits(6, 9, 500, "bf16", 0, 0)
    dev, _ = to_cuda(x, "bf16", 500, 0)
    tok = torch.arange(9, dtype=torch.int32, device="cuda")
    full = run_forward(sga_lib, dev, 500, tok, 4)
    ids = torch.empty_like(full[3])
    sga_lib.sga_token_logprobs(dev, 500, out_top_ids=ids)
    assert torch.equal(ids, full[3])
    lp = torch.empty_like(full[4])
    sga_lib.sga_token_logprobs(dev, 500, out_top_logprobs=lp)
    assert torch.equal(lp, full[4])
    lse = torch.empty_like(full[2])
    sga_lib.sga_token_logprobs(dev, 500, out_lse=lse)
    assert torch.equal(lse, full[2])
    sga_lib.sga_token_logprobs(dev[:0], 500, tok[:0], full[0][:0])   # no rows: nothing to do


@pytest.mark.gpu
def test_own_stream_and_graph_replay(sga_lib):
    rows, vocab, k = 12, 5000, 5
    dev = torch.empty((rows, vocab), dtype=torch.bfloat16, device="cuda")
    tok = torch.zeros(rows, dtype=torch.int32, device="cuda")
    grad = torch.empty_like(dev)
    up = torch.ones(rows, device="cuda")
    out = run_forward(sga_lib, dev.zero_(), vocab, tok, k)

    def step():
        sga_lib.sga_token_logprobs(dev, vocab, tok, *out)
        sga_lib.sga_token_logprobs_grad(dev, 0, vocab, tok, out[2], out[1], up, grad)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        x, _ = make_logits(seed, rows, vocab, "bf16", 0, 0)
        src, x64 = to_cuda(x, "bf16", vocab, 0)
        tokens = make_tokens(rows, vocab, vocab, seed)
        dev.copy_(src)
        tok.copy_(torch.from_numpy(tokens))
        graph.replay()
        check_outputs(x64, vocab, tokens, k, out)
        first = grad.clone()
        step()
        assert torch.equal(first, grad)


@pytest.mark.gpu
def test_row_offsets_past_32_bits(sga_lib):
    rows, ld, vocab = 3, (1 << 31) // 2 + 8, 700     # byte offsets past 2^31 and 2^32
    buf = torch.zeros((rows, ld), dtype=torch.bfloat16, device="cuda")
    x, _ = make_logits(8, rows, vocab, "bf16", 0, 0)
    src, x64 = to_cuda(x, "bf16", vocab, 0)
    buf[:, :vocab] = src
    tokens = np.array([5, 699, 0], np.int32)
    tok = torch.from_numpy(tokens).cuda()
    out = run_forward(sga_lib, buf[:, :vocab], vocab, tok, 3)
    check_outputs(x64, vocab, tokens, 3, out)
    up = torch.ones(rows, device="cuda")
    a = torch.empty((rows, vocab), dtype=torch.bfloat16, device="cuda")
    sga_lib.sga_token_logprobs_grad(src, 0, vocab, tok, out[2], out[1], up, a)
    sga_lib.sga_token_logprobs_grad(buf[:, :vocab], 0, vocab, tok, out[2], out[1], up,
                                    buf[:, :vocab])
    assert torch.equal(a, buf[:, :vocab])


# ----------------------------------------------------------------- gradient

GRAD_CASES = [  # rows, vocab, org, dtype, k, x pad, x offset, grad pad, grad offset
    (1, 1, 1, "f32", 0, 0, 0, 0, 0), (30, 40, 37, "f32", 5, 1, 3, 0, 0),
    (30, 257, 257, "bf16", 3, 3, 5, 3, 5), (30, 1001, 990, "bf16", 20, 0, 0, 7, 1),
    (30, 4099, 4099, "f32", 1, 0, 0, 0, 0), (4, 50257, 50250, "bf16", 0, 0, 0, 0, 0),
    (3, 33000, 33000, "bf16", 5, 8, 0, 8, 0), (9, 64, 8, "bf16", 2, 0, 0, 0, 0),
]


def grad_inputs(rows, org, k, seed):
    rng = np.random.default_rng(seed)
    f = lambda *s: rng.standard_normal(s).astype(np.float32)   # noqa: E731
    ids = rng.integers(0, org, (rows, k)).astype(np.int32)     # repeats are allowed
    if k:
        ids[::5, 0] = -1
    return f(rows), f(rows), ids, f(rows, k)


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("with_entropy", [False, True])
@pytest.mark.parametrize("case", GRAD_CASES, ids=str)
def test_gradient_matches_the_formula(sga_lib, case, with_entropy, in_place):
    rows, vocab, org, dtype, k, pad, offset, gpad, goffset = case
    x, _ = make_logits(rows + vocab, rows, vocab, dtype, pad, offset)
    for r, f in ((1, lambda v: v.fill(NEG)), (3, lambda v: v.__setitem__(slice(0, vocab, 3), NEG)),
                 (5, lambda v: v.__setitem__(slice(1, vocab), LOWEST[dtype])),
                 (7, lambda v: v.fill(2.0))):
        if r < rows:
            f(x[r, :vocab])
    dev, x64 = to_cuda(x, dtype, vocab, offset)
    tokens = make_tokens(rows, org, vocab, 11)
    gl, ge, ids, gt = grad_inputs(rows, org, k, 12)
    if k and rows > 8:
        ids[8, -1] = tokens[8]
    tok = torch.from_numpy(tokens).cuda()
    lse = torch.empty(rows, device="cuda")
    ent = torch.empty(rows, device="cuda")
    sga_lib.sga_token_logprobs(dev, org, tok, None, ent, lse)
    if in_place:
        out = dev
    else:
        out, _ = to_cuda(np.full((rows, vocab + gpad), 3.0, np.float32), dtype, vocab, goffset)
    sga_lib.sga_token_logprobs_grad(
        dev, 0, org, tok, lse, ent if with_entropy else None, torch.from_numpy(gl).cuda(), out,
        grad_entropy=torch.from_numpy(ge).cuda() if with_entropy else None,
        top_ids=torch.from_numpy(ids).cuda() if k else None,
        grad_top=torch.from_numpy(gt).cuda() if k else None)
    got = out.double().cpu().numpy()
    lse, ent = lse.double().cpu().numpy(), ent.double().cpu().numpy()
    for r in range(rows):
        exp, tol = plain_grad_row(x64[r, :org], vocab, int(tokens[r]), lse[r], ent[r], gl[r],
                                  ge[r] if with_entropy else 0.0, ids[r], gt[r])
        if dtype == "bf16":
            tol = tol + 2.0 ** -8 * np.abs(exp) + 1e-38
        close(got[r], exp, tol + 1e-37)


@pytest.mark.gpu
@pytest.mark.parametrize("shards", [2, 3])
def test_gradient_of_shards_is_the_whole_gradient(sga_lib, shards):
    rows, vocab, org, k = 10, 999, 960, 4
    x, _ = make_logits(4, rows, vocab, "f32", 0, 0)
    dev, _ = to_cuda(x, "f32", vocab, 0)
    tok = torch.from_numpy(make_tokens(rows, org, vocab, 5)).cuda()
    gl, ge, ids, gt = (torch.from_numpy(a).cuda() for a in grad_inputs(rows, org, k, 6))
    lse, ent = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    sga_lib.sga_token_logprobs(dev, org, tok, None, ent, lse)
    whole = torch.full_like(dev, 4.0)
    sga_lib.sga_token_logprobs_grad(dev, 0, org, tok, lse, ent, gl, whole, ge, ids, gt)
    split = torch.full_like(dev, 5.0)
    for o, w in wl.even_shards(vocab, shards):
        sga_lib.sga_token_logprobs_grad(dev[:, o:o + w], o, org, tok, lse, ent, gl,
                                        split[:, o:o + w], ge, ids, gt)
    assert torch.equal(whole, split)


@pytest.mark.gpu
def test_gradient_against_differences(sga_lib):
    """Central differences of the kernels' own forward pass.  With h = 1/32 the
    truncation is h^2 / 6 times a third derivative of at most about 10 of the
    upstream size (1.6e-3) and the rounding 4e-5 * 6 terms / 2h = 4e-3."""
    rows, vocab, k, h = 4, 24, 3, 2.0 ** -5
    x, _ = make_logits(14, rows, vocab, "f32", 0, 0, sigma=1.5)
    dev, _ = to_cuda(x, "f32", vocab, 0)
    tok = torch.tensor([3, 0, 23, 7], dtype=torch.int32, device="cuda")
    gl, ge, _, gt = (torch.from_numpy(a).cuda() for a in grad_inputs(rows, vocab, k, 15))
    base = run_forward(sga_lib, dev, vocab, tok, k)
    grad = torch.empty_like(dev)
    sga_lib.sga_token_logprobs_grad(dev, 0, vocab, tok, base[2], base[1], gl, grad, ge, base[3], gt)

    def loss(d):
        out = run_forward(sga_lib, d, vocab, tok, vocab)
        # the log probabilities of the base point's alternatives
        where = (out[3][:, None, :] == base[3][:, :, None]).double()
        tops = (where * out[4].double()[:, None, :]).sum(2)
        return gl.double() * out[0].double() + ge.double() * out[1].double() + (
            gt.double() * tops).sum(1)

    for j in range(vocab):
        up, down = dev.clone(), dev.clone()
        up[:, j] += h
        down[:, j] -= h
        diff = (loss(up) - loss(down)) / (up[:, j] - down[:, j]).double()
        size = 1.0 + gl.abs() + ge.abs() * 4 + gt.abs().sum(1)
        assert ((diff - grad[:, j].double()).abs() <= 6e-3 * size).all(), j


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [0, 1])
def test_masked_ids_stay_zero_under_a_huge_entropy_gradient(sga_lib, pad):
    """p = 0 times a finite factor, however large.  Error of the others: p and
    the factor b (log p + H) are each off by a few 2^-23 of |b| times log p and
    H, which are below 5: 2^-18 |b| bounds it."""
    b = 1e12
    x = torch.full((3, 64 + pad), -1e30)
    x[0, :4] = torch.tensor([0.5, 1.0, float("-inf"), -2.0])
    x[1, 5:30] = torch.linspace(-1, 1, 25)
    x[1, 40:] = float("-inf")
    x[2, 63] = 3.0
    x = x.cuda()[:, :64]
    tok = torch.tensor([1, 7, 63], dtype=torch.int32, device="cuda")
    lse, ent = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    sga_lib.sga_token_logprobs(x, 64, tok, None, ent, lse)
    grad = torch.empty((3, 64), device="cuda")
    ge = torch.full((3,), b, device="cuda")
    sga_lib.sga_token_logprobs_grad(x, 0, 64, tok, lse, ent, None, grad, ge)
    lp = x.double() - lse.double()[:, None]
    exp = torch.where(lp < -200, 0.0, -b * lp.exp() * (lp.clamp(min=-300) + ent.double()[:, None]))
    assert (grad[lp < -200] == 0).all()
    assert ((grad.double() - exp).abs() <= 2.0 ** -18 * b).all()


# ----------------------------------------------------------------- refusals


def test_token_logprobs_validation(sga_lib):
    f = sga_lib.lib().sga_token_logprobs

    def call(**kw):
        a = dict(dict(x=FAKE, dtype=1, rows=4, ld=10, vocab=10, org=10, tok=FAKE, k=2, lp=FAKE,
                      en=FAKE, ls=FAKE, ids=FAKE, tl=FAKE), **kw)
        return f(a["x"], a["dtype"], a["rows"], a["ld"], a["vocab"], a["org"], a["tok"], a["k"],
                 a["lp"], a["en"], a["ls"], a["ids"], a["tl"], None)

    assert call(dtype=2) == -5
    assert call(rows=-1) == -2 and call(rows=(1 << 28) + 1) == -2
    assert call(k=-1) == -2 and call(k=33) == -2
    assert call(vocab=0) == -3 and call(ld=9) == -3
    assert call(org=0) == -4 and call(vocab=(1 << 24) + 1, ld=1 << 25) == -4
    assert call(x=None) == -1
    for name in ("x", "tok", "lp", "en", "ls", "ids", "tl"):
        assert call(**{name: ODD}) == -6, name
    assert call(rows=0) == 0 and call(rows=0, x=None) == 0


def test_local_and_reduce_validation(sga_lib):
    f = sga_lib.lib().sga_local_logprobs

    def call(**kw):
        a = dict(dict(x=FAKE, dtype=0, rows=4, ld=10, start=0, width=10, org=10, tok=FAKE, k=2,
                      parts=FAKE, top=FAKE), **kw)
        return f(a["x"], a["dtype"], a["rows"], a["ld"], a["start"], a["width"], a["org"],
                 a["tok"], a["k"], a["parts"], a["top"], None)

    assert call(dtype=-1) == -5 and call(rows=-1) == -2 and call(k=33) == -2
    assert call(start=-1) == -3 and call(width=0) == -3 and call(ld=9) == -3
    assert call(org=0) == -4 and call(start=(1 << 24) - 9) == -4
    assert call(parts=None) == -1 and call(top=None) == -1 and call(x=None) == -1
    assert call(parts=ODD) == -6 and call(top=ctypes.c_void_p(0x10004)) == -6
    assert call(rows=0) == 0
    g = sga_lib.lib().sga_logprob_reduce

    def reduce(**kw):
        a = dict(dict(parts=FAKE, tops=FAKE, n=2, rows=4, k=2, tok=FAKE, lp=FAKE, ids=FAKE), **kw)
        return g(a["parts"], a["tops"], a["n"], a["rows"], a["k"], a["tok"], a["lp"], None, None,
                 a["ids"], None, None)

    assert reduce(n=0) == -2 and reduce(n=4097) == -2 and reduce(rows=-1) == -2
    assert reduce(k=33) == -2 and reduce(parts=None) == -1 and reduce(tops=None) == -1
    assert reduce(parts=ODD) == -6 and reduce(lp=ODD) == -6 and reduce(rows=0) == 0


def test_logprobs_grad_validation(sga_lib):
    f = sga_lib.lib().sga_token_logprobs_grad

    def call(**kw):
        a = dict(dict(x=FAKE, dtype=1, rows=4, ld=10, start=0, width=10, org=10, tok=FAKE,
                      lse=FAKE, ent=FAKE, gl=FAKE, ge=FAKE, k=2, ids=FAKE, gt=FAKE, out=FAKE,
                      ldg=10), **kw)
        return f(a["x"], a["dtype"], a["rows"], a["ld"], a["start"], a["width"], a["org"],
                 a["tok"], a["lse"], a["ent"], a["gl"], a["ge"], a["k"], a["ids"], a["gt"],
                 a["out"], a["ldg"], None)

    assert call(dtype=9) == -5 and call(rows=-1) == -2 and call(k=33) == -2
    assert call(ld=9) == -3 and call(ldg=9) == -3 and call(width=0) == -3
    assert call(org=0) == -4
    for name in ("x", "lse", "out", "ent", "ids", "gt"):
        assert call(**{name: None}) == -1, name
    for name in ("x", "lse", "ent", "gl", "ge", "ids", "gt", "out", "tok"):
        assert call(**{name: ODD}) == -6, name
    assert call(rows=0) == 0


def test_binding_refuses_wrong_tensors(sga_lib):
    x = torch.zeros(3, 8)
    f32, i32 = torch.zeros(3), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        sga_lib.sga_token_logprobs(x.t(), 3, i32, f32)
    with pytest.raises(ValueError):
        sga_lib.sga_token_logprobs(x, 8, i32.long(), f32)
    with pytest.raises(ValueError):
        sga_lib.sga_token_logprobs(x, 8, i32, f32.double())
    with pytest.raises(ValueError):
        sga_lib.sga_token_logprobs(x, 8, i32[:2], f32)
    with pytest.raises(TypeError):
        sga_lib.sga_token_logprobs(x.half(), 8, i32, f32)
    with pytest.raises(ValueError):
        sga_lib.sga_local_logprobs(x, 0, 9, 9, i32, torch.zeros(3, 4))
    with pytest.raises(ValueError):
        sga_lib.sga_token_logprobs_grad(x, 0, 8, i32, f32, f32, f32, x[:, :4])
    with pytest.raises(ValueError):
        sga_lib.sga_token_logprobs_grad(x, 0, 8, i32, f32, f32, f32, x.bfloat16())


def test_binding_refuses_host_tensors(sga_lib):
    x = torch.zeros(3, 8)
    f32, i32 = torch.zeros(3), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sga_lib.sga_token_logprobs(x, 8, i32, f32)
    with pytest.raises(ValueError, match="CUDA"):
        sga_lib.sga_local_logprobs(x, 0, 8, 8, i32, torch.zeros(3, 4))
    with pytest.raises(ValueError, match="CUDA"):
        sga_lib.sga_logprob_reduce(torch.zeros(1, 3, 4), None, 1, i32, f32)
    with pytest.raises(ValueError, match="CUDA"):
        sga_lib.sga_token_logprobs_grad(x, 0, 8, i32, f32, f32, f32, torch.zeros(3, 8))


def test_binding_refuses_numbers_of_shards_below_one(sga_lib):
    parts, f32 = torch.zeros(2, 3, 4), torch.zeros(3)
    for n in (0, -1):
        with pytest.raises(ValueError, match="num_shards"):
            sga_lib.sga_logprob_reduce(parts, None, n, None, f32)
