"""Probabilities of logits rows and the sampled verification that reads them,
against plain implementations, at the sizes, masks and alignments where the
kernels change path, and the entry points' refusals.

The probabilities' tolerance, by counting roundings: t = (x - max) log2(e) / T has
five of 2^-24 relative to itself (the difference, the constant, its quotient,
the product, and bf16's none), so 2^t is off by 5 ln2 2^-24 |t|, and by 2^-22 as
computed; the row's sum of n positive terms, taken by 256 threads or more in two
halves each, has at most n / 256 + 64 additions along any path, 2^-24 each (rows of up
to 48 KB by 64 threads: n / 128 + 16, less up to n = 12288); the last product and
the reciprocal add 2^-22.  Terms below 2^-126 may be flushed.

What sga_sampled_verify emits is whole numbers defined exactly (units of 2^-38,
fp32 products and differences rounded once), so it is compared for equality.
"""
import ctypes
import math

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
    """(buffer, matrix): a matrix of row stride cols + pad, `offset` elements into
    a buffer that is otherwise (and at first) GUARD, with a row more."""
    ld = cols + pad
    buf = torch.full((offset + (rows + 1) * ld + 8,), GUARD, dtype=dtype, device="cuda")
    return buf, buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]


def check_guard(buf, rows, cols, pad, offset):
    seen = torch.ones(buf.numel(), dtype=torch.bool, device="cuda")
    seen[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = False
    assert (buf[seen] == GUARD).all(), "written outside of the rows"


# ------------------------------------------------------------- probabilities


def plain_probs(x, org, t):
    """x: logits; (probabilities in 64 bits, the exponents log2(e) (x - max) / T)."""
    rows, width = x.shape
    out = torch.zeros((rows, width), dtype=torch.float64, device=x.device)
    expo = torch.zeros_like(out)
    y = x[:, :org].double()
    for r in range(rows):
        tr = 1.0 if t is None else float(t[r])
        row = y[r]
        if tr == 0.0:
            nan = torch.isnan(row).nonzero()
            best = nan[0, 0] if len(nan) else (row == row.max()).nonzero()[0, 0]
            out[r, best] = 1.0
        elif not tr > 0.0 or torch.isnan(row).any() or (row == math.inf).any():
            out[r, :org] = math.nan
        elif (row > NEG).any():
            d = (row - row.max()) / tr
            e = torch.exp(d)
            out[r, :org] = e / e.sum()
            expo[r, :org] = torch.where(row == NEG, 0.0, d / math.log(2.0))
    return out, expo


def check_probs(got, x, org, t):
    exp, expo = plain_probs(x, org, t)
    rel = (5 * math.log(2.0) * expo.abs() + org / 256 + 64 + 8) * 2.0 ** -24
    tol = torch.nan_to_num(exp) * rel + 2.0 ** -125
    assert torch.equal(torch.isnan(got), torch.isnan(exp))
    bad = (got.double() - exp).abs() > tol
    assert not bad.any(), (bad.nonzero()[:4].tolist(), got[bad][:4], exp[bad][:4])
    if t is not None:                   # greedy rows and what is 0 are exact
        z = t == 0
        assert torch.equal(got[z].double(), exp[z])
    assert (got[:, org:] == 0).all()


def plant(x, org):
    """Special rows, as many as there is room for."""
    lowest = torch.finfo(x.dtype).min
    if x.size(0) > 2:
        x[2] = NEG
    if x.size(0) > 4:
        x[3, 1:org] = lowest
        x[4] = lowest
    if x.size(0) > 6:
        x[5, org // 2] = math.nan
        x[6, org // 3] = math.inf
    if x.size(0) > 8:
        x[7] = 3.0
        x[8] = NEG
        x[8, org - 1] = -5.0
    if x.size(0) > 10:
        x[9] += 1e6 if x.dtype == torch.float32 else 1e3
        x[10] -= 1e6 if x.dtype == torch.float32 else 1e3
        x[10, ::2] = NEG


PROBS = [  # rows, vocab, org, dtype, temperature, pad, offset
    (1, 1, 1, "bf16", "none", 0, 0), (1, 2, 1, "f32", "mixed", 0, 0),
    (3, 7, 5, "bf16", "row", 2, 3), (12, 1000, 1000, "bf16", "mixed", 0, 0),
    (12, 4099, 4090, "bf16", "mixed", 0, 1), (12, 4099, 4090, "f32", "mixed", 1, 1),
    (14, 50257, 50257, "f32", "none", 1, 2), (333, 5003, 5003, "bf16", "row", 0, 7),
    (2, 152064, 151936, "bf16", "row", 0, 0), (40, 152064, 151936, "bf16", "mixed", 8, 0),
    (11, 202048, 202048, "f32", "mixed", 0, 0), (700, 1531, 1500, "f32", "none", 3, 1),
    # longer than the shared memory of a cluster, at aligned and odd rows
    (3, 900001, 900001, "bf16", "row", 0, 0), (11, 480003, 480000, "f32", "mixed", 1, 1),
    (2000, 333, 333, "bf16", "mixed", 1, 0),
    # several such rows per cluster, and short rows longer than a small ring
    (60, 900001, 900001, "bf16", "mixed", 0, 0), (2000, 24001, 24000, "bf16", "mixed", 0, 0),
    (2000, 12001, 12001, "f32", "row", 1, 1),
]


def temperatures(kind, rows, g):
    if kind == "none":
        return None
    t = 0.2 + 1.5 * torch.rand(rows, generator=g, device="cuda")
    if kind == "mixed":
        t[1::3] = 0.0
    return t


@pytest.mark.gpu
@pytest.mark.parametrize("case", PROBS, ids=str)
def test_probs_match_64_bits(sga_lib, case):
    rows, vocab, org, dtype, kind, pad, offset = case
    g = gen(vocab + rows)
    xbuf, x = guarded(rows, vocab, pad, offset, DT[dtype])
    x.normal_(0.0, 4.0, generator=g)
    plant(x, org)
    before = xbuf.clone()
    t = temperatures(kind, rows, g)
    for opad, ooff in ((0, 0), (1, 1), (pad, offset)):
        obuf, out = guarded(rows, vocab, opad, ooff, torch.float32)
        sga_lib.sga_probs(x, org, out, temperature=t)
        check_probs(out, x, org, t)
        check_guard(obuf, rows, vocab, opad, ooff)
    assert torch.equal(xbuf.view(torch.int16), before.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("t", [1e-30, 1e-3, 30.0, 1e30])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_probs_at_extreme_temperatures(sga_lib, dtype, t):
    x = torch.empty((12, 3001), dtype=DT[dtype], device="cuda").normal_(0.0, 4.0, generator=gen(1))
    plant(x, 3001)
    if t == 1e30:                       # lowest values are worth something there
        x[3:5] = 0.0
    temps = torch.full((12,), t, device="cuda")
    out = torch.empty((12, 3001), device="cuda")
    sga_lib.sga_probs(x, 3001, out, temperature=temps)
    check_probs(out, x, 3001, temps)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,vocab,dtype,pad", [
    (64, 5, "bf16", 1), (64, 1003, "f32", 1), (700, 9001, "bf16", 0), (40, 70001, "bf16", 3),
    (40, 70001, "f32", 1), (30, 900001, "bf16", 1), (30, 480003, "f32", 0)])
def test_greedy_rows_take_the_lowest_of_equal_logits(sga_lib, rows, vocab, dtype, pad):
    """Logits of four values, NaN among them in some rows, -inf alone in others."""
    g = gen(vocab)
    _, x = guarded(rows, vocab, pad, 1, DT[dtype])
    x.copy_(torch.randint(-2, 2, (rows, vocab), generator=g, device="cuda"))
    x[1::4] = torch.where(torch.rand((len(x[1::4]), vocab), generator=g, device="cuda") < 3 / vocab,
                          5.0, x[1::4].float()).to(x.dtype)
    x[2::8, vocab // 3:] = math.nan
    x[3::8] = NEG
    x[5::8, :-1] = NEG
    out = torch.empty((rows, vocab), device="cuda")
    sga_lib.sga_probs(x, vocab, out, temperature=torch.zeros(rows, device="cuda"))
    xf = x.float()
    nan = torch.isnan(xf)
    best = xf.masked_fill(nan, NEG).amax(1, keepdim=True)
    hit = torch.where(nan.any(1, keepdim=True), nan, xf == best)
    first = hit.to(torch.uint8).argmax(1)      # the first of equal ones
    exp = torch.zeros_like(out)
    exp[torch.arange(rows, device="cuda"), first] = 1.0
    assert torch.equal(out, exp)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_probs_of_the_largest_vocabulary(sga_lib, dtype):
    vocab = sga_lib.SGA_MAX_VOCAB
    x = torch.empty((2, vocab), dtype=DT[dtype], device="cuda").normal_(0.0, 4.0, generator=gen(3))
    x[1, vocab - 1] = 50.0
    out = torch.full((2, vocab), GUARD, device="cuda")
    for t in (None, torch.tensor([0.7, 0.0], device="cuda")):
        sga_lib.sga_probs(x, vocab, out, temperature=t)
        check_probs(out, x, vocab, t)
    with pytest.raises(sga_lib.SgaError):
        sga_lib.sga_probs(torch.empty((1, vocab + 1), dtype=DT[dtype], device="cuda"), vocab + 1,
                          torch.empty((1, vocab + 1), device="cuda"))


@pytest.mark.gpu
def test_a_negative_or_nan_temperature_makes_the_row_nan(sga_lib):
    x = torch.randn((4, 100), device="cuda")
    x[3] = NEG
    temps = torch.tensor([-1.0, math.nan, 1.0, -0.5], device="cuda")
    out = torch.empty_like(x)
    sga_lib.sga_probs(x, 90, out, temperature=temps)
    check_probs(out, x, 90, temps)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,vocab", [(3, 5000), (40, 50257), (2, 480003)])
def test_probs_in_place(sga_lib, rows, vocab):
    x = torch.randn((rows, vocab + 1), generator=gen(2), device="cuda")[:, :vocab]
    org = vocab - 3
    out = torch.empty((rows, vocab + 1), device="cuda")[:, :vocab]
    sga_lib.sga_probs(x, org, out)
    sga_lib.sga_probs(x, org, x)
    assert torch.equal(x, out)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,vocab", [(13, 5000), (40, 50257), (12, 480003), (40, 480003),
                                        (700, 9001), (3, 1 << 22)])
def test_probs_in_place_at_temperatures(sga_lib, rows, vocab):
    """Greedy rows among them, with equal best logits: in rows longer than the rings
    their place is found by a second look at the logits, before they are written over."""
    x = torch.randn((rows, vocab + 1), generator=gen(2), device="cuda")[:, :vocab]
    org, g = vocab - 3, gen(4)
    plant(x, org)
    t = temperatures("mixed", rows, g)
    for r in range(1, rows, 6):                          # every other greedy row
        x[r, torch.randint(0, org, (3,), generator=g, device="cuda")] = 90.0
    was = x.clone()
    out = torch.empty((rows, vocab + 1), device="cuda")[:, :vocab]
    sga_lib.sga_probs(x, org, out, temperature=t)
    sga_lib.sga_probs(x, org, x, temperature=t)
    assert torch.equal(x.nan_to_num(9.0), out.nan_to_num(9.0))
    check_probs(x, was, org, t)


@pytest.mark.gpu
def test_probs_rows_past_32_bits(sga_lib):
    """Row offsets of 2^31 elements and more, in and out."""
    stride = (1 << 31) // 3 + 5
    buf = torch.empty(3 * stride + 4096, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (4, 4000), (stride, 1))
    x.normal_(0.0, 3.0, generator=gen(3))
    obuf = torch.empty(3 * stride + 4096, device="cuda")
    out = torch.as_strided(obuf, (4, 4000), (stride, 1))
    sga_lib.sga_probs(x, 4000, out)
    check_probs(out, x, 4000, None)


# -------------------------------------------------------------- verification


def plain_verify(target, draft, cu, tokens, au, su, max_k, prefill=None):
    """Request by request, from the definition; numpy on the host."""
    n, vocab = len(cu) - 1, target.shape[1]
    sampled = np.full((n, max_k + 1), -1, np.int32)
    num, rej, last = np.zeros(n, np.int32), np.zeros(n, np.int32), np.full(n, -1, np.int32)

    def units(w):
        w = np.nan_to_num(w.astype(np.float64), nan=0.0)
        return np.rint(np.clip(w, 0.0, 1.0) * 2.0 ** 38).astype(np.int64)

    for i in range(n):
        if prefill is not None and prefill[i]:
            continue
        k, a = cu[i + 1] - cu[i], 0
        q = np.zeros(vocab, np.float32)
        while a < k:
            t, d = tokens[cu[i] + a], cu[i] + a
            row = target[cu[i] + i + a]
            if 0 <= t < vocab:
                qt = draft[d, t] if draft is not None else np.float32(1)
                if np.float32(au[d]) * qt < row[t]:
                    a += 1
                    continue
                if draft is not None:
                    q = draft[d]
                else:
                    q[t] = 1
            break
        p = target[cu[i] + i + a]
        token = -1
        for w in ([p - q] if a < k else []) + [p]:
            sums = np.cumsum(units(w))
            if sums[-1] > 0:
                u = np.float64(su[i])
                edge = min(math.floor(u * np.float64(sums[-1])) if u > 0 else 0, sums[-1] - 1)
                token = int(np.searchsorted(sums, edge, side="right"))
                break
        sampled[i, :a] = tokens[cu[i]:cu[i] + a]
        sampled[i, a] = last[i] = token
        num[i], rej[i] = a + 1, k - a
    return sampled, num, rej, last


def gpu_verify(sga_lib, target, draft, cu, tokens, au, su, max_k, prefill=None, stream=None):
    n = len(cu) - 1
    dev = dict(dtype=torch.int32, device="cuda")
    outs = [torch.full((n, max_k + 1), -99, **dev)] + [torch.full((n,), -99, **dev)
                                                       for _ in range(3)]
    sga_lib.sga_sampled_verify(
        target, draft, torch.tensor(cu, **dev), torch.tensor(tokens, **dev),
        torch.tensor(au, dtype=torch.float32, device="cuda"),
        torch.tensor(su, dtype=torch.float32, device="cuda"), max_k, *outs,
        in_prefill=prefill,
        stream=stream)
    return outs


def verify_case(seed, n, max_k, vocab, drafts, pad, offset, ragged=True):
    """Guarded probabilities, drafts of assorted quality, uniforms with the
    ends of their range among them."""
    rng = np.random.default_rng(seed)
    g = gen(seed)
    counts = rng.integers(0, max_k + 1, n) if ragged else np.full(n, max_k)
    cu = np.concatenate([[0], np.cumsum(counts)]).tolist()
    d = cu[-1]
    _, target = guarded(d + n, vocab, pad, offset, torch.float32)
    _, draft = guarded(d, vocab, pad + 1, offset + 1, torch.float32)
    x = torch.randn((d, vocab), generator=g, device="cuda") * 2.0
    draft.copy_(torch.softmax(x, 1))
    of = [cu[i] + i + j for i in range(n) for j in range(cu[i + 1] - cu[i])]
    target.copy_(torch.softmax(torch.randn((d + n, vocab), generator=g, device="cuda") * 2.0, 1))
    if d:
        target[of] = torch.softmax(x + 0.7 * torch.randn(x.shape, generator=g, device="cuda"), 1)
        same = of[::5]
        target[same] = draft[::5]                       # nothing left of p - q
        tokens = torch.multinomial(draft[:, :1 << 23], 1, generator=g)[:, 0].cpu().numpy()
    else:
        tokens = np.zeros(0, np.int64)
    target[::7, vocab // 2:] = 0.0                      # cut rows
    if d + n > 11:
        target[11] = 0.0                                # no weight at all
    au = rng.random(d, dtype=np.float32)
    su = rng.random(n, dtype=np.float32)
    au[3::11] = 1.0 - 2.0 ** -24
    su[2::9] = 0.0
    su[4::9] = 1.0 - 2.0 ** -24
    tokens[5::13] = -1
    tokens[6::13] = vocab
    return (target, draft if drafts == "probs" else None, cu, tokens.astype(np.int32).tolist(),
            au.tolist(), su.tolist(), max_k)


def host(case):
    target, draft, cu, tokens, au, su, max_k = case
    return (target.cpu().numpy(), None if draft is None else draft.cpu().numpy(), cu, tokens,
            np.float32(au), np.float32(su), max_k)


def check_same(got, exp):
    for name, a, b in zip(("sampled", "num_sampled", "num_rejected", "last"), got, exp):
        assert np.array_equal(a.cpu().numpy(), b), name


VERIFY = [  # requests, max_k, vocab, drafts, pad, offset
    (1, 1, 1, "probs", 0, 0), (5, 2, 2, "tokens", 0, 0), (7, 15, 33, "probs", 3, 1),
    (40, 15, 1000, "probs", 0, 0), (40, 15, 1000, "tokens", 1, 3), (3, 3, 4099, "probs", 1, 1),
    (37, 5, 50257, "probs", 0, 0), (37, 5, 50257, "tokens", 5, 1), (1, 3, 152064, "probs", 0, 0),
    (24, 3, 200064, "probs", 0, 0), (2, 1, 1000003, "probs", 0, 0), (700, 2, 600, "probs", 0, 0),
    (5000, 1, 64, "tokens", 0, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", VERIFY, ids=str)
def test_verify_matches_the_definition(sga_lib, case):
    n, max_k, vocab, drafts, pad, offset = case
    c = verify_case(n * 31 + vocab, n, max_k, vocab, drafts, pad, offset)
    check_same(gpu_verify(sga_lib, *c), plain_verify(*host(c)))
    assert sga_lib.sga_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("n,max_k,vocab", [
    (85, 2, 40003), (6, 3, 30011), (120, 1, 20012), (100, 2, 24579), (200, 1, 9001),
    (20, 5, 16383), (400, 1, 152064), (310, 3, 9999)])
@pytest.mark.parametrize("drafts", ["probs", "tokens"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (1, 3)])
def test_every_number_of_ctas_per_request(sga_lib, n, max_k, vocab, drafts, pad, offset):
    """Requests that 6, 4 or 2 CTAs share, or that one takes in segments of several steps
    (aligned rows: vocabularies of a multiple of four)."""
    c = verify_case(n * 17 + vocab, n, max_k, vocab, drafts, pad, offset)
    check_same(gpu_verify(sga_lib, *c), plain_verify(*host(c)))
    assert sga_lib.sga_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(6))
def test_every_end_of_the_uniforms(sga_lib, seed):
    """Draws at the first and last weighted ids and at sums' borders."""
    rng = np.random.default_rng(seed)
    vocab, n = 2000 + 31 * seed, 64
    p = np.zeros((n, vocab), np.float32)
    for r in range(n):                       # a few ids of 1/2^b each: borders are exact
        ids = np.sort(rng.choice(vocab, 8, replace=False))
        p[r, ids] = np.array([.125] * 8, np.float32)
    su = (np.arange(n) % 9 / 8).astype(np.float32)       # 1.0 among them: the last id
    su[60:] = [math.nan, -1.0, 2.0, math.inf]
    c = (torch.from_numpy(p).cuda(), None, list(np.zeros(n + 1, np.int64)), [], [], su.tolist(), 1)
    got = gpu_verify(sga_lib, *c)
    last = got[3].cpu().numpy()
    for r in range(n):
        ids = np.flatnonzero(p[r])
        at = {60: 0, 61: 0, 62: 7, 63: 7}.get(r, min(r % 9, 7))
        assert last[r] == ids[at], r


@pytest.mark.gpu
@pytest.mark.parametrize("fill", ["ones", "sparse"])
def test_verify_of_the_largest_vocabulary(sga_lib, fill):
    """Sums of 2^62 units (every weight 1), and weights at both ends alone."""
    vocab = sga_lib.SGA_MAX_VOCAB
    target = torch.zeros((3, vocab), device="cuda")
    if fill == "ones":
        target += 1.0
    else:
        target[:, 0], target[:, vocab - 1] = 0.25, 0.5
    cu = torch.tensor([0, 0, 0, 0], dtype=torch.int32, device="cuda")
    none_i = torch.empty(0, dtype=torch.int32, device="cuda")
    none_f = torch.empty(0, device="cuda")
    su = torch.tensor([0.0, 0.4, 1.0 - 2.0 ** -24], device="cuda")
    out = [torch.empty(m, dtype=torch.int32, device="cuda") for m in (6, 3, 3, 3)]
    sga_lib.sga_sampled_verify(target, None, cu, none_i, none_f, su, 1, *out)
    u = [float(v) for v in su]
    if fill == "ones":
        # the first j with (j + 1) 2^38 > floor(u 2^62): floor(u 2^24)
        want = [int(math.floor(v * 2.0 ** 24)) for v in u]
    else:
        want = [0 if v * 0.75 < 0.25 else vocab - 1 for v in u]
    assert out[3].tolist() == want
    assert out[1].tolist() == [1, 1, 1] and out[2].tolist() == [0, 0, 0]


@pytest.mark.gpu
def test_nan_and_negative_weights_are_not_drawn(sga_lib):
    p = torch.full((3, 100), math.nan, device="cuda")
    p[0, 50] = 0.5
    p[1, 20:30] = -1.0
    p[1, 99] = 7.0
    got = gpu_verify(sga_lib, p, None, [0, 0, 0, 0], [], [], [0.9, 0.1, 0.5], 1)
    assert got[3].tolist() == [50, 99, -1]


@pytest.mark.gpu
@pytest.mark.parametrize("flag", [torch.bool, torch.uint8])
def test_requests_in_prefill_emit_nothing(sga_lib, flag):
    c = verify_case(5, 20, 4, 900, "probs", 0, 0)
    pre = np.arange(20) % 3 == 0
    got = gpu_verify(sga_lib, *c, prefill=torch.tensor(pre, device="cuda").to(flag))
    check_same(got, plain_verify(*host(c), prefill=pre))


@pytest.mark.gpu
def test_a_request_outside_of_the_layout_is_reported(sga_lib):
    c = list(verify_case(6, 4, 3, 500, "probs", 0, 0, ragged=False))
    good = plain_verify(*host(c))
    sga_lib.sga_clear_device_error()
    for cu, fine in (([0, 3, 6, 9, 40], 3), ([0, 3, 6, 5, 12], 2), ([-3, 0, 3, 6, 9], 0)):
        c[2] = cu
        got = gpu_verify(sga_lib, *c)
        assert sga_lib.sga_device_error() == sga_lib.SGA_DEVERR_K_RANGE
        sga_lib.sga_clear_device_error()
        check_same([g[:fine] for g in got], [e[:fine] for e in good])
        off = fine if fine else 0
        assert got[0][off].tolist() == [-1] * 4 and int(got[1][off]) == 0 and int(got[3][off]) == -1
    assert sga_lib.sga_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("with_draft_rows", [False, True])
def test_greedy_rows_give_the_greedy_result(sga_lib, with_draft_rows):
    """Temperature 0 through sga_probs and sga_sampled_verify, against
    sga_greedy_verify on the same logits."""
    g = gen(8)
    n, max_k, vocab, org = 30, 5, 3000, 2950
    rng = np.random.default_rng(8)
    cu = np.concatenate([[0], np.cumsum(rng.integers(0, max_k + 1, n))]).tolist()
    d = cu[-1]
    x = torch.randn((d + n, vocab), generator=g, device="cuda").bfloat16()
    x[::4, 100:200] = 9.0                                # ties
    x[1, 7] = math.nan
    stats = sga_lib.new_stats(d + n)
    sga_lib.sga_local_argmax(x, 0, vocab, org, stats)
    best = sga_lib.stat_ids(stats).cpu().numpy()
    of = [cu[i] + i + j for i in range(n) for j in range(cu[i + 1] - cu[i])]
    tokens = np.where(rng.random(d) < 0.7, best[of], rng.integers(0, org, d)).astype(np.int32)
    probs = torch.empty((d + n, vocab), device="cuda")
    sga_lib.sga_probs(x, org, probs, temperature=torch.zeros(d + n, device="cuda"))
    draft = None
    if with_draft_rows:
        draft = torch.zeros((d, vocab), device="cuda")
        draft[torch.arange(d), torch.from_numpy(tokens).long()] = 1.0
    got = gpu_verify(sga_lib, probs, draft, cu, tokens.tolist(), rng.random(d).tolist(),
                     rng.random(n).tolist(), max_k)
    dev = dict(dtype=torch.int32, device="cuda")
    exp = [torch.empty((n, max_k + 1), **dev)] + [torch.empty(n, **dev) for _ in range(3)]
    sga_lib.sga_greedy_verify(stats, 1, torch.tensor(cu, **dev), torch.tensor(tokens, **dev),
                              max_k, *exp)
    for a, b in zip(got, exp):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_emitted_tokens_have_the_targets_distribution(sga_lib):
    """200000 requests of one draft each over 8 ids: the first emitted token and,
    after an accepted draft, the second.  Five standard deviations of a count."""
    n, vocab = 200000, 8
    g = gen(9)
    p = torch.tensor([.3, .05, .2, .0, .15, .1, .15, .05], device="cuda")
    q = torch.tensor([.1, .3, .2, .1, .05, .05, .1, .1], device="cuda")
    bonus = torch.tensor([.02, .5, .08, .1, .1, .1, .05, .05], device="cuda")
    target = torch.stack([p, bonus]).repeat(n, 1)
    draft = q.repeat(n, 1)
    tokens = torch.multinomial(draft, 1, generator=g)[:, 0].to(torch.int32)
    dev = dict(dtype=torch.int32, device="cuda")
    outs = [torch.empty((n, 2), **dev)] + [torch.empty(n, **dev) for _ in range(3)]
    sga_lib.sga_sampled_verify(target, draft, torch.arange(n + 1, **dev), tokens,
                               torch.rand(n, generator=g, device="cuda"),
                               torch.rand(n, generator=g, device="cuda"), 1, *outs)
    first = torch.bincount(outs[0][:, 0].long(), minlength=vocab).double()
    sd = (n * p.double() * (1 - p.double())).sqrt()
    assert ((first - n * p.double()).abs() <= 5 * sd).all(), first
    both = outs[1] == 2
    m = int(both.sum())
    # an accepted draft has probability sum_j min(p_j, q_j)
    acc = float(torch.minimum(p, q).double().sum())
    assert abs(m - n * acc) <= 5 * math.sqrt(n * acc * (1 - acc))
    second = torch.bincount(outs[0][both, 1].long(), minlength=vocab).double()
    sd = (m * bonus.double() * (1 - bonus.double())).sqrt()
    assert ((second - m * bonus.double()).abs() <= 5 * sd).all(), second


@pytest.mark.gpu
def test_verify_rows_past_32_bits(sga_lib):
    """Row offsets of 2^31 elements and more in both matrices."""
    stride = (1 << 31) // 3 + 5
    vocab = 3000
    tb = torch.empty(4 * stride + vocab, device="cuda")
    target = torch.as_strided(tb, (5, vocab), (stride, 1))
    target.copy_(torch.softmax(torch.randn((5, vocab), generator=gen(10), device="cuda"), 1))
    db = torch.empty(3 * stride + vocab, device="cuda")
    draft = torch.as_strided(db, (4, vocab), (stride, 1))
    draft.copy_(torch.softmax(torch.randn((4, vocab), generator=gen(11), device="cuda"), 1))
    for au in ([0, 0, 0, 0], [0, 0, 0, 1], [0, 1, 0, 1]):
        c = (target, draft, [0, 4], [7, 2900, 1000, 1500], au, [0.6], 4)
        check_same(gpu_verify(sga_lib, *c), plain_verify(*host(c)))


@pytest.mark.gpu
def test_logits_to_tokens_on_a_stream_and_in_a_graph(sga_lib):
    """Both distributions and the verification as one captured step, replayed
    with other inputs in the same buffers, on a stream of its own."""
    n, k, vocab, org = 6, 3, 8000, 7990
    d = n * k
    g = gen(12)
    x = torch.empty((d + n, vocab), dtype=torch.bfloat16, device="cuda")
    y = torch.empty((d, vocab), dtype=torch.bfloat16, device="cuda")
    t, td = torch.empty(d + n, device="cuda"), torch.empty(d, device="cuda")
    p, q = torch.empty((d + n, vocab), device="cuda"), torch.empty((d, vocab), device="cuda")
    dev = dict(dtype=torch.int32, device="cuda")
    cu, tokens = torch.arange(0, d + 1, k, **dev), torch.zeros(d, **dev)
    au, su = torch.empty(d, device="cuda"), torch.empty(n, device="cuda")
    outs = [torch.empty((n, k + 1), **dev)] + [torch.empty(n, **dev) for _ in range(3)]
    row_of = torch.arange(d, device="cuda") + torch.arange(n, device="cuda").repeat_interleave(k)

    def fill(seed):
        h = gen(seed)
        y.normal_(0.0, 3.0, generator=h)
        x.normal_(0.0, 3.0, generator=h)
        x[row_of] = (y.float() + 0.3 * torch.randn(y.shape, generator=h, device="cuda")).bfloat16()
        t.uniform_(0.3, 1.2, generator=h)
        td.copy_(t[row_of])
        tokens.copy_(torch.multinomial(torch.softmax(y.float() / td[:, None], 1), 1,
                                       generator=h)[:, 0])
        au.uniform_(generator=h)
        su.uniform_(generator=h)

    def step():
        sga_lib.sga_probs(x, org, p, temperature=t)
        sga_lib.sga_probs(y, org, q, temperature=td)
        sga_lib.sga_sampled_verify(p, q, cu, tokens, au, su, k, *outs)

    def check():
        check_probs(p, x, org, t)
        exp = plain_verify(p.cpu().numpy(), q.cpu().numpy(), cu.tolist(), tokens.cpu().numpy(),
                           au.cpu().numpy(), su.cpu().numpy(), k)
        check_same(outs, exp)

    s = torch.cuda.Stream()
    fill(1)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for seed in (2, 3):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        check()
    del g


@pytest.mark.gpu
def test_two_graphs_at_once(sga_lib):
    """Two graphs of the same calls on other data, replayed on two streams at the
    same time, again and again: each has its own results every time."""
    steps = []
    for seed in (1, 2):
        g = gen(seed)
        n, k, vocab = 6, 3, 30011
        logits = torch.empty((n * (k + 1), vocab), device="cuda").normal_(0.0, 3.0, generator=g)
        target = torch.empty_like(logits)
        draft = torch.softmax(torch.randn((n * k, vocab), generator=g, device="cuda") * 3.0, 1)
        cu = torch.arange(n + 1, device="cuda", dtype=torch.int32) * k
        tokens = torch.randint(0, vocab, (n * k,), generator=g, device="cuda").to(torch.int32)
        au, su = (torch.rand(m, generator=g, device="cuda") for m in (n * k, n))
        out = [torch.empty(m, dtype=torch.int32, device="cuda") for m in (n * (k + 1), n, n, n)]

        def step(logits=logits, target=target, draft=draft, cu=cu, tokens=tokens, au=au, su=su,
                 out=out):
            sga_lib.sga_probs(logits, vocab, target)
            sga_lib.sga_sampled_verify(target, draft, cu, tokens, au, su, k, *out)

        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (target, *out)]
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=stream):
            for _ in range(20):
                step()
        for t in (target, *out):
            t.fill_(-7)
        steps.append((graph, stream, want, (target, *out), step))    # (step holds the inputs)
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, stream, *_ in steps:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for _, _, want, got, _ in steps:
            assert all(torch.equal(a, b) for a, b in zip(want, got))


# ------------------------------------------------------------------ refusals


def test_probs_validation(sga_lib):
    f = sga_lib.lib().sga_probs
    ok = dict(logits=FAKE, dtype=1, rows=4, ld=10, vocab=10, org=10, t=FAKE, out=FAKE, ldp=10)

    def call(**kw):
        a = dict(ok, **kw)
        return f(a["logits"], a["dtype"], a["rows"], a["ld"], a["vocab"], a["org"], a["t"],
                 a["out"], a["ldp"], None)

    assert call(dtype=2) == -5
    assert call(rows=-1) == -2 and call(rows=(1 << 28) + 1) == -2
    assert call(vocab=0) == -3 and call(ld=9) == -3 and call(ldp=9) == -3
    assert call(vocab=(1 << 24) + 1, ld=1 << 25, ldp=1 << 25) == -4
    assert call(org=0) == -4 and call(org=(1 << 24) + 1) == -4
    assert call(logits=None) == -1 and call(out=None) == -1
    assert call(out=ODD) == -6 and call(t=ODD) == -6 and call(dtype=0, logits=ODD) == -6
    assert call(rows=0, logits=None, out=None) == 0


def test_sampled_verify_validation(sga_lib):
    f = sga_lib.lib().sga_sampled_verify
    names = ("target", "rows", "ldt", "draft", "ldd", "vocab", "n", "cu", "tokens", "pre", "au",
             "su", "max_k", "o0", "o1", "o2", "o3")
    ok = dict(zip(names, (FAKE, 7, 10, FAKE, 10, 10, 3, FAKE, FAKE, FAKE, FAKE, FAKE, 3, FAKE,
                          FAKE, FAKE, FAKE)))

    def call(**kw):
        a = dict(ok, **kw)
        return f(*(a[n] for n in names), None)

    assert call(max_k=0) == -8 and call(max_k=16) == -8
    assert call(n=-1) == -2 and call(rows=2) == -2 and call(rows=(1 << 28) + 1) == -2
    assert call(vocab=0) == -4 and call(vocab=(1 << 24) + 1) == -4
    assert call(ldt=9) == -3 and call(ldd=9) == -3
    for name in ("target", "cu", "tokens", "au", "su", "o0", "o1", "o2", "o3"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: ODD}) == -6, name
    assert call(draft=ODD) == -6
    assert call(n=0, rows=0, target=None, cu=None) == 0


def test_binding_refuses_wrong_tensors(sga_lib):
    f32, i32, i64 = torch.float32, torch.int32, torch.int64

    def t(*shape, dtype=f32):
        return torch.zeros(shape, dtype=dtype)

    with pytest.raises(ValueError):                         # host memory
        sga_lib.sga_probs(t(2, 8), 8, t(2, 8))
    with pytest.raises(ValueError):                         # another shape
        sga_lib.sga_probs(t(2, 8), 8, t(2, 9))
    with pytest.raises(ValueError):                         # not fp32
        sga_lib.sga_probs(t(2, 8), 8, t(2, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError):                         # not unit stride
        sga_lib.sga_probs(t(2, 8), 8, t(8, 2).t())
    with pytest.raises(TypeError):
        sga_lib.sga_probs(t(2, 8, dtype=torch.float16), 8, t(2, 8))

    ok = dict(target_probs=t(5, 8), draft_probs=t(3, 8), cu_num_draft=t(3, dtype=i32),
              draft_tokens=t(3, dtype=i32), accept_u=t(3), sample_u=t(2), max_k=3,
              out_sampled=t(2, 4, dtype=i32), out_num_sampled=t(2, dtype=i32),
              out_num_rejected=t(2, dtype=i32), out_last=t(2, dtype=i32))
    for wrong in (dict(target_probs=t(1, 8)), dict(draft_probs=t(2, 8)), dict(draft_probs=t(3, 9)),
                  dict(target_probs=t(5, 8, dtype=torch.float64)), dict(cu_num_draft=t(0, dtype=i32)),
                  dict(in_prefill=t(2, dtype=i32)), dict()):
        with pytest.raises(ValueError):
            sga_lib.sga_sampled_verify(**dict(ok, **wrong))


@pytest.mark.gpu
def test_binding_refuses_wrong_sizes_on_the_device(sga_lib):
    f32, i32 = torch.float32, torch.int32

    def t(*shape, dtype=f32):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    ok = dict(target_probs=t(5, 8), draft_probs=t(3, 8),
              cu_num_draft=torch.tensor([0, 2, 3], dtype=i32, device="cuda"),
              draft_tokens=t(3, dtype=i32), accept_u=t(3), sample_u=t(2), max_k=3,
              out_sampled=t(2, 4, dtype=i32), out_num_sampled=t(2, dtype=i32),
              out_num_rejected=t(2, dtype=i32), out_last=t(2, dtype=i32))
    sga_lib.sga_sampled_verify(**ok)
    for wrong in (dict(draft_tokens=t(4, dtype=i32)), dict(draft_tokens=t(3, dtype=torch.int64)),
                  dict(accept_u=t(2)), dict(sample_u=t(3)), dict(out_sampled=t(2, 3, dtype=i32)),
                  dict(out_last=t(1, dtype=i32)), dict(accept_u=torch.zeros(3))):
        with pytest.raises(ValueError):
            sga_lib.sga_sampled_verify(**dict(ok, **wrong))
    with pytest.raises(ValueError):
        sga_lib.sga_probs(t(2, 8), 8, t(2, 8), temperature=t(3))
