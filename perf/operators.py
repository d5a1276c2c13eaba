"""Measured cases of the draft-head and log-probability operators.

Four operators: the matrix product with bias, activation and residual
(sga_linear), its gradient (sga_linear_grad), the log probability of a given
token with entropy and top alternatives (sga_token_logprobs, or
sga_local_logprobs per vocab shard and sga_logprob_reduce), and the gradient
of those with respect to the logits (sga_token_logprobs_grad).

`listed()` are the named cases, `draw(rng)` one more case of the same ranges;
`prepare` makes a case's inputs from a seed, `run` is one pass, in plain torch
operations or (own = True) through the library, `exact` the same outputs from
the definitions in 64 bits, `work` the bytes and operations of a pass.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
NEG = float("-inf")


def listed():
    return [
        # one token through a draft head's residual block, x + silu(W x + b)
        dict(name="linear_1", op="linear", M=1, N=4096, K=4096, act="silu", bias="f32",
             residual=True, train=False, pad=0),
        # a speculative batch (24 requests x 4 rows) through a wide layer
        dict(name="linear_96", op="linear", M=96, N=8192, K=4096, act="gelu_tanh", bias="bf16",
             residual=False, train=False, pad=64),
        # a mid-size batch on odd sizes, rows of a wider buffer
        dict(name="linear_odd", op="linear", M=333, N=1531, K=2056, act="gelu", bias="bf16",
             residual=True, train=False, pad=8),
        # a training batch, the pre-activation kept for the gradient
        dict(name="linear_4096", op="linear", M=4096, N=8192, K=4096, act="silu", bias="bf16",
             residual=False, train=True, pad=0),
        # gradient of the residual block on a short training batch
        dict(name="linear_grad_512", op="linear_grad", M=512, N=4096, K=4096, act="silu",
             bias="f32", pad=0),
        # odd sizes, the layer without an activation
        dict(name="linear_grad_odd", op="linear_grad", M=777, N=1001, K=1336, act="none",
             bias="bf16", pad=8),
        # a full training batch
        dict(name="linear_grad_4096", op="linear_grad", M=4096, N=4096, K=4096, act="gelu_tanh",
             bias="bf16", pad=0),
        # one decode row over the padded vocabulary, the 20 best alternatives
        dict(name="logprobs_1", op="logprobs", rows=1, vocab=152064, org=151936, dtype="bf16",
             k=20, shards=1, pad=0),
        # a verify batch on four vocab shards: per-shard statistics, then the reduce
        dict(name="logprobs_96_shards", op="logprobs", rows=96, vocab=200064, org=200064,
             dtype="bf16", k=5, shards=4, pad=0),
        # prompt log probabilities of a long batch
        dict(name="logprobs_4096", op="logprobs", rows=4096, vocab=202048, org=202048,
             dtype="bf16", k=5, shards=1, pad=0),
        # fine-tuning rows in fp32 on an odd vocabulary (every row at another alignment)
        dict(name="logprobs_grad_odd", op="logprobs_grad", rows=333, vocab=50257, org=50257,
             dtype="f32", k=0, pad=0),
        # distillation on a training batch: token, entropy and alternatives all carry gradients
        dict(name="logprobs_grad_4096", op="logprobs_grad", rows=4096, vocab=152064, org=151936,
             dtype="bf16", k=5, pad=0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    op = rng.choice(("linear", "linear_grad", "logprobs", "logprobs_grad"))
    if op in ("linear", "linear_grad"):
        while True:
            M = _log_int(rng, 1, 4096)
            N = _log_int(rng, 64, 16384)
            K = 8 * _log_int(rng, 8, 1024)
            most = 4096 * 8192 * 4096 // (1 if op == "linear" else 2)
            if M * N * K <= most and 3072 not in (M, N, K):
                break
        case = dict(op=op, M=M, N=N, K=K, act=rng.choice(ACTS), pad=rng.choice((0, 8, 72)),
                    bias=rng.choice(("none", "f32", "bf16")))
        if op == "linear":
            case.update(residual=rng.random() < 0.5, train=rng.random() < 0.3)
        return case
    while True:
        rows = _log_int(rng, 1, 4096)
        vocab = _log_int(rng, 1000, 202048)
        dtype = rng.choice(("bf16", "bf16", "f32"))
        if rows * vocab * (2 if dtype == "bf16" else 4) <= 4096 * 152064 * 2 and 3072 not in (
                rows, vocab):
            break
    org = vocab - rng.choice((0, 0, 1, 128))
    case = dict(op=op, rows=rows, vocab=vocab, org=org, dtype=dtype,
                k=rng.choice((0, 1, 5, 20)), pad=rng.choice((0, 0, 1, 64)))
    if op == "logprobs":
        case.update(shards=rng.choice((1, 1, 2, 4)))
    return case


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + 17)
    return g


def _normal(g, rows, cols, sigma, dtype, pad=0):
    """rows x cols draws of N(0, sigma^2), a column slice of a buffer `pad` wider."""
    t = torch.empty((rows, cols + pad), dtype=dtype, device="cuda")
    t.normal_(0.0, sigma, generator=g)
    return t[:, :cols]


def _linear_inputs(case, seed):
    g = _gen(seed)
    M, N, K, pad = case["M"], case["N"], case["K"], case["pad"]
    s = {"x": _normal(g, M, K, 1.0, torch.bfloat16, pad),
         "weight": _normal(g, N, K, K ** -0.5, torch.bfloat16)}
    if case["op"] == "linear":
        s["bias"] = None if case["bias"] == "none" else _normal(
            g, 1, N, 0.5, DTYPES[case["bias"]])[0]
        s["residual"] = _normal(g, M, N, 1.0, torch.bfloat16, pad) if case["residual"] else None
    else:
        s["grad_out"] = _normal(g, M, N, 1.0, torch.bfloat16, pad)
        s["preact"] = None if case["act"] == "none" else _normal(g, M, N, 1.2, torch.bfloat16, pad)
    return s


def _logits_inputs(case, seed):
    """Logits of N(0, 2.5^2) with one raised id per row; every eighth row keeps
    about 1 % of its ids (a grammar mask), row 13 none; a few rows have no
    token (-1)."""
    g = _gen(seed)
    rows, vocab, org = case["rows"], case["vocab"], case["org"]
    x = _normal(g, rows, vocab, 2.5, DTYPES[case["dtype"]], case["pad"])
    r = torch.arange(rows, device="cuda")
    best = torch.randint(0, org, (rows,), generator=g, device="cuda")
    lift = torch.rand(rows, generator=g, device="cuda") * 14.0
    x[r, best] = (x[r, best].float() + lift).to(x.dtype)
    for row in range(5, rows, 8):
        keep = torch.rand(vocab, generator=g, device="cuda") < 0.01
        x[row].masked_fill_(~keep, NEG)
    if rows > 13:
        x[13].fill_(NEG)
    other = torch.randint(0, org, (rows,), generator=g, device="cuda")
    pick = torch.rand(rows, generator=g, device="cuda")
    tokens = torch.where(pick < 0.7, best, other)
    tokens[9::64] = -1
    s = {"logits": x, "tokens": tokens.to(torch.int32)}
    if case["op"] == "logprobs_grad":
        # the statistics that the forward pass saved, and the upstream gradients
        xs = x[:, :org].float()
        m = xs.amax(1)
        lse = torch.logsumexp(xs, 1)
        p = torch.exp(xs - torch.where(m == NEG, 0.0, lse)[:, None])
        h = torch.where(m == NEG, 0.0, lse - (p * torch.where(xs == NEG, 0.0, xs)).sum(1))
        s["lse"], s["entropy"] = lse, h
        del xs, p
        s["grad_logprob"] = torch.randn(rows, generator=g, device="cuda")
        k = case["k"]
        s["grad_entropy"] = torch.randn(rows, generator=g, device="cuda") if k != 1 else None
        if k:
            first = torch.randint(0, org, (rows, 1), generator=g, device="cuda")
            step = org // k
            ids = (first + step * torch.arange(k, device="cuda")) % org
            s["top_ids"] = ids.to(torch.int32)
            s["grad_top"] = torch.randn((rows, k), generator=g, device="cuda")
        else:
            s["top_ids"] = s["grad_top"] = None
    return s


def _shards(case):
    """(start, width) of each vocab shard, the first ones one id wider."""
    base, extra = divmod(case["vocab"], case["shards"])
    out, start = [], 0
    for i in range(case["shards"]):
        out.append((start, base + (i < extra)))
        start += out[-1][1]
    return out


def prepare(case, seed):
    """Inputs, and the output buffers that a program keeps from call to call."""
    op = case["op"]
    out = {}
    if op == "linear":
        s = _linear_inputs(case, seed)
        out["y"] = torch.empty((case["M"], case["N"]), dtype=torch.bfloat16, device="cuda")
        out["z"] = torch.empty_like(out["y"]) if case["train"] else None
    elif op == "linear_grad":
        s = _linear_inputs(case, seed)
        out["grad_x"] = torch.empty((case["M"], case["K"]), dtype=torch.bfloat16, device="cuda")
        out["grad_weight"] = torch.empty((case["N"], case["K"]), dtype=torch.bfloat16,
                                         device="cuda")
        out["grad_bias"] = None if case["bias"] == "none" else torch.empty(
            case["N"], dtype=DTYPES[case["bias"]], device="cuda")
        out["ws"] = None
    elif op == "logprobs":
        s = _logits_inputs(case, seed)
        rows, k = case["rows"], case["k"]
        for name in ("logprob", "entropy", "lse"):
            out[name] = torch.empty(rows, dtype=torch.float32, device="cuda")
        out["top_ids"] = torch.empty((rows, k), dtype=torch.int32, device="cuda") if k else None
        out["top_logprobs"] = torch.empty((rows, k), dtype=torch.float32,
                                          device="cuda") if k else None
        n = case["shards"]
        out["parts"] = torch.empty((n, rows, 4), dtype=torch.float32, device="cuda")
        out["tops"] = torch.empty((n, rows, k, 2), dtype=torch.int32, device="cuda")
        s["shards"] = _shards(case)
    else:
        s = _logits_inputs(case, seed)
        out["grad"] = torch.empty((case["rows"], case["vocab"]), dtype=DTYPES[case["dtype"]],
                                  device="cuda")
    s["case"], s["out"] = case, out
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    op = s["case"]["op"]
    if own:
        return {"linear": _own_linear, "linear_grad": _own_linear_grad, "logprobs": _own_logprobs,
                "logprobs_grad": _own_logprobs_grad}[op](s)
    return {"linear": _plain_linear, "linear_grad": _plain_linear_grad,
            "logprobs": _plain_logprobs, "logprobs_grad": _plain_logprobs_grad}[op](s)


def _own_linear(s):
    import greedy_spec_decode_gb300 as sga
    c, o = s["case"], s["out"]
    sga.sga_linear(s["x"], s["weight"], o["y"], bias=s["bias"], act=ACTS.index(c["act"]),
                   residual=s["residual"], out_preact=o["z"])
    return {"y": o["y"], "z": o["z"]} if c["train"] else {"y": o["y"]}


def _own_linear_grad(s):
    import greedy_spec_decode_gb300 as sga
    c, o = s["case"], s["out"]
    if o["ws"] is None:
        o["ws"] = torch.empty(sga.sga_linear_grad_workspace(c["M"], c["N"], c["K"]),
                              dtype=torch.uint8, device="cuda")
    sga.sga_linear_grad(s["grad_out"], s["x"], s["weight"], o["ws"], act=ACTS.index(c["act"]),
                        preact=s["preact"], grad_x=o["grad_x"], grad_weight=o["grad_weight"],
                        grad_bias=o["grad_bias"])
    got = {"grad_x": o["grad_x"], "grad_weight": o["grad_weight"]}
    if o["grad_bias"] is not None:
        got["grad_bias"] = o["grad_bias"]
    return got


def _own_logprobs(s):
    import greedy_spec_decode_gb300 as sga
    c, o = s["case"], s["out"]
    if c["shards"] == 1:
        sga.sga_token_logprobs(s["logits"], c["org"], s["tokens"], o["logprob"], o["entropy"],
                               o["lse"], o["top_ids"], o["top_logprobs"])
    else:
        tops = o["tops"] if c["k"] else None
        for i, (start, width) in enumerate(s["shards"]):
            sga.sga_local_logprobs(s["logits"][:, start:start + width], start, width, c["org"],
                                   s["tokens"], o["parts"][i], None if tops is None else tops[i])
        sga.sga_logprob_reduce(o["parts"], tops, c["shards"], s["tokens"], o["logprob"],
                               o["entropy"], o["lse"], o["top_ids"], o["top_logprobs"])
    got = {"logprob": o["logprob"], "entropy": o["entropy"], "lse": o["lse"]}
    if c["k"]:
        got.update(top_ids=o["top_ids"], top_logprobs=o["top_logprobs"])
    return got


def _own_logprobs_grad(s):
    import greedy_spec_decode_gb300 as sga
    c, o = s["case"], s["out"]
    sga.sga_token_logprobs_grad(s["logits"], 0, c["org"], s["tokens"], s["lse"], s["entropy"],
                                s["grad_logprob"], o["grad"], grad_entropy=s["grad_entropy"],
                                top_ids=s["top_ids"], grad_top=s["grad_top"])
    return {"grad": o["grad"]}


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return torch.where(z > 0, 1.0, 0.0)
    if act == "silu":
        q = 1.0 / (1.0 + torch.exp(-z))
        return q * (1.0 + z * (1.0 - q))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(
            -0.5 * z * z) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)


def _plain_linear(s):
    c = s["case"]
    z = s["x"].float() @ s["weight"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    y = y.to(torch.bfloat16)
    return {"y": y, "z": z.to(torch.bfloat16)} if c["train"] else {"y": y}


def _plain_linear_grad(s):
    c = s["case"]
    dz = s["grad_out"].float()
    if c["act"] != "none":
        dz = dz * _act_grad(s["preact"].float(), c["act"])
    got = {"grad_x": (dz @ s["weight"].float()).to(torch.bfloat16),
           "grad_weight": (dz.t() @ s["x"].float()).to(torch.bfloat16)}
    if c["bias"] != "none":
        got["grad_bias"] = dz.sum(0).to(DTYPES[c["bias"]])
    return got


def _plain_logprobs(s):
    """A row with no value above -inf has log-sum-exp -inf, entropy 0 and every
    log probability -inf; a row without a token has log probability 0.  The
    alternatives come in descending order, equal values by ascending id."""
    c = s["case"]
    x = s["logits"][:, :c["org"]].float()
    m = x.amax(1)
    empty = m == NEG
    e = torch.exp(x - torch.where(empty, 0.0, m)[:, None])
    total = e.sum(1)
    lse = torch.where(empty, NEG, m + torch.log(total))
    mean = (e * torch.where(x == NEG, 0.0, x - m[:, None])).sum(1) / total
    got = {"entropy": torch.where(empty, 0.0, torch.log(total) - mean), "lse": lse}
    del e
    t = s["tokens"].long()
    xt = torch.gather(x, 1, t.clamp(min=0)[:, None])[:, 0]
    got["logprob"] = torch.where(t < 0, 0.0, torch.where(xt == NEG, NEG, xt - lse))
    if c["k"]:
        # one 64-bit key per id: the value's order above, the lower id first below
        b = (x + 0.0).view(torch.int32)
        b = b ^ ((b >> 31) & 0x7fffffff)
        ids = torch.arange(c["org"], device="cuda")
        key = (b.long() << 32) | (0x7fffffff - ids)
        del b
        top = 0x7fffffff - (torch.topk(key, c["k"], dim=1).values & 0xffffffff)
        v = torch.gather(x, 1, top)
        got["top_ids"] = top.to(torch.int32)
        got["top_logprobs"] = torch.where(v == NEG, NEG, v - lse[:, None])
    return {n: got[n] for n in ("logprob", "entropy", "lse", "top_ids", "top_logprobs")
            if n in got}


def _plain_logprobs_grad(s):
    c = s["case"]
    org = c["org"]
    x = s["logits"][:, :org].float()
    t = s["tokens"].long()
    gl = torch.where(t < 0, 0.0, s["grad_logprob"])
    total = gl if s["grad_top"] is None else gl + s["grad_top"].sum(1)
    none = x == NEG
    lp = torch.where(none, 0.0, x - s["lse"][:, None])
    p = torch.where(none, 0.0, torch.exp(lp))
    d = -total[:, None] * p
    if s["grad_entropy"] is not None:
        d = d - s["grad_entropy"][:, None] * p * (lp + s["entropy"][:, None])
    del p, lp
    live = s["lse"] > NEG
    d.scatter_add_(1, t.clamp(min=0)[:, None], torch.where(live, gl, 0.0)[:, None])
    if s["grad_top"] is not None:
        d.scatter_add_(1, s["top_ids"].long(), torch.where(live[:, None], s["grad_top"], 0.0))
    grad = torch.zeros((c["rows"], c["vocab"]), dtype=s["logits"].dtype, device="cuda")
    grad[:, :org] = d.to(grad.dtype)
    return {"grad": grad}


# ------------------------------------------------------------------ work


def work(case):
    op = case["op"]
    if op in ("linear", "linear_grad"):
        M, N, K = case["M"], case["N"], case["K"]
        bias = {"none": 0, "f32": 4, "bf16": 2}[case["bias"]] * N
        if op == "linear":
            outs = M * N * (1 + case["residual"] + case["train"])
            return {"bytes": 2 * (M * K + N * K + outs) + bias, "flops": 2 * M * N * K}
        ins = M * N * (1 if case["act"] == "none" else 2)
        return {"bytes": 2 * (ins + 2 * M * K + 2 * N * K) + bias, "flops": 4 * M * N * K}
    elt = 2 if case["dtype"] == "bf16" else 4
    rows, k, org = case["rows"], case["k"], case["org"]
    if op == "logprobs":
        return {"bytes": rows * (elt * org + 4 + 12 + 8 * k), "flops": 5 * rows * org}
    small = rows * (4 + 8 + 4 + (4 if k != 1 else 0) + 8 * k)
    return {"bytes": rows * elt * (org + case["vocab"]) + small, "flops": 6 * rows * org}


# ------------------------------------------------------------------ 64 bits


def _exact_act(z, act):
    """(value, derivative) in 64 bits."""
    one = torch.ones_like(z)
    if act == "none":
        return z, one
    if act == "relu":
        return z.clamp(min=0.0), (z > 0).double()
    if act == "silu":
        q = torch.sigmoid(z)
        return z * q, q + z * q * (1.0 - q)
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z ** 2 / 2.0) / math.sqrt(2.0 * math.pi)
    a = math.sqrt(2.0 / math.pi)
    q = torch.sigmoid(2.0 * a * (z + 0.044715 * z ** 3))     # (1 + tanh u) / 2 = sigmoid(2 u)
    return z * q, q + 2.0 * z * q * (1.0 - q) * a * (1.0 + 0.134145 * z ** 2)


def _exact_linear(case, seed):
    s = _linear_inputs(case, seed)
    w, x = s["weight"].double(), s["x"].double()
    if case["op"] == "linear_grad":
        dz = s["grad_out"].double()
        if s["preact"] is not None:
            dz = dz * _exact_act(s["preact"].double(), case["act"])[1]
        got = {"grad_x": torch.matmul(dz, w), "grad_weight": torch.matmul(dz.T, x)}
        if case["bias"] != "none":
            got["grad_bias"] = dz.sum(0)
        return got
    z = torch.matmul(x, w.T)
    if s["bias"] is not None:
        z += s["bias"].double()
    y = _exact_act(z, case["act"])[0]
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return {"y": y, "z": z} if case["train"] else {"y": y}


def _exact_logprobs_rows(x, tokens, k):
    """Some rows, in 64 bits: the definitions term by term."""
    live = (x > NEG).any(1)
    lse = torch.logsumexp(x, 1)
    lp = x - torch.where(live, lse, 0.0)[:, None]
    ent = -(torch.exp(lp) * lp.masked_fill(lp == NEG, 0.0)).sum(1)
    at = torch.gather(lp, 1, tokens.clamp(min=0)[:, None])[:, 0].masked_fill(tokens < 0, 0.0)
    top = torch.topk(lp, k, dim=1).values if k else None
    return at, ent, lse, top


def _exact_grad_rows(x, s, a, b):
    org = x.shape[1]
    lse, h = s["lse"][a:b].double(), s["entropy"][a:b].double()
    live = lse > NEG
    lp = x - torch.where(live, lse, 0.0)[:, None]
    p = torch.exp(lp)
    onehot_sum = torch.zeros_like(x)      # the upstream gradient of each id's log probability
    t = s["tokens"][a:b].long()
    gl = s["grad_logprob"][a:b].double() * (t >= 0)
    onehot_sum.scatter_add_(1, t.clamp(min=0)[:, None], gl[:, None])
    if s["grad_top"] is not None:
        onehot_sum.scatter_add_(1, s["top_ids"][a:b].long(), s["grad_top"][a:b].double())
    d = onehot_sum - p * onehot_sum.sum(1, keepdim=True)
    if s["grad_entropy"] is not None:
        plogp = p * lp.masked_fill(lp == NEG, 0.0)
        d = d - s["grad_entropy"][a:b].double()[:, None] * (plogp + p * h[:, None])
    return d * live[:, None]


def exact(case, seed):
    if case["op"] in ("linear", "linear_grad"):
        return _exact_linear(case, seed)
    s = _logits_inputs(case, seed)
    rows, org, k = case["rows"], case["org"], case["k"]
    cuts = range(0, rows, 256)            # rows in blocks: 64-bit logits of all would be 5 GB
    if case["op"] == "logprobs_grad":
        d = torch.zeros((rows, case["vocab"]), dtype=torch.float64, device="cuda")
        for a in cuts:
            b = min(rows, a + 256)
            d[a:b, :org] = _exact_grad_rows(s["logits"][a:b, :org].double(), s, a, b)
        return {"grad": d}
    parts = [_exact_logprobs_rows(s["logits"][a:a + 256, :org].double(),
                                  s["tokens"][a:a + 256].long(), k) for a in cuts]
    got = {n: torch.cat([p[i] for p in parts]) for i, n in enumerate(("logprob", "entropy", "lse"))}
    if k:
        got["top_ids"] = None
        got["top_logprobs"] = torch.cat([p[3] for p in parts])
    return got
