"""Measured cases of the sampled-verification and distillation operators.

Four operators: the probabilities of logits rows at a temperature (sga_probs),
the verification of drafted tokens by rejection sampling against those
probabilities (sga_sampled_verify), the divergence of a draft model from a
teacher's top logits, with or without its gradient in the same pass
(sga_distill), and that gradient from the saved sums (sga_distill_grad).

`listed()` are the named cases, `draw(rng)` one more case of the same ranges;
`prepare` makes a case's inputs from a seed, `run` is one pass, in plain torch
operations or (own = True) through the library, `exact` the same outputs from
the definitions in 64 bits, `work` the bytes and operations of a pass.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
NEG = float("-inf")
UNIT = 2.0 ** 38          # probabilities are summed in units of 2^-38


def listed():
    return [
        # sampling one decode row of a padded vocabulary
        dict(name="probs_1", op="probs", rows=1, vocab=152064, org=151936, dtype="bf16",
             temperature="row", pad=0),
        # fp32 logits of an odd vocabulary, rows of a wider buffer, temperature 1
        dict(name="probs_odd", op="probs", rows=333, vocab=50257, org=50257, dtype="f32",
             temperature="none", pad=1),
        # every target row of 512 requests with three drafts, greedy ones (temperature 0) among
        # them
        dict(name="probs_2048", op="probs", rows=2048, vocab=202048, org=202048, dtype="bf16",
             temperature="mixed", pad=0),
        # one request with three drafts
        dict(name="verify_1", op="verify", reqs=1, max_k=3, vocab=152064, drafts="probs",
             ragged=False, pad=0),
        # a speculative batch
        dict(name="verify_24", op="verify", reqs=24, max_k=3, vocab=200064, drafts="probs",
             ragged=False, pad=0),
        # drafts without probabilities (proposed greedily or by n-grams), 0 to 15 a request,
        # some requests still in prefill, odd vocabulary
        dict(name="verify_ragged", op="verify", reqs=37, max_k=15, vocab=50257, drafts="tokens",
             ragged=True, pad=3),
        # a large batch
        dict(name="verify_512", op="verify", reqs=512, max_k=3, vocab=152064, drafts="probs",
             ragged=False, pad=0),
        # a validation batch: the loss alone
        dict(name="distill_256", op="distill", rows=256, vocab=32000, org=32000, dtype="bf16",
             k=20, rest=True, temperature=1.0, grad=False, pad=0),
        # a training batch: loss and gradient at once
        dict(name="distill_4096", op="distill", rows=4096, vocab=152064, org=151936, dtype="bf16",
             k=20, rest=True, temperature=1.0, grad=True, pad=0),
        # fp32 logits of an odd vocabulary, a softened teacher's list by itself
        dict(name="distill_odd", op="distill", rows=333, vocab=50257, org=50257, dtype="f32",
             k=64, rest=False, temperature=2.0, grad=True, pad=1),
        # the backward call of a step whose loss is combined with others
        dict(name="distill_grad_96", op="distill_grad", rows=96, vocab=32000, org=32000,
             dtype="bf16", k=5, rest=True, temperature=1.0, grad=True, pad=0),
        # the same of a full batch, softened
        dict(name="distill_grad_2048", op="distill_grad", rows=2048, vocab=200064, org=200064,
             dtype="bf16", k=32, rest=True, temperature=1.5, grad=True, pad=64),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    op = rng.choice(("probs", "verify", "distill", "distill_grad"))
    vocab = _log_int(rng, 1000, 202048)
    if op == "verify":
        max_k = rng.choice((1, 2, 3, 5, 8, 15))
        most = min(512, 512 * 152064 // vocab, 512 * 7 * 152064 // ((2 * max_k + 1) * vocab))
        return dict(op=op, reqs=_log_int(rng, 1, max(1, most)), max_k=max_k, vocab=vocab,
                    drafts=rng.choice(("probs", "probs", "tokens")), ragged=rng.random() < 0.5,
                    pad=rng.choice((0, 0, 1, 64)))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    most = (2048 * 202048 if op == "probs" else 4096 * 152064) // (vocab * (
        1 if dtype == "bf16" else 2))
    case = dict(op=op, rows=_log_int(rng, 1, min(4096, most)), vocab=vocab,
                org=vocab - rng.choice((0, 0, 1, 128)), dtype=dtype, pad=rng.choice((0, 0, 1, 64)))
    if op == "probs":
        case.update(temperature=rng.choice(("none", "row", "mixed")))
    else:
        case.update(k=rng.choice((1, 5, 20, 32, 64)), rest=rng.random() < 0.6,
                    temperature=rng.choice((1.0, 1.0, 0.7, 2.0)),
                    grad=op == "distill_grad" or rng.random() < 0.6)
    return case


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + 29)
    return g


def _logits(g, rows, vocab, dtype, pad):
    """N(0, 2.5^2) logits with one raised id a row, a column slice of a buffer
    `pad` wider."""
    x = torch.empty((rows, vocab + pad), dtype=dtype, device="cuda")
    x.normal_(0.0, 2.5, generator=g)
    x = x[:, :vocab]
    r = torch.arange(rows, device="cuda")
    best = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    lift = torch.rand(rows, generator=g, device="cuda") * 14.0
    x[r, best] = (x[r, best].float() + lift).to(dtype)
    return x


def _probs_inputs(case, seed):
    """Every eighth row keeps about 1 % of its ids (a grammar mask), row 13
    none (it then has no distribution)."""
    g = _gen(seed)
    rows, vocab = case["rows"], case["vocab"]
    x = _logits(g, rows, vocab, DTYPES[case["dtype"]], case["pad"])
    for row in range(5, rows, 8):
        keep = torch.rand(vocab, generator=g, device="cuda") < 0.01
        x[row].masked_fill_(~keep, NEG)
    if rows > 13:
        x[13].fill_(NEG)
    t = None
    if case["temperature"] != "none":
        t = 0.3 + 1.2 * torch.rand(rows, generator=g, device="cuda")
        if case["temperature"] == "mixed":
            t[torch.rand(rows, generator=g, device="cuda") < 0.3] = 0.0
    return {"logits": x, "temperature": t}


def _verify_inputs(case, seed):
    """The target's distribution of a draft row is the draft's, moved: about
    three in four drafts are accepted; every eighth target row is cut to some
    of its ids (top-p)."""
    g = _gen(seed)
    n, vocab, pad = case["reqs"], case["vocab"], case["pad"]
    if case["ragged"]:
        h = torch.Generator()
        h.manual_seed(int(seed) + 5)
        counts = torch.randint(0, case["max_k"] + 1, (n,), generator=h)
    else:
        counts = torch.full((n,), case["max_k"])
    cu = torch.zeros(n + 1, dtype=torch.int64)
    cu[1:] = counts.cumsum(0)
    drafts = int(cu[-1])
    cu = cu.to(device="cuda", dtype=torch.int32)
    rows = drafts + n
    target = torch.empty((rows, vocab + pad), device="cuda")[:, :vocab]
    draft = torch.empty((drafts, vocab + pad), device="cuda")[:, :vocab]
    tokens = torch.zeros(drafts, dtype=torch.int32, device="cuda")
    # the draft row of each target row, -1 for a bonus row
    of = torch.full((rows,), -1, device="cuda")
    req = torch.repeat_interleave(torch.arange(n), counts).cuda()
    of[torch.arange(drafts, device="cuda") + req] = torch.arange(drafts, device="cuda")
    for a in range(0, rows, 256):
        b = min(rows, a + 256)
        x = _logits(g, b - a, vocab, torch.float32, 0)
        y = x + 0.5 * torch.randn(x.shape, generator=g, device="cuda")
        cut = torch.arange(a, b, device="cuda") % 8 == 3
        y.masked_fill_(cut[:, None] & (y < 2.0), NEG)
        target[a:b] = torch.softmax(y, 1)
        d = of[a:b]
        sel = d >= 0
        draft[d[sel]] = torch.softmax(x[sel], 1)
        race = torch.empty_like(x).exponential_(generator=g)
        tokens[d[sel]] = (x - torch.log(race)).argmax(1)[sel].to(torch.int32)
    s = {"target": target, "draft": draft if case["drafts"] == "probs" else None, "cu": cu,
         "tokens": tokens, "accept_u": torch.rand(drafts, generator=g, device="cuda"),
         "sample_u": torch.rand(n, generator=g, device="cuda"), "prefill": None}
    if case["ragged"]:
        s["prefill"] = torch.rand(n, generator=g, device="cuda") < 0.1
    return s


def _distill_inputs(case, seed):
    """A teacher's list holds most of its probability, on ids that the student
    partly raises too; every sixteenth list is shorter (-1), every 32nd row has
    none (prompt tokens); every eighth row of the student is masked outside of
    the list."""
    g = _gen(seed)
    rows, vocab, org, k = case["rows"], case["vocab"], case["org"], case["k"]
    x = _logits(g, rows, vocab, DTYPES[case["dtype"]], case["pad"])
    first = torch.randint(0, org, (rows, 1), generator=g, device="cuda")
    ids = (first + org // k * torch.arange(k, device="cuda")) % org
    z = torch.randn((rows, k), generator=g, device="cuda") * 3.0 + 12.0
    z = z.sort(dim=1, descending=True).values
    for row in range(5, rows, 8):
        keep = torch.rand(vocab, generator=g, device="cuda") < 0.5
        keep[ids[row]] = True
        x[row].masked_fill_(~keep, NEG)
    at = torch.gather(x, 1, ids).float()
    x.scatter_(1, ids, (at + 0.7 * z).to(x.dtype))
    ids = ids.to(torch.int32)
    ids[7::16, k // 2:] = -1
    ids[9::32] = -1
    t = case["temperature"]
    s = {"logits": x, "ids": ids, "teacher": z, "teacher_lse": None,
         "grad_loss": torch.randn(rows, generator=g, device="cuda") / rows}
    if case["rest"]:
        s["teacher_lse"] = torch.logsumexp(z / t, 1) + 0.3 * torch.rand(
            rows, generator=g, device="cuda")
    if case["op"] == "distill_grad":
        # what the forward pass saved
        s["lse"], s["lse_rest"] = _lse_pair(s, case)
    return s


def prepare(case, seed):
    """Inputs, and the output buffers that a program keeps from call to call."""
    op = case["op"]
    out = {}
    if op == "probs":
        s = _probs_inputs(case, seed)
        out["probs"] = torch.empty((case["rows"], case["vocab"]), device="cuda")
    elif op == "verify":
        s = _verify_inputs(case, seed)
        n = case["reqs"]
        out["sampled"] = torch.empty((n, case["max_k"] + 1), dtype=torch.int32, device="cuda")
        for name in ("num_sampled", "num_rejected", "last"):
            out[name] = torch.empty(n, dtype=torch.int32, device="cuda")
    else:
        s = _distill_inputs(case, seed)
        rows = case["rows"]
        if op == "distill":
            for name in ("loss", "lse", "lse_rest"):
                out[name] = torch.empty(rows, device="cuda")
        if case["grad"]:
            out["grad"] = torch.empty((rows, case["vocab"]), dtype=DTYPES[case["dtype"]],
                                      device="cuda")
    s["case"], s["out"] = case, out
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    op = s["case"]["op"]
    if own:
        return {"probs": _own_probs, "verify": _own_verify, "distill": _own_distill,
                "distill_grad": _own_distill_grad}[op](s)
    return {"probs": _plain_probs, "verify": _plain_verify, "distill": _plain_distill,
            "distill_grad": _plain_distill_grad}[op](s)


def _own_probs(s):
    import greedy_spec_decode_gb300 as sga
    sga.sga_probs(s["logits"], s["case"]["org"], s["out"]["probs"], temperature=s["temperature"])
    return {"probs": s["out"]["probs"]}


def _own_verify(s):
    import greedy_spec_decode_gb300 as sga
    o = s["out"]
    sga.sga_sampled_verify(s["target"], s["draft"], s["cu"], s["tokens"], s["accept_u"],
                           s["sample_u"], s["case"]["max_k"], o["sampled"], o["num_sampled"],
                           o["num_rejected"], o["last"], in_prefill=s["prefill"])
    return dict(o)


def _own_distill(s):
    import greedy_spec_decode_gb300 as sga
    c, o = s["case"], s["out"]
    sga.sga_distill(s["logits"], c["org"], s["ids"], s["teacher"], o["loss"],
                    teacher_lse=s["teacher_lse"], temperature=c["temperature"], out_lse=o["lse"],
                    out_lse_rest=o["lse_rest"], grad_loss=s["grad_loss"] if c["grad"] else None,
                    out_grad=o["grad"] if c["grad"] else None)
    return dict(o)


def _own_distill_grad(s):
    import greedy_spec_decode_gb300 as sga
    c, o = s["case"], s["out"]
    sga.sga_distill_grad(s["logits"], c["org"], s["ids"], s["teacher"], s["lse"], s["lse_rest"],
                         o["grad"], teacher_lse=s["teacher_lse"], temperature=c["temperature"],
                         grad_loss=s["grad_loss"])
    return {"grad": o["grad"]}


def _plain_probs(s):
    """Columns past org_vocab are 0, and so is a row with nothing above -inf;
    temperature 0 is a one at the row's best id (the lowest of equal ones; id 0
    in a row with nothing above -inf)."""
    c, t = s["case"], s["temperature"]
    x = s["logits"][:, :c["org"]].float()
    m = x.amax(1, keepdim=True)
    d = x - torch.where(m == NEG, 0.0, m)
    if t is not None:
        d = d / torch.where(t > 0, t, 1.0)[:, None]
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    p = e / torch.where(total == 0, 1.0, total)
    if t is not None:
        ids = torch.arange(c["org"], device="cuda")
        best = torch.where(x == m, ids, c["org"]).amin(1)
        p = torch.where((t > 0)[:, None], p, (ids == best[:, None]).float())
    out = torch.zeros((c["rows"], c["vocab"]), device="cuda")
    out[:, :c["org"]] = p
    return {"probs": out}


def _plain_verify(s):
    """Draft t of a row with probabilities p, q and uniform u is accepted when
    u q(t) < p(t), up to the first that is not; there a token is drawn from
    max(p - q, 0) (from p where that is 0 everywhere), after all drafts from
    the bonus row: the first id whose cumulative sum passes u times the total,
    sums being of whole units of 2^-38."""
    c, cu = s["case"], s["cu"].long()
    n, width = c["reqs"], c["max_k"] + 1
    k = cu[1:] - cu[:-1]
    j = torch.arange(width, device="cuda")
    is_draft = j < k[:, None]
    if s["tokens"].numel():
        at = torch.where(is_draft, cu[:-1, None] + j, 0)
        row = torch.where(is_draft, cu[:-1, None] + torch.arange(n, device="cuda")[:, None] + j, 0)
        t = s["tokens"][at].long()
        p = s["target"][row, t]
        q = s["draft"][at, t] if s["draft"] is not None else torch.ones_like(p)
        fails = is_draft & ~(s["accept_u"][at] * q < p)
        a = torch.where(fails, j, width).amin(1).minimum(k)
    else:
        at, t = torch.zeros((n, width), dtype=torch.long, device="cuda"), None
        a = torch.zeros_like(k)
    r = torch.arange(n, device="cuda")
    p = s["target"][cu[:-1] + r + a]
    w = p
    if s["tokens"].numel():
        rejected = a < k
        d = at[r, a.clamp(max=c["max_k"])]
        if s["draft"] is not None:
            q = s["draft"][d]
        else:
            q = torch.zeros_like(p)
            q[r, t[r, a.clamp(max=c["max_k"])]] = 1.0
        w = torch.where(rejected[:, None], p - q, p)
    w = torch.round(w.clamp(0.0, 1.0) * UNIT).long()
    nothing = w.sum(1, keepdim=True) == 0
    w = torch.where(nothing, torch.round(p.clamp(0.0, 1.0) * UNIT).long(), w)
    cum = w.cumsum(1)
    total = cum[:, -1]
    # in 64 bits: the sums have up to 62
    edge = torch.floor(s["sample_u"].double() * total.double()).long().minimum(total - 1)
    last = torch.searchsorted(cum, edge[:, None], right=True)[:, 0]
    last = torch.where(total == 0, -1, last).to(torch.int32)
    sampled = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    if s["tokens"].numel():
        sampled = torch.where(j < a[:, None], t.to(torch.int32), sampled)
    sampled[r, a] = last
    got = {"sampled": sampled, "num_sampled": (a + 1).to(torch.int32),
           "num_rejected": (k - a).to(torch.int32), "last": last}
    if s["prefill"] is not None:
        for name, empty in (("sampled", -1), ("num_sampled", 0), ("num_rejected", 0),
                            ("last", -1)):
            off = s["prefill"][:, None] if name == "sampled" else s["prefill"]
            got[name] = torch.where(off, empty, got[name]).to(torch.int32)
    return got


def _listed_mask(s, org):
    """True at the ids of each row's list."""
    hit = torch.zeros((s["ids"].size(0), org + 1), dtype=torch.bool, device="cuda")
    ids = s["ids"].long()
    hit.scatter_(1, torch.where(ids < 0, org, ids), True)
    return hit[:, :org]


def _lse_of(x):
    m = x.amax(1)
    none = m == NEG
    total = torch.exp(x - torch.where(none, 0.0, m)[:, None]).sum(1)
    return torch.where(none, NEG, m + torch.log(total))


def _lse_pair(s, c):
    """log-sum-exp of logits / temperature, of all ids and of those off the list."""
    x = s["logits"][:, :c["org"]].float() / c["temperature"]
    return _lse_of(x), _lse_of(torch.where(_listed_mask(s, c["org"]), NEG, x))


def _teacher(s, c, lse_rest):
    """The list's probabilities and the rest's, in 64 bits (the rest is 1 less
    a sum near 1); a list without ids has none."""
    z = s["teacher"].double() / c["temperature"]
    z = torch.where(s["ids"] < 0, NEG, z)
    if s["teacher_lse"] is None:
        lse = torch.logsumexp(z, 1)
    else:
        lse = s["teacher_lse"].double()
    live = (s["ids"] >= 0).any(1)
    logp = torch.where(live[:, None], z - lse[:, None], NEG)
    p = torch.exp(logp)
    rest = torch.zeros_like(lse)
    if s["teacher_lse"] is not None:
        rest = (1.0 - p.sum(1)).clamp(min=0.0)
        rest = torch.where(live & (lse_rest > NEG), rest, 0.0)
    return p, logp, rest


def _plain_grad(s, lse, lse_rest):
    c = s["case"]
    x = s["logits"][:, :c["org"]].float() / c["temperature"]
    p, _, rest = _teacher(s, c, lse_rest)
    total = (p.sum(1) + rest).float()
    d = total[:, None] * torch.exp(x - lse[:, None])
    if s["teacher_lse"] is not None:
        off = torch.exp(x - torch.where(lse_rest == NEG, 0.0, lse_rest)[:, None])
        off = rest.float()[:, None] * off
        d = d - torch.where(_listed_mask(s, c["org"]), 0.0, off)
        del off
    d.scatter_add_(1, s["ids"].clamp(min=0).long(), -torch.where(s["ids"] < 0, 0.0, p).float())
    d *= (s["grad_loss"] / c["temperature"])[:, None]
    grad = torch.zeros((c["rows"], c["vocab"]), dtype=s["logits"].dtype, device="cuda")
    grad[:, :c["org"]] = d.to(grad.dtype)
    return grad


def _plain_distill(s):
    c = s["case"]
    lse, lse_rest = _lse_pair(s, c)
    p, logp, rest = _teacher(s, c, lse_rest)
    at = torch.gather(s["logits"], 1, s["ids"].clamp(min=0).long()).double() / c["temperature"]
    term = p * (logp - (at - lse[:, None]))
    loss = torch.where(p > 0, term, 0.0).sum(1)
    term = rest * (torch.log(rest) - (lse_rest - lse))
    loss = loss + torch.where(rest > 0, term, 0.0)
    got = {"loss": loss.float(), "lse": lse, "lse_rest": lse_rest}
    if c["grad"]:
        got["grad"] = _plain_grad(s, lse, lse_rest)
    return got


def _plain_distill_grad(s):
    return {"grad": _plain_grad(s, s["lse"], s["lse_rest"])}


# ------------------------------------------------------------------ work


def work(case):
    op, vocab = case["op"], case["vocab"]
    if op == "verify":
        # the row that the last token is drawn from, and in about half of the requests
        # (those with a rejection) the draft's row beside it
        rows = case["reqs"] * (1.5 if case["drafts"] == "probs" else 1.0)
        return {"bytes": int(rows * vocab * 4), "flops": int(3 * rows * vocab)}
    rows, org = case["rows"], case["org"]
    elt = 2 if case["dtype"] == "bf16" else 4
    if op == "probs":
        return {"bytes": rows * (elt * org + 4 * vocab), "flops": 4 * rows * org}
    small = rows * (8 * case["k"] + (4 if case["rest"] else 0) + 12)
    if not case["grad"]:
        return {"bytes": rows * elt * org + small, "flops": 4 * rows * org}
    return {"bytes": rows * elt * (org + vocab) + small,
            "flops": (4 if op == "distill_grad" else 8) * rows * org}


# ------------------------------------------------------------------ 64 bits


def _exact_probs(case, seed):
    s = _probs_inputs(case, seed)
    out = torch.zeros((case["rows"], case["vocab"]), dtype=torch.float64, device="cuda")
    for a in range(0, case["rows"], 256):
        x = s["logits"][a:a + 256, :case["org"]].double()
        t = torch.ones(x.size(0), dtype=torch.float64, device="cuda")
        if s["temperature"] is not None:
            t = s["temperature"][a:a + 256].double()
        p = torch.softmax(x / t.masked_fill(t == 0, 1.0)[:, None], 1)
        p[~(x > NEG).any(1)] = 0.0
        for row in (t == 0).nonzero()[:, 0].tolist():
            p[row] = 0.0
            p[row, int((x[row] == x[row].max()).nonzero()[0, 0])] = 1.0
        out[a:a + 256, :case["org"]] = p
    return {"probs": out}


def _exact_verify(case, seed):
    """Request by request, from the definition."""
    s = _verify_inputs(case, seed)
    n, width = case["reqs"], case["max_k"] + 1
    cu, tokens = s["cu"].tolist(), s["tokens"].tolist()
    sampled = torch.full((n, width), -1, dtype=torch.int32)
    num = torch.zeros(n, dtype=torch.int32)
    rejected, last = torch.zeros_like(num), torch.full_like(num, -1)
    drafts = len(tokens)
    req = torch.repeat_interleave(torch.arange(n), torch.tensor(cu).diff()).cuda()
    t = s["tokens"].long()
    p_t = s["target"][torch.arange(drafts, device="cuda") + req, t]
    q_t = torch.ones_like(p_t)
    if s["draft"] is not None:
        q_t = s["draft"][torch.arange(drafts, device="cuda"), t]
    ok = (s["accept_u"] * q_t < p_t).tolist()
    off = s["prefill"].tolist() if s["prefill"] is not None else [False] * n
    u = s["sample_u"].tolist()
    for i in range(n):
        if off[i]:
            continue
        a = 0
        while a < cu[i + 1] - cu[i] and ok[cu[i] + a]:
            a += 1
        p = s["target"][cu[i] + i + a]
        weights = [p]
        if a < cu[i + 1] - cu[i]:
            q = torch.zeros_like(p)
            if s["draft"] is not None:
                q = s["draft"][cu[i] + a]
            else:
                q[tokens[cu[i] + a]] = 1.0
            weights = [p - q, p]
        token = -1
        for w in weights:
            sums = (w.clamp(0.0, 1.0).double() * UNIT).round().long().cumsum(0)
            if int(sums[-1]) > 0:
                edge = min(int(u[i] * float(int(sums[-1]))), int(sums[-1]) - 1)
                token = int((sums <= edge).sum())
                break
        sampled[i, :a] = torch.tensor(tokens[cu[i]:cu[i] + a], dtype=torch.int32)
        sampled[i, a] = last[i] = token
        num[i], rejected[i] = a + 1, cu[i + 1] - cu[i] - a
    return {"sampled": sampled.cuda(), "num_sampled": num.cuda(), "num_rejected": rejected.cuda(),
            "last": last.cuda()}


def _exact_distill(case, seed):
    """The gradient by automatic differentiation of the loss, or (with the sums
    of the forward pass given) from their own values."""
    s = _distill_inputs(case, seed)
    rows, vocab, org, t = case["rows"], case["vocab"], case["org"], case["temperature"]
    got = {n: torch.zeros(rows, dtype=torch.float64, device="cuda")
           for n in ("loss", "lse", "lse_rest")}
    if case["grad"]:
        got["grad"] = torch.zeros((rows, vocab), dtype=torch.float64, device="cuda")
    for a in range(0, rows, 256):
        b = min(rows, a + 256)
        x = s["logits"][a:b, :org].double()
        if case["grad"] and case["op"] == "distill":
            x.requires_grad_()
        ids, z = s["ids"][a:b].long(), s["teacher"][a:b].double() / t
        some = ids >= 0
        slot = torch.where(some, ids, org)
        on = torch.zeros((b - a, org + 1), dtype=torch.bool, device="cuda").scatter_(1, slot, True)
        on = on[:, :org]
        y = x / t
        if case["op"] == "distill":
            lse = torch.logsumexp(y, 1)
            lse_rest = torch.logsumexp(y.masked_fill(on, NEG), 1)
        else:
            lse, lse_rest = s["lse"][a:b].double(), s["lse_rest"][a:b].double()
        if case["rest"]:
            norm = s["teacher_lse"][a:b].double()
        else:
            norm = torch.logsumexp(z.masked_fill(~some, NEG), 1).masked_fill(~some.any(1), 0.0)
        p = torch.exp(z - norm[:, None]).masked_fill(~some, 0.0)
        pr = torch.zeros(b - a, dtype=torch.float64, device="cuda")
        if case["rest"]:
            pr = (1.0 - p.sum(1)).clamp(min=0.0).masked_fill(
                ~some.any(1) | (lse_rest.detach() == NEG), 0.0)
        if case["op"] == "distill":
            log_s = torch.gather(y, 1, slot.clamp(max=org - 1)) - lse[:, None]
            loss = torch.where(p > 0, p * (torch.log(p.clamp(min=1e-300)) - log_s), 0.0).sum(1)
            loss = loss + torch.where(
                pr > 0, pr * (torch.log(pr.clamp(min=1e-300)) - lse_rest + lse), 0.0)
            if case["grad"]:
                (loss * s["grad_loss"][a:b].double()).sum().backward()
                got["grad"][a:b, :org] = x.grad
            got["loss"][a:b], got["lse"][a:b] = loss.detach(), lse.detach()
            got["lse_rest"][a:b] = lse_rest.detach()
        else:
            d = (p.sum(1) + pr)[:, None] * torch.exp(y - lse[:, None])
            d = d - torch.where(on, 0.0, pr[:, None] * torch.exp(y - lse_rest[:, None]))
            d.scatter_add_(1, slot.clamp(max=org - 1), -p)
            got["grad"][a:b, :org] = d * (s["grad_loss"][a:b].double() / t)[:, None]
    if case["op"] == "distill_grad":
        return {"grad": got["grad"]}
    return got


def exact(case, seed):
    if case["op"] == "probs":
        return _exact_probs(case, seed)
    if case["op"] == "verify":
        return _exact_verify(case, seed)
    return _exact_distill(case, seed)
