"""Operators on rows of logits: what is measured, in plain torch operations and
through the library.

Three operators that belong together: the token draw of a rollout (`sample`),
the top logits of a scored position (`top_logprobs`, the teacher's side of a
distillation) and the distillation loss against a teacher's top logits with
its gradient (`distill`, `distill_step`).

A case is a dict of plain values; prepare() makes its inputs on the GPU from a
seed, run() is one pass as a program calls it (own = False: elementary torch
operations; own = True: the library's calls), exact() the operator's
definition in 64 bits, work() the bytes and operations that it cannot do
without.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # One request being decoded: latency counts. A chat request's usual
        # filters, on the fp32 logits of an engine.
        dict(name="sample_decode_1", op="sample", rows=1, vocab=151936, pad=0, dtype="float32",
             temperature=0.7, top_k=20, top_p=0.8, min_p=0.0, mixed=False, masked=0.0),
        # A decode batch of requests with settings of their own (greedy rows
        # among them), bf16 logits.
        dict(name="sample_decode_64_mixed", op="sample", rows=64, vocab=151936, pad=0,
             dtype="bfloat16", temperature=0.8, top_k=50, top_p=0.9, min_p=0.02, mixed=True,
             masked=0.0),
        # A rollout batch: nucleus only, so the kept set spans the vocabulary.
        dict(name="sample_rollout_512", op="sample", rows=512, vocab=151936, pad=0,
             dtype="float32", temperature=1.0, top_k=0, top_p=0.95, min_p=0.0, mixed=False,
             masked=0.0),
        # An odd vocabulary in padded rows, a tenth of the tokens masked out by
        # a grammar, min-p only.
        dict(name="sample_odd_37", op="sample", rows=37, vocab=32003, pad=61, dtype="float16",
             temperature=1.3, top_k=0, top_p=1.0, min_p=0.05, mixed=False, masked=0.1),
        # The top logprobs that an engine returns beside a decode batch.
        dict(name="top_decode_8", op="top", rows=8, vocab=151936, pad=0, dtype="float32",
             temperature=1.0, k=20),
        # A teacher's replay of one long response: its top logits at every
        # position, for the distillation below.
        dict(name="top_teacher_2304", op="top", rows=2304, vocab=151936, pad=0,
             dtype="bfloat16", temperature=1.0, k=64),
        # A small vocabulary with an odd size and a temperature.
        dict(name="top_odd_300", op="top", rows=300, vocab=50021, pad=3, dtype="float16",
             temperature=2.0, k=100),
        # The loss alone on a short evaluation batch.
        dict(name="distill_eval_7", op="distill", rows=7, vocab=151936, pad=0, dtype="bfloat16",
             temperature=1.0, k=32, renormalize=True, masked_rows=0.0),
        # The loss alone on a training-sized batch (a validation pass).
        dict(name="distill_eval_4096", op="distill", rows=4096, vocab=151936, pad=0,
             dtype="bfloat16", temperature=1.0, k=64, renormalize=True, masked_rows=0.0),
        # A training step through autograd: loss forward, gradient backward;
        # a tenth of the rows (the prompt) have no weight.
        dict(name="distill_autograd_1100", op="distill_grad", rows=1100, vocab=151936, pad=0,
             dtype="bfloat16", temperature=2.0, k=64, renormalize=True, masked_rows=0.1),
        # Loss and gradient in one call, the row weights known beforehand.
        dict(name="distill_step_2048", op="distill_step", rows=2048, vocab=151936, pad=0,
             dtype="bfloat16", temperature=1.0, k=64, renormalize=True, masked_rows=0.1),
        # fp32 logits of an odd vocabulary; the teacher's logprobs are taken
        # as they are, and a fifth of the rows are padding.
        dict(name="distill_step_odd_500", op="distill_step", rows=500, vocab=50021, pad=0,
             dtype="float32", temperature=1.0, k=100, renormalize=False, masked_rows=0.2),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "top", "distill", "distill_grad", "distill_step"])
    dtype = rng.choice(list(DTYPES))
    vocab = _log_uniform(rng, 1000, 160000) | rng.choice([0, 1])
    pad = rng.choice([0, 0, 1, 13, 64])
    # Rows limited so that no drawn case passes the largest listed one.
    cells = {"sample": 512 * 151936, "top": 512 * 151936, "distill": 1024 * 151936,
             "distill_grad": 512 * 151936, "distill_step": 512 * 151936}[op]
    rows = _log_uniform(rng, 1, min(2304, max(1, cells // (vocab + pad))))
    case = dict(op=op, rows=rows, vocab=vocab, pad=pad, dtype=dtype,
                temperature=rng.choice([0.5, 0.7, 1.0, 1.0, 1.5, 2.0]))
    if op == "sample":
        case.update(top_k=rng.choice([0, 0, 1, _log_uniform(rng, 2, 900)]),
                    top_p=rng.choice([1.0, 0.5, 0.9, 0.95, 0.99]),
                    min_p=rng.choice([0.0, 0.0, 0.01, 0.1]), mixed=rng.choice([False, True]),
                    masked=rng.choice([0.0, 0.0, 0.3]))
    else:
        case["k"] = min(_log_uniform(rng, 1, 256), vocab)
        if op != "top":
            case.update(renormalize=rng.choice([True, True, False]),
                        masked_rows=rng.choice([0.0, 0.1, 0.5]))
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _lm_logits(g, rows, columns, dtype):
    """Rows like a language model's: a normal bulk, and a head of raised
    tokens whose height differs from row to row (confident and open rows).
    Made in blocks of rows, so no fp32 copy of a large case is ever held."""
    out = torch.empty(rows, columns, dtype=dtype, device=DEV)
    head = min(48, columns)
    for a in range(0, rows, 256):
        b = min(a + 256, rows)
        z = torch.randn(b - a, columns, generator=g, device=DEV).mul_(2.2)
        at = torch.randint(0, columns, (b - a, head), generator=g, device=DEV)
        height = 12.0 * torch.rand(b - a, 1, generator=g, device=DEV)
        fall = torch.rand(b - a, head, generator=g, device=DEV)
        z.scatter_add_(1, at, height * fall * fall)
        out[a:b] = z.to(dtype)
    return out


def _teacher(g, logits, vocab, k, renormalize, temperature):
    """A teacher near the student: its top k of perturbed logits, in blocks of
    rows. Some of its lists are shorter (id -1 from there on)."""
    rows = logits.shape[0]
    ids = torch.empty(rows, k, dtype=torch.int64, device=DEV)
    values = torch.empty(rows, k, dtype=torch.float32, device=DEV)
    for a in range(0, rows, 256):
        z = logits[a:a + 256, :vocab].float()
        z = z + 0.7 * torch.randn(z.shape, generator=g, device=DEV)
        v, i = torch.topk(z, k, dim=1)
        if not renormalize:
            v = v / temperature - torch.logsumexp(z / temperature, dim=1, keepdim=True)
        ids[a:a + 256], values[a:a + 256] = i, v
    length = torch.randint(max(1, k // 2), 2 * k + 1, (rows, 1), generator=g, device=DEV)
    short = torch.arange(k, device=DEV)[None, :] >= length
    return ids.masked_fill_(short, -1), values


def prepare(case, seed):
    g = _generator(seed)
    rows, vocab, op = case["rows"], case["vocab"], case["op"]
    logits = _lm_logits(g, rows, vocab + case["pad"], DTYPES[case["dtype"]])
    state = dict(case=case, logits=logits)
    if op == "sample":
        if case["masked"] > 0:
            for a in range(0, rows, 256):
                block = logits[a:a + 256]
                gone = torch.rand(block.shape, generator=g, device=DEV) < case["masked"]
                block.masked_fill_(gone, -math.inf)
        state["u"] = torch.rand(rows, generator=g, device=DEV)

        def setting(name, dtype, others):
            """The case's value in every row, or each request's own choice."""
            if not case["mixed"]:
                return torch.full((rows,), case[name], dtype=dtype, device=DEV)
            options = torch.tensor([case[name]] + others, dtype=dtype, device=DEV)
            return options[torch.randint(0, len(options), (rows,), generator=g, device=DEV)]

        state["temperature"] = setting("temperature", torch.float32, [0.0, 0.6, 1.0, 1.2])
        state["top_k"] = setting("top_k", torch.int32, [0, 1, 20, 400])
        state["top_p"] = setting("top_p", torch.float32, [0.5, 0.95, 1.0])
        state["min_p"] = setting("min_p", torch.float32, [0.0, 0.1])
    elif op != "top":
        state["ids"], state["teacher"] = _teacher(g, logits, vocab, case["k"],
                                                  case["renormalize"], case["temperature"])
        if op != "distill":
            weight = torch.rand(rows, generator=g, device=DEV) >= case["masked_rows"]
            state["weight"] = weight.float() / max(1, rows)
        if op == "distill_grad":
            state["logits"] = logits.requires_grad_(True)
    return state


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    case = state["case"]
    return (_run_own if own else _run_plain)(state, case, case["op"])


def _run_own(state, case, op):
    import rollout_logprob_consistency_amd as lp

    if op == "sample":
        return lp.sample(state["logits"], state["u"], state["temperature"], state["top_k"],
                         state["top_p"], state["min_p"], v_true=case["vocab"])
    if op == "top":
        return lp.top_logprobs(state["logits"], case["k"], case["temperature"],
                               v_true=case["vocab"])
    args = (state["ids"], state["teacher"])
    more = dict(temperature=case["temperature"], renormalize=case["renormalize"],
                v_true=case["vocab"])
    if op == "distill":
        return lp.distill(state["logits"], *args, **more)
    if op == "distill_step":
        return lp.distill_step(state["logits"], *args, state["weight"], **more)
    loss = lp.distill(state["logits"], *args, **more)
    grad, = torch.autograd.grad(loss, state["logits"], state["weight"])
    return loss.detach(), grad


def _run_plain(state, case, op):
    if op == "sample":
        return _plain_sample(state, case)
    if op == "top":
        return _plain_top(state, case)
    return _plain_distill(state, case, op != "distill")


def _plain_sample(state, case):
    """Sorted probabilities and their running sums, in 64 bits: a draw next to
    a border between two tokens is decided by digits that 32 bits lose."""
    z = state["logits"][:, :case["vocab"]].double()
    tau = state["temperature"].double()[:, None]
    greedy = tau == 0
    z, order = torch.sort(z, dim=1, descending=True, stable=True)
    s = z / torch.where(greedy, torch.ones_like(tau), tau)
    s = s - s[:, :1]
    w = torch.exp(s)
    lse = torch.log(w.sum(dim=1, keepdim=True))
    rank = torch.arange(z.shape[1], device=z.device)[None, :]
    finite = (z > -math.inf).sum(dim=1, keepdim=True)
    top_k = state["top_k"].long()[:, None]
    first = torch.where(top_k > 0, torch.minimum(top_k, finite), finite)
    c = torch.cumsum(w * (rank < first), dim=1)
    before = torch.cat([torch.zeros_like(c[:, :1]), c[:, :-1]], dim=1)
    top_p = state["top_p"].double()[:, None]
    keep = (rank < first) & ((top_p >= 1) | (before < top_p * c[:, -1:]))
    keep &= w >= state["min_p"].double()[:, None]
    kept = keep.sum(dim=1, keepdim=True).clamp(min=1)
    kept = torch.where(greedy, torch.ones_like(kept), kept)
    mass = c.gather(1, kept - 1)
    r = ((c <= state["u"].double()[:, None] * mass) & (rank < kept)).sum(dim=1, keepdim=True)
    r = torch.minimum(r, kept - 1)
    token = order.gather(1, r)
    logprob = s.gather(1, r) - lse
    processed = torch.log(w.gather(1, r) / mass)
    return (token[:, 0], logprob[:, 0].float(), processed[:, 0].float(),
            kept[:, 0].to(torch.int32))


def _plain_top(state, case):
    z = state["logits"][:, :case["vocab"]].float()
    best = z.max(dim=1, keepdim=True).values
    scale = 1.0 / case["temperature"]
    lse = torch.log(torch.exp((z - best) * scale).sum(dim=1, keepdim=True))
    z, order = torch.sort(z, dim=1, descending=True, stable=True)
    z, order = z[:, :case["k"]], order[:, :case["k"]]
    return order.contiguous(), z.contiguous(), (z - best) * scale - lse


def _plain_distill(state, case, with_grad):
    logits, ids, t = state["logits"].detach(), state["ids"], state["teacher"]
    scale = 1.0 / case["temperature"]
    s = logits[:, :case["vocab"]].float() * scale
    best = s.max(dim=1, keepdim=True).values
    e = torch.exp(s - best)
    total = e.sum(dim=1, keepdim=True)
    there = ids >= 0
    at = ids.clamp(min=0)
    if case["renormalize"]:
        t = (t * scale).masked_fill(~there, -math.inf)
        t = t - t.max(dim=1, keepdim=True).values
        t = t - torch.log(torch.exp(t).sum(dim=1, keepdim=True))
    q = torch.exp(t) * there
    logp = s.gather(1, at) - best - torch.log(total)
    loss = torch.where(q > 0, q * (t - logp), torch.zeros_like(q)).sum(dim=1)
    if not with_grad:
        return loss
    grad = e / total * q.sum(dim=1, keepdim=True)
    grad.scatter_add_(1, at, -q)
    grad *= state["weight"][:, None] * scale
    out = torch.zeros_like(logits)
    out[:, :case["vocab"]] = grad.to(logits.dtype)
    return loss, out


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    rows, vocab, op = case["rows"], case["vocab"], case["op"]
    size = 4 if case["dtype"] == "float32" else 2
    read = rows * vocab * size
    if op == "sample":
        # settings and the random number in; token, two logprobs, count out;
        # a scaled difference, an exponential and a sum for each logit
        return {"bytes": read + rows * (20 + 20), "flops": 4 * rows * vocab}
    if op == "top":
        return {"bytes": read + rows * case["k"] * 16, "flops": 4 * rows * vocab}
    lists = rows * case["k"] * 12
    if op == "distill":
        return {"bytes": read + lists + rows * 4, "flops": 4 * rows * vocab}
    written = rows * (vocab + case["pad"]) * size
    return {"bytes": read + written + lists + rows * 8, "flops": 8 * rows * vocab}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    state = prepare(case, seed)
    logits, vocab, op = state["logits"].detach(), case["vocab"], case["op"]
    if op == "sample":
        return _exact_sample(state, vocab)
    if op == "top":
        return _exact_top(logits, vocab, case)
    return _exact_distill(state, logits, vocab, case)


def _exact_sample(state, vocab):
    """Row by row: the tokens in order, the filters as lengths of a prefix."""
    tokens, raw, processed, counts = [], [], [], []
    u, tau, top_k, top_p, min_p = (state[n].cpu().tolist() for n in
                                   ("u", "temperature", "top_k", "top_p", "min_p"))
    for row in range(len(u)):
        z = state["logits"][row, :vocab].to(torch.float64)
        order = torch.argsort(-z, stable=True)
        t = tau[row] if tau[row] > 0 else 1.0
        gap = (z[order] - z[order[0]]) / t
        p = torch.exp(gap)
        log_total = math.log(float(p.sum()))
        n = int((z > -math.inf).sum())
        if top_k[row] > 0:
            n = min(n, top_k[row])
        c = torch.cumsum(p[:n], 0)
        if tau[row] == 0:
            keep = 1
        else:
            keep = n
            if top_p[row] < 1:
                keep = 1 + int(torch.searchsorted(c, top_p[row] * c[-1:], right=False))
            keep = max(1, min(keep, n, int((p >= min_p[row]).sum())))
        mass = c[keep - 1]
        r = min(keep - 1, int(torch.searchsorted(c[:keep], u[row] * mass[None], right=True)))
        tokens.append(int(order[r]))
        raw.append(float(gap[r]) - log_total)
        processed.append(float(gap[r]) - math.log(float(mass)))
        counts.append(keep)
    return (torch.tensor(tokens, device=DEV), torch.tensor(raw, dtype=torch.float64, device=DEV),
            torch.tensor(processed, dtype=torch.float64, device=DEV),
            torch.tensor(counts, dtype=torch.int32, device=DEV))


def _exact_top(logits, vocab, case):
    rows, k = logits.shape[0], case["k"]
    ids = torch.empty(rows, k, dtype=torch.int64, device=DEV)
    values = torch.empty(rows, k, dtype=torch.float64, device=DEV)
    logprobs = torch.empty(rows, k, dtype=torch.float64, device=DEV)
    for a in range(0, rows, 128):
        z = logits[a:a + 128, :vocab].to(torch.float64)
        order = torch.argsort(-z, dim=1, stable=True)[:, :k]
        s = z / case["temperature"]
        ids[a:a + 128] = order
        values[a:a + 128] = z.gather(1, order)
        logprobs[a:a + 128] = s.gather(1, order) - torch.logsumexp(s, dim=1, keepdim=True)
    return ids, values, logprobs


def _exact_distill(state, logits, vocab, case):
    rows, tau = logits.shape[0], case["temperature"]
    loss = torch.empty(rows, dtype=torch.float64, device=DEV)
    grad = None
    if case["op"] != "distill":
        grad = torch.zeros(logits.shape, dtype=torch.float64, device=DEV)
    for a in range(0, rows, 128):
        b = min(a + 128, rows)
        z = logits[a:b, :vocab].to(torch.float64) / tau
        ids, t = state["ids"][a:b], state["teacher"][a:b].to(torch.float64)
        gone = ids < 0
        t = (t / tau if case["renormalize"] else t).masked_fill(gone, -math.inf)
        log_q = torch.log_softmax(t, dim=1) if case["renormalize"] else t
        q = torch.exp(log_q)
        # The teacher's distribution over the whole vocabulary.
        target = torch.zeros_like(z)
        rows_of = torch.arange(b - a, device=DEV)[:, None].expand_as(ids)
        target.index_put_((rows_of[~gone], ids[~gone]), q[~gone], accumulate=True)
        log_p = torch.log_softmax(z, dim=1)
        entropy = torch.where(q > 0, q * log_q, torch.zeros_like(q)).sum(dim=1)
        loss[a:b] = entropy - (target * log_p).sum(dim=1)
        if grad is not None:
            g = state["weight"][a:b].to(torch.float64)[:, None] / tau
            grad[a:b, :vocab] = g * (target.sum(dim=1, keepdim=True) * torch.exp(log_p) - target)
    return loss if grad is None else (loss, grad)
