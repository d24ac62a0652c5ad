"""Operators on next-token logits as they are timed and compared: log
probabilities of given tokens with the entropy and the top alternatives, the
gradient of log probability and entropy, and distillation from a teacher's top
logits (the divergence alone, or the loss with the gradient of its logits).

``own`` selects the form: False computes each operator from elementary torch
operations in float32 (float64 for the long sums), True calls the library.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4}


def listed():
    return [
        # one request's next token with its 5 alternatives: the smallest call, where latency counts
        dict(name="top-one", op="top", tokens=1, vocab=128256, k=5, dtype="bf16", temperature=1.0, prompt=0.0, pad=0,
             targets=True),
        # a serving batch: the tokens sampled for 256 requests, 20 alternatives each, the vocabulary padded to 128512
        dict(name="top-decode", op="top", tokens=256, vocab=128512, k=20, dtype="bf16", temperature=1.0, prompt=0.0,
             pad=256, targets=True),
        # a teacher's pass over a batch: its 64 top tokens at temperature 2, no targets
        dict(name="top-teacher", op="top", tokens=4096, vocab=128256, k=64, dtype="bf16", temperature=2.0, prompt=0.0,
             pad=0, targets=False),
        # evaluation on float32 logits of an odd vocabulary, prompts masked
        dict(name="top-eval-odd", op="top", tokens=2043, vocab=32003, k=8, dtype="f32", temperature=1.0, prompt=0.3,
             pad=3, targets=True),
        # the forward pass of a policy update with an entropy term, at the sampling temperature
        dict(name="top-entropy", op="top", tokens=8192, vocab=128256, k=0, dtype="bf16", temperature=0.75, prompt=0.3,
             pad=0, targets=True),
        # its backward pass for a few sampled tokens of one rollout
        dict(name="top-grad-short", op="grad", tokens=40, vocab=128256, dtype="bf16", temperature=1.0, prompt=0.2,
             pad=0),
        # the backward pass of the whole batch
        dict(name="top-grad-train", op="grad", tokens=8192, vocab=128256, dtype="bf16", temperature=0.75, prompt=0.3,
             pad=0),
        # the same for float32 logits of an odd vocabulary
        dict(name="top-grad-odd", op="grad", tokens=2043, vocab=32003, dtype="f32", temperature=1.0, prompt=0.3, pad=3),
        # one short sequence distilled: the smallest training step
        dict(name="distill-short", op="distill", tokens=96, vocab=128256, k=32, dtype="bf16", temperature=1.0,
             prompt=0.3, rest=True),
        # a full batch: loss and the gradient of its 8192 x 128256 logits from the teacher's 64 top tokens
        dict(name="distill-train", op="distill", tokens=8192, vocab=128256, k=64, dtype="bf16", temperature=2.0,
             prompt=0.3, rest=True),
        # float32 logits of an odd vocabulary, the teacher's 100 top tokens taken for all of its distribution
        dict(name="distill-odd", op="distill", tokens=1021, vocab=32003, k=100, dtype="f32", temperature=1.0,
             prompt=0.0, rest=False),
        # evaluation: the tokens' divergence from the teacher, no gradient
        dict(name="distill-eval", op="kl", tokens=2048, vocab=128256, k=64, dtype="bf16", temperature=1.0, prompt=0.3,
             rest=True),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["top", "grad", "distill", "kl"])
    case = dict(op=op, tokens=spread(1, 4096), vocab=spread(500, 131072), dtype=rng.choice(["bf16", "f32"]),
                temperature=rng.choice([0.7, 1.0, 1.5, 2.0]), prompt=rng.choice([0.0, 0.3]))
    if op in ("top", "grad"):
        case["pad"] = rng.choice([0, 0, 1, 64])
    if op == "top":
        return dict(case, k=rng.choice([0, spread(1, 128), spread(1, 128)]), targets=rng.random() < 0.7)
    if op == "grad":
        return case
    return dict(case, k=spread(1, 128), rest=rng.random() < 0.7)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _masked(case):
    """How many tokens of each sequence (of up to 512, packed one after the other) are its prompt, and so masked."""
    length = min(case["tokens"], 512)
    return length, int(length * case["prompt"])


def _live_rows(case):
    length, prompt = _masked(case)
    full, rest = divmod(case["tokens"], length)
    return full * (length - prompt) + max(0, rest - prompt)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = torch.device("cuda")
    T, V = case["tokens"], case["vocab"]

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(*shape, device=dev, dtype=dtype, generator=g).mul_(std)

    logits = normal(T, V, std=2.0, dtype=_DT[case["dtype"]])
    pad = case.get("pad", 0)
    if pad:  # columns past the last token of a vocabulary that was padded
        logits[:, V - pad:] = -math.inf
    rows = torch.arange(T, device=dev)
    targets = torch.randint(0, V - pad, (T,), device=dev, dtype=torch.int32, generator=g)
    # the model favours one token in each place
    logits[rows, targets.long()] += normal(T, std=3.0).add_(9.0).to(logits.dtype)
    length, prompt = _masked(case)
    masked = rows % length < prompt
    state = dict(case=case, logits=logits)
    if case["op"] in ("top", "grad"):
        state["targets"] = None
        if case.get("targets", True):
            state["targets"] = torch.where(masked, torch.full_like(targets, -100), targets)
        if case["op"] == "grad":
            # what the forward pass keeps of each row
            m, r, gap = [], [], []
            for x in logits.split(512):
                top, at = x.max(1, keepdim=True)
                d = (x.double() - top.double()) / case["temperature"]
                e = torch.exp(d)
                gap.append(-torch.where(e > 0, e * d, 0.0).sum(1) / e.sum(1))
                r.append(e.scatter_(1, at, 0.0).sum(1))
                m.append(top[:, 0].double())
            state["stats"] = torch.stack([torch.cat(m), torch.cat(r), torch.cat(gap)], 1).float()
            if prompt:
                state["stats"][masked] = 0.0
            state["dlogp"] = normal(T, std=1e-3)
            state["dentropy"] = normal(T, std=1e-4)
        return state
    # a teacher that mostly agrees with the model
    ids, logp = [], []
    for x in logits.split(1024):
        t = (x.float() + normal(*x.shape, std=0.7)) / case["temperature"]
        at = _top(t, case["k"])
        logp.append((t.gather(1, at).double() - torch.logsumexp(t, 1, keepdim=True).double()).float())
        ids.append(at.to(torch.int32))
    state["top_ids"], state["top_logp"] = torch.cat(ids), torch.cat(logp)
    state["top_ids"][masked] = -1
    state["top_logp"][masked] = -math.inf
    state["weights"] = torch.full((T,), case["temperature"] ** 2 / max(1, _live_rows(case)), device=dev)
    return state


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _top(x, k):
    """Columns of the k largest values of each row (float32), ties to the lowest column."""
    bits = (x + 0.0).view(torch.int32)  # + 0.0: -0 equals 0
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).to(torch.int64)
    last = 0xFFFFFFFF - torch.arange(x.shape[1], device=x.device)
    return 0xFFFFFFFF - (order.mul_(1 << 32).add_(last).topk(k, 1).values & 0xFFFFFFFF)


def _plain_top(state):
    case = state["case"]
    raw = state["logits"].float()
    T, V = raw.shape
    x = raw / case["temperature"]
    m = x.amax(1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    s = e.sum(1, keepdim=True)
    log_s = torch.log(s)
    out = {"entropy": (log_s - torch.where(e > 0, e * d, 0.0).sum(1, keepdim=True) / s)[:, 0]}
    ok = None
    if state["targets"] is not None:
        y = state["targets"].long()
        ok = (y >= 0) & (y < V)
        out["logp"] = torch.where(ok, (d.gather(1, torch.where(ok, y, 0)[:, None]) - log_s)[:, 0], 0.0)
        out["entropy"] = torch.where(ok, out["entropy"], 0.0)
    if case["k"]:
        k = min(case["k"], V)
        ids = _top(raw, k)
        top = d.gather(1, ids) - log_s
        ids = torch.nn.functional.pad(ids, (0, case["k"] - k), value=-1)
        top = torch.nn.functional.pad(top, (0, case["k"] - k), value=-math.inf)
        if ok is not None:
            ids = torch.where(ok[:, None], ids, -1)
            top = torch.where(ok[:, None], top, -math.inf)
        out["top_ids"], out["top_logp"] = ids.to(torch.int32), top
    return out


def _plain_grad(state):
    case = state["case"]
    m, r, gap = (state["stats"][:, i:i + 1] for i in range(3))
    d = (state["logits"].float() - m) / case["temperature"]
    V = d.shape[1]
    y = state["targets"].long()
    ok = ((y >= 0) & (y < V))[:, None]
    p = torch.exp(d) / (1 + r)
    # dlogp * (one at the target - p) - dentropy * p * (log p + entropy), with log p + entropy = d + gap
    by_logp = torch.where(ok, state["dlogp"][:, None], 0.0)
    by_entropy = torch.where(ok, state["dentropy"][:, None], 0.0)
    grad = torch.where(p > 0, -p * (by_logp + by_entropy * (d + gap)), 0.0)
    at = torch.where(ok, y[:, None], 0)
    grad.scatter_(1, at, grad.gather(1, at) + by_logp)
    return {"dlogits": (grad / case["temperature"]).to(state["logits"].dtype)}


def _plain_distill(state):
    """The divergence of the tokens, and what its gradient takes: softmax of the logits, the teacher's weights at its
    tokens, the factor of the others."""
    case = state["case"]
    x = state["logits"].float() / case["temperature"]
    V = x.shape[1]
    ids = state["top_ids"].long()
    ok = (ids >= 0) & (ids < V)
    live = ok.any(1, keepdim=True)
    at = torch.where(ok, ids, ids[:, :1].clamp(0, V - 1))
    logq = torch.where(ok, state["top_logp"].double(), -math.inf)
    if not case["rest"]:
        logq = logq - torch.logsumexp(torch.where(live, logq, 0.0), 1, keepdim=True)
    q = torch.exp(logq)
    x = x - x.amax(1, keepdim=True)
    e = torch.exp(x)
    others = e.scatter(1, at, 0.0).sum(1, keepdim=True).double()
    total = others + e.gather(1, at).double().sum(1, keepdim=True)
    logp = x.gather(1, at).double() - torch.log(total)
    each = torch.where(q > 0, q * (logq - logp), 0.0)
    kl = each.sum(1, keepdim=True)
    factor = torch.ones_like(kl)
    if case["rest"]:
        q_rest = (1 - q.sum(1, keepdim=True)).clamp_min(0.0)
        p_rest = others / total
        kl = kl + torch.where(q_rest > 0, q_rest * torch.log(q_rest / p_rest), 0.0)
        factor = q.sum(1, keepdim=True) + q_rest - q_rest / p_rest
    kl = torch.where(live, kl, 0.0)
    return kl[:, 0], e, total, at, q, factor, live


def _plain_step(state):
    case = state["case"]
    kl, e, total, at, q, factor, live = _plain_distill(state)
    w = state["weights"]
    p_top = e.gather(1, at).double() / total
    all_q = q.sum(1, keepdim=True) + (1 - q.sum(1, keepdim=True)).clamp_min(0.0) if case["rest"] else 1.0
    grad = e.mul_((factor / total).float())
    grad.scatter_(1, at, (all_q * p_top - q).float())
    grad.mul_(torch.where(live, w[:, None] / case["temperature"], 0.0))
    return {"loss": (w.double() * kl).sum().float(), "kl": kl.float(), "dlogits": grad.to(state["logits"].dtype)}


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        if op == "kl":
            return {"kl": _plain_distill(state)[0].float()}
        return {"top": _plain_top, "grad": _plain_grad, "distill": _plain_step}[op](state)
    import lora_rank_adapter_amd as L
    if op == "top":
        logp, entropy, ids, top, _ = L.lora_token_top(state["logits"], state["targets"], k=case["k"],
                                                      temperature=case["temperature"])
        out = {"entropy": entropy}
        if logp is not None:
            out["logp"] = logp
        if case["k"]:
            out["top_ids"], out["top_logp"] = ids, top
        return out
    if op == "grad":
        return {"dlogits": L.lora_token_top_grad(state["logits"], state["targets"], state["stats"],
                                                 dlogp=state["dlogp"], dentropy=state["dentropy"],
                                                 temperature=case["temperature"])}
    if op == "kl":
        return {"kl": L.lora_distill_kl(state["logits"], state["top_ids"], state["top_logp"],
                                        temperature=case["temperature"], rest=case["rest"])[0]}
    loss, kl, dlogits = L.lora_distill_step(state["logits"], state["top_ids"], state["top_logp"], state["weights"],
                                            temperature=case["temperature"], rest=case["rest"])
    return {"loss": loss, "kl": kl, "dlogits": dlogits}


# ---------------------------------------------------------------------------
# the definitions in float64
# ---------------------------------------------------------------------------

def _exact_top(state, case, logits, part):
    logprob = torch.log_softmax(logits.double() / case["temperature"], 1)
    terms = torch.exp(logprob) * logprob
    out = {"entropy": -terms.nan_to_num(nan=0.0).sum(1)}
    hide = torch.zeros(len(logits), dtype=torch.bool, device=logits.device)
    if state["targets"] is not None:
        y = state["targets"][part]
        hide = (y < 0) | (y >= case["vocab"])
        out["logp"] = logprob[torch.arange(len(y), device=y.device), y.clamp(0, case["vocab"] - 1).long()]
        out["logp"][hide] = 0.0
        out["entropy"][hide] = 0.0
    if case["k"]:
        ids = torch.sort(logits.float(), dim=1, descending=True, stable=True).indices[:, :case["k"]]
        top = torch.full((len(logits), case["k"]), -math.inf, dtype=torch.float64, device=logits.device)
        names = torch.full((len(logits), case["k"]), -1, dtype=torch.int32, device=logits.device)
        top[:, :ids.shape[1]] = logprob.gather(1, ids)
        names[:, :ids.shape[1]] = ids.int()
        top[hide] = -math.inf
        names[hide] = -1
        out["top_ids"], out["top_logp"] = names, top
    return out


def _exact_grad(state, case, logits, part):
    # through torch's own differentiation of log probability and entropy
    y = state["targets"][part]
    on = (y >= 0) & (y < case["vocab"])
    finite = torch.isfinite(logits)
    x = torch.where(finite, logits.double(), 0.0).requires_grad_()
    lp = torch.log_softmax(torch.where(finite, x, -math.inf) / case["temperature"], 1)
    safe = torch.where(finite, lp, 0.0)
    entropy = -(torch.exp(safe) * safe * finite).sum(1)
    picked = safe[torch.arange(len(y), device=y.device), y.clamp(0, case["vocab"] - 1).long()]
    total = ((state["dlogp"][part].double() * picked + state["dentropy"][part].double() * entropy) * on).sum()
    dx, = torch.autograd.grad(total, x)
    return {"dlogits": dx}


def _exact_distill(state, case, logits, part):
    ids, logq = state["top_ids"][part], state["top_logp"][part].double()
    rows = torch.nonzero((ids >= 0).any(1))[:, 0]
    kl = torch.zeros(len(logits), dtype=torch.float64, device=logits.device)
    dx = torch.zeros(logits.shape, dtype=torch.float64, device=logits.device)
    if len(rows):
        at, logq = ids[rows].long(), logq[rows]
        x = logits[rows].double().requires_grad_()
        z = x / case["temperature"]
        hidden = torch.zeros_like(z, dtype=torch.bool).scatter_(1, at, True)
        lse = torch.logsumexp(z, 1, keepdim=True)
        if not case["rest"]:
            logq = torch.log_softmax(logq, 1)
        loss = (torch.exp(logq) * (logq - (z.gather(1, at) - lse))).sum(1)
        if case["rest"]:
            left = 1.0 - torch.exp(logq).sum(1)
            others = torch.logsumexp(z.masked_fill(hidden, -math.inf), 1) - lse[:, 0]
            loss = loss + torch.where(left > 0, left * (torch.log(left.clamp_min(1e-300)) - others), 0.0)
        kl[rows] = loss.detach()
        if case["op"] == "distill":
            dx[rows], = torch.autograd.grad((state["weights"][part][rows].double() * loss).sum(), x)
    if case["op"] == "kl":
        return {"kl": kl}
    return {"loss": (state["weights"][part].double() * kl).sum()[None], "kl": kl, "dlogits": dx}


def exact(case, seed):
    state = prepare(case, seed)
    T, V = state["logits"].shape
    form = {"top": _exact_top, "grad": _exact_grad}.get(case["op"], _exact_distill)
    parts = []
    for a in range(0, T, 512):
        part = slice(a, min(T, a + 512))
        one = form(state, case, state["logits"][part], part)
        if T * V > 1 << 28 and "dlogits" in one:
            # kept in 32 bits: half a step of 2^-24 is far below what the outputs' types allow
            one["dlogits"] = one["dlogits"].float()
        parts.append(one)
    out = {name: torch.cat([p[name] for p in parts]) for name in parts[0]}
    if "loss" in out:
        out["loss"] = out["loss"].sum()
    return out


def work(case):
    T, V, es, op = case["tokens"], case["vocab"], _ES[case["dtype"]], case["op"]
    live = T if op == "top" and not case["targets"] else _live_rows(case)  # masked rows need not be read
    size = {"bytes": live * V * es, "flops": 6 * live * V}
    if op in ("grad", "distill"):
        size["bytes"] += T * V * es
        size["flops"] += 2 * live * V
    # ids and values of the alternatives, and the vectors of each token
    return {"bytes": size["bytes"] + T * (8 * case.get("k", 0) + 16), "flops": size["flops"]}
