"""The operators of an adapter training step that surround the adapter linears,
as they are timed and compared: embedding lookup and its gradient, the
preference loss over paired sequences, the clipped policy loss with a KL term,
and the AdamW step over many tensors.

``own`` selects the form: False computes each operator from elementary torch
operations in float32 (float64 for the long sums), True calls the library.
"""
import math
import random

import numpy as np
import torch

own = False

# fields of one batch that every loss case shares
BETA, SMOOTHING = 0.1, 0.05
CLIP_LOW, CLIP_HIGH, KL_COEF = 0.2, 0.28, 0.04
# AdamW settings of the step cases; the step is taken after STEP earlier ones
LR, BETA1, BETA2, EPS, DECAY, STEP = 2e-4, 0.9, 0.999, 1e-8, 0.01, 20
BLOCK = 256  # elements that share one scale in an 8-bit state
FP8_MAX, FP8_MIN = 448.0, 2.0 ** -9  # largest and smallest positive e4m3 value

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4}


def listed():
    return [
        # a serving batch: one new token for each of 256 requests
        dict(name="embed-decode", op="embed", tokens=256, rows=128256, cols=4096, dtype="bf16", out="bf16", scale=1.0),
        # a prefill batch, the float32 residual stream, embeddings scaled by sqrt(cols)
        dict(name="embed-prefill", op="embed", tokens=16731, rows=128256, cols=8192, dtype="bf16", out="f32",
             scale=math.sqrt(8192.0)),
        # the gradient of an embedding adapter's table (rank 64): dY*B^T summed over each id's tokens
        dict(name="embed-grad-adapter", op="embed_grad", tokens=16384, rows=128256, cols=64, dtype="f32", out="f32",
             scale=0.5),
        # the gradient of a whole embedding table in bfloat16
        dict(name="embed-grad-table", op="embed_grad", tokens=8192, rows=128256, cols=4096, dtype="bf16", out="bf16",
             scale=1.0),
        # one short preference pair: the smallest training step, where latency counts
        dict(name="pref-one-pair", op="pref", pairs=1, tokens=96, vocab=128256, dtype="bf16", train=True),
        # a full preference batch: loss and the gradient of its 8192 x 128256 logits
        dict(name="pref-train", op="pref", pairs=8, tokens=8192, vocab=128256, dtype="bf16", train=True),
        # evaluation on float32 logits of an odd vocabulary, no gradient
        dict(name="pref-eval-odd", op="pref", pairs=5, tokens=2043, vocab=32003, dtype="f32", train=False),
        # a few sampled tokens of one rollout
        dict(name="policy-short", op="policy", seqs=2, tokens=40, vocab=128256, dtype="bf16"),
        # a full rollout batch: loss and the gradient of its 8192 x 128256 logits
        dict(name="policy-train", op="policy", seqs=16, tokens=8192, vocab=128256, dtype="bf16"),
        # one adapter pair (rank 8, 512 features) trained in bfloat16
        dict(name="adamw-one-adapter", op="adamw", layers=1, rank=8, width=512, out=512, bits=32, param="bf16",
             grad="f32", shadow=False),
        # a model's adapters, rank 16: float32 weights, the bfloat16 copies that the forward reads, 32-bit states
        dict(name="adamw-32bit", op="adamw", layers=32, rank=16, width=4096, out=14336, bits=32, param="f32",
             grad="f32", shadow=True),
        # the same at rank 64 with 8-bit states
        dict(name="adamw-8bit", op="adamw", layers=32, rank=64, width=4096, out=14336, bits=8, param="f32",
             grad="f32", shadow=True),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["embed", "embed_grad", "pref", "policy", "adamw"])
    if op in ("embed", "embed_grad"):
        dtype = rng.choice(["bf16", "f32"])
        return dict(op=op, tokens=spread(1, 16384), rows=spread(500, 131072), cols=spread(8, 4096), dtype=dtype,
                    out="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]),
                    scale=rng.choice([0.5, 1.0, 8.0, 64.0]))
    if op == "adamw":
        param = rng.choice(["f32", "bf16"])
        return dict(op=op, layers=spread(1, 32), rank=spread(4, 64), width=spread(256, 4096), out=spread(256, 8192),
                    bits=rng.choice([8, 32]), param=param, grad=rng.choice(["f32", "bf16"]),
                    shadow=param == "f32" and rng.random() < 0.5)
    case = dict(op=op, tokens=spread(16, 4096), vocab=spread(1000, 131072), dtype=rng.choice(["bf16", "f32"]))
    if op == "pref":
        return dict(case, pairs=rng.randint(1, 8), train=rng.random() < 0.7)
    return dict(case, seqs=rng.randint(1, 16))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _sequences(case):
    """[(prompt, response)] of the packed sequences: the tokens cut at random, a
    prompt of a tenth to a half of each; in a batch of 8 sequences or more the
    fourth was cut short before its response."""
    n = 2 * case["pairs"] if case["op"] == "pref" else case["seqs"]
    rng = random.Random("%d %d" % (case["tokens"], n))
    weights = [rng.uniform(0.5, 1.5) for _ in range(n)]
    cuts = [int(case["tokens"] * sum(weights[:i]) / sum(weights)) for i in range(n)] + [case["tokens"]]
    out = []
    for i in range(n):
        length = cuts[i + 1] - cuts[i]
        prompt = length if n >= 8 and i == 3 else int(length * rng.uniform(0.1, 0.5))
        out.append((prompt, length - prompt))
    return out


def _tensor_sizes(case):
    """Elements of each adapter weight: per layer A and B of the fused
    projection's slices (width, width/4, width/4) and of the wide projection."""
    r, width = case["rank"], case["width"]
    if case["layers"] == 1:
        return [r * width, case["out"] * r]
    layer = []
    for outs in (width, width // 4, width // 4, case["out"]):
        layer += [r * width, outs * r]
    return layer * case["layers"]


def _zipf(tokens, rows, g):
    """Ids with the law of token frequencies: P(id < v) = log(v + 1) / log(rows + 1)."""
    u = torch.rand(tokens, device="cuda", dtype=torch.float64, generator=g)
    return torch.exp(u * math.log(rows + 1)).sub_(1).floor_().clamp_(0, rows - 1).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = torch.device("cuda")
    op = case["op"]

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(*shape, device=dev, dtype=dtype, generator=g).mul_(std)

    if op in ("embed", "embed_grad"):
        ids = _zipf(case["tokens"], case["rows"], g)
        # one position in a hundred holds no token of the table (an image's place)
        ids[torch.rand(case["tokens"], device=dev, generator=g) < 0.01] = -1
        n = case["rows"] if op == "embed" else case["tokens"]
        data = normal(n, case["cols"], std=0.02 if op == "embed" else 1.0, dtype=_DT[case["dtype"]])
        return dict(case=case, ids=ids, data=data)

    if op in ("pref", "policy"):
        T, V = case["tokens"], case["vocab"]
        seqs = _sequences(case)
        logits = normal(T, V, std=2.0, dtype=_DT[case["dtype"]])
        targets = torch.randint(0, V, (T,), device=dev, dtype=torch.int32, generator=g)
        rows = torch.arange(T, device=dev)
        # the model favours the token that follows
        logits[rows, targets.long()] += normal(T, std=3.0).add_(9.0).to(logits.dtype)
        lp = torch.cat([x.double().gather(1, t.long()[:, None])[:, 0] - torch.logsumexp(x.float(), 1).double()
                        for x, t in zip(logits.split(1024), targets.split(1024))])
        mask, offsets = [], [0]
        for prompt, response in seqs:
            mask += [0] * prompt + [1] * response
            offsets.append(offsets[-1] + prompt + response)
        mask = torch.tensor(mask, device=dev, dtype=torch.bool)
        targets = torch.where(mask, targets, torch.full_like(targets, -100))
        offsets = torch.tensor(offsets, device=dev, dtype=torch.int32)
        state = dict(case=case, logits=logits, targets=targets, offsets=offsets)
        if op == "pref":
            total = torch.cat([lp.new_zeros(1), torch.where(mask, lp, 0.0).cumsum(0)])[offsets.long()]
            state["ref_logp"] = (total[1:] - total[:-1]).float() + normal(len(seqs), std=4.0)
            return state
        state["old_logp"] = lp.float() + normal(T, std=0.15)
        state["ref_logp"] = lp.float() + normal(T, std=0.3)
        lengths = torch.tensor([p + r for p, r in seqs], device=dev)
        state["advantages"] = normal(len(seqs)).repeat_interleave(lengths)
        state["weights"] = torch.full((T,), 1.0 / max(1, int(sum(r for _, r in seqs))), device=dev)
        return state

    # AdamW: each weight is a view of one buffer, starting at a multiple of BLOCK elements
    sizes = _tensor_sizes(case)
    starts = np.concatenate([[0], np.cumsum([-(-n // BLOCK) * BLOCK for n in sizes])]).tolist()
    total = starts[-1]
    live = torch.zeros(total, device=dev, dtype=torch.bool)
    for s, n in zip(starts, sizes):
        live[s:s + n] = True
    pads = ~live
    p = normal(total, std=0.02)
    grad = normal(total, std=1e-3)
    m = normal(total, std=3e-4)
    v = normal(total, std=1e-3).square_()
    for t in (p, grad, m, v):
        t[pads] = 0.0
    p, grad = p.to(_DT[case["param"]]), grad.to(_DT[case["grad"]])
    state = dict(case=case, p=p, grad=grad, step=torch.full((1,), STEP, device=dev, dtype=torch.int32))
    if case["shadow"]:
        state["shadow"] = p.to(torch.bfloat16)
    if case["bits"] == 8:
        state["m"], state["m_scale"] = _quantise(m, False)
        state["v"], state["v_scale"] = _quantise(v.sqrt_(), True)
    else:
        state["m"], state["v"] = m, v
    if own:
        import lora_rank_adapter_amd as L

        def views(t):
            return [t[s:s + n] for s, n in zip(starts, sizes)]

        held = {k: state[k] for k in ("step", "m", "v", "m_scale", "v_scale") if k in state}
        state["opt"] = L.AdamW(views(p), views(grad), lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY,
                               state_bits=case["bits"], state=held,
                               shadows=views(state["shadow"]) if case["shadow"] else None)
    return state


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _quantise(x, positive):
    """Blocks of 256 elements as e4m3 codes times a float32 scale (the block's
    largest magnitude over 448; a block below 1e-30 is stored as zeros).
    positive: an element above zero keeps at least the smallest code."""
    b = x.view(-1, BLOCK)
    amax = b.abs().amax(1, keepdim=True)
    some = amax >= 1e-30
    scaled = b * torch.where(some, FP8_MAX / amax, torch.zeros_like(amax))
    code = scaled.to(torch.float8_e4m3fn)
    if positive:
        least = torch.full_like(scaled, FP8_MIN).to(torch.float8_e4m3fn)
        keep = (scaled > 0) & (scaled <= FP8_MIN / 2)
        code = torch.where(keep, least.view(torch.uint8), code.view(torch.uint8)).view(torch.float8_e4m3fn)
    return code.view(-1), torch.where(some, amax / FP8_MAX, torch.zeros_like(amax)).view(-1)


def _values(code, scale):
    return (code.float().view(-1, BLOCK) * scale[:, None]).view(-1)


def _plain_embed(state):
    case, ids, table = state["case"], state["ids"].long(), state["data"]
    ok = (ids >= 0) & (ids < case["rows"])
    out = table[torch.where(ok, ids, 0)].float() * case["scale"]
    return {"out": torch.where(ok[:, None], out, 0.0).to(_DT[case["out"]])}


def _plain_embed_grad(state):
    case, ids, dy = state["case"], state["ids"].long(), state["data"]
    ok = (ids >= 0) & (ids < case["rows"])
    grad = torch.zeros(case["rows"] + 1, case["cols"], device=dy.device)
    grad.index_add_(0, torch.where(ok, ids, case["rows"]), dy.float())
    return {"dtable": (grad[:-1] * case["scale"]).to(_DT[case["out"]])}


def _plain_logp(state):
    """The masked tokens' log probabilities (0 where masked), the softmax's
    exponentials and their sums, the mask and the targets with 0 where masked."""
    x = state["logits"].float()
    t = state["targets"].long()
    ok = (t >= 0) & (t < x.shape[1])
    at = torch.where(ok, t, 0)[:, None]
    top = x.amax(1, keepdim=True)
    picked = x.gather(1, at) - top
    e = x.sub_(top).exp_() if x.dtype != state["logits"].dtype else torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    logp = torch.where(ok, (picked - torch.log(total))[:, 0], 0.0)
    return logp, e, total, ok, at


def _plain_logit_grad(e, total, ok, at, coef, dtype):
    """coef * (one at the target - softmax), zero rows where masked."""
    c = torch.where(ok, coef, 0.0)[:, None]
    grad = e.mul_(-c / total)
    grad.scatter_(1, at, grad.gather(1, at) + c)
    return grad.to(dtype)


def _plain_pref(state):
    case, off = state["case"], state["offsets"].long()
    logp, e, total, ok, at = _plain_logp(state)
    sums = torch.cat([torch.zeros(1, device=logp.device, dtype=torch.float64), logp.double().cumsum(0)])[off]
    seq = sums[1:] - sums[:-1]
    gain = (seq - state["ref_logp"].double()).view(-1, 2)
    z = BETA * (gain[:, 0] - gain[:, 1])
    loss = ((1 - SMOOTHING) * torch.log1p(torch.exp(-z.abs())) + SMOOTHING * torch.log1p(torch.exp(-z.abs()))
            + (1 - SMOOTHING) * (-z).clamp_min(0) + SMOOTHING * z.clamp_min(0)).mean()
    out = {"loss": loss.float(), "seq_logp": seq.float(), "logp": logp}
    if case["train"]:
        # d loss / d z = smoothing * sigmoid(z) - (1 - smoothing) * sigmoid(-z)
        dz = (SMOOTHING - 1 / (1 + torch.exp(z))) * BETA / case["pairs"]
        per_seq = torch.stack([dz, -dz], 1).view(-1).float()
        coef = per_seq[torch.bucketize(torch.arange(len(logp), device=logp.device), off[1:], right=True)]
        out["dlogits"] = _plain_logit_grad(e, total, ok, at, coef, state["logits"].dtype)
    return out


def _plain_policy(state):
    logp, e, total, ok, at = _plain_logp(state)
    adv, w = state["advantages"], state["weights"]
    ratio = torch.exp(logp - state["old_logp"])
    held = ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH)
    free = ~(ratio * adv > held * adv)
    k = state["ref_logp"] - logp
    each = -torch.where(free, ratio * adv, held * adv) + KL_COEF * (torch.expm1(k) - k)
    loss = torch.where(ok, w * each, 0.0).double().sum()
    coef = w * (-torch.where(free, ratio * adv, 0.0) - KL_COEF * torch.expm1(k))
    return {"loss": loss.float(), "logp": logp,
            "dlogits": _plain_logit_grad(e, total, ok, at, coef, state["logits"].dtype)}


def _plain_adamw(state):
    case = state["case"]
    state["step"] += 1
    t = state["step"].double()
    alpha = (LR / (1 - BETA1 ** t)).float()
    root = torch.sqrt(1 - BETA2 ** t).float()
    g = state["grad"].float()
    if case["bits"] == 8:
        m, v = _values(state["m"], state["m_scale"]), _values(state["v"], state["v_scale"]).square_()
    else:
        m, v = state["m"], state["v"]
    m = m.mul_(BETA1).add_(g * (1 - BETA1))
    v = v.mul_(BETA2).add_(g * g * (1 - BETA2))
    p = state["p"].float() * (1 - LR * DECAY) - alpha * m / (torch.sqrt(v) / root + EPS)
    state["p"].copy_(p)
    if case["shadow"]:
        state["shadow"].copy_(p)
    if case["bits"] == 8:
        code, scale = _quantise(m, False)
        state["m"].copy_(code)
        state["m_scale"].copy_(scale)
        code, scale = _quantise(torch.sqrt(v), True)
        state["v"].copy_(code)
        state["v_scale"].copy_(scale)


def run(state):
    case = state["case"]
    op = case["op"]
    if op == "adamw":
        if own:
            state["opt"].step()
        else:
            _plain_adamw(state)
        return {k: state[k] for k in ("p", "shadow", "m", "v", "m_scale", "v_scale", "step") if k in state}
    if not own:
        return {"embed": _plain_embed, "embed_grad": _plain_embed_grad, "pref": _plain_pref,
                "policy": _plain_policy}[op](state)
    import lora_rank_adapter_amd as L
    if op == "embed":
        return {"out": L.lora_embed(state["ids"], state["data"], case["scale"], dtype=_DT[case["out"]])}
    if op == "embed_grad":
        return {"dtable": L.lora_embed_grad(state["ids"], state["data"], case["rows"], case["scale"],
                                            dtype=_DT[case["out"]])}
    if op == "policy":
        loss, logp, dlogits = L.lora_policy_step(state["logits"], state["targets"], state["old_logp"],
                                                 state["advantages"], state["weights"], CLIP_LOW, CLIP_HIGH,
                                                 ref_logp=state["ref_logp"], kl_coef=KL_COEF)
        return {"loss": loss, "logp": logp, "dlogits": dlogits}
    if case["train"]:
        loss, seq, logp, dlogits = L.lora_pref_step(state["logits"], state["targets"], state["offsets"],
                                                    state["ref_logp"], BETA, SMOOTHING)
        return {"loss": loss, "seq_logp": seq, "logp": logp, "dlogits": dlogits}
    logp, _ = L.lora_token_logp(state["logits"], state["targets"])
    loss, seq, _ = L.lora_pref_loss(logp, state["offsets"], state["ref_logp"], BETA, SMOOTHING)
    return {"loss": loss, "seq_logp": seq, "logp": logp}


# ---------------------------------------------------------------------------
# the definitions in float64
# ---------------------------------------------------------------------------

def _round_e4m3(x):
    """Nearest e4m3 value (ties to even): 3 fraction bits, exponents from -6, subnormals of 2^-9."""
    _, ex = torch.frexp(x)
    step = torch.exp2((ex - 1).clamp(min=-6).double() - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    op = case["op"]
    state = prepare(case, seed)
    if op == "embed":
        rows = torch.cat([state["data"], state["data"].new_zeros(1, case["cols"])])
        ids = state["ids"].long()
        ids[(ids < 0) | (ids >= case["rows"])] = case["rows"]
        return {"out": rows[ids].double() * case["scale"]}
    if op == "embed_grad":
        # the running sum over the tokens in order of their ids, taken at each id's last token
        ids = state["ids"].long()
        keep = (ids >= 0) & (ids < case["rows"])
        ids, order = torch.sort(ids[keep])
        ends = torch.searchsorted(ids, torch.arange(case["rows"], device=ids.device), right=True)
        cols = []
        for part in state["data"][keep].split(512, 1):
            run_sum = torch.cumsum(part[order].double(), 0)
            run_sum = torch.cat([run_sum.new_zeros(1, part.shape[1]), run_sum])[ends]
            cols.append(torch.diff(run_sum, dim=0, prepend=run_sum.new_zeros(1, part.shape[1])) * case["scale"])
        return {"dtable": torch.cat(cols, 1)}
    if op in ("pref", "policy"):
        T, V = case["tokens"], case["vocab"]
        logits, targets = state["logits"], state["targets"].tolist()
        logp = torch.zeros(T, dtype=torch.float64, device="cuda")
        probs_of = []
        for a in range(0, T, 512):
            x = logits[a:a + 512].double()
            probs_of.append(torch.logsumexp(x, 1))
            for i, t in enumerate(targets[a:a + 512]):
                if 0 <= t < V:
                    logp[a + i] = x[i, t] - probs_of[-1][i]
        lse = torch.cat(probs_of)
        bounds = state["offsets"].tolist()
        coef = torch.zeros(T, dtype=torch.float64, device="cuda")
        if op == "pref":
            seq = torch.stack([logp[a:b].sum() for a, b in zip(bounds[:-1], bounds[1:])])
            ref = state["ref_logp"].double()
            loss = 0.0
            for p in range(case["pairs"]):
                z = BETA * ((seq[2 * p] - ref[2 * p]) - (seq[2 * p + 1] - ref[2 * p + 1]))
                loss = loss - ((1 - SMOOTHING) * torch.nn.functional.logsigmoid(z)
                               + SMOOTHING * torch.nn.functional.logsigmoid(-z)) / case["pairs"]
                d = BETA / case["pairs"] * (SMOOTHING * torch.sigmoid(z) - (1 - SMOOTHING) * torch.sigmoid(-z))
                coef[bounds[2 * p]:bounds[2 * p + 1]] = d
                coef[bounds[2 * p + 1]:bounds[2 * p + 2]] = -d
            out = {"loss": loss, "seq_logp": seq, "logp": logp}
            if not case["train"]:
                return out
        else:
            old, ref, adv, w = (state[k].double() for k in ("old_logp", "ref_logp", "advantages", "weights"))
            on = torch.tensor([0 <= t < V for t in targets], device="cuda")
            x = logp.clone().requires_grad_()
            r = torch.exp(x - old)
            term = -torch.minimum(r * adv, torch.clamp(r, 1 - CLIP_LOW, 1 + CLIP_HIGH) * adv)
            term = term + KL_COEF * (torch.exp(ref - x) - (ref - x) - 1)
            loss = (w * term)[on].sum()
            coef, = torch.autograd.grad(loss, x)
            out = {"loss": loss.detach(), "logp": logp}
        grads = []
        for a in range(0, T, 512):
            b = min(T, a + 512)
            d = -torch.softmax(logits[a:b].double(), 1)
            hit = torch.tensor([[i, t] for i, t in enumerate(targets[a:b]) if 0 <= t < V], device="cuda")
            off = torch.tensor([not 0 <= t < V for t in targets[a:b]], device="cuda")
            if len(hit):
                d[hit[:, 0], hit[:, 1]] += 1.0
            d *= coef[a:b, None]
            d[off] = 0.0
            # kept in 32 bits: half a step of 2^-24 is far below what the outputs' types allow
            grads.append(d.float() if T * V > 1 << 28 else d)
        out["dlogits"] = torch.cat(grads)
        return out
    # AdamW
    t = STEP + 1
    g, p = state["grad"].double(), state["p"].double()
    m, v = state["m"].double(), state["v"].double()
    if case["bits"] == 8:
        m = (m.view(-1, BLOCK) * state["m_scale"].double()[:, None]).view(-1)
        v = ((v.view(-1, BLOCK) * state["v_scale"].double()[:, None]) ** 2).view(-1)
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g ** 2
    p = p - LR * DECAY * p - LR * (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + EPS)
    out = {"p": p, "step": t}
    if case["shadow"]:
        out["shadow"] = p
    if case["bits"] == 32:
        return dict(out, m=m, v=v)
    for name, x in (("m", m), ("v", v.sqrt())):
        b = x.view(-1, BLOCK)
        scale = b.abs().amax(1) / FP8_MAX
        q = _round_e4m3(b / torch.where(scale > 0, scale, 1.0)[:, None])
        if name == "v":
            q = torch.where((b > 0) & (q == 0), FP8_MIN, q)
        out[name], out[name + "_scale"] = q.view(-1), scale
    return out


def work(case):
    op = case["op"]
    if op in ("embed", "embed_grad"):
        T, V, D = case["tokens"], case["rows"], case["cols"]
        if op == "embed":  # each row that occurs is read once
            share = np.diff(np.log(np.arange(1, V + 2))) / math.log(V + 1)
            rows = float(np.sum(1 - (1 - share) ** T))
            return {"bytes": 4 * T + rows * D * _ES[case["dtype"]] + T * D * _ES[case["out"]], "flops": T * D}
        return {"bytes": 4 * T + T * D * _ES[case["dtype"]] + V * D * _ES[case["out"]], "flops": 2 * T * D}
    if op in ("pref", "policy"):
        live = sum(r for _, r in _sequences(case))  # masked rows need not be read
        grad = case["op"] == "policy" or case["train"]
        size = case["vocab"] * _ES[case["dtype"]]
        return {"bytes": live * size + (case["tokens"] * size if grad else 0) + 24 * case["tokens"],
                "flops": (7 if grad else 4) * live * case["vocab"]}
    n = sum(_tensor_sizes(case))
    state_bytes = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    per = 2 * _ES[case["param"]] + _ES[case["grad"]] + (2 if case["shadow"] else 0) + state_bytes
    return {"bytes": n * per, "flops": 16 * n}
