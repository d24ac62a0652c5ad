"""Fine-tunes an adapter and an embedding table on synthetic preference pairs.

One step runs the library's operators as a training loop would: the embedding
lookup, a linear layer with its adapter, the loss on the next token's logits
with their gradient, the adapter's backward, the table's gradient and one
AdamW step over all three weights. The frozen projections around them are
torch products. Two vocabularies of tokens answer the prompts; the preference
and the policy loss learn to prefer the first, distillation learns the top
tokens of a teacher, a model with other weights.

    python examples/adapter_training.py --loss pref --steps 40
    python examples/adapter_training.py --loss policy --state-bits 8
    python examples/adapter_training.py --loss distill
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import lora_rank_adapter_amd as L  # noqa: E402


def make_batch(pairs, length, vocab, device, seed=0):
    """Packed sequences of odd lengths, a third of each a prompt (masked in the targets): the preferred one of a
    pair answers with tokens of the vocabulary's lower half, the other with the upper half's."""
    g = torch.Generator().manual_seed(seed)
    ids, targets, offsets = [], [], [0]
    for s in range(2 * pairs):
        n = length - s % 3
        half = vocab // 2
        answer = torch.randint(0, half, (n,), generator=g) + (half if s % 2 else 0)
        prompt = n // 3
        answer[:prompt] = torch.randint(0, vocab, (prompt,), generator=g)
        follows = torch.cat([answer[1:], answer[:1]])
        follows[:prompt] = -100
        follows[-1] = -100
        ids.append(answer)
        targets.append(follows)
        offsets.append(offsets[-1] + n)

    def dev(x):
        return torch.as_tensor(x, dtype=torch.int32).to(device)

    return dev(torch.cat(ids)), dev(torch.cat(targets)), dev(offsets)


class AdapterTrainer:
    """Weights in float32, the copies that the forward reads in `dtype` (bfloat16, or float32 itself)."""

    def __init__(self, vocab, width, rank, lr=2e-3, state_bits=32, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, std):
            return torch.randn(*shape, device=device, generator=g) * std

        self.vocab, self.scale, self.dtype = vocab, 2.0, dtype
        self.base = normal(width, width, std=width ** -0.5).to(dtype)  # frozen: y = x base
        self.head = normal(width, vocab, std=width ** -0.5).to(dtype)  # frozen: logits = y head
        # A: width x rank, B: rank x width, the layouts of their gradients
        self.weights = [normal(width, rank, std=width ** -0.5), normal(rank, width, std=0.02),
                        normal(vocab, width, std=1.0)]
        half = dtype is torch.bfloat16
        self.read = [w.to(dtype) for w in self.weights] if half else self.weights
        self.grads = [torch.empty_like(w) for w in self.weights]
        self.opt = L.AdamW(self.weights, self.grads, lr, weight_decay=0.0, state_bits=state_bits,
                           shadows=self.read if half else None)

    def logits(self, ids):
        """(embedded tokens, logits)"""
        A, B, table = self.read
        x = L.lora_embed(ids, table)
        y = (x @ self.base).float()
        L.lora_fwd(x, A, B, y, self.scale)
        return x, y.to(self.dtype) @ self.head

    def logp(self, ids, targets):
        return L.lora_token_logp(self.logits(ids)[1], targets)[0]

    def backward(self, ids, x, dlogits):
        """The gradients of A, B and the table into self.grads."""
        A, B, _ = self.read
        dy = dlogits @ self.head.t()
        dx = (dy @ self.base.t()).float()
        L.lora_bwd_dx_da_accumulate(x.t(), dy, B.t(), A.t(), self.scale, dx, dA=self.grads[0])
        L.lora_bwd_db(A.t(), x.t(), dy, self.scale, dB=self.grads[1])
        L.lora_embed_grad(ids, dx, self.vocab, dtable=self.grads[2])

    def pref_step(self, ids, targets, offsets, ref_logp, beta=0.1):
        x, logits = self.logits(ids)
        loss, _, _, dlogits = L.lora_pref_step(logits, targets, offsets, ref_logp, beta, dlogits=logits)
        self.backward(ids, x, dlogits)
        self.opt.step()
        return loss

    def policy_step(self, ids, targets, old_logp, advantages, weights, ref_logp, kl_coef=0.02):
        x, logits = self.logits(ids)
        loss, _, dlogits = L.lora_policy_step(logits, targets, old_logp, advantages, weights, 0.2, 0.28, ref_logp,
                                              kl_coef, dlogits=logits)
        self.backward(ids, x, dlogits)
        self.opt.step()
        return loss

    def top(self, ids, targets, k, temperature):
        """What a student is given of this model: its k top tokens of each unmasked place at a temperature."""
        return L.lora_token_top(self.logits(ids)[1], targets, k, temperature)[2:4]

    def distill_step(self, ids, top_ids, top_logp, weights, temperature):
        x, logits = self.logits(ids)
        loss, _, dlogits = L.lora_distill_step(logits, top_ids, top_logp, weights, temperature, dlogits=logits)
        self.backward(ids, x, dlogits)
        self.opt.step()
        return loss


def sequence_sums(logp, offsets):
    o = offsets.tolist()
    return torch.stack([logp[a:b].sum() for a, b in zip(o[:-1], o[1:])])


def train(loss="pref", steps=40, state_bits=32, pairs=6, length=40, vocab=1000, width=256, rank=8, seed=0):
    """Returns (the losses, the pairs' log-probability gains of the preferred answer over the other)."""
    t = AdapterTrainer(vocab, width, rank, state_bits=state_bits, seed=seed)
    ids, targets, offsets = make_batch(pairs, length, vocab, "cuda", seed)
    start = t.logp(ids, targets)  # the reference model is the model before training
    ref = sequence_sums(start, offsets)
    losses = []
    if loss == "policy":
        lengths = (offsets[1:] - offsets[:-1]).long()
        advantages = torch.tensor([1.0, -1.0], device="cuda").repeat(pairs).repeat_interleave(lengths)
        weights = torch.full_like(start, 1.0 / int((targets >= 0).sum()))
    for step in range(steps):
        if loss == "pref":
            losses.append(t.pref_step(ids, targets, offsets, ref))
        else:
            if step % 4 == 0:  # four steps on what the policy of the first one sampled
                old = t.logp(ids, targets)
            losses.append(t.policy_step(ids, targets, old, advantages, weights, start))
    gain = (sequence_sums(t.logp(ids, targets), offsets) - ref).view(pairs, 2)
    return torch.stack(losses).tolist(), (gain[:, 0] - gain[:, 1]).tolist()


def distill(steps=40, state_bits=32, pairs=6, length=40, vocab=1000, width=256, rank=8, k=16, temperature=2.0, seed=0):
    """A student learns from a teacher that differs from it in the table and the adapter. Returns the losses."""
    t = AdapterTrainer(vocab, width, rank, state_bits=state_bits, seed=seed)
    teacher = AdapterTrainer(vocab, width, rank, seed=seed + 1)
    teacher.base, teacher.head = t.base, t.head
    ids, targets, _ = make_batch(pairs, length, vocab, "cuda", seed)
    top_ids, top_logp = teacher.top(ids, targets, k, temperature)
    weights = torch.full((len(ids),), temperature ** 2 / int((targets >= 0).sum()), device="cuda")
    return torch.stack([t.distill_step(ids, top_ids, top_logp, weights, temperature) for _ in range(steps)]).tolist()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--loss", choices=("pref", "policy", "distill"), default="pref")
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--state-bits", type=int, choices=(8, 32), default=32)
    a = ap.parse_args()
    if a.loss == "distill":
        losses, gains = distill(a.steps, a.state_bits), None
    else:
        losses, gains = train(a.loss, a.steps, a.state_bits)
    for i in range(0, a.steps, max(1, a.steps // 10)):
        print(f"step {i:4d}  loss {losses[i]:.4f}")
    print(f"step {a.steps - 1:4d}  loss {losses[-1]:.4f}")
    if gains is not None:
        print("log-probability gain of the preferred answers:", " ".join(f"{g:.1f}" for g in gains))


if __name__ == "__main__":
    main()
