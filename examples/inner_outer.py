"""DiLoCo on one GPU: K learners take inner steps, then one outer step merges them.

Every learner trains its own copy of a small residual model (embedding, blocks of
layer norm and MLP, with --attention also of causal attention on rotary queries and
keys, final norm, output layer) on its own synthetic data. The inner step is the
library's: layer norms, rotary positions and the tokens' log probabilities forward and
backward, clipping by the global gradient norm, AdamW over the learner's flat fragments
with 8- or 32-bit states.
After H of them the outer step quantises the learners' pseudo-gradients, merges them
and applies the outer Nesterov update to the global parameters, from which the
learners go on.

    python examples/inner_outer.py [--learners 3] [--rounds 5] [--inner 20] [--bits 8]
                                   [--attention]

The memory layout is what makes the two halves meet without a copy: a learner's fp32
parameters are one flat buffer per fragment; the model's bf16 weights are views into
the rounded copy that AdamW writes beside them, and their .grad views into one flat
gradient buffer.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import pseudo_grad_sync_gb300 as dl  # noqa: E402

VOCAB, WIDTH, HIDDEN, BLOCKS = 512, 192, 512, 3
TOKENS, SEQ = 512, 64                 # of an inner step; of a sequence
HEADS, KV_HEADS, HEAD = 4, 2, 48      # of the attention: query heads, key and value heads


def shapes(attention=False):
    """name -> shape of every tensor of the model, in order."""
    out = {"embed": (VOCAB, WIDTH)}
    for i in range(BLOCKS):
        if attention:
            out |= {f"{i}.att_norm.w": (WIDTH,), f"{i}.qkv": ((HEADS + 2 * KV_HEADS) * HEAD, WIDTH),
                    f"{i}.att_out": (WIDTH, HEADS * HEAD)}
        out |= {f"{i}.norm.w": (WIDTH,), f"{i}.norm.b": (WIDTH,), f"{i}.up": (HIDDEN, WIDTH),
                f"{i}.down": (WIDTH, HIDDEN)}
    return out | {"norm.w": (WIDTH,), "out": (VOCAB, WIDTH)}


def attend(x, p, i, rotary):
    """Causal attention of sequences of SEQ tokens, on rotary queries and keys."""
    h = dl.layer_norm(x, p[f"{i}.att_norm.w"], rms=True)
    qkv = (h @ p[f"{i}.qkv"].t()).view(-1, SEQ, HEADS + 2 * KV_HEADS, HEAD)
    q, k, v = qkv.split([HEADS, KV_HEADS, KV_HEADS], 2)
    q, k = dl.rotary((q, k), rotary)
    k, v = (t.repeat_interleave(HEADS // KV_HEADS, 2) for t in (k, v))
    a = torch.einsum("bshd,bthd->bhst", q, k).float() * HEAD ** -0.5
    later = torch.ones(SEQ, SEQ, dtype=torch.bool, device=x.device).triu(1)
    a = a.masked_fill(later, float("-inf")).softmax(-1).to(v.dtype)
    y = torch.einsum("bhst,bthd->bshd", a, v).reshape(len(x), -1)
    return y @ p[f"{i}.att_out"].t()


def loss_of(p, tokens, targets, rotary=None):
    x = p["embed"][tokens]
    for i in range(BLOCKS):
        if rotary is not None:
            x = x + attend(x, p, i, rotary)
        h = dl.layer_norm(x, p[f"{i}.norm.w"], p[f"{i}.norm.b"])
        x = x + torch.nn.functional.gelu(h @ p[f"{i}.up"].t()) @ p[f"{i}.down"].t()
    h = dl.layer_norm(x, p["norm.w"], rms=True)
    return -dl.token_logprobs(h @ p["out"].t(), targets).logp.mean()


class Learner:
    """A replica: flat buffers per fragment, the model's views into them, and
    its inner optimiser."""

    def __init__(self, frags, names, theta_g, bits, seed, attention=False):
        sh = shapes(attention)
        self.rotary = dl.RotaryFrequencies(HEAD) if attention else None
        self.theta = [t.clone() for t in theta_g]
        self.copy = [t.to(torch.bfloat16) for t in self.theta]
        self.grad = [torch.zeros_like(c) for c in self.copy]
        self.p = {}
        for F, in_frag, c, g in zip(frags, names, self.copy, self.grad):
            for name, a, b in zip(in_frag, F.offsets, F.offsets[1:]):
                w = c[a:b].view(sh[name]).requires_grad_()
                w.grad = g[a:b].view(sh[name])
                self.p[name] = w
        decay = [[float(len(sh[n]) > 1) for n in in_frag] for in_frag in names]
        self.opt = dl.InnerAdamW(frags, self.theta, self.grad, bits=bits, lr=2e-3,
                                 weight_decay=0.01, decay=decay, theta_bf16=self.copy,
                                 max_norm=1.0, seed=seed)

    def inner_step(self, tokens, targets):
        for g in self.grad:
            g.zero_()
        loss = loss_of(self.p, tokens, targets, self.rotary)
        loss.backward()
        self.opt.step()
        return loss.detach()

    def restart(self, theta_g):
        with torch.no_grad():
            for t, c, g in zip(self.theta, self.copy, theta_g):
                t.copy_(g)
                c.copy_(g)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--learners", type=int, default=3)
    ap.add_argument("--rounds", type=int, default=5)
    ap.add_argument("--inner", type=int, default=20, help="inner steps per outer step")
    ap.add_argument("--bits", type=int, default=8, choices=(8, 32), help="AdamW state width")
    ap.add_argument("--fragments", type=int, default=2)
    ap.add_argument("--attention", action="store_true", help="blocks with rotary attention")
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    sh = shapes(a.attention)
    order = list(sh)
    numel = [torch.Size(sh[n]).numel() for n in order]
    of, _ = dl.plan_fragments(numel, a.fragments)
    names = [[n for n, f in zip(order, of) if f == j] for j in range(a.fragments)]
    frags = [dl.Fragment([torch.Size(sh[n]).numel() for n in f]) for f in names]

    theta_g = []
    for f in names:
        parts = [torch.ones(sh[n]) if n.endswith("norm.w") else torch.zeros(sh[n])
                 if n.endswith("norm.b") else torch.randn(sh[n]) * 0.05 for n in f]
        theta_g.append(torch.cat([t.reshape(-1) for t in parts]).cuda())
    momentum = [torch.zeros_like(t) for t in theta_g]
    learners = [Learner(frags, names, theta_g, a.bits, k, a.attention) for k in range(a.learners)]
    sync = dl.ModelSync(frags, a.learners)

    table = torch.randperm(VOCAB).cuda()      # the task: token -> its partner
    data = torch.Generator(device="cuda").manual_seed(1)
    losses = []
    for r in range(a.rounds):
        total = torch.zeros((), device="cuda")
        for L in learners:
            for _ in range(a.inner):
                tokens = torch.randint(0, VOCAB, (TOKENS,), generator=data, device="cuda")
                total += L.inner_step(tokens, table[tokens])
        sync.step(theta_g, momentum, [[L.theta[j] for L in learners] for j in range(len(frags))])
        for L in learners:
            L.restart(theta_g)
        losses.append(float(total) / (a.learners * a.inner))
        print(f"round {r}: mean inner loss {losses[-1]:.4f}, last gradient norm "
              f"{float(learners[0].opt.clip[0]):.3f}")
    return losses


if __name__ == "__main__":
    main()
