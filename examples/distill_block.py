"""Distil a teacher into a one-block GPT-2-type student, with every product, the
attention, the loss and their gradients in this library's kernels.

    python examples/distill_block.py [--steps 60]

The student: token embeddings, a causal self-attention block (qkv, attention,
projection with residual), a feed-forward block (GELU, residual) and an LM head
whose vocabulary is padded to whole 16-byte units. The teacher is synthetic: for
every token a list of likely next tokens with their logits, as a file of a large
model's top logits would give them. A step:

    logits  = head(block(x))
    loss, dlogits = tll.distill_forward_backward(...)   # in place of the logits
    ... backward products ...
    dqkv    = tll.attention_backward(qkv, a, lse, da, ...)

and after training tll.token_logprobs scores the teacher's first choice under the
student, with the entropy of its distribution and its own first choices.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import transformer_linear_layer_gb300 as tll  # noqa: E402


class Student:
    """Weights out x in, fp32 masters with bf16 copies for the products."""

    def __init__(self, V, H, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        C = 64 * H
        self.V, self.H, self.C = V, H, C
        pad = (V + 7) // 8 * 8  # rows of the logits in whole 16-byte units
        sizes = {"embed": (V, C), "qkv": (3 * C, C), "proj": (C, C), "fc1": (4 * C, C), "fc2": (C, 4 * C), "head": (pad, C)}
        self.master = {k: (torch.randn(s, generator=g) * (1.0 if k == "embed" else s[1] ** -0.5)).to(device)
                       for k, s in sizes.items()}
        self.master["head"][V:] = 0  # padded tokens: logits 0, never read
        self.refresh()

    def refresh(self):
        self.w = {k: v.bfloat16() for k, v in self.master.items()}

    def logits(self, tokens):
        """The padded logits ((B*T) x padded vocabulary) and what backward needs."""
        B, T = tokens.shape
        w = self.w
        x0 = w["embed"][tokens.reshape(-1)]
        qkv = tll.forward(x0, w["qkv"])
        a, lse = tll.attention_forward(qkv, B, T, self.H, causal=True, with_lse=True)
        x1 = tll.forward_residual(a, w["proj"], x0)
        z = tll.forward(x1, w["fc1"])
        h = torch.nn.functional.gelu(z, approximate="tanh")
        x2 = tll.forward_residual(h, w["fc2"], x1)
        return tll.forward(x2, w["head"]), (tokens, x0, qkv, a, lse, x1, z, h, x2)

    def backward(self, dlogits, saved):
        """Gradients of the masters from the padded logits' gradient."""
        tokens, x0, qkv, a, lse, x1, z, h, x2 = saved
        B, T = tokens.shape
        w, grad = self.w, {}
        grad["head"], _ = tll.backward_weight(dlogits, x2)
        dx2 = tll.backward_data(dlogits, w["head"])
        grad["fc2"], _ = tll.backward_weight(dx2, h)
        dz = tll.backward_data_gelu(dx2, w["fc2"], z)
        grad["fc1"], _ = tll.backward_weight(dz, x1)
        dx1 = dx2 + tll.backward_data(dz, w["fc1"])
        grad["proj"], _ = tll.backward_weight(dx1, a)
        da = tll.backward_data(dx1, w["proj"])
        dqkv = tll.attention_backward(qkv, a, lse, da, B, T, self.H, causal=True)
        grad["qkv"], _ = tll.backward_weight(dqkv, x0)
        dx0 = dx1 + tll.backward_data(dqkv, w["qkv"])
        grad["embed"] = torch.zeros_like(self.master["embed"]).index_add_(0, tokens.reshape(-1), dx0.float())
        return grad

    def step(self, tokens, ids, teacher, temperature=1.0):
        """(mean loss, gradients) of one batch."""
        buf, saved = self.logits(tokens)
        rows = buf.shape[0]
        z = buf[:, :self.V]
        weight = torch.full((rows,), 1.0 / rows, device=buf.device)
        # the gradient takes the logits' place; the padding stays 0
        loss, _ = tll.distill_forward_backward(z, ids, teacher, weight=weight, temperature=temperature, out=z)
        return loss.mean(), self.backward(buf, saved)


def make_teacher(V, K, seed=1, device="cuda"):
    """For every token K distinct next tokens with logits, most likely first."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(V)])
    logits = (torch.randn(V, K, generator=g) * 2).sort(dim=1, descending=True).values
    return ids.int().to(device), logits.to(device)


def train(steps=60, V=1003, H=2, B=16, T=64, K=16, lr=3e-3, temperature=1.0, seed=0, log=print):
    """Losses of every step and the final evaluation (a TokenLogprobs)."""
    student = Student(V, H, seed)
    ids, teacher = make_teacher(V, K)
    g = torch.Generator().manual_seed(seed + 2)
    moments = {k: (torch.zeros_like(v), torch.zeros_like(v)) for k, v in student.master.items()}
    losses = []
    for n in range(1, steps + 1):
        tokens = torch.randint(0, V, (B, T), generator=g).cuda()
        flat = tokens.reshape(-1)
        loss, grad = student.step(tokens, ids[flat], teacher[flat], temperature)
        for k, v in student.master.items():  # Adam
            m, s = moments[k]
            d = grad[k].float()
            m.mul_(0.9).add_(d, alpha=0.1)
            s.mul_(0.99).addcmul_(d, d, value=0.01)
            v.sub_(lr * (m / (1 - 0.9 ** n)) / ((s / (1 - 0.99 ** n)).sqrt() + 1e-8))
        student.refresh()
        losses.append(loss)
        if n % 20 == 0 or n == 1:
            log(f"step {n:4d}  loss {loss.item():.4f}")
    tokens = torch.randint(0, V, (B, T), generator=g).cuda()
    best = ids[tokens.reshape(-1), 0].contiguous()
    buf, _ = student.logits(tokens)
    score = tll.token_logprobs(buf[:, :V], best, top=5)
    log(f"teacher's first choice: mean log probability {score.logprob.mean().item():.3f}, "
        f"among the student's first five {(score.top_ids == best[:, None]).any(1).float().mean().item():.2f}; "
        f"entropy {score.entropy.mean().item():.3f} nats")
    tll.default_context(0).check()
    return [x.item() for x in losses], score


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    train(ap.parse_args().steps)
