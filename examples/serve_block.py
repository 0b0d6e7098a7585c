"""A one-block decoder with rotary positions: its training pass over whole
sequences, and serving it from a paged cache, prompts in chunks and then token by
token in a captured graph. Every product, the rotations, the attention and their
gradients run in this library's kernels.

    python examples/serve_block.py [--prompts 5] [--steps 24]

Training pass (Block.logits, Block.backward):

    qkv = x Wqkv';  q and k columns rotated in place (rotary_forward)
    a, lse = attention_forward(qkv);  ...;  dqkv = attention_backward(...)
    dq and dk columns turned back in place (rotary_backward)

Serving (Server): new tokens of all sequences are rows of one batch.

    qkv = x Wqkv';  q = cache_append(q, k, v, cache, batch, rotary)   # k rotated on the way into its page
    a = paged_attention(q, cache, batch)

The served logits are those of the training pass over the same tokens, up to the
roundings on the way.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import transformer_linear_layer_gb300 as tll  # noqa: E402

D = 64  # width of a head


class Block:
    """Token embeddings, attention, feed-forward and LM head; weights out x in, bf16."""

    def __init__(self, V, H, rotary, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        C = D * H
        self.V, self.H, self.C, self.rotary = V, H, C, rotary
        sizes = {"embed": (V, C), "qkv": (3 * C, C), "proj": (C, C), "fc1": (4 * C, C), "fc2": (C, 4 * C),
                 "head": ((V + 7) // 8 * 8, C)}
        self.w = {k: (torch.randn(s, generator=g) * (1.0 if k == "embed" else s[1] ** -0.5)).bfloat16().to(device)
                  for k, s in sizes.items()}

    def rest(self, a, x0):
        """From the attention's output to the (padded) logits, and what backward needs."""
        w = self.w
        x1 = tll.forward_residual(a, w["proj"], x0)
        z = tll.forward(x1, w["fc1"])
        h = torch.nn.functional.gelu(z, approximate="tanh")
        x2 = tll.forward_residual(h, w["fc2"], x1)
        return tll.forward(x2, w["head"]), (x1, z, h, x2)

    def heads(self, qkv):
        """The q and k columns of a qkv matrix as rows of heads."""
        return qkv[:, :2 * self.C].unflatten(1, (2 * self.H, D))

    def logits(self, tokens):
        B, T = tokens.shape
        x0 = self.w["embed"][tokens.reshape(-1)]
        positions = torch.arange(T, device=x0.device).repeat(B)
        qkv = tll.forward(x0, self.w["qkv"])
        turned = self.heads(qkv)
        tll.rotary_forward(turned, positions, self.rotary, out=turned)
        a, lse = tll.attention_forward(qkv, B, T, self.H, causal=True, with_lse=True)
        out, saved = self.rest(a, x0)
        return out, (tokens, positions, x0, qkv, a, lse, *saved)

    def backward(self, dlogits, saved):
        """Gradients of the weights from the padded logits' gradient."""
        tokens, positions, x0, qkv, a, lse, x1, z, h, x2 = saved
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
        turned = self.heads(dqkv)
        tll.rotary_backward(turned, positions, self.rotary, out=turned)
        grad["qkv"], _ = tll.backward_weight(dqkv, x0)
        dx0 = dx1 + tll.backward_data(dqkv, w["qkv"])
        grad["embed"] = torch.zeros(w["embed"].shape, device=dx0.device).index_add_(0, tokens.reshape(-1), dx0.float())
        return grad


class Server:
    """Sequences served from a paged cache; every sequence may grow to `longest` tokens."""

    def __init__(self, block, sequences, longest, page=16, seed=0, device="cuda"):
        self.block, self.B = block, sequences
        each = -(-longest // page)
        kv = torch.zeros(sequences * each + 1, 2, block.H, page, D, dtype=torch.bfloat16, device=device)
        self.cache = tll.KVCache(kv[:, 0], kv[:, 1])
        pages = torch.randperm(sequences * each + 1, generator=torch.Generator().manual_seed(seed))[:sequences * each]
        self.held = torch.zeros(sequences, dtype=torch.int32, device=device)
        self.q_start = torch.zeros(sequences + 1, dtype=torch.int32, device=device)
        self.batch = tll.KVBatch(self.q_start, self.held, pages.int().reshape(sequences, each).to(device))

    def rows(self, tokens, longest):
        """Logits of the rows that q_start and held describe."""
        b = self.block
        x0 = b.w["embed"][tokens]
        qkv = tll.forward(x0, b.w["qkv"]).unflatten(1, (3 * b.H, D))
        q = tll.cache_append(qkv[:, :b.H], qkv[:, b.H:2 * b.H], qkv[:, 2 * b.H:], self.cache, self.batch, rotary=b.rotary)
        a = tll.paged_attention(q, self.cache, self.batch, max_new=longest)
        return b.rest(a.flatten(1), x0)[0]

    def extend(self, new):
        """Logits of lists of new tokens, one (perhaps empty) per sequence."""
        lengths = torch.tensor([len(t) for t in new], dtype=torch.int32)
        self.held += lengths.to(self.held.device)
        self.q_start[1:] = lengths.cumsum(0).to(self.held.device)
        tokens = torch.tensor([t for row in new for t in row], device=self.held.device)
        return self.rows(tokens, int(lengths.max()))

    def capture(self):
        """One step for one token of each sequence as a graph: tokens in, logits and the likeliest
        next tokens out, in place."""
        self.q_start.copy_(torch.arange(self.B + 1))
        tokens = torch.zeros(self.B, dtype=torch.int64, device=self.held.device)

        def step():
            self.held.add_(1)
            logits = self.rows(tokens, 1)
            best = tll.token_logprobs(logits[:, :self.block.V], top=1)
            tokens.copy_(best.top_ids[:, 0])
            return logits, best

        kept = self.held.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()  # first launches; what it leaves in the cache is written again
        torch.cuda.current_stream().wait_stream(side)
        self.held.copy_(kept)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            logits, best = step()
        self.held.copy_(kept)
        return graph, tokens, logits, best


def serve(prompts=5, steps=24, V=1003, H=4, chunk=50, seed=0, log=print):
    """Greedy continuations of random prompts; (sequences, the logits of every generated place, block)."""
    rotary = tll.Rotary(D, scaling="yarn", factor=4.0, original_length=256)
    block = Block(V, H, rotary, seed)
    g = torch.Generator().manual_seed(seed + 1)
    text = [torch.randint(0, V, (int(torch.randint(1, 3 * chunk, (1,), generator=g)),), generator=g).tolist()
            for _ in range(prompts)]
    server = Server(block, prompts, max(map(len, text)) + steps + 1)
    last = [None] * prompts
    for at in range(0, max(map(len, text)), chunk):  # prompts in chunks; a finished one has no rows
        parts = [t[at:at + chunk] for t in text]
        logits, row = server.extend(parts), 0
        for b, part in enumerate(parts):
            row += len(part)
            if part:
                last[b] = logits[row - 1]
    first = torch.stack(last)
    graph, tokens, logits, best = server.capture()
    tokens.copy_(tll.token_logprobs(first[:, :V].contiguous(), top=1).top_ids[:, 0])
    seen = [first.clone()]
    for _ in range(steps):
        for t, n in zip(text, tokens.tolist()):
            t.append(n)
        graph.replay()
        seen.append(logits.clone())
    tll.default_context(0).check()
    log(f"{prompts} sequences of {min(map(len, text))} to {max(map(len, text))} tokens, {steps} of them generated")
    return text, torch.stack(seen, 1), block


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--prompts", type=int, default=5)
    ap.add_argument("--steps", type=int, default=24)
    args = ap.parse_args()
    serve(args.prompts, args.steps)
