"""Rotary positions, the cache's append and attention over it together, as
examples/serve_block.py trains and serves with them."""
import importlib.util
import os

import pytest
import torch

import transformer_linear_layer_gb300 as tll

pytestmark = pytest.mark.gpu

spec = importlib.util.spec_from_file_location(
    "serve_block", os.path.join(os.path.dirname(__file__), "..", "examples", "serve_block.py"))
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)


def test_served_logits_are_those_of_the_whole_sequence():
    """Prompts in chunks, then a captured step per token, against the training pass over each finished sequence.
    About eight bf16 roundings lie on either way to a row of logits, at different places: 4 % of its norm."""
    text, seen, block = example.serve(prompts=5, steps=24, log=lambda *_: None)
    for t, rows in zip(text, seen):
        whole, _ = block.logits(torch.tensor([t], device="cuda"))
        want = whole[len(t) - 25:, :block.V].double()
        got = rows[:, :block.V].double()
        assert got.shape == want.shape
        assert ((got - want).norm(dim=1) <= 0.04 * want.norm(dim=1)).all()
        # the token that was taken is the likeliest of the logits that were served
        assert torch.equal(got[:-1].argmax(1).cpu(), torch.tensor(t[len(t) - 24:]))


def test_any_cut_of_a_prompt_gives_the_same_rows():
    """One prompt whole, in uneven chunks, and token by token."""
    block = example.Block(503, 3, tll.Rotary(32, interleaved=True), seed=3)
    prompt = torch.randint(0, 503, (150,), generator=torch.Generator().manual_seed(1)).tolist()
    rows = []
    for cuts in ([150], [1, 16, 17, 64, 52], [1] * 150):
        server, at, got = example.Server(block, 1, 150), 0, []
        for n in cuts:
            got.append(server.extend([prompt[at:at + n]]))
            at += n
        rows.append(torch.cat(got)[:, :503].double())
    tll.default_context(0).check()
    for other in rows[1:]:
        assert ((other - rows[0]).norm(dim=1) <= 0.04 * rows[0].norm(dim=1)).all()


def autograd(block, tokens, dlogits):
    """The same gradients by torch in float64, from the bf16 weights."""
    w = {k: v.double().requires_grad_() for k, v in block.w.items()}
    B, T = tokens.shape
    H, C = block.H, block.C
    x0 = w["embed"][tokens.reshape(-1)]
    q, k, v = (x0 @ w["qkv"].T).reshape(B, T, 3, H, 64).permute(2, 0, 3, 1, 4)
    r = block.rotary
    theta = torch.outer(torch.arange(T, dtype=torch.float64, device=q.device),
                        torch.tensor(r.frequencies, dtype=torch.float64, device=q.device))
    turn = torch.polar(torch.full_like(theta, r.scale), theta)

    def rotate(x):
        a, b = x[..., :r.dim // 2], x[..., r.dim // 2:r.dim]
        z = torch.complex(a, b) * turn
        return torch.cat([z.real, z.imag, x[..., r.dim:]], -1)

    a = torch.nn.functional.scaled_dot_product_attention(rotate(q), rotate(k), v, is_causal=True)
    x1 = a.transpose(1, 2).reshape(-1, C) @ w["proj"].T + x0
    x2 = torch.nn.functional.gelu(x1 @ w["fc1"].T, approximate="tanh") @ w["fc2"].T + x1
    ((x2 @ w["head"].T) * dlogits.double()).sum().backward()
    return {k: x.grad for k, x in w.items()}


@pytest.mark.parametrize("rot", [64, 32])
def test_gradients_match_autograd(rot):
    """Activations and gradients pass through about twelve bf16 roundings on the way: each gradient's error
    stays within 4 % of its norm."""
    block = example.Block(503, 3, tll.Rotary(rot, scaling="linear", factor=2.0), seed=2)
    g = torch.Generator().manual_seed(0)
    tokens = torch.randint(0, 503, (3, 70), generator=g).cuda()
    _, saved = block.logits(tokens)
    dlogits = (torch.randn(210, 504, generator=g) * 0.01).bfloat16().cuda()
    got = block.backward(dlogits, saved)
    want = autograd(block, tokens, dlogits)
    for k, d in got.items():
        assert (d.double() - want[k]).norm() <= 0.04 * want[k].norm(), k


def test_two_threads_call_at_once():
    """Append and attention from two threads, each with its own stream, cache and batch, sharing the context."""
    import threading

    r = tll.Rotary(64)
    want, got, errors = {}, {}, []

    def work(n, out):
        try:
            torch.manual_seed(n)
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                g = torch.Generator(device="cuda").manual_seed(n)
                kv = torch.randn(80, 2, 2, 16, 64, device="cuda", generator=g).bfloat16()
                cache = tll.KVCache(kv[:, 0], kv[:, 1])
                i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
                batch = tll.KVBatch(i32(0, 1, 4), i32(600, 333), torch.arange(80, dtype=torch.int32, device="cuda").reshape(2, 40))
                qkv = torch.randn(4, 8, 64, device="cuda", generator=g).bfloat16()
                for _ in range(200):
                    q = tll.cache_append(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], cache, batch, rotary=r)
                    a, lse = tll.paged_attention(q, cache, batch, with_lse=True, max_new=3 + 100 * (n % 2))
                out[n] = a.clone(), lse.clone()
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    for n in range(2):
        work(n, want)
    threads = [threading.Thread(target=work, args=(n, got)) for n in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for n in range(2):
        assert torch.equal(want[n][0], got[n][0]) and torch.equal(want[n][1], got[n][1])
