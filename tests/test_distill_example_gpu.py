"""The operators together, as examples/distill_block.py trains with them."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

spec = importlib.util.spec_from_file_location(
    "distill_block", os.path.join(os.path.dirname(__file__), "..", "examples", "distill_block.py"))
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)


def autograd_step(student, tokens, ids, teacher):
    """The same loss and gradients by torch in float64, from the bf16 weights."""
    w = {k: v.double().requires_grad_() for k, v in student.w.items()}
    B, T = tokens.shape
    C, H, V = student.C, student.H, student.V
    x0 = w["embed"][tokens.reshape(-1)]
    q, k, v = (x0 @ w["qkv"].T).reshape(B, T, 3, H, 64).permute(2, 0, 3, 1, 4)
    a = torch.nn.functional.scaled_dot_product_attention(q, k, v, is_causal=True).transpose(1, 2).reshape(-1, C)
    x1 = a @ w["proj"].T + x0
    x2 = torch.nn.functional.gelu(x1 @ w["fc1"].T, approximate="tanh") @ w["fc2"].T + x1
    logp = torch.log_softmax((x2 @ w["head"].T)[:, :V], -1)
    p = torch.softmax(teacher.double(), -1)
    loss = (p * (p.log() - logp.gather(1, ids.long()))).sum(-1).mean()
    loss.backward()
    return loss.item(), {k: x.grad for k, x in w.items()}


def test_a_step_matches_autograd():
    """Activations and gradients pass through about ten bf16 roundings on the way:
    each gradient's error stays within 4 % of its norm, the loss within 2 %."""
    student = example.Student(1003, 2)
    ids, teacher = example.make_teacher(1003, 16)
    tokens = torch.randint(0, 1003, (4, 50), generator=torch.Generator().manual_seed(0)).cuda()
    flat = tokens.reshape(-1)
    loss, grad = student.step(tokens, ids[flat], teacher[flat])
    want_loss, want = autograd_step(student, tokens, ids[flat], teacher[flat])
    assert abs(loss.item() - want_loss) <= 0.02 * want_loss
    for k, g in grad.items():
        assert (g.double() - want[k]).norm() <= 0.04 * want[k].norm(), k
    assert (grad["head"][1003:] == 0).all()


def test_the_student_learns():
    losses, score = example.train(steps=60, log=lambda *_: None)
    assert losses[-1] < 0.6 * losses[0], (losses[0], losses[-1])
    assert torch.isfinite(score.logprob).all() and torch.isfinite(score.entropy).all()
