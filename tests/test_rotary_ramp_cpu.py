""""yarn" is the ramp over turns; the one over the pair's index is passed as frequencies, as the docstring writes it."""
import math
import textwrap

import pytest

import transformer_linear_layer_gb300 as tll


def documented(**names):
    """The plan that the lines of the docstring make."""
    lines = tll.Rotary.__doc__.split("pass::\n", 1)[1].split("    (without", 1)[0]
    code = textwrap.dedent(lines).strip().replace("\nRotary(", "\nplan = Rotary(")
    space = {"math": math, "Rotary": lambda *a, **k: tll.Rotary(*a, device="cpu", **k), **names}
    exec(code, space)
    return space["plan"]


def test_the_ramps_differ_in_the_middle():
    dim, base, length, factor = 128, 10000.0, 4096, 8.0
    turns = tll.Rotary(dim, scaling="yarn", factor=factor, original_length=length, device="cpu")
    index = documented(dim=dim, base=base, original_length=length, factor=factor, fast=32.0, slow=1.0)
    plain = tll.Rotary(dim, device="cpu").frequencies
    assert index.scale == turns.scale == pytest.approx(0.1 * math.log(8) + 1)
    # pairs 20 and 46 are the first beyond 32 turns and 1 turn in the length
    assert length * plain[21] / (2 * math.pi) < 32 < length * plain[20] / (2 * math.pi)
    assert length * plain[46] / (2 * math.pi) < 1 < length * plain[45] / (2 * math.pi)
    for i, (f, a, b) in enumerate(zip(plain, turns.frequencies, index.frequencies)):
        ramp = (min(1, max(0, (length * f / (2 * math.pi) - 1) / 31)), min(1, max(0, (46 - i) / 26)))
        assert a == pytest.approx(f * ramp[0] + f / factor * (1 - ramp[0]), rel=1e-12)
        assert b == pytest.approx(f * ramp[1] + f / factor * (1 - ramp[1]), rel=1e-12)
    assert min(a / b for a, b in zip(turns.frequencies, index.frequencies)) == pytest.approx(0.434, abs=1e-3)
    assert turns.frequencies[36] / index.frequencies[36] == pytest.approx(0.434, abs=1e-3)
