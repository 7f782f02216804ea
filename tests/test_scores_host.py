"""The bound of the tests of running maxima: exact scores stay inside, results
that are scaled wrongly, zeroed or negated do not."""
import math

import pytest
import torch

import scores_common as sc

LOG2E = 1 / math.log(2)


def test_scores_are_exact_in_every_type():
    z = torch.arange(-1023, 1024).double() / 8
    k = sc.keys(z, 64)
    assert torch.equal(k.to(torch.bfloat16).double(), k)
    for s in (0.5, 1.0, 2.0):
        assert torch.equal((k / s).to(torch.float8_e4m3fn).double() * s, k)
    for f in sc.FACTORS:
        q = torch.zeros(64, dtype=torch.float64)
        q[:sc.DIGITS] = f
        assert torch.equal((k.float() @ q.float()).double(), f * z)


@pytest.mark.parametrize("step,slack", [(2.0 ** -8, 8 / LOG2E), (2.0 ** -11, 4 / LOG2E)])
@pytest.mark.parametrize("hd", [64, 256])
def test_the_bound_holds_rounded_probabilities_and_nothing_worse(step, slack, hd):
    caught = {}
    for kind in sc.KINDS:
        g = torch.Generator().manual_seed(1)
        z = sc.scores(kind, 640, g)
        v = torch.randn((640, hd), generator=g, dtype=torch.float64)
        ref, mass = sc.plain(z, v)
        tol = sc.bound(ref, mass, float(z.abs().max()), 640, step)
        # probabilities rounded once, and the result
        p = torch.exp(z - z.max())
        low = p.to(torch.bfloat16 if step > 2.0 ** -10 else torch.float16).double() if step > 2.0 ** -10 else (p * 2048).half().double() / 2048
        got = (low @ v / p.sum()).to(torch.bfloat16).double()
        assert ((got - ref).abs() <= tol).all(), kind
        for wrong in (torch.zeros_like(ref), -ref):
            assert ((wrong - ref).abs() > tol).double().mean() > 0.9, kind
        for mistake in ("accumulator", "sum", "half"):
            got, moved = sc.by_tiles(z, v, slack, mistake)
            if moved:
                caught.setdefault(mistake, []).append(bool(((got - ref).abs() > tol).any()))
        good, _ = sc.by_tiles(z, v, slack, "none")
        assert ((good - ref).abs() <= tol).all(), kind
    for mistake, seen in caught.items():
        assert len(seen) >= 4 and sum(seen) >= len(seen) - 1, (mistake, seen)
