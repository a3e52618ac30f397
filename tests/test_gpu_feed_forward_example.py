"""The example's step against the formulas: its second loss is that of the parameters after a step by the gradients in 64 bits.

The block's outputs are off by 6 h of their 2-norm (h = eps / 2 of BF16; see test_gpu_feed_forward), the teacher's as much, and
the difference of the two, whose square the loss is, by 6 h of both; the gradients by 6 h of theirs, which moves the
parameters by 6 h of the step.  2 * 6 h of the loss for the first two, and for the step 12 h of how far the loss is from where it
would be without one."""

import pytest
import torch

import gemm16_ref as ref
from dense_fp32_gemm_sm_gb300.feed_forward import main
from test_gpu_feed_forward import reference
from test_gpu_gemm16 import _cuda  # noqa: F401

pytestmark = pytest.mark.gpu


def run(M, K, N, E, sign):
    """The two losses, the second after a step of `sign` times the gradients."""
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    make = lambda: [(rand(E, K, N) / K**0.5), (rand(E, N, K) / N**0.5), 0.1 * rand(E, N), torch.zeros(E, K, device="cuda")]  # noqa: E731
    target, params, losses = make(), make(), []
    target, params = [p.cpu() for p in target], [p.cpu() for p in params]
    for _ in range(2):
        at = [0]
        for n in torch.bincount(torch.randint(0, E, (M,), generator=g, device="cuda"), minlength=E).tolist():
            at.append(at[-1] + n)
        x = rand(M, K).bfloat16().cpu()
        total, steps = 0.0, []
        for e in range(E):
            rows, zero = x[at[e]:at[e + 1]], torch.zeros(at[e + 1] - at[e], K)
            own = [p[e].bfloat16() if i < 2 else p[e] for i, p in enumerate(params)]
            others = [p[e].bfloat16() if i < 2 else p[e] for i, p in enumerate(target)]
            diff = reference(rows, zero, *own, "gelu", False)[0] - reference(rows, zero, *others, "gelu", False)[0]
            total += float(diff.square().sum())
            steps.append(reference(rows, diff * (2.0 / M), *own, "gelu", False)[2:])
        losses.append(total / (M * K))
        for e, step in enumerate(steps):
            for p, d in zip(params, step):
                p[e] -= (0.25 * sign * d).float()
    return losses


def test_a_step():
    sizes = dict(M=192, K=64, N=128, E=3)
    got = main(steps=2, **sizes)
    want, still, back = run(**sizes, sign=1), run(**sizes, sign=0), run(**sizes, sign=-1)
    h = torch.finfo(torch.bfloat16).eps / 2
    assert abs(got[0] - want[0]) <= 12 * h * want[0]
    bound = 12 * h * want[1] + 12 * h * abs(want[1] - still[1])
    assert abs(got[1] - want[1]) <= bound
    assert min(abs(still[1] - want[1]), abs(back[1] - want[1])) > 2 * bound  # (another step would show)
