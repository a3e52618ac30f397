"""The feed-forward block on 16-bit calls: forward and backward against 64 bits, alike for one weight and for experts.

Tolerances.  The block rounds H, Z, dZ and the outputs to 16 bits (half a step each, h = eps / 2) and keeps its sums in FP32
(K u at most of the sums of magnitudes, u = 2^-23).  Written as how far an output may be off in the 2-norm: with
independent roundings of relative size h of each factor of a sum of n products, the sum is off by h of its 2-norm over
random operands; three such roundings and the output's own are at most 4 h, GELU's and SiLU's slope at most 1.13 each:
6 h in all, of the norm of the output's larger part."""

import pytest
import torch

import dense_fp32_gemm_sm_gb300 as fg
import gemm16_ref as ref
from dense_fp32_gemm_sm_gb300.feed_forward import FeedForward, main
from test_gpu_gemm16 import _cuda  # noqa: F401

pytestmark = pytest.mark.gpu


def block(K, N, E, dt, act, bias, residual, seed=0):
    g = torch.Generator().manual_seed(seed)
    lead = () if E is None else (E,)
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    w1, w2 = (rand(*lead, K, N) / K**0.5).to(dt), (rand(*lead, N, K) / N**0.5).to(dt)
    b1, b2 = (0.3 * rand(*lead, N), 0.3 * rand(*lead, K)) if bias else (None, None)
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    return FeedForward(cuda(w1), cuda(w2), cuda(b1), cuda(b2), act, residual), (w1, w2, b1, b2), g


def reference(x, g, w1, w2, b1, b2, act, residual):
    """(y, dx, dw1, dw2, db1, db2) in 64 bits."""
    x, g, w1, w2 = (t.double() for t in (x, g, w1, w2))
    z = x @ w1 + (b1.double() if b1 is not None else 0)
    h = ref.act(z, act)[0]
    y = h @ w2 + (b2.double() if b2 is not None else 0) + (x if residual else 0)
    dz = (g @ w2.t()) * ref.slope(z, act)[0]
    return y, dz @ w1.t() + (g if residual else 0), x.t() @ dz, h.t() @ g, dz.sum(0), g.sum(0)


def near(got, want, h):
    off = (got.double().cpu() - want).norm()
    assert off <= 6 * h * want.norm() + 1e-30, float(off / want.norm())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act,bias,residual", [("gelu", True, True), ("silu", False, False), ("gelu", True, False), ("none", False, True)])
@pytest.mark.parametrize("M,K,N", [(1, 64, 128), (50, 72, 136), (300, 130, 257), (777, 256, 512)])
def test_block(M, K, N, act, bias, residual, dt):
    ff, params, g = block(K, N, None, dt, act, bias, residual)
    x, gr = torch.randn(M, K, generator=g).to(dt), torch.randn(M, K, generator=g).to(dt)
    y, saved = ff.forward(x.cuda())
    assert torch.equal(ff(x.cuda()), y)
    got = (y, *ff.backward(gr.cuda(), saved))
    want = reference(x, gr, *params, act, residual)
    h = torch.finfo(dt).eps / 2
    for a, b in zip(got, want):
        if a is not None:
            near(a, b, h)
    assert (got[4] is None) == (got[5] is None) == (not bias)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,K,N", [([3, 0, 40, 1, 130], 72, 136), ([0, 0, 7], 33, 65), ([200, 300], 256, 512), ([1] * 30, 64, 128)])
@pytest.mark.parametrize("act,bias,residual", [("gelu", True, True), ("silu", False, False)])
def test_experts(rows, K, N, act, bias, residual, dt):
    E, M = len(rows), sum(rows) + 9  # nine rows of no expert
    ff, params, g = block(K, N, E, dt, act, bias, residual)
    x, gr = torch.randn(M, K, generator=g).to(dt), torch.randn(M, K, generator=g).to(dt)
    at = torch.tensor([0] + rows).cumsum(0)
    offsets = at.int().cuda()
    y, saved = ff.forward(x.cuda(), offsets)
    assert torch.equal(ff(x.cuda(), offsets), y)
    dx, dw1, dw2, db1, db2 = ff.backward(gr.cuda(), saved)
    assert not y[at[-1]:].any() and not dx[at[-1]:].any()
    h = torch.finfo(dt).eps / 2
    for e in range(E):
        p = slice(int(at[e]), int(at[e + 1]))
        w1, w2, b1, b2 = (None if t is None else t[e] for t in params)
        want = reference(x[p], gr[p], w1, w2, b1, b2, act, residual)
        for a, b in zip((y[p], dx[p], dw1[e], dw2[e], None if db1 is None else db1[e], None if db2 is None else db2[e]), want):
            if a is not None:
                near(a, b, h)


def test_gradients_against_differences():
    """The block's own outputs, a step to either side along random directions: (f(p + s d) - f(p - s d)) / 2 s.  F16 weights
    and tokens move by steps they hold exactly; f sums outputs times fixed numbers in 64 bits.  The outputs are
    off by h each, at random: sqrt(M K) h |y| |g| / s of the difference (six of them allowed); the gradient's elements
    by a few h; and Z moves by s sqrt(64 / 20) |w| or so, 0.06, whose square times GELU's third derivative over six is
    less than a hundredth of the slope."""
    M, K, N, s = 96, 64, 128, 2.0**-5
    ff, (w1, w2, b1, b2), g = block(K, N, None, torch.float16, "gelu", True, True, seed=4)
    grid = lambda t: (t * 256).round() / 256  # noqa: E731
    x = grid(torch.randn(M, K, generator=g)).half()
    w1, w2 = grid(w1.float()).half(), grid(w2.float()).half()
    gr = torch.randn(M, K, generator=g).half()

    def f(x_, w1_, w2_, b1_):
        return (FeedForward(w1_.cuda(), w2_.cuda(), b1_.cuda(), b2.cuda(), "gelu", True)(x_.cuda()).double().cpu() * gr.double()).sum()

    ff = FeedForward(w1.cuda(), w2.cuda(), b1.cuda(), b2.cuda(), "gelu", True)
    y, saved = ff.forward(x.cuda())
    dx, dw1, dw2, db1, _ = ff.backward(gr.cuda(), saved)
    noise = (M * K) ** 0.5 * torch.finfo(torch.float16).eps * float(y.abs().mean()) / s
    for i, d in ((0, dx), (1, dw1), (2, dw2), (3, db1)):
        p = [x, w1, w2, b1]
        direction = torch.randint(0, 2, p[i].shape, generator=g).float() * 2 - 1
        direction *= (torch.rand(p[i].shape, generator=g) < 0.05)
        up, down = list(p), list(p)
        up[i], down[i] = (p[i].float() + s * direction).to(p[i].dtype), (p[i].float() - s * direction).to(p[i].dtype)
        along = (f(*up) - f(*down)) / (2 * s)
        want = float((d.double().cpu() * direction).sum())
        assert abs(float(along) - want) <= 6 * noise + 6 * 2.0**-11 * float((d.double().cpu() * direction).norm()) + 0.01 * abs(want), i


def test_two_streams_and_several_forwards():
    ff, _, g = block(64, 128, 4, torch.bfloat16, "silu", True, False)
    offsets = torch.tensor([0, 10, 10, 60, 100], dtype=torch.int32).cuda()
    xs = [torch.randn(100, 64, generator=g).bfloat16().cuda() for _ in range(4)]
    want = [(y, *ff.backward(x, saved)) for x in xs for y, saved in [ff.forward(x, offsets)]]
    torch.cuda.synchronize()
    streams, kept, got = [torch.cuda.Stream() for _ in xs], [], []
    for x, s in zip(xs, streams):
        with torch.cuda.stream(s):
            kept.append(ff.forward(x, offsets))
    for x, s, (y, saved) in zip(xs, streams, kept):
        with torch.cuda.stream(s):
            got.append((y, *ff.backward(x, saved)))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(i, j) for i, j in zip(a, b))


def test_captured():
    ff, _, g = block(64, 128, 3, torch.bfloat16, "gelu", True, True)
    x, offsets = torch.randn(70, 64, generator=g).bfloat16().cuda(), torch.tensor([0, 20, 20, 66], dtype=torch.int32).cuda()

    def step():
        y, saved = ff.forward(x, offsets)
        return (y, *ff.backward(y, saved))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (1, 2):
        x.copy_(torch.randn(70, 64, generator=torch.Generator().manual_seed(seed)).bfloat16())
        offsets.copy_(torch.tensor([0, 5 * seed, 30, 66], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step()))


def test_example_runs():
    losses = main(steps=3, M=64, K=64, N=128, E=3)
    assert len(losses) == 3 and all(l == l for l in losses)
