"""MXFP4 calls one after the other: on a stream, between other work, in a CUDA graph, on two
streams.  Each kernel may come to the GPU before the one before it has ended, so every call
here reads what the call before it writes (or overwrites what it reads), nothing waits in
between, and the results have to equal those of the same calls with a wait after each.
"""

import pytest
import torch

import dense_fp32_gemm_sm_gb300 as fg
import mxfp4_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    fg.library()
    fg.device_status(clear=True)
    yield
    assert fg.device_status() == fg.OK


def room(rows, cols):
    return (torch.empty(rows, 16 * ref.blocks(cols), dtype=torch.uint8, device="cuda"),
            torch.empty(fg.mxfp4_scales_size(rows, cols), dtype=torch.uint8, device="cuda"))


class Steps:
    """A training step's calls on buffers that the steps share."""

    def __init__(self, M, N, K, seed, dt=torch.float32):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.t = fg.F32 if dt == torch.float32 else fg.BF16
        self.M, self.N, self.K = M, N, K
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.x, self.w = rand(M, K).to(dt), (rand(K, N) / K**0.5).to(dt)
        self.y, self.dx, self.dw = (torch.empty(*s, dtype=dt, device="cuda") for s in ((M, N), (M, K), (K, N)))
        self.xr, self.xc, self.wr, self.wc = room(M, K), room(K, M), room(K, N), room(N, K)
        self.gr, self.gc = room(M, N), room(N, M)
        self.b, self.db = rand(N), torch.empty(N, device="cuda")
        self.ws = torch.empty(max(fg.mxfp4_quantize_grad_workspace_size(M, N), 16, fg.mxfp4_linear_workspace_size(M, N, K)),
                              dtype=torch.uint8, device="cuda")

    def calls(self, stream=None):
        M, N, K, t = self.M, self.N, self.K, self.t
        lk, ln, lm = (16 * ref.blocks(n) for n in (K, N, M))
        yield lambda: fg.mxfp4_quantize(t, M, K, self.x, K, self.xr[0], lk, self.xr[1], self.xc[0], lm, self.xc[1], stream=stream)
        yield lambda: fg.mxfp4_quantize(t, K, N, self.w, N, self.wr[0], ln, self.wr[1], self.wc[0], lk, self.wc[1], stream=stream)
        yield lambda: fg.mxfp4_gemm(t, M, N, K, 1.0, self.xr[0], lk, self.xr[1], self.wc[0], lk, self.wc[1], 0.0, self.y, N, self.b,
                                    True, stream=stream)
        yield lambda: fg.mxfp4_quantize_grad(t, M, N, self.y, N, self.y, N, self.gr[0], ln, self.gr[1], self.gc[0], lm, self.gc[1],
                                             self.db, self.ws, self.ws.numel(), stream=stream)
        yield lambda: fg.mxfp4_gemm(t, M, K, N, 1.0, self.gr[0], ln, self.gr[1], self.wr[0], ln, self.wr[1], 0.0, self.dx, K,
                                    stream=stream)
        yield lambda: fg.mxfp4_gemm(t, K, N, M, -2.0**-6, self.xc[0], lm, self.xc[1], self.gc[0], lm, self.gc[1], 1.0, self.w, N,
                                    stream=stream)  # the weights change under the next step
        yield lambda: fg.mxfp4_gemm(fg.F32, 1, N, K, 0.0, None, lk, None, None, lk, None, 0.5, self.b, N, self.db, False,
                                    stream=stream)  # b = b / 2 + db, with no products
        # the next step's tokens: this one's, through the layer and back
        yield lambda: fg.mxfp4_linear(t, M, N, K, self.x, K, self.wc[0], lk, self.wc[1], None, True, self.y, N, self.ws,
                                      self.ws.numel(), stream=stream)
        yield lambda: fg.mxfp4_dequantize(t, M, K, self.xr[0], lk, self.xr[1], self.x, K, stream=stream)
        yield lambda: fg.mxfp4_gemm(t, M, K, N, 2.0**-8, self.gr[0], ln, self.gr[1], self.wr[0], ln, self.wr[1], 0.5, self.x, K,
                                    stream=stream)

    def results(self):
        return [v.clone() for v in (self.x, self.w, self.y, self.dx, self.b, self.db, self.gr[0], self.gc[1], self.xc[0])]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


SHAPES = [(1, 300, 200), (3, 1001, 520), (40, 256, 300), (130, 500, 1000), (600, 1500, 700), (2000, 2300, 1100)]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_calls_in_a_row_equal_calls_one_by_one(M, N, K, dt):
    a, b = Steps(M, N, K, 1, dt), Steps(M, N, K, 1, dt)
    torch.cuda.synchronize()
    for _ in range(6):
        for call in a.calls():
            call()
            torch.cuda.synchronize()
    for _ in range(6):
        for call in b.calls():
            call()
    torch.cuda.synchronize()
    assert same(a.results(), b.results())
    assert torch.isfinite(a.x).all()


def test_between_other_kernels_of_the_library():
    # the FP32 product's own launches follow one another early too; each call's input is the
    # output of the one before
    n = 700
    outs = []
    for wait in (True, False):
        g = torch.Generator(device="cuda").manual_seed(3)
        x = torch.randn(n, n, generator=g, device="cuda") / n**0.5
        a = torch.randn(n, n, generator=g, device="cuda")
        y, q = torch.empty_like(a), room(n, n)
        torch.cuda.synchronize()
        for _ in range(10):
            fg.mxfp4_quantize(fg.F32, n, n, a, n, q[0], q[0].shape[1], q[1], None, 0, None)
            if wait:
                torch.cuda.synchronize()
            fg.mxfp4_dequantize(fg.F32, n, n, q[0], q[0].shape[1], q[1], y, n)
            if wait:
                torch.cuda.synchronize()
            fg.sgemm(0, 0, n, n, n, 1.0, y, n, x, n, 0.0, a, n)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        outs.append(a)
    assert torch.equal(outs[0], outs[1]) and torch.isfinite(outs[0]).all()


@pytest.mark.parametrize("M,N,K", SHAPES[1:5])
def test_in_a_graph_after_copies_and_fills(M, N, K):
    a, b = Steps(M, N, K, 2), Steps(M, N, K, 2)
    x0, w0, b0 = a.x.clone(), a.w.clone(), a.b.clone()
    torch.cuda.synchronize()
    for call in a.calls():
        call()
    torch.cuda.synchronize()
    want = a.results()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            b.y.fill_(float("nan"))
            b.w.copy_(w0)
            b.b.copy_(b0)
            b.x.copy_(x0)  # a copy, right before the first call that reads it
            for call in b.calls():
                call()
            kept = b.x.clone()
        for _ in range(3):
            b.x.fill_(float("nan"))
            graph.replay()
        stream.synchronize()
    assert same(b.results(), want) and torch.equal(kept, want[0])


def test_two_streams():
    one, two = Steps(600, 1500, 700, 4), Steps(130, 500, 1000, 5)
    want = [Steps(600, 1500, 700, 4), Steps(130, 500, 1000, 5)]
    torch.cuda.synchronize()
    for s in want:
        for _ in range(4):
            for call in s.calls():
                call()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        for c1, c2 in zip(one.calls(s1), two.calls(s2)):
            c1()
            c2()
    torch.cuda.synchronize()
    assert same(one.results(), want[0].results()) and same(two.results(), want[1].results())
