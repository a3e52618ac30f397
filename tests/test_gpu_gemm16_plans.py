"""Every kernel that a 16-bit product may be planned for, at sizes that reach it: exact on integers, with copies that never
arrive, one after the other without a wait, captured, on two streams."""

import time

import pytest
import torch

import dense_fp32_gemm_sm_gb300 as fg
from test_gpu_gemm16 import CODE, _cuda  # noqa: F401

pytestmark = pytest.mark.gpu

PAIR, TURNS = 8192, 16384

# M, N, K and what they are planned as: rows of a tile, ranks (0: pairs).  (With 152 SMs.)
SHAPES = []
_seen = set()
for _m in (1, 9, 24, 40, 64, 120, 200, 260, 300, 500, 700, 900, 1300, 1900, 2500):
    for _n in (64, 100, 300, 520, 1000, 1304, 2048, 3000):
        for _k in (40, 200, 520, 1032, 2056, 4100):
            if _m * _n * _k > 3 << 30:
                continue
            _v = fg.gemm16_plan(fg.BF16, 0, 1, _m, _n, _k, 0, 152)
            _kind = (bool(_v & PAIR), (_v & 8191) // 16, _v % 16)
            if _kind not in _seen:
                _seen.add(_kind)
                SHAPES.append((_m, _n, _k, *_kind))
# pairs with a longer depth than those sizes gave them
for _m, _n, _k in ((260, 2048, 4100), (500, 2048, 2056), (900, 3000, 1032), (1300, 2048, 1032), (2500, 3000, 520), (1900, 2048, 776)):
    _v = fg.gemm16_plan(fg.BF16, 0, 1, _m, _n, _k, 0, 152)
    SHAPES.append((_m, _n, _k, bool(_v & PAIR), (_v & 8191) // 16, _v % 16))


def ints(g, *shape, dtype=torch.bfloat16):
    return torch.randint(-3, 4, shape, generator=g, device="cuda").to(dtype)


def test_all_kinds_are_here():
    kinds = {(pair, rows) for *_, pair, rows, _ in SHAPES}
    assert {(False, 16), (False, 32), (False, 64), (True, 64), (True, 96), (True, 128)} <= kinds and len(kinds) >= 8
    assert {ranks for *_, pair, _, ranks in SHAPES if not pair} >= {1, 2, 3, 4, 5, 8}


def operands(g, M, N, K, ta, tb):
    a, b = ints(g, K, M) if ta else ints(g, M, K), ints(g, N, K) if tb else ints(g, K, N)
    return a, b, (a.t() if ta else a).double() @ (b.t() if tb else b).double()


@pytest.mark.parametrize("M,N,K,pair,rows,ranks", SHAPES)
@pytest.mark.parametrize("ta,tb", [(0, 0), (0, 1), (1, 0), (1, 1)])
def test_exact(M, N, K, pair, rows, ranks, ta, tb):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    a, b, want = operands(g, M, N, K, ta, tb)
    bias, r = ints(g, N, dtype=torch.float32), ints(g, M, N, dtype=torch.float32)
    ws = torch.empty(fg.gemm16_copy_workspace_size(ta, tb, 1, M, N, K) + fg.gemm16_sums_workspace_size(1, M, N), dtype=torch.uint8,
                     device="cuda")
    want = want + bias.double()
    for out in (torch.float32, torch.bfloat16):
        # a few integers that BF16 holds are compared as they are rounded
        y, z = torch.full((M, N), float("nan"), dtype=out, device="cuda"), torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        code = fg.F32 if out == torch.float32 else fg.BF16
        res = r.to(out)
        fg.gemm16(fg.BF16, code, ta, tb, M, N, K, 1.0, a, a.shape[1], b, b.shape[1], bias, fg.ACT_RELU, z, N, 2.0, res, N, y, N, ws,
                  ws.numel())
        assert torch.equal(y, (want.clamp(min=0) + 2 * r.double()).to(out))
        assert torch.equal(z, want.to(torch.bfloat16))
        # without anything but the bias (a kernel instance of its own)
        fg.gemm16(fg.BF16, code, ta, tb, M, N, K, 1.0, a, a.shape[1], b, b.shape[1], bias, fg.ACT_NONE, None, 0, 0.0, None, 0, y, N, ws,
                  ws.numel())
        assert torch.equal(y, want.to(out))
        s = torch.full((N,), float("nan"), device="cuda")
        fg.gemm16_grad(fg.BF16, code, ta, tb, M, N, K, 1.0, a, a.shape[1], b, b.shape[1], fg.ACT_RELU, z, N, y, N, s, ws, ws.numel())
        grad = torch.where(z.double() > 0, want - bias.double(), 0.0)
        assert torch.equal(y, grad.to(out)) and torch.equal(s.double(), grad.sum(0))


# Groups: experts' rows, columns, depth and the spread of the groups' sizes.
GROUPED = [(64, 16, 520, 264, 1), (300, 24, 256, 1032, 1), (1000, 7, 712, 200, 1), (2000, 3, 1304, 520, 2), (3000, 16, 1000, 776, 1),
           (5000, 5, 520, 1304, 2), (777, 1, 300, 300, 1), (900, 600, 136, 72, 0), (2500, 1024, 64, 64, 0)]


def groups(g, M, E, spread):
    share = torch.softmax(spread * torch.randn(E, generator=g, device="cuda"), 0)
    rows = torch.bincount(torch.multinomial(share, M, replacement=True, generator=g), minlength=E)
    return torch.cat((torch.zeros(1, dtype=torch.int64, device="cuda"), rows.cumsum(0))).int()


@pytest.mark.parametrize("M,E,N,K,spread", GROUPED)
@pytest.mark.parametrize("tb", [0, 1])
def test_groups_exact(M, E, N, K, spread, tb):
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    off = groups(g, M, E, spread)
    at = off.tolist()
    a, b, gr = ints(g, M + 11, K), ints(g, E, N, K) if tb else ints(g, E, K, N), ints(g, M + 11, N)
    ws = torch.empty(max(fg.gemm16_copy_workspace_size(0, tb, E, M + 11, N, K) + fg.gemm16_sums_workspace_size(E, M + 11, N),
                         fg.gemm16_copy_workspace_size(1, 0, 1, K, N, M + 11)), dtype=torch.uint8, device="cuda")
    y = torch.full((M + 11, N), 7.0, device="cuda")
    fg.gemm16_grouped(fg.BF16, fg.F32, tb, E, M + 11, N, K, off, 1.0, a, K, b, b.shape[2], N * K, None, fg.ACT_NONE, None, 0, 0.0, None,
                      0, y, N, ws, ws.numel())
    d, s = torch.full((M + 11, N), 7.0, device="cuda"), torch.full((E, N), float("nan"), device="cuda")
    fg.gemm16_grouped_grad(fg.BF16, fg.F32, tb, E, M + 11, N, K, off, 1.0, a, K, b, b.shape[2], N * K, fg.ACT_RELU, gr, N, d, N, s, ws,
                           ws.numel())
    c = torch.full((E, K, N), float("nan"), device="cuda")
    fg.gemm16_weight_grad(fg.BF16, fg.F32, E, M + 11, N, K, off, 1.0, a, K, gr, N, 0.0, c, N, K * N, ws, ws.numel())
    for e in range(E):
        p = slice(at[e], at[e + 1])
        want = a[p].double() @ (b[e].t() if tb else b[e]).double()
        grad = torch.where(gr[p] > 0, want, 0.0)
        assert torch.equal(y[p].double(), want) and torch.equal(d[p].double(), grad), e
        assert torch.equal(s[e].double(), grad.sum(0)), e
        assert torch.equal(c[e].double(), a[p].double().t() @ gr[p].double()), e
    assert (y[M:] == 7).all() and (d[M:] == 7).all()


LIMIT_NS = 200_000_000  # 0.2 s a wait


def calls():
    """One call for each kind of kernel: a name, the call, its output."""
    g = torch.Generator(device="cuda").manual_seed(0)
    for M, N, K in ((9, 300, 4100), (40, 520, 1032), (120, 1000, 520), (500, 2048, 1032), (2500, 1000, 2056)):
        K = K // 8 * 8
        a, b, y = ints(g, M, K), ints(g, N // 8 * 8, K), torch.empty(M, N // 8 * 8, device="cuda")
        N = N // 8 * 8
        yield "%d %d %d" % (M, N, K), lambda M=M, N=N, K=K, a=a, b=b, y=y: fg.gemm16(
            fg.BF16, fg.F32, 0, 1, M, N, K, 1.0, a, K, b, K, None, 0, None, 0, 0.0, None, 0, y, N), y, a.double() @ b.double().t()
    for M, E, N, K in ((3000, 5, 1000, 776), (200, 12, 136, 264)):
        off = groups(g, M, E, 1)
        at = off.tolist()
        a, gr, c, w = ints(g, M, K), ints(g, M, N), torch.empty(E, K, N, device="cuda"), ints(g, E, K, N)
        yield "weights %d" % M, lambda M=M, E=E, N=N, K=K, off=off, a=a, gr=gr, c=c: fg.gemm16_weight_grad(
            fg.BF16, fg.F32, E, M, N, K, off, 1.0, a, K, gr, N, 0.0, c, N, K * N), c, torch.stack(
                [a[i:j].double().t() @ gr[i:j].double() for i, j in zip(at, at[1:])])
        y = torch.empty(M, N, device="cuda")
        yield "groups %d" % M, lambda M=M, E=E, N=N, K=K, off=off, a=a, w=w, y=y: fg.gemm16_grouped(
            fg.BF16, fg.F32, 0, E, M, N, K, off, 1.0, a, K, w, N, K * N, None, 0, None, 0, 0.0, None, 0, y, N), y, torch.cat(
                [a[i:j].double() @ w[e].double() for e, (i, j) in enumerate(zip(at, at[1:]))])


@pytest.mark.parametrize("withheld", [0, 1, 4])
def test_a_copy_that_never_arrives_times_out_and_the_context_survives(withheld):
    for name, call, out, want in calls():
        torch.cuda.synchronize()
        fg.device_status(clear=True)
        try:
            fg.debug_withhold_tensor_core(withheld, LIMIT_NS)
            t0 = time.perf_counter()
            call()
            torch.cuda.synchronize()
            elapsed = time.perf_counter() - t0
        finally:
            fg.debug_withhold_tensor_core(-1)
        status = fg.device_status(clear=True)
        assert elapsed < 5.0, (name, elapsed)
        out.fill_(float("nan"))
        call()
        torch.cuda.synchronize()
        assert fg.device_status() == fg.OK and torch.equal(out.double(), want), name
        if withheld == 0:
            assert status == fg.ERR_TIMEOUT, name


def test_captured_and_replayed_and_on_two_streams():
    """All kinds in one graph, replayed; and two graphs on two streams at a time, with buffers of their own."""
    sets = [list(calls()), list(calls())]
    graphs = []
    for one in sets:
        for _, call, _, _ in one:
            call()
        torch.cuda.synchronize()
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=stream):
            for _, call, _, _ in one:
                call()
        graphs.append((graph, stream))
    for _ in range(3):
        for one in sets:
            for _, _, out, _ in one:
                out.fill_(float("nan"))
        torch.cuda.synchronize()
        for graph, stream in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
                graph.replay()
        torch.cuda.synchronize()
        for one in sets:
            for name, _, out, want in one:
                assert torch.equal(out.double(), want), name


@pytest.mark.parametrize("M,N,K", [(3, 512, 1024), (40, 520, 776), (300, 1000, 512), (1500, 1304, 776)])
def test_outputs_as_the_next_calls_inputs(M, N, K):
    """Tokens, bias, residual, Z and offsets that the call before has just written, with nothing in between, have to
    give what the same calls give with a wait after each."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x0 = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    w = [(torch.randn(K, N, generator=g, device="cuda") / K**0.5).bfloat16(), (torch.randn(N, K, generator=g, device="cuda") / N**0.5).bfloat16()]
    b0 = torch.randn(N, generator=g, device="cuda")

    def run(after):
        x, bias, outs = x0.clone(), b0.clone(), []
        z, h = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(fg.gemm16_sums_workspace_size(4, M, N), dtype=torch.uint8, device="cuda")
        dw = torch.zeros(4, K, N, device="cuda")
        off = torch.empty(5, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        for i in range(8):
            fg.gemm16(fg.BF16, fg.BF16, 0, 0, M, N, K, 1.0, x, K, w[0], N, bias, fg.ACT_GELU, z, N, 0.0, None, 0, h, N)
            after()
            fg.gemm16(fg.BF16, fg.BF16, 0, 0, M, K, N, 0.5, h, N, w[1], K, None, fg.ACT_NONE, None, 0, 0.5, x, K, x, K)  # in place
            after()
            fg.gemm16_grad(fg.BF16, fg.BF16, 0, 0, M, N, K, 1.0, x, K, w[0], N, fg.ACT_SILU, z, N, h, N, bias, ws, ws.numel())
            after()
            fg.act16_grad(fg.BF16, 1, M, N, None, fg.ACT_GELU, h, N, z, N, h, N, bias, ws, ws.numel())
            after()
            off.copy_(torch.tensor([0, M // 5, M // 3, M // 3, M - i], dtype=torch.int32).cuda())
            fg.gemm16_weight_grad(fg.BF16, fg.F32, 4, M, N, K, off, 1.0, x, K, h, N, 0.5, dw, N, K * N)
            after()
            bias.mul_(0.01)
            outs += [x.clone(), h.clone(), bias.clone(), dw.clone()]
        return outs

    one, row = run(torch.cuda.synchronize), run(lambda: None)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(one, row)) and all(a.isfinite().all() for a in one)


def test_past_two_to_the_31_elements():
    """Rows, groups and outputs further apart than 32 bits tell, in elements."""
    g = torch.Generator(device="cuda").manual_seed(2)
    K, N, far = 72, 136, (1 << 30) + 8
    x = torch.zeros(3 * far, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(3 * far, dtype=torch.bfloat16, device="cuda")
    rows, w = ints(g, 3, K), ints(g, 3, K, N)
    for i in range(3):
        x[i * far:i * far + K] = rows[i]
    fg.gemm16(fg.BF16, fg.BF16, 0, 0, 3, N, K, 1.0, x, far, w[0], N, None, 0, None, 0, 0.0, None, 0, y, far)
    got = torch.stack([y[i * far:i * far + N] for i in range(3)])
    assert torch.equal(got, (rows.double() @ w[0].double()).bfloat16())
    for i in range(3):  # three experts' weights as far apart, a row for each
        x[i * far:i * far + K * N] = w[i].flatten()
    off = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    out = torch.empty(3, N, dtype=torch.bfloat16, device="cuda")
    fg.gemm16_grouped(fg.BF16, fg.BF16, 0, 3, 3, N, K, off, 1.0, rows, K, x, N, far, None, 0, None, 0, 0.0, None, 0, out, N)
    assert torch.equal(out, torch.stack([rows[i].double() @ w[i].double() for i in range(3)]).bfloat16())
    gr = ints(g, 3, N)
    fg.gemm16_weight_grad(fg.BF16, fg.BF16, 3, 3, N, K, off, 1.0, rows, K, gr, N, 0.0, y, N, far)
    for i in range(3):
        assert torch.equal(y[i * far:i * far + K * N].view(K, N), (rows[i].double()[:, None] * gr[i].double()[None]).bfloat16())
    d = torch.empty(3, N, dtype=torch.bfloat16, device="cuda")
    y[far:far + N], y[:N], y[2 * far:2 * far + N] = gr[1], gr[0], gr[2]
    fg.act16_grad(fg.BF16, 1, 3, N, None, fg.ACT_RELU, y, far, gr, N, d, N)
    assert torch.equal(d, torch.where(gr > 0, gr, 0))


def test_many_rows_and_columns():
    """More tiles than a grid has CTAs many times over, and an output of more than 2^31 elements."""
    M, N, K = 70000, 34000, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    a, b = ints(g, M, K), ints(g, N, K)
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    fg.gemm16(fg.BF16, fg.BF16, 0, 1, M, N, K, 1.0, a, K, b, K, None, fg.ACT_RELU, None, 0, 0.0, None, 0, y, N)
    for r in (0, 1, 33333, 69999):
        assert torch.equal(y[r].double(), (a[r].double() @ b.double().t()).clamp(min=0))
    for c in (0, 17777, 33999):
        assert torch.equal(y[:, c].double(), (a.double() @ b[c].double()).clamp(min=0))


def test_one_weight_for_all_groups():
    g = torch.Generator(device="cuda").manual_seed(4)
    M, N, K, E = 200, 136, 72, 3
    x, w = ints(g, M, K), ints(g, K, N)
    off = torch.tensor([0, 70, 71, M], dtype=torch.int32, device="cuda")
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    fg.gemm16_grouped(fg.BF16, fg.BF16, 0, E, M, N, K, off, 1.0, x, K, w, N, 0, None, 0, None, 0, 0.0, None, 0, y, N)
    assert torch.equal(y, (x.double() @ w.double()).bfloat16())


@pytest.mark.parametrize("E,full", [(64, 17), (1024, 1023), (33, 32)])
def test_all_rows_in_one_of_many_groups(E, full):
    """Sums of integers, exact: the slices of a gradient are counted through all groups."""
    g = torch.Generator(device="cuda").manual_seed(5)
    M, N = 5000, 264
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[full + 1:] = M
    x, z = ints(g, M, N), ints(g, M, N)
    d, s = torch.full_like(x, 9), torch.full((E, N), float("nan"), device="cuda")
    ws = torch.full((fg.gemm16_sums_workspace_size(E, M, N),), 255, dtype=torch.uint8, device="cuda")
    fg.act16_grad(fg.BF16, E, M, N, off, fg.ACT_RELU, x, N, z, N, d, N, s, ws, ws.numel())
    want = torch.where(z > 0, x, 0)
    assert torch.equal(d, want) and torch.equal(s[full].double(), want.double().sum(0))
    assert not s[:full].any() and not s[full + 1:].any()


def test_depths_near_the_limit():
    """2^31 - 256: one tile's sums take seconds, in one go and in turns."""
    K = (1 << 31) - 256
    a, b = (torch.zeros(K, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for i, k in enumerate((0, 767, 768, 1 << 30, K - 129, K - 1)):
        a[k], b[k] = i + 1, 1
    y, s = torch.zeros(1, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, device="cuda")
    ws = torch.empty(fg.gemm16_sums_workspace_size(1, 1, 1), dtype=torch.uint8, device="cuda")
    fg.gemm16_grad(fg.BF16, fg.BF16, 0, 1, 1, 1, K, 1.0, a, K, b, K, fg.ACT_NONE, None, 0, y, 1, s, ws, ws.numel())
    assert y.item() == 21 and s.item() == 21
    del a, b
    x, g = (torch.zeros(K, 8, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for i, k in enumerate((0, 1, 127, 128, 1 << 30, K - 129, K - 1)):
        x[k, i], g[k, 7 - i] = i + 1, 1
    off = torch.tensor([0, K], dtype=torch.int32, device="cuda")
    c = torch.full((8, 8), 5.0, dtype=torch.bfloat16, device="cuda")
    fg.gemm16_weight_grad(fg.BF16, fg.BF16, 1, K, 8, 8, off, 1.0, x, 8, g, 8, 0.0, c, 8, 64)
    want = torch.zeros(8, 8)
    for i in range(7):
        want[i, 7 - i] = i + 1
    assert torch.equal(c.cpu().float(), want)
    assert fg.device_status() == fg.OK


# Rounds of tiles whose last one has few (for 152 SMs: tiles of 160 to 256 rows, by 2 and 4; a last tile of 4 rows).
DIVIDED = [(5000, 5000, 72), (1500, 8200, 520), (3100, 6000, 520), (5000, 7700, 72), (4100, 8200, 1032), (4130, 8200, 1032),
           (3000, 8200, 1032), (5000, 7700, 1032)]


def room(size):
    return torch.empty(size, dtype=torch.uint8, device="cuda"), size


@pytest.mark.parametrize("M,N,K", DIVIDED)
def test_last_rounds_of_few_tiles(M, N, K):
    """Every row once: added in place, stored across and along the depth, through a gate."""
    g = torch.Generator(device="cuda").manual_seed(6)
    x, w, y0 = ints(g, M, K), ints(g, N, K), ints(g, M, N, dtype=torch.float32)
    want = x.float() @ w.float().t()  # integers below 2^24
    y = y0.clone()
    fg.gemm16(fg.BF16, fg.F32, 0, 1, M, N, K, 1.0, x, K, w, K, None, 0, None, 0, 1.0, y, N, y, N)
    assert torch.equal(y, want + y0)
    xt, wt = torch.zeros(K, (M + 7) // 8 * 8, dtype=torch.bfloat16, device="cuda"), w.t().contiguous()
    xt[:, :M] = x.t()
    h, z = torch.full((M + 1, N), 9.0, dtype=torch.bfloat16, device="cuda"), torch.full((M + 1, N), 9.0, dtype=torch.bfloat16, device="cuda")
    fg.gemm16(fg.BF16, fg.BF16, 1, 0, M, N, K, 1.0, xt, xt.shape[1], wt, N, None, fg.ACT_RELU, z, N, 0.0, None, 0, h, N,
              *room(fg.gemm16_copy_workspace_size(1, 0, 1, M, N, K)))
    assert torch.equal(h[:M], want.clamp(min=0).bfloat16()) and torch.equal(z[:M], want.bfloat16())
    assert (h[M] == 9).all() and (z[M] == 9).all()
    gate = ints(g, M, N)
    fg.gemm16_grad(fg.BF16, fg.BF16, 0, 1, M, N, K, 1.0, x, K, w, K, fg.ACT_RELU, gate, N, h, N)
    assert torch.equal(h[:M], torch.where(gate > 0, want, 0).bfloat16()) and (h[M] == 9).all()


@pytest.mark.parametrize("rows,N,K", [((700, 3, 900, 0, 1400, 260, 31), 4000, 520), ((1, 5000), 5000, 72), ((600, 600, 600), 7700, 1032),
                                      ((257, 255, 1025, 2), 8200, 264)])
def test_last_rounds_of_few_tiles_of_groups(rows, N, K):
    g = torch.Generator(device="cuda").manual_seed(7)
    E, M = len(rows), sum(rows)
    at = [0]
    for n in rows:
        at.append(at[-1] + n)
    off = torch.tensor(at, dtype=torch.int32, device="cuda")
    x, w, y = ints(g, M + 2, K), ints(g, E, K, N), torch.full((M + 2, N), 9.0, device="cuda")
    y0 = ints(g, M + 2, N, dtype=torch.float32)
    y.copy_(y0)
    fg.gemm16_grouped(fg.BF16, fg.F32, 0, E, M + 2, N, K, off, 1.0, x, K, w, N, K * N, None, 0, None, 0, 1.0, y, N, y, N,
                      *room(fg.gemm16_copy_workspace_size(0, 0, E, M + 2, N, K)))
    want = torch.cat([x[i:j].float() @ w[e].float() for e, (i, j) in enumerate(zip(at, at[1:]))])
    assert torch.equal(y[:M], want + y0[:M]) and torch.equal(y[M:], y0[M:])
    gr, c = ints(g, M + 2, N), ints(g, E, K, N, dtype=torch.float32)
    sums = c + torch.stack([x[i:j].float().t() @ gr[i:j].float() for i, j in zip(at, at[1:])])
    fg.gemm16_weight_grad(fg.BF16, fg.F32, E, M + 2, N, K, off, 1.0, x, K, gr, N, 1.0, c, N, K * N,
                          *room(fg.gemm16_copy_workspace_size(1, 0, 1, K, N, M + 2)))
    assert torch.equal(c, sums)


def test_calls_from_two_threads():
    """Each with its own stream and workspace, sizes in turn: what a thread keeps of its plans is its own."""
    import threading

    sizes = [(1, 264, 520), (300, 1001, 72), (700, 1304, 1032), (64, 200, 264)]
    failures = []

    def work(seed):
        try:
            g = torch.Generator(device="cuda").manual_seed(seed)
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for i in range(24):
                    M, N, K = sizes[(i + seed) % len(sizes)]
                    x, w, y = ints(g, M, K), ints(g, K, N), torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
                    fg.gemm16(fg.BF16, fg.BF16, 0, 0, M, N, K, 1.0, x, K, w, N, None, 0, None, 0, 0.0, None, 0, y, N,
                              *room(fg.gemm16_copy_workspace_size(0, 0, 1, M, N, K)))
                    want = (x.double() @ w.double()).bfloat16()
                    stream.synchronize()
                    if not torch.equal(y, want):
                        failures.append((seed, M, N, K))
        except Exception as e:  # noqa: BLE001
            failures.append(e)

    threads = [threading.Thread(target=work, args=(s,)) for s in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures
