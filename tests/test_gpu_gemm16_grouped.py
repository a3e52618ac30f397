"""16-bit products by groups of rows on the GPU against 64 bits (tolerances: gemm16_ref)."""

import pytest
import torch

import dense_fp32_gemm_sm_gb300 as fg
import gemm16_ref as ref
from test_gpu_gemm16 import ACT, CODE, _cuda, values  # noqa: F401

pytestmark = pytest.mark.gpu

# Rows of each group, rows before the first and behind the last one.
GROUPS = {
    "one": ([50], 0, 0),
    "one_empty": ([0], 3, 4),
    "few": ([3, 0, 1, 17, 0], 0, 0),
    "single_rows": ([1] * 40, 2, 1),
    "uneven": ([200, 1, 0, 33, 64, 129, 16], 5, 9),
    "last_only": ([0, 0, 0, 77], 0, 30),
    "many": ([(7 * e) % 23 for e in range(70)], 0, 13),
}


def offsets_of(name):
    rows, before, behind = GROUPS[name]
    at = [before]
    for n in rows:
        at.append(at[-1] + n)
    return at, at[-1] + behind


def stacked(mats, pad, offset, gap):
    """Matrices of one shape `gap` elements apart inside a NaN buffer: (tensor, address, ld, stride)."""
    rows, cols = mats[0].shape
    ld = cols + pad
    stride = rows * ld + gap
    flat = torch.full((len(mats) * stride + offset + 16,), float("nan"), dtype=mats[0].dtype)
    for e, m in enumerate(mats):
        flat[offset + e * stride:offset + e * stride + rows * ld].view(rows, ld)[:, :cols] = m
    data = flat.cuda()
    return data, data.data_ptr() + offset * data.element_size(), ld, stride


def grouped(name, t, N, K, out=None, tb=False, alpha=1.0, bias=False, act="none", keep=False, beta=0.0, grad=False, sums=False,
            pads=(0, 0, 0, 0, 0), offset=0, gap=0, ints=False, seed=0):
    at, M = offsets_of(name)
    E = len(at) - 1
    g = torch.Generator().manual_seed(seed)
    dt, ot = ref.TYPES[t], ref.TYPES[out or t]
    a = values(g, M, K, dt, ints)
    if not ints:
        a[:at[0]], a[at[-1]:] = float("nan"), float("nan")  # rows of no group must not count
    b = [values(g, K, N, dt, ints, max(K, 1) ** -0.5) for _ in range(E)]
    A = ref.Buffer(a, pads[0], offset)
    B, b_ptr, ldb, stride = stacked([m.t() if tb else m for m in b], pads[1], offset, gap)
    bi = torch.randint(-8, 9, (E, N), generator=g) / 4.0 if bias else None
    r, z = values(g, M, N, ot, ints), values(g, M, N, dt)
    offs = torch.tensor(at, dtype=torch.int32).cuda()
    size = fg.gemm16_copy_workspace_size(0, tb, E, M, N, K) + fg.gemm16_sums_workspace_size(E, M, N)
    ws = torch.full((size,), 255, dtype=torch.uint8).cuda()
    Y = ref.output(M, N, ot, pads[4], offset)
    common = (CODE[t], CODE[out or t], tb, E, M, N, K, offs, alpha, A.ptr, A.ld, b_ptr, ldb, stride)
    R, Zin = ref.Buffer(r, pads[3], offset), ref.Buffer(z, pads[2], offset)
    Z = ref.output(M, N, dt, pads[2], offset) if keep else None
    s = torch.full((E, N), float("nan")).cuda() if sums else None
    if grad:
        fg.gemm16_grouped_grad(*common, ACT[act], Zin.ptr, Zin.ld, Y.ptr, Y.ld, s, ws, size)
    else:
        fg.gemm16_grouped(*common, bi.cuda() if bias else None, ACT[act], Z.ptr if keep else None, Z.ld if keep else 0, beta,
                          R.ptr if beta else None, R.ld, Y.ptr, Y.ld, ws, size)
    torch.cuda.synchronize()
    y, dy = torch.full((M, N), ref.Buffer.SENTINEL, dtype=torch.float64), torch.zeros(M, N, dtype=torch.float64)
    zw, dz = y.clone(), dy.clone()
    for e in range(E):
        p = slice(at[e], at[e + 1])
        if grad:
            (y[p], dy[p]), (cs, dcs) = ref.layer_grad(a[p].double(), b[e].double(), alpha, act, z[p].double())
            if sums:
                assert not ref.outside(s[e].cpu(), cs, dcs, torch.float32).any(), e
        else:
            (y[p], dy[p]), (zw[p], dz[p]) = ref.layer(a[p].double(), b[e].double(), alpha, bi[e].double() if bias else None, act,
                                                      beta, r[p].double())
    if ints:
        dy, dz = 0 * dy, 0 * dz
    got = Y.result()
    bad = ref.outside(got, y, dy, ot)
    assert not bad.any(), "%d of %d wrong, first at %s: %s for %s" % (
        bad.sum(), bad.numel(), bad.nonzero()[0].tolist(), got[bad][0], y[bad][0])
    if keep:
        assert not ref.outside(Z.result(), zw, dz, dt).any()


@pytest.mark.parametrize("name", GROUPS)
@pytest.mark.parametrize("tb", [0, 1])
@pytest.mark.parametrize("N,K", [(128, 64), (129, 65), (7, 5), (300, 200), (1, 1030)])
def test_integers_are_exact(name, tb, N, K):
    grouped(name, "bf16", N, K, out="f32", tb=tb, ints=True)


@pytest.mark.parametrize("name", GROUPS)
@pytest.mark.parametrize("t,act", [("bf16", "gelu"), ("f16", "silu"), ("bf16", "relu")])
def test_layer(name, t, act):
    grouped(name, t, 200, 136, bias=True, act=act, keep=True)
    grouped(name, t, 131, 71, out="f32", tb=True, bias=True, act=act, keep=True, beta=-1.5, alpha=0.5)


@pytest.mark.parametrize("name", ["few", "uneven", "many"])
@pytest.mark.parametrize("pads,offset,gap", [((1, 0, 3, 5, 7), 1, 0), ((8, 8, 2, 2, 2), 8, 8), ((0, 0, 0, 0, 0), 0, 3),
                                             ((0, 8, 1, 1, 1), 4, 16)])
def test_strides_and_alignment(name, pads, offset, gap):
    grouped(name, "f16", 136, 72, bias=True, act="silu", keep=True, beta=1.0, pads=pads, offset=offset, gap=gap)
    grouped(name, "bf16", 133, 77, tb=True, grad=True, sums=True, act="gelu", pads=pads, offset=offset, gap=gap)


@pytest.mark.parametrize("name", GROUPS)
@pytest.mark.parametrize("act", ref.ACTS)
def test_gradient_through_an_activation(name, act):
    grouped(name, "bf16", 200, 136, tb=True, grad=True, sums=True, act=act)
    grouped(name, "f16", 65, 130, out="f32", grad=True, sums=True, act=act)


def weight_grad(name, t, N, K, out=None, alpha=1.0, beta=0.0, pads=(0, 0, 0), offset=0, gap=0, ints=False, seed=0, nan=True):
    at, M = offsets_of(name)
    E = len(at) - 1
    gen = torch.Generator().manual_seed(seed)
    dt, ot = ref.TYPES[t], ref.TYPES[out or t]
    a, g = values(gen, M, K, dt, ints), values(gen, M, N, dt, ints)
    if nan:  # rows of no group must not count
        for x in (a, g):
            x[:at[0]], x[at[-1]:] = float("nan"), float("nan")
    A, G = ref.Buffer(a, pads[0], offset), ref.Buffer(g, pads[1], offset)
    c0 = [values(gen, K, N, ot, ints) for _ in range(E)]
    ld, stride = N + pads[2], K * (N + pads[2]) + gap
    flat = torch.full((E * stride + offset,), ref.Buffer.SENTINEL, dtype=ot)
    inside = torch.zeros_like(flat, dtype=torch.bool)
    place = lambda f, e: f[offset + e * stride:offset + e * stride + K * ld].view(K, ld)[:, :N]  # noqa: E731
    for e in range(E):
        place(flat, e)[:] = c0[e] if beta else float("nan")
        place(inside, e)[:] = True
    data = flat.cuda()
    offs = torch.tensor(at, dtype=torch.int32).cuda()
    size = fg.gemm16_copy_workspace_size(1, 0, 1, K, N, max(M, 1))
    ws = torch.full((size,), 255, dtype=torch.uint8).cuda()
    fg.gemm16_weight_grad(CODE[t], CODE[out or t], E, M, N, K, offs, alpha, A.ptr, A.ld, G.ptr, G.ld, beta,
                          data.data_ptr() + offset * data.element_size(), ld, stride, ws, size)
    torch.cuda.synchronize()
    got = data.cpu()
    assert (got[~inside] == ref.Buffer.SENTINEL).all(), "written outside C"
    for e in range(E):
        p = slice(at[e], at[e + 1])
        (y, dy), _ = ref.layer(a[p].double().t(), g[p].double(), alpha, None, "none", beta, c0[e].double())
        bad = ref.outside(place(got, e), y, 0 * dy if ints else dy, ot)
        assert not bad.any(), (e, at[e], at[e + 1], int(bad.sum()), place(got, e)[bad][:3], y[bad][:3])


@pytest.mark.parametrize("name", GROUPS)
@pytest.mark.parametrize("N,K", [(128, 128), (64, 300), (257, 33), (1, 1), (520, 600)])
def test_weights_gradient_of_integers_is_exact(name, N, K):
    weight_grad(name, "bf16", N, K, out="f32", ints=True)
    weight_grad(name, "f16", N, K, out="f32", ints=True, beta=1.0)


@pytest.mark.parametrize("name", GROUPS)
@pytest.mark.parametrize("t,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32")])
def test_weights_gradient(name, t, out):
    weight_grad(name, t, 130, 200, out=out, alpha=0.5)
    weight_grad(name, t, 136, 72, out=out, beta=-2.0, pads=(1, 3, 5), offset=1, gap=7)


def test_infinities_of_the_next_group_stay_there():
    """A group's last stage holds rows of the next one: no 0 * inf."""
    rows = [5, 1, 18, 40, 3]
    at = [0]
    for n in rows:
        at.append(at[-1] + n)
    M, K, N = at[-1], 70, 150
    gen = torch.Generator().manual_seed(0)
    a, g = values(gen, M, K, torch.bfloat16, True), values(gen, M, N, torch.bfloat16, True)
    a[at[1]:at[2]] = float("inf")
    g[at[3]:at[4]] = float("nan")
    c = torch.full((len(rows), K, N), 7.0).cuda()
    ws = torch.empty(fg.gemm16_copy_workspace_size(1, 0, 1, K, N, M), dtype=torch.uint8).cuda()
    fg.gemm16_weight_grad(fg.BF16, fg.F32, len(rows), M, N, K, torch.tensor(at, dtype=torch.int32).cuda(), 1.0, a.cuda(), K,
                          g.cuda(), N, 0.0, c, N, K * N, ws, ws.numel())
    for e in (0, 2, 4):
        want = a[at[e]:at[e + 1]].double().t() @ g[at[e]:at[e + 1]].double()
        assert torch.equal(c[e].cpu().double(), want), e


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("name", [None, "one_empty", "few", "uneven", "many"])
@pytest.mark.parametrize("N,pads,offset", [(256, (0, 0, 0), 0), (300, (4, 4, 4), 8), (77, (1, 0, 3), 1), (1, (0, 0, 0), 0)])
def test_act_grad(t, act, name, N, pads, offset):
    at, M = offsets_of(name) if name else ([0, 333], 333)
    E, dt = len(at) - 1, ref.TYPES[t]
    gen = torch.Generator().manual_seed(1)
    g, z = values(gen, M, N, dt), values(gen, M, N, dt, scale=2.0)
    G, Z, D = ref.Buffer(g, pads[0], offset), ref.Buffer(z, pads[1], offset), ref.output(M, N, dt, pads[2], offset)
    offs = torch.tensor(at, dtype=torch.int32).cuda() if name else None
    s = torch.full((E, N), float("nan")).cuda()
    ws = torch.full((fg.gemm16_sums_workspace_size(E, M, N),), 255, dtype=torch.uint8).cuda()
    fg.act16_grad(CODE[t], E, M, N, offs, ACT[act], G.ptr, G.ld, Z.ptr, Z.ld, D.ptr, D.ld, s, ws, ws.numel())
    torch.cuda.synchronize()
    got = D.result()
    p = slice(at[0], at[-1])
    assert (got[:at[0]] == ref.Buffer.SENTINEL).all() and (got[at[-1]:] == ref.Buffer.SENTINEL).all()
    sl, ds = ref.slope(z.double(), act)
    y, dy = g.double() * sl, g.double().abs() * ds + ref.U * (g.double() * sl).abs()
    assert not ref.outside(got[p], y[p], dy[p], dt).any()
    for e in range(E):
        q = slice(at[e], at[e + 1])
        tol = dy[q].sum(0) + (at[e + 1] - at[e] + 1) * ref.U * (y[q].abs() + dy[q]).sum(0)
        assert not ref.outside(s[e].cpu(), y[q].sum(0), tol, torch.float32).any(), e
    # sums alone, and in place
    s2 = torch.full((E, N), float("nan")).cuda()
    fg.act16_grad(CODE[t], E, M, N, offs, ACT[act], G.ptr, G.ld, Z.ptr, Z.ld, None, 0, s2, ws, ws.numel())
    assert torch.equal(s, s2)
    fg.act16_grad(CODE[t], E, M, N, offs, ACT[act], G.ptr, G.ld, Z.ptr, Z.ld, G.ptr, G.ld)
    assert torch.equal(G.data[offset:offset + M * G.ld].view(M, G.ld)[p, :N].cpu(), got[p])


@pytest.mark.parametrize("at", [[5, 3, 60, 20, 100], [-7, 10, 1 << 30, 40, 50], [90, 80, 70, 60, 50], [-(1 << 31), (1 << 31) - 1, 0, 0, 9]])
def test_offsets_out_of_order_reach_no_other_memory(at):
    """What such a call computes is not defined; that it stays inside its matrices is."""
    M, N, K, E = 64, 136, 72, 4
    offs = torch.tensor(at, dtype=torch.int32).cuda()
    A = ref.Buffer(torch.ones(M, K, dtype=torch.bfloat16))
    B = torch.ones(E, K, N, dtype=torch.bfloat16).cuda()
    Y, Z = ref.output(M, N, torch.bfloat16), ref.output(M, N, torch.bfloat16)
    ws_size = fg.gemm16_sums_workspace_size(E, M, N)
    ws = torch.full((ws_size + 4096,), 99, dtype=torch.uint8).cuda()
    s = torch.zeros(E + 1, N).cuda()
    fg.gemm16_grouped(fg.BF16, fg.BF16, 0, E, M, N, K, offs, 1.0, A.ptr, K, B, N, K * N, None, fg.ACT_NONE, Z.ptr, N, 0.0, None, N,
                      Y.ptr, N)
    fg.gemm16_grouped_grad(fg.BF16, fg.BF16, 0, E, M, N, K, offs, 1.0, A.ptr, K, B, N, K * N, fg.ACT_GELU, Z.ptr, N, Y.ptr, N, s, ws,
                           ws_size)
    C = torch.full((E * K * N + 100,), -77.0).cuda()
    fg.gemm16_weight_grad(fg.BF16, fg.F32, E, M, N, K, offs, 1.0, A.ptr, K, Y.ptr, N, 0.0, C, N, K * N)
    fg.act16_grad(fg.BF16, E, M, N, offs, fg.ACT_SILU, Y.ptr, N, Z.ptr, N, Y.ptr, N, s, ws, ws_size)
    torch.cuda.synchronize()
    Y.result(), Z.result(), A.result()
    assert (ws[ws_size:] == 99).all() and (C[E * K * N:] == -77).all() and not s[E].any()
