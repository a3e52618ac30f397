"""The library's 16-bit layers (BF16 and F16 operands, FP32 sums) as they are called, case by case.

A layer is Y = act(X W + b) + R with act none, ReLU, GELU (z Phi(z)) or SiLU (z sigma(z)); training
keeps Z = X W + b.  The cases are the layer forward; its backward pass from the gradient of its
output; the layer by groups of rows, each with a weight of its own (experts: rows offsets[e] up to
offsets[e+1] take W[e], b[e]); and the backward pass through an inner layer of such experts, which
ends at the pre-activation of the layer before.  ``own`` selects the library's entry points or a
plain evaluation in elementary torch operations; both take the same inputs.
"""

import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # One token through the benchmark's fully-connected layer: decoding, the weight's bytes alone count.
        dict(name="linear_one_token", op="linear", type="bf16", out="bf16", M=1, N=11008, K=4096, wt=False, act="relu",
             bias=True, keep=False, residual=False, pad=0),
        # The smallest square of the benchmark, where latency counts.
        dict(name="linear_square256", op="linear", type="f16", out="f16", M=256, N=256, K=256, wt=False, act="gelu",
             bias=True, keep=False, residual=False, pad=0),
        # A short batch of odd sizes whose rows follow each other without padding, with the block's input added.
        dict(name="linear_ragged", op="linear", type="f16", out="f16", M=333, N=1001, K=1237, wt=False, act="silu",
             bias=True, keep=False, residual=True, pad=0),
        # Back to the width behind the layer: the weight stored N x K, the residual stream added.
        dict(name="linear_residual", op="linear", type="bf16", out="bf16", M=2048, N=4096, K=11008, wt=True, act="none",
             bias=True, keep=False, residual=True, pad=0),
        # The benchmark's fully-connected layer for a full batch in training: Z is kept.  The largest.
        dict(name="linear_layer", op="linear", type="bf16", out="bf16", M=8192, N=11008, K=4096, wt=False, act="gelu",
             bias=True, keep=True, residual=False, pad=0),
        # The layer's whole backward pass for a micro-batch, the weight's gradient in FP32.
        dict(name="backward_layer", op="backward", type="bf16", out="f32", M=2048, N=11008, K=4096, act="gelu", pad=0),
        # The same for a short batch and odd widths, rows padded by three elements.
        dict(name="backward_ragged", op="backward", type="f16", out="f16", M=77, N=1237, K=1001, act="silu", pad=3),
        # A few decoding requests, each with two of sixteen experts: the experts' weights are what is read.
        dict(name="grouped_decode", op="grouped", type="bf16", out="bf16", M=64, E=16, N=4096, K=2048, wt=False,
             act="silu", bias=False, keep=False, residual=False, pad=0, spare=0),
        # A batch sorted by expert in training: Z is kept.
        dict(name="grouped_batch", op="grouped", type="bf16", out="bf16", M=8192, E=16, N=4096, K=2048, wt=False,
             act="gelu", bias=True, keep=True, residual=False, pad=0, spare=0),
        # Odd sizes, weights stored N x K, FP32 out on top of what is there, rows behind the last group.
        dict(name="grouped_ragged", op="grouped", type="f16", out="f32", M=777, E=7, N=1001, K=515, wt=True, act="none",
             bias=True, keep=False, residual=True, pad=0, spare=23),
        # Backward through the experts' second layer to the pre-activation of their first one.
        dict(name="grouped_backward", op="grouped_backward", type="bf16", out="f32", M=8192, E=16, N=2048, K=4096,
             act="gelu", pad=0, spare=0),
        # The same for a few rows of small experts, some of them without any.
        dict(name="grouped_backward_few", op="grouped_backward", type="f16", out="f16", M=300, E=24, N=256, K=1024,
             act="silu", pad=0, spare=5),
    ]


def _size(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n - n % 32 if n >= 64 and rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["linear", "linear", "backward", "grouped", "grouped", "grouped_backward"])
    t = rng.choice(["bf16", "f16"])
    out = rng.choice([t, t, "f32"])
    act = rng.choice(["none", "relu", "gelu", "silu"])
    pad = rng.choice([0, 0, 1, 8])
    flag = lambda: rng.random() < 0.5  # noqa: E731
    case = dict(op=op, type=t, out=out)
    if op == "linear":
        case.update(M=_size(rng, 1, 8192), N=_size(rng, 8, 11008), K=_size(rng, 8, 4096), wt=flag())
    elif op == "backward":
        case.update(M=_size(rng, 1, 2048), N=_size(rng, 8, 11008), K=_size(rng, 8, 4096))
    else:
        E = _size(rng, 1, 64)
        case.update(M=_size(rng, 1, 8192), E=E, N=_size(rng, 8, 4096 if E <= 16 else 2048), K=_size(rng, 8, 2048),
                    spare=rng.choice([0, 0, 17]))
    if op in ("linear", "grouped"):
        case.update(wt=flag(), bias=flag(), keep=flag(), residual=flag())
    return dict(case, act=act, pad=pad)


# ---- the plain form: 32-bit elementary operations --------------------------------------


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _slope(z, act):
    """The activation's derivative."""
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * torch.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def _layer(x, w, bias, r, act):
    z = x.float() @ w.float()
    if bias is not None:
        z = z + bias
    y = _act(z, act)
    return z, y if r is None else y + r.float()


def _plain(state):
    case = state["case"]
    op, act = case["op"], case["act"]
    dt, ot = TYPES[case["type"]], TYPES[case["out"]]
    if op == "linear":
        w = state["w"].t() if case["wt"] else state["w"]
        z, y = _layer(state["x"], w, state["bias"], state["r"], act)
        return {"y": y.to(ot), "z": z.to(dt)} if case["keep"] else {"y": y.to(ot)}
    if op == "backward":
        d = state["g"].float() * _slope(state["z"].float(), act)
        dz = d.to(dt)
        return {"dz": dz, "db": d.sum(0), "dx": (dz.float() @ state["w"].float().t()).to(dt),
                "dw": (state["x"].float().t() @ dz.float()).to(ot)}
    ends, spare = state["ends"], case["spare"]
    if op == "grouped":
        y = torch.zeros(case["M"] + spare, case["N"], dtype=ot, device="cuda")
        z = torch.zeros_like(y, dtype=dt)
        for e in range(case["E"]):
            a, b = ends[e], ends[e + 1]
            w = state["w"][e].t() if case["wt"] else state["w"][e]
            r = None if state["r"] is None else state["r"][a:b]
            ze, ye = _layer(state["x"][a:b], w, None if state["bias"] is None else state["bias"][e], r, act)
            y[a:b], z[a:b] = ye.to(ot), ze.to(dt)
        return {"y": y, "z": z} if case["keep"] else {"y": y}
    E, N, K = case["E"], case["N"], case["K"]
    dz = torch.zeros(case["M"] + spare, K, dtype=dt, device="cuda")
    db = torch.zeros(E, K, device="cuda")
    dw = torch.zeros(E, K, N, dtype=ot, device="cuda")
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        g = state["g"][a:b].float()
        d = (g @ state["w"][e].float().t()) * _slope(state["z"][a:b].float(), act)
        dz[a:b], db[e] = d.to(dt), d.sum(0)
        dw[e] = (state["x"][a:b].float().t() @ g).to(ot)
    return {"dz": dz, "db": db, "dw": dw}


# ---- the library's calls ---------------------------------------------------------------


def _own(state):
    import dense_fp32_gemm_sm_gb300 as fg

    case, out, ws = state["case"], state["out"], state["workspace"]
    op, M, N, K = case["op"], case["M"], case["N"], case["K"]
    types = {"f32": fg.F32, "bf16": fg.BF16, "f16": fg.F16}
    t, ot = types[case["type"]], types[case["out"]]
    act = {"none": fg.ACT_NONE, "relu": fg.ACT_RELU, "gelu": fg.ACT_GELU, "silu": fg.ACT_SILU}[case["act"]]
    size = 0 if ws is None else ws.numel()
    if op == "linear":
        x, w, r = state["x"], state["w"], state["r"]
        fg.gemm16(t, ot, fg.OP_N, fg.OP_T if case["wt"] else fg.OP_N, M, N, K, 1.0, x, x.stride(0), w, w.stride(0),
                  state["bias"], act, out.get("z"), N, 1.0 if r is not None else 0.0, r, N, out["y"], N, ws, size)
        return out
    if op == "backward":
        g, z, x, w = state["g"], state["z"], state["x"], state["w"]
        dz = out["dz"]
        fg.act16_grad(t, 1, M, N, None, act, g, g.stride(0), z, z.stride(0), dz, dz.stride(0), out["db"], ws, size)
        fg.gemm16(t, t, fg.OP_N, fg.OP_T, M, K, N, 1.0, dz, dz.stride(0), w, w.stride(0), None, fg.ACT_NONE, None, 0,
                  0.0, None, 0, out["dx"], K, ws, size)
        fg.gemm16(t, ot, fg.OP_T, fg.OP_N, K, N, M, 1.0, x, x.stride(0), dz, dz.stride(0), None, fg.ACT_NONE, None, 0,
                  0.0, None, 0, out["dw"], N, ws, size)
        return out
    E, offsets, w, x = case["E"], state["offsets"], state["w"], state["x"]
    rows = M + case["spare"]
    if op == "grouped":
        r = state["r"]
        fg.gemm16_grouped(t, ot, fg.OP_T if case["wt"] else fg.OP_N, E, rows, N, K, offsets, 1.0, x, x.stride(0), w,
                          w.stride(1), w.stride(0), state["bias"], act, out.get("z"), N,
                          1.0 if r is not None else 0.0, r, N, out["y"], N, ws, size)
        return out
    g, z = state["g"], state["z"]
    fg.gemm16_grouped_grad(t, t, fg.OP_T, E, rows, K, N, offsets, 1.0, g, g.stride(0), w, w.stride(1), w.stride(0), act,
                           z, z.stride(0), out["dz"], K, out["db"], ws, size)
    fg.gemm16_weight_grad(t, ot, E, rows, N, K, offsets, 1.0, x, x.stride(0), g, g.stride(0), 0.0, out["dw"], N, K * N,
                          ws, size)
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---- inputs ----------------------------------------------------------------------------


def _up(n, m):
    return -(-n // m)


def _ld(n):
    """Leading dimension of a matrix that the program lays out for the products: rows on 16 bytes."""
    return 8 * _up(n, 8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, M, N, K, pad = case["op"], case["M"], case["N"], case["K"], case["pad"]
    dt, ot = TYPES[case["type"]], TYPES[case["out"]]

    def normal(rows, cols, std=1.0):
        return std * torch.randn(rows, cols, device="cuda", generator=gen)

    def tokens(rows, cols):
        # activations: N(0, 1) with a few channels much larger than the rest; rows of cols + pad elements
        x = normal(rows, cols + pad)
        loud = torch.rand(cols + pad, device="cuda", generator=gen) < 0.005
        return torch.where(loud, 16 * x, x).to(dt)[:, :cols]

    def padded(rows, cols, std=1.0):
        return normal(rows, cols + pad, std).to(dt)[:, :cols]

    def empty(rows, cols, d=dt):
        return torch.empty(rows, cols, dtype=d, device="cuda")

    # gradients: a thousandth of the activations; in F16 as a scaled loss leaves them
    small = 1e-3 if case["type"] == "bf16" else 1.0
    state = {"case": case}
    space = 0  # copies of the operands that do not start their rows on 16 bytes, and partial column sums
    if op in ("linear", "grouped"):
        rows, E = M + case.get("spare", 0), case.get("E", 1)
        # the inner width is scaled for its louder channels, so that Z stays near one
        std = (K * (1 + 0.005 * 255)) ** -0.5
        shape = (N, K) if case["wt"] else (K, N)
        state["x"] = tokens(rows, K)
        w = torch.stack([normal(*shape, std).to(dt) for _ in range(E)])
        state["w"] = w[0] if op == "linear" else w
        bias = torch.rand(E, N, device="cuda", generator=gen) * 0.2 - 0.1 if case["bias"] else None
        state["bias"] = bias[0] if bias is not None and op == "linear" else bias
        state["r"] = normal(rows, N).to(ot) if case["residual"] else None
        state["out"] = {"y": torch.zeros(rows, N, dtype=ot, device="cuda")}
        if case["keep"]:
            state["out"]["z"] = torch.zeros(rows, N, dtype=dt, device="cuda")
        if state["x"].stride(0) % 8:
            space += 2 * rows * _ld(K)
        if shape[1] % 8:
            space += 2 * E * shape[0] * _ld(shape[1])
    elif op == "backward":
        state["g"], state["z"] = padded(M, N, small), padded(M, N)
        state["x"], state["w"] = tokens(M, K), normal(K, N, N ** -0.5).to(dt)
        state["out"] = {"dz": empty(M, _ld(N))[:, :N], "db": torch.empty(N, device="cuda"), "dx": empty(M, K),
                        "dw": empty(K, N, ot)}
        space = max(4 * N * 2 * (_up(M, 32) + 1), (0 if N % 8 == 0 else 2 * K * _ld(N)),
                    (0 if state["x"].stride(0) % 8 == 0 else 2 * M * _ld(K)))
    else:
        rows, E = M + case["spare"], case["E"]
        state["g"], state["z"] = padded(rows, N, small), padded(rows, K)
        state["x"] = tokens(rows, K)
        state["w"] = torch.stack([normal(K, N, N ** -0.5).to(dt) for _ in range(E)])
        state["out"] = {"dz": torch.zeros(rows, K, dtype=dt, device="cuda"), "db": torch.empty(E, K, device="cuda"),
                        "dw": torch.empty(E, K, N, dtype=ot, device="cuda")}
        g = 0 if state["g"].stride(0) % 8 == 0 else 2 * rows * _ld(N)
        space = max(4 * K * 2 * (_up(rows, 32) + E) + g + (0 if N % 8 == 0 else 2 * E * K * _ld(N)),
                    g + (0 if state["x"].stride(0) % 8 == 0 else 2 * rows * _ld(K)))
    if "E" in case:
        # a router's choice: experts differ in how often they are taken, and some may go without rows
        E = case["E"]
        share = torch.softmax(torch.randn(E, device="cuda", generator=gen), 0)
        counts = torch.bincount(torch.multinomial(share, M, replacement=True, generator=gen), minlength=E)
        offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        offsets[1:] = counts.cumsum(0)
        state["offsets"], state["ends"] = offsets, offsets.tolist()
    # pieces of the workspace start on 256 bytes
    state["workspace"] = torch.empty(space + 1024, dtype=torch.uint8, device="cuda") if space else None
    return state


def work(case):
    op, M, N, K, E = case["op"], case["M"], case["N"], case["K"], case.get("E", 1)
    es, os = SIZE[case["type"]], SIZE[case["out"]]
    # experts that have rows, where each row takes any of them alike
    met = E if E == 1 else min(E, max(1, round(E * (1 - (1 - 1 / E) ** M))))
    if op in ("linear", "grouped"):
        size = (M * K + met * K * N) * es + M * N * os * (2 if case["residual"] else 1)
        size += (M * N * es if case["keep"] else 0) + (4 * met * N if case["bias"] else 0)
        return {"bytes": size, "flops": 2.0 * M * N * K}
    if op == "backward":
        return {"bytes": 3 * M * N * es + 2 * M * K * es + K * N * (es + os) + 4 * N, "flops": 4.0 * M * N * K}
    return {"bytes": M * N * es + 3 * M * K * es + met * K * N * es + E * (K * N * os + 4 * K), "flops": 4.0 * M * N * K}


# ---- the definition in 64 bits ---------------------------------------------------------


def _exact_act(z, act):
    """(activation, derivative) in float64."""
    if act == "relu":
        return torch.relu(z), torch.where(z > 0, 1.0, 0.0).double()
    if act == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z.square() / 2) * 0.3989422804014327
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    return z, torch.ones_like(z)


def exact(case, seed):
    state = prepare(case, seed)
    op, act, dt = case["op"], case["act"], TYPES[case["type"]]
    if op == "backward":
        d = state["g"].double() * _exact_act(state["z"].double(), act)[1]
        dz = d.to(dt).double()  # the products take the gradient as it is kept
        return {"dz": d, "db": torch.einsum("mn->n", d), "dx": torch.einsum("mn,kn->mk", dz, state["w"].double()),
                "dw": torch.einsum("mk,mn->kn", state["x"].double(), dz)}
    grouped = "E" in case
    ends = state["ends"] if grouped else [0, case["M"]]
    parts = []
    for e in range(len(ends) - 1):
        at = slice(ends[e], ends[e + 1])
        w = state["w"][e].double() if grouped else state["w"].double()
        x = state["x"][at].double()
        if op == "grouped_backward":
            g = state["g"][at].double()
            d = torch.einsum("mn,kn->mk", g, w) * _exact_act(state["z"][at].double(), act)[1]
            parts.append((d, torch.einsum("mk->k", d), torch.einsum("mk,mn->kn", x, g)))
            continue
        z = torch.einsum("mk,nk->mn" if case["wt"] else "mk,kn->mn", x, w)
        if state["bias"] is not None:
            z = z + (state["bias"][e] if grouped else state["bias"]).double()
        y = _exact_act(z, act)[0]
        if state["r"] is not None:
            y = y + state["r"][at].double()
        parts.append((y, z))
    rest = torch.zeros(case.get("spare", 0), parts[0][0].shape[1], dtype=torch.float64, device="cuda")
    first = torch.cat([p[0] for p in parts] + [rest])
    if op == "grouped_backward":
        return {"dz": first, "db": torch.stack([p[1] for p in parts]), "dw": torch.stack([p[2] for p in parts])}
    return {"y": first, "z": torch.cat([p[1] for p in parts] + [rest])} if case["keep"] else {"y": first}
