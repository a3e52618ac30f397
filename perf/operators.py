"""The microscaled 4-bit (MXFP4) operators of the library as they are called, case by case.

A quantised matrix holds 4-bit E2M1 codes in blocks of 32 along its rows, with one power-of-two
scale (E8M0) a block.  The cases are the parts of a fully-connected layer Y = ReLU(X W + b) in that
format: quantising tokens and weights, the products, the layer for a few tokens with X quantised
on the way, and the layer's backward pass.  ``own`` selects the library's entry points or a plain
evaluation in elementary torch operations; both take the same inputs, quantised matrices included,
in the library's layout.
"""

import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
LUT = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    return [
        # The layer's tokens before its product: the widest read, one direction (inference).
        dict(name="quantize_tokens", op="quantize", type="f32", M=8192, N=4096, rows=True, cols=False, pad=0),
        # A small weight of odd sizes in both directions (training keeps both), padded rows.
        dict(name="quantize_ragged_both", op="quantize", type="f16", M=333, N=1001, rows=True, cols=True, pad=3),
        # The layer's output gradient behind ReLU, both directions and the bias's gradient.
        dict(name="grad_layer", op="grad", type="bf16", M=8192, N=11008, gate=True, bias=True, pad=0),
        # The same for a short batch and an odd width.
        dict(name="grad_ragged", op="grad", type="f32", M=77, N=1237, gate=True, bias=True, pad=1),
        # The smallest square of the benchmark, where latency counts.
        dict(name="gemm_square256", op="gemm", type="f32", M=256, N=256, K=256, alpha=1.0, beta=0.0, bias=False, relu=False, pad=0),
        # The benchmark's headline square, in the type that a network's activations have.
        dict(name="gemm_square4096", op="gemm", type="bf16", M=4096, N=4096, K=4096, alpha=1.0, beta=0.0, bias=False, relu=False, pad=0),
        # The benchmark's fully-connected layer for a full batch of tokens: the largest.
        dict(name="gemm_layer", op="gemm", type="f32", M=8192, N=11008, K=4096, alpha=1.0, beta=0.0, bias=True, relu=True, pad=0),
        # A long sum into few outputs, odd sizes, added to what is there (gradient accumulation).
        dict(name="gemm_long_sum", op="gemm", type="f32", M=130, N=1001, K=11013, alpha=0.5, beta=1.0, bias=False, relu=False, pad=2),
        # One token through the layer: decoding.
        dict(name="linear_one_token", op="linear", type="f32", M=1, N=11008, K=4096, bias=True, relu=True, pad=0),
        # A few tokens (a draft to verify) through a small layer of odd sizes.
        dict(name="linear_seven_ragged", op="linear", type="bf16", M=7, N=1001, K=1237, bias=True, relu=False, pad=1),
        # A batch of decoding requests through the layer that brings the width back.
        dict(name="linear_batch32", op="linear", type="bf16", M=32, N=4096, K=11008, bias=False, relu=False, pad=0),
        # The layer's whole backward pass for a micro-batch: dX, dW and the bias's gradient.
        dict(name="backward_layer", op="backward", type="bf16", M=2048, N=11008, K=4096, pad=0),
    ]


def _size(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = n - n % 32 if n >= 64 and rng.random() < 0.4 else n
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["quantize", "grad", "gemm", "linear", "backward"])
    t = rng.choice(["f32", "bf16", "f16"] if op in ("quantize", "gemm", "linear") else ["f32", "bf16"])
    pad = rng.choice([0, 0, 1, 3, 8])
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op == "quantize":
        rows, cols = rng.choice([(True, False), (False, True), (True, True)])
        return dict(op=op, type=t, M=_size(rng, 1, 8192), N=_size(rng, 1, 11008), rows=rows, cols=cols, pad=pad)
    if op == "grad":
        return dict(op=op, type=t, M=_size(rng, 1, 8192), N=_size(rng, 1, 11008), gate=flag(), bias=flag(), pad=pad)
    if op == "gemm":
        return dict(op=op, type=t, M=_size(rng, 16, 8192), N=_size(rng, 16, 11008), K=_size(rng, 32, 4096),
                    alpha=rng.choice([1.0, 0.5]), beta=rng.choice([0.0, 0.0, 1.0]), bias=flag(), relu=flag(), pad=pad)
    if op == "linear":
        return dict(op=op, type=t, M=_size(rng, 1, 64), N=_size(rng, 64, 11008), K=_size(rng, 64, 11008), bias=flag(), relu=flag(), pad=pad)
    return dict(op=op, type=t, M=_size(rng, 32, 2048), N=_size(rng, 64, 11008), K=_size(rng, 64, 4096), pad=pad)


# ---- sizes of a quantised matrix ------------------------------------------------------


def _up(n, m):
    return -(-n // m)


def _ld(cols):
    """Bytes of a row of codes: whole blocks of 32."""
    return 16 * _up(cols, 32)


def _scale_bytes(rows, cols):
    return 512 * _up(rows, 128) * _up(_up(cols, 32), 4)


# ---- the plain form: 32-bit elementary operations --------------------------------------


def _encode(x):
    """x (rows x cols, float32) -> (codes 0..15 rows x 32 nb, scale bytes rows x nb)."""
    rows, cols = x.shape
    nb = _up(cols, 32)
    b = torch.nn.functional.pad(x, (0, 32 * nb - cols)).reshape(rows, nb, 32)
    bits = b.view(torch.int32)
    field = ((bits & 0x7FFFFFFF) >> 23).amax(2)
    s = (field - 2).clamp(min=0)
    s = torch.where(field == 255, torch.full_like(s, 255), s)
    inverse = ((254 - s.clamp(max=252)) << 23).view(torch.float32)  # 2^(127 - s)
    v = (b * inverse[:, :, None]).abs().clamp(max=6.0)
    code = torch.where(v < 2, (2 * v).round(), torch.where(v < 4, v.round() + 2, (v / 2).round() + 4))
    code = code.nan_to_num(0.0).to(torch.int32) + ((bits >> 28) & 8)
    code = torch.where(s[:, :, None] == 255, torch.zeros_like(code), code)
    return code.reshape(rows, 32 * nb), s


def _values(code, s, cols):
    """What codes and scale bytes stand for, as float32."""
    lut = torch.tensor(LUT, device=code.device)
    scale = torch.where(s > 0, s << 23, torch.full_like(s, 1 << 22)).view(torch.float32)
    scale = torch.where(s == 255, torch.full_like(scale, float("nan")), scale)
    v = lut[code.long()].reshape(code.shape[0], -1, 32) * scale[:, :, None]
    return v.reshape(code.shape[0], -1)[:, :cols]


def _pack(x):
    """x (float32) as a quantised matrix in the library's layout: (codes, scales) bytes."""
    code, s = _encode(x)
    rows, nb = s.shape
    codes = (code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8)
    full = torch.zeros(_up(rows, 128) * 128, _up(nb, 4) * 4, dtype=torch.uint8, device=x.device)
    full[:rows, :nb] = s.to(torch.uint8)
    atoms = full.reshape(-1, 4, 32, _up(nb, 4), 4).permute(0, 3, 2, 1, 4)
    return codes.contiguous(), atoms.contiguous().reshape(-1)


def _unpack(codes, scales, rows, cols):
    """The values of a quantised matrix in the library's layout, as float32."""
    nb = _up(cols, 32)
    c = codes.to(torch.int32)
    code = torch.stack((c & 15, c >> 4), 2).reshape(rows, -1)
    s = scales.reshape(-1, _up(nb, 4), 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, 4 * _up(nb, 4))
    return _values(code, s[:rows, :nb].to(torch.int32), cols)


def _through(x):
    """Quantised and back."""
    code, s = _encode(x)
    return _values(code, s, x.shape[1])


def _layer(a, b, alpha, beta, c, bias, relu):
    y = alpha * (a @ b.t())
    if beta:
        y = y + beta * c[:, :b.shape[0]].float()
    if bias is not None:
        y = y + bias
    return y.clamp(min=0) if relu else y


def _plain(state):
    case = state["case"]
    dt = TYPES[case["type"]]
    op = case["op"]
    if op == "quantize":
        x = state["x"].float()
        out = {}
        if case["rows"]:
            out["rows"] = _through(x).to(dt)
        if case["cols"]:
            out["cols"] = _through(x.t().contiguous()).to(dt)
        return out
    if op in ("grad", "backward"):
        g = state["g"].float()
        if state["y"] is not None:
            g = torch.where(state["y"] > 0, g, torch.zeros_like(g))
        rows, cols = _through(g), _through(g.t().contiguous())
        if op == "grad":
            out = {"rows": rows.to(dt), "cols": cols.to(dt)}
            if case["bias"]:
                out["bias"] = g.sum(0)
            return out
        w = _unpack(*state["w"], case["K"], case["N"])
        x = _unpack(*state["x"], case["K"], case["M"])
        return {"dx": (rows @ w.t()).to(dt), "dw": (x @ cols.t()).to(dt), "bias": g.sum(0)}
    if op == "gemm":
        a = _unpack(*state["a"], case["M"], case["K"])
        b = _unpack(*state["b"], case["N"], case["K"])
        return _layer(a, b, case["alpha"], case["beta"], state["c"], state["bias"], case["relu"]).to(dt)
    w = _unpack(*state["w"], case["N"], case["K"])
    return _layer(_through(state["x"].float()), w, 1.0, 0.0, None, state["bias"], case["relu"]).to(dt)


# ---- the library's calls ---------------------------------------------------------------


def _own(state):
    import dense_fp32_gemm_sm_gb300 as fg

    case = state["case"]
    op, out = case["op"], state["out"]
    t = {"f32": fg.F32, "bf16": fg.BF16, "f16": fg.F16}[case["type"]]
    M, N = case["M"], case["N"]
    if op == "quantize":
        r, c = state["r"], state["c"]
        fg.mxfp4_quantize(t, M, N, state["x"], N + case["pad"], r and r[0], _ld(N), r and r[1], c and c[0], _ld(M), c and c[1])
        if r:
            fg.mxfp4_dequantize(t, M, N, r[0], _ld(N), r[1], out["rows"], N)
        if c:
            fg.mxfp4_dequantize(t, N, M, c[0], _ld(M), c[1], out["cols"], M)
        return out
    if op in ("grad", "backward"):
        r, c, ws = state["r"], state["c"], state["workspace"]
        fg.mxfp4_quantize_grad(t, M, N, state["g"], N + case["pad"], state["y"], N + case["pad"], r[0], _ld(N), r[1],
                               c[0], _ld(M), c[1], out.get("bias"), ws, ws.numel())
        if op == "grad":
            fg.mxfp4_dequantize(t, M, N, r[0], _ld(N), r[1], out["rows"], N)
            fg.mxfp4_dequantize(t, N, M, c[0], _ld(M), c[1], out["cols"], M)
            return out
        K, w, x = case["K"], state["w"], state["x"]
        fg.mxfp4_gemm(t, M, K, N, 1.0, r[0], _ld(N), r[1], w[0], _ld(N), w[1], 0.0, out["dx"], K)
        fg.mxfp4_gemm(t, K, N, M, 1.0, x[0], _ld(M), x[1], c[0], _ld(M), c[1], 0.0, out["dw"], N)
        return out
    K = case["K"]
    if op == "gemm":
        a, b = state["a"], state["b"]
        if case["beta"]:
            out.copy_(state["c"])  # the call adds to its C: each pass starts from the same one
        fg.mxfp4_gemm(t, M, N, K, case["alpha"], a[0], _ld(K), a[1], b[0], _ld(K), b[1], case["beta"], out, N + case["pad"],
                      state["bias"], case["relu"])
        return out[:, :N]
    w, ws = state["w"], state["workspace"]
    fg.mxfp4_linear(t, M, N, K, state["x"], K + case["pad"], w[0], _ld(K), w[1], state["bias"], case["relu"], out, N, ws, ws.numel())
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---- inputs ----------------------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, op, M, N, pad = TYPES[case["type"]], case["op"], case["M"], case["N"], case["pad"]

    def normal(rows, cols, std=1.0):
        return std * torch.randn(rows, cols, device="cuda", generator=g)

    def tokens(rows, cols, extra=0):
        # activations: N(0, 1) with a few channels much larger than the rest
        x = normal(rows, cols + extra)
        loud = torch.rand(cols + extra, device="cuda", generator=g) < 0.005
        return torch.where(loud, 16 * x, x)

    def empty(rows, cols, d=dt):
        return torch.empty(rows, cols, dtype=d, device="cuda")

    def quantised(rows, cols):  # room for a quantised matrix
        return (torch.empty(rows, _ld(cols), dtype=torch.uint8, device="cuda"),
                torch.empty(_scale_bytes(rows, cols), dtype=torch.uint8, device="cuda"))

    state = {"case": case}
    if op == "quantize":
        state["x"] = tokens(M, N, pad).to(dt)[:, :N]
        state["r"] = quantised(M, N) if case["rows"] else None
        state["c"] = quantised(N, M) if case["cols"] else None
        state["out"] = {k: empty(*s) for k, s in (("rows", (M, N)), ("cols", (N, M))) if case[k]}
    elif op in ("grad", "backward"):
        # a gradient a thousandth the size of the activations, and the layer's ReLU output
        state["g"] = normal(M, N + pad, 1e-3).to(dt)[:, :N]
        state["y"] = normal(M, N + pad).clamp(min=0).to(dt)[:, :N] if case.get("gate", True) else None
        state["r"], state["c"] = quantised(M, N), quantised(N, M)
        # one partial sum of each column for every 128 rows
        state["workspace"] = torch.empty(4 * N * _up(M, 128), dtype=torch.uint8, device="cuda")
        out = {"bias": torch.empty(N, device="cuda")} if case.get("bias", True) else {}
        if op == "grad":
            out.update(rows=empty(M, N), cols=empty(N, M))
        else:
            K = case["K"]
            state["w"] = _pack(normal(K, N, K ** -0.5))
            state["x"] = _pack(tokens(M, K).t().contiguous())
            out.update(dx=empty(M, K), dw=empty(K, N))
        state["out"] = out
    else:
        K = case["K"]
        state["bias"] = torch.rand(N, device="cuda", generator=g) * 0.2 - 0.1 if case["bias"] else None
        if op == "gemm":
            state["a"], state["b"] = _pack(tokens(M, K)), _pack(normal(N, K, K ** -0.5))
            state["out"] = empty(M, N + pad)
            state["c"] = normal(M, N + pad).to(dt) if case["beta"] else None
        else:
            state["x"] = tokens(M, K, pad).to(dt)[:, :K]
            state["w"] = _pack(normal(N, K, K ** -0.5))
            state["out"] = empty(M, N)
            # room for the tokens' codes and scales, where the call quantises them first
            state["workspace"] = torch.empty(M * _ld(K) + _scale_bytes(M, K) + 256, dtype=torch.uint8, device="cuda")
    return state


def work(case):
    op, M, N, es = case["op"], case["M"], case["N"], SIZE[case["type"]]
    q = lambda rows, cols: rows * _ld(cols) + rows * _up(cols, 32)  # noqa: E731
    if op == "quantize":
        ways = [q(M, N)] * case["rows"] + [q(N, M)] * case["cols"]
        return {"bytes": M * N * es + sum(2 * w + M * N * es for w in ways), "flops": 0}
    read = M * N * es * (2 if case.get("gate", True) else 1)
    if op == "grad":
        return {"bytes": read + 2 * (q(M, N) + q(N, M)) + 2 * M * N * es + (4 * N if case["bias"] else 0), "flops": 0}
    K = case["K"]
    if op == "backward":
        return {"bytes": read + q(K, N) + q(K, M) + (M * K + K * N) * es + 4 * N, "flops": 4.0 * M * N * K}
    out = M * N * es * (2 if op == "gemm" and case["beta"] else 1) + (4 * N if case["bias"] else 0)
    a = q(M, K) if op == "gemm" else M * K * es
    return {"bytes": a + q(N, K) + out, "flops": 2.0 * M * N * K}


# ---- the definition in 64 bits ---------------------------------------------------------


def _power_of_two(e):
    """2^e in float64 for whole e from -1022 to 1023, by its exponent field."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_through(x):
    """The definition block by block: the scale from the exponent of the largest magnitude, the
    nearest of the eight magnitudes by their midpoints, ties to the even one."""
    rows, cols = x.shape
    pad = -cols % 32
    b = torch.cat((x, x.new_zeros(rows, pad)), 1).reshape(rows, -1, 32)
    top = b.abs().max(2, keepdim=True).values
    exponent = (torch.frexp(top).exponent - 3).clamp(min=-127)
    scale = _power_of_two(torch.where(top == 0, torch.full_like(exponent, -127), exponent))
    v = b / scale
    middle = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=x.device)
    below = torch.bucketize(v.abs(), middle)
    above = torch.bucketize(v.abs(), middle, right=True)
    index = torch.where(below % 2 == 0, below, above)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    return (torch.sign(v) * grid[index] * scale).reshape(rows, -1)[:, :cols]


def _exact_matrix(codes, scales, rows, cols):
    """Element (r, k): bits 1 + 2 + 1 of its code, times the scale found at its byte's address."""
    r = torch.arange(rows, device=codes.device)[:, None]
    k = torch.arange(cols, device=codes.device)[None, :]
    code = (codes[r, k // 2].short() >> (4 * (k % 2)).short()) & 15
    e, m = (code >> 1) & 3, code & 1
    value = torch.where(e == 0, 0.5 * m.double(), (1 + 0.5 * m.double()) * _power_of_two(e - 1))
    value = torch.where(code >= 8, -value, value)
    block = torch.arange(_up(cols, 32), device=codes.device)[None, :]
    at = 512 * ((r // 128) * _up(_up(cols, 32), 4) + block // 4) + 16 * (r % 32) + 4 * ((r % 128) // 32) + block % 4
    scale = _power_of_two(scales[at].long() - 127)
    return value * scale.repeat_interleave(32, 1)[:, :cols]


def exact(case, seed):
    op, M, N = case["op"], case["M"], case["N"]
    state = prepare(case, seed)
    if op == "quantize":
        x = state["x"].double()
        return {k: _exact_through(v) for k, v in (("rows", x), ("cols", x.t())) if case[k]}
    if op in ("grad", "backward"):
        g = state["g"].double()
        if state["y"] is not None:
            g = g * (state["y"] > 0)
        rows, cols = _exact_through(g), _exact_through(g.t())
        out = {"bias": g.sum(0)} if case.get("bias", True) else {}
        if op == "grad":
            return dict(out, rows=rows, cols=cols)
        w = _exact_matrix(*state["w"], case["K"], N)
        x = _exact_matrix(*state["x"], case["K"], M)
        return dict(out, dx=torch.einsum("mn,kn->mk", rows, w), dw=torch.einsum("km,nm->kn", x, cols))
    K = case["K"]
    if op == "gemm":
        a, b = _exact_matrix(*state["a"], M, K), _exact_matrix(*state["b"], N, K)
    else:
        a, b = _exact_through(state["x"].double()), _exact_matrix(*state["w"], N, K)
    y = torch.einsum("mk,nk->mn", a, b)
    if op == "gemm":
        y = case["alpha"] * y
        if case["beta"]:
            y = y + case["beta"] * state["c"][:, :N].double()
    if state["bias"] is not None:
        y = y + state["bias"].double()
    return torch.relu(y) if case["relu"] else y
