"""A fully-connected layer Y = ReLU(X W + b) in MXFP4, trained and served.

The package's MXFP4 calls as they go together: the master weight W (K x N) is quantised both
ways in one pass, along its columns for the product forward and along its rows for the
gradient of X; tokens X (M x K) along their rows forward and their columns for the gradient
of W; the output's gradient both ways behind ReLU's gate, with the bias's gradient.  A few
tokens at a time go through ``decode``, which quantises them on the way.

``forward`` and ``backward`` work in buffers of the layer (those of the last few sizes met), so they are used on
one stream at a time.
``python -m dense_fp32_gemm_sm_gb300.mxfp4_layer`` fits a small layer to another one's outputs.
"""

from __future__ import annotations

import weakref

import torch

from . import _binding as fg

SIZES = 4  # numbers of tokens whose buffers a layer keeps

_TYPES = {torch.float32: fg.F32, torch.bfloat16: fg.BF16, torch.float16: fg.F16}


class Quantised:
    """Codes and scales of a quantised matrix of rows x cols.  Rows of codes start on 64 bytes: products
    read them in pieces of 128 (4096 x 4096 x 4000 with ld 2000: 36 us, with 2048: 27)."""

    def __init__(self, rows: int, cols: int, device):
        self.shape = (rows, cols)
        self.ld = 64 * max(1, -(-cols // 128))
        self.codes = torch.empty(rows, self.ld, dtype=torch.uint8, device=device)
        self.scales = torch.empty(fg.mxfp4_scales_size(rows, cols), dtype=torch.uint8, device=device)

    @property
    def args(self):
        return self.codes, self.ld, self.scales


class Saved:
    """What a forward leaves for its backward: its tokens, quantised along their columns (a K x M matrix), and
    where its output is."""

    def __init__(self, layer: "Mxfp4Layer", tokens: Quantised, output: int):
        self.of, self.tokens, self.output = weakref.ref(layer), tokens, output
        self.kept = False  # a caller has it, so later forwards leave its tokens alone


class Mxfp4Layer:
    """``weight`` (K x N) and ``bias`` (N floats, or None) stay the caller's; call ``update`` after
    changing the weight.  The element type of weight, tokens and gradients is the weight's."""

    def __init__(self, weight: torch.Tensor, bias: torch.Tensor | None = None, relu: bool = True):
        if weight.dtype not in _TYPES or weight.dim() != 2 or weight.stride(1) != 1:
            raise ValueError("weight: a K x N matrix of float32, bfloat16 or float16, rows contiguous")
        if bias is not None and not (isinstance(bias, torch.Tensor) and bias.dtype == torch.float32 and bias.is_contiguous()
                                     and bias.numel() == weight.shape[1] and bias.device == weight.device):
            raise ValueError("bias: %d consecutive float32 on %s" % (weight.shape[1], weight.device))
        self.weight, self.bias, self.relu = weight, bias, relu
        self.type = _TYPES[weight.dtype]
        self.K, self.N = weight.shape
        self.w_rows = Quantised(self.K, self.N, weight.device)
        self.w_cols = Quantised(self.N, self.K, weight.device)
        self._sized = {}      # rows -> buffers of the last sizes met, the latest last
        self._latest = None   # what the latest forward left (None for no tokens)
        self.update()

    def update(self) -> None:
        """Quantise the weight both ways."""
        fg.mxfp4_quantize(self.type, self.K, self.N, self.weight, self.weight.stride(0), *self.w_rows.args,
                          *self.w_cols.args)

    def _buffers(self, M: int):
        b = self._sized.pop(M, None)
        if b is None:
            dev, K, N = self.weight.device, self.K, self.N
            if len(self._sized) == SIZES:
                del self._sized[next(iter(self._sized))]
            b = dict(x_rows=Quantised(M, K, dev), g_rows=Quantised(M, N, dev), g_cols=Quantised(N, M, dev), saved=None,
                     workspace=torch.empty(fg.mxfp4_quantize_grad_workspace_size(M, N), dtype=torch.uint8, device=dev))
        self._sized[M] = b
        return b

    def _tokens(self, x: torch.Tensor, cols: int):
        """Rows and leading dimension of a matrix given to a call."""
        if x.dtype != self.weight.dtype or x.dim() != 2 or x.shape[1] != cols or (x.shape[0] and x.stride(1) != 1):
            raise ValueError("a matrix of %s with %d contiguous columns" % (self.weight.dtype, cols))
        M = x.shape[0]
        if M > 1 and x.stride(0) < cols:  # expanded rows, windows: the kernels read rows of their own
            raise ValueError("rows that overlap (row stride %d for %d columns): pass .contiguous()" % (x.stride(0), cols))
        return M, max(x.stride(0) if M > 1 else cols, 1)

    def decode(self, x: torch.Tensor) -> torch.Tensor:
        """Y for tokens x (M x K): quantised on the way, nothing kept."""
        M, ldx = self._tokens(x, self.K)
        y = torch.empty(M, self.N, dtype=x.dtype, device=x.device)
        need = fg.mxfp4_linear_workspace_size(M, self.N, self.K)  # 0 for a few tokens
        space = torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
        fg.mxfp4_linear(self.type, M, self.N, self.K, x, ldx, *self.w_cols.args, self.bias, self.relu, y, self.N,
                        space, need)
        return y

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """Y for tokens x (M x K), which stay quantised along their columns for ``backward``: the layer keeps
        those of the last forward for each of the last ``SIZES`` numbers of tokens, and ``saved`` is what
        the caller keeps where more forwards come before their backwards.  (``decode`` keeps nothing.)"""
        M, ldx = self._tokens(x, self.K)
        y = torch.empty(M, self.N, dtype=x.dtype, device=x.device)
        self._latest = None
        if M:
            b = self._buffers(M)
            last, b["saved"] = b["saved"], None
            cols = last.tokens if last and not last.kept else Quantised(self.K, M, self.weight.device)
            fg.mxfp4_quantize(self.type, M, self.K, x, ldx, *b["x_rows"].args, *cols.args)
            fg.mxfp4_gemm(self.type, M, self.N, self.K, 1.0, *b["x_rows"].args, *self.w_cols.args, 0.0, y, self.N, self.bias,
                          self.relu)
            self._latest = b["saved"] = Saved(self, cols, y.data_ptr())
        return y

    @property
    def saved(self) -> Saved | None:
        """What the latest forward left for its backward, the caller's from here on."""
        if self._latest:
            self._latest.kept = True
        return self._latest

    def backward(self, g: torch.Tensor, y: torch.Tensor | None, saved: Saved | None = None):
        """(dX, dW, db) for the gradient g of the output y (None will do without ReLU) of the forward that left
        ``saved``, or else of the last forward with as many tokens, whose output y then has to be."""
        M, ldg = self._tokens(g, self.N)
        rows, ldy = self._tokens(y, self.N) if self.relu else (M, 0)
        if rows != M:  # y is read as the gate of every row of g
            raise ValueError("%d outputs for %d gradients" % (rows, M))
        if saved is not None:
            if not isinstance(saved, Saved) or saved.of() is not self or saved.tokens.shape[1] != M:
                raise ValueError("saved: what a forward of this layer with %d tokens left" % M)
        elif M:
            saved = self._sized[M]["saved"] if M in self._sized else None
            if saved is None:  # there are no tokens to multiply the gradient with
                raise ValueError("no forward with %d tokens before this backward" % M)
            if y is not None and y.data_ptr() != saved.output:  # another forward's tokens have taken its place
                raise ValueError("y is not the output of the last forward with %d tokens: keep the layer's `saved` after "
                                 "its forward and pass it" % M)
        dev, dt = g.device, g.dtype
        dx = torch.empty(M, self.K, dtype=dt, device=dev)
        dw = torch.zeros(self.K, self.N, dtype=dt, device=dev) if M == 0 else torch.empty(self.K, self.N, dtype=dt, device=dev)
        db = torch.empty(self.N, device=dev) if M else torch.zeros(self.N, device=dev)
        if M:
            b = self._buffers(M)
            ws = b["workspace"]
            fg.mxfp4_quantize_grad(self.type, M, self.N, g, ldg, y if self.relu else None, ldy, *b["g_rows"].args,
                                   *b["g_cols"].args, db, ws, ws.numel())
            fg.mxfp4_gemm(self.type, M, self.K, self.N, 1.0, *b["g_rows"].args, *self.w_rows.args, 0.0, dx, self.K)
            fg.mxfp4_gemm(self.type, self.K, self.N, M, 1.0, *saved.tokens.args, *b["g_cols"].args, 0.0, dw, self.N)
        return dx, dw, db


def main(steps: int = 60, M: int = 512, K: int = 256, N: int = 384) -> list[float]:
    """Fit a layer to another one's outputs; prints and returns the losses."""
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    target_w, target_b = rand(K, N) / K**0.5, 0.1 * rand(N)
    w, b = rand(K, N) / K**0.5, torch.zeros(N, device="cuda")
    layer, losses = Mxfp4Layer(w, b), []
    for step in range(steps):
        x = rand(M, K)
        want = (x @ target_w + target_b).clamp(min=0)
        y = layer.forward(x)
        diff = y - want
        losses.append(float(diff.square().mean()))
        _, dw, db = layer.backward(diff * (2.0 / M), y)
        w -= 0.25 * dw
        b -= 0.25 * db
        layer.update()
        if step % 10 == 0 or step + 1 == steps:
            print("step %d: loss %.4f" % (step, losses[-1]))
    x = rand(3, K)
    print("three tokens through decode: largest difference from forward %.2g"
          % float((layer.decode(x) - layer.forward(x)).abs().max()))
    return losses


if __name__ == "__main__":
    main()
