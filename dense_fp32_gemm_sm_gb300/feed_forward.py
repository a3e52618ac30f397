"""A feed-forward block in BF16 or F16, Y = act(X W1 + b1) W2 + b2 (+ X), and the same by experts.

The package's 16-bit calls as they go together: the first layer keeps its pre-activation Z for the
backward pass; the second adds the residual in its epilogue.  Backward, the gradient of the second layer's
input goes through act'(Z) in the product's epilogue, which also gives the gradient of b1.
With weights of E experts (E x K x N, E x N x K) rows offsets[e] .. offsets[e+1] - 1 of X belong to
expert e; the offsets stay on the device.

Calls allocate their outputs and workspaces from torch on the current stream, and may run on any streams of one device.
A backward on another stream than its forward's has to come after it (``wait_stream``); what the forward left is then
not given out again before that stream is done with it.  The caller's own tensors are the caller's to ``record_stream``.
``python -m dense_fp32_gemm_sm_gb300.feed_forward`` fits a small block of experts to another one's outputs.
"""

from __future__ import annotations

import torch

from . import _binding as fg

_TYPES = {torch.float32: fg.F32, torch.bfloat16: fg.BF16, torch.float16: fg.F16}
ACTIVATIONS = {"none": fg.ACT_NONE, "relu": fg.ACT_RELU, "gelu": fg.ACT_GELU, "silu": fg.ACT_SILU}


class Saved:
    """What a forward leaves for its backward."""

    def __init__(self, x, z, h, offsets, stream=None):
        self.x, self.z, self.h, self.offsets = x, z, h, offsets
        self.stream = stream  # that they were made on

    def used_on(self, stream):
        if self.stream is not None and stream != self.stream:
            for t in (self.x, self.z, self.h, self.offsets):
                if t is not None:
                    t.record_stream(stream)


class FeedForward:
    """``w1`` (K x N), ``w2`` (N x K), or E of each; biases are float32 (N, K; E x N, E x K) or None.  All
    stay the caller's.  ``grad_type``: of the weights' gradients.  Rows of no expert are 0 in Y and in dX, with
    ``residual`` too (X and the gradient are added to rows of experts alone)."""

    def __init__(self, w1, w2, b1=None, b2=None, act: str = "gelu", residual: bool = False, grad_type=torch.float32):
        if w1.dtype not in (torch.bfloat16, torch.float16) or w1.dim() not in (2, 3) or not w1.is_contiguous():
            raise ValueError("w1: K x N, or E x K x N, of bfloat16 or float16, contiguous")
        self.experts = w1.shape[0] if w1.dim() == 3 else None
        self.K, self.N = w1.shape[-2:]
        lead = w1.shape[:-2]
        if w2.dtype != w1.dtype or tuple(w2.shape) != (*lead, self.N, self.K) or not w2.is_contiguous() or w2.device != w1.device:
            raise ValueError("w2: %s of %s on %s, contiguous" % ((*lead, self.N, self.K), w1.dtype, w1.device))
        for name, b, n in (("b1", b1, self.N), ("b2", b2, self.K)):
            if b is not None and (b.dtype != torch.float32 or tuple(b.shape) != (*lead, n) or not b.is_contiguous()
                                  or b.device != w1.device):
                raise ValueError("%s: %s of float32 on %s, contiguous" % (name, (*lead, n), w1.device))
        if act not in ACTIVATIONS or grad_type not in (torch.float32, w1.dtype):
            raise ValueError("act: one of %s; grad_type: float32 or the weights'" % ", ".join(ACTIVATIONS))
        self.w1, self.w2, self.b1, self.b2 = w1, w2, b1, b2
        self.act, self.residual, self.grad_type = ACTIVATIONS[act], residual, grad_type
        self.type, self.dtype = _TYPES[w1.dtype], w1.dtype

    def _rows(self, x, cols):
        if x.dtype != self.dtype or x.dim() != 2 or x.shape[1] != cols or (x.shape[0] and cols > 1 and x.stride(1) != 1):
            raise ValueError("a matrix of %s with %d contiguous columns" % (self.dtype, cols))
        if x.shape[0] > 1 and x.stride(0) < cols:
            raise ValueError("rows that overlap (row stride %d for %d columns): pass .contiguous()" % (x.stride(0), cols))
        return max(x.stride(0) if x.shape[0] > 1 else cols, 1)

    def _offsets(self, offsets):
        if self.experts is None:
            if offsets is not None:
                raise ValueError("offsets: of experts only")
        elif offsets is None or offsets.dtype != torch.int32 or tuple(offsets.shape) != (self.experts + 1,) or not offsets.is_contiguous():
            raise ValueError("offsets: %d int32, the first row of each expert and the end" % (self.experts + 1))
        return offsets

    def _space(self, copies, sums=0):
        """A workspace of so many bytes; copies are of operands whose rows are not on 16 bytes."""
        size = sums + copies
        return torch.empty(size, dtype=torch.uint8, device=self.w1.device) if size else None, size

    def _empty(self, *shape, dtype=None):
        # (rows of no expert stay as they are: zeros, not what was there before)
        make = torch.empty if self.experts is None else torch.zeros
        return make(*shape, dtype=dtype or self.dtype, device=self.w1.device)

    @staticmethod
    def _copied(*matrices):
        return any(m.data_ptr() % 16 or (m.shape[-2] > 1 and m.stride(-2) % 8) or
                   (m.dim() == 3 and m.shape[0] > 1 and m.stride(0) % 8) for m in matrices if m.numel())

    def _layer(self, x, w, b, act, z, r, y, offsets):
        """z = x w + b, y = act(z) + r."""
        M, (K, N) = x.shape[0], w.shape[-2:]
        ws, size = self._space(fg.gemm16_copy_workspace_size(fg.OP_N, fg.OP_N, self.experts or 1, M, N, K)
                               if self._copied(x, w) else 0)
        rest = (b, act, z, N, 1.0 if r is not None else 0.0, r, self._rows(r, N) if r is not None else 0, y, N, ws, size)
        if self.experts is None:
            fg.gemm16(self.type, self.type, fg.OP_N, fg.OP_N, M, N, K, 1.0, x, self._rows(x, K), w, N, *rest)
        else:
            fg.gemm16_grouped(self.type, self.type, fg.OP_N, self.experts, M, N, K, offsets, 1.0, x, self._rows(x, K), w, N,
                              K * N, *rest)
        return y

    def _through(self, g, w, act, z, r, sums, offsets):
        """(g w^T) act'(z) + r, and its column sums.  (r without an activation or sums.)"""
        M, (N, K) = g.shape[0], w.shape[-2:]  # of the result M x N
        y = self._empty(M, N)
        copies = fg.gemm16_copy_workspace_size(fg.OP_N, fg.OP_T, self.experts or 1, M, N, K) if self._copied(g, w) else 0
        ws, size = self._space(copies, fg.gemm16_sums_workspace_size(self.experts or 1, M, N) if sums is not None else 0)
        ldg = self._rows(g, K)
        if r is not None:
            epilogue = (None, fg.ACT_NONE, None, 0, 1.0, r, self._rows(r, N), y, N, ws, size)
        else:
            epilogue = (act, z, N, y, N, sums, ws, size)
        if self.experts is None:
            call = fg.gemm16 if r is not None else fg.gemm16_grad
            call(self.type, self.type, fg.OP_N, fg.OP_T, M, N, K, 1.0, g, ldg, w, K, *epilogue)
        else:
            call = fg.gemm16_grouped if r is not None else fg.gemm16_grouped_grad
            call(self.type, self.type, fg.OP_T, self.experts, M, N, K, offsets, 1.0, g, ldg, w, K, N * K, *epilogue)
        return y

    def _weight_grad(self, x, g, offsets):
        """x^T g, for each expert's rows."""
        M, K, N = x.shape[0], x.shape[1], g.shape[1]
        t = _TYPES[self.grad_type]
        lead = () if self.experts is None else (self.experts,)
        dw = torch.empty(*lead, K, N, dtype=self.grad_type, device=self.w1.device)
        ws, size = self._space(fg.gemm16_copy_workspace_size(fg.OP_T, fg.OP_N, 1, K, N, M) if self._copied(x, g) else 0)
        ldx, ldg = self._rows(x, K), self._rows(g, N)
        if self.experts is None:
            fg.gemm16(self.type, t, fg.OP_T, fg.OP_N, K, N, M, 1.0, x, ldx, g, ldg, None, fg.ACT_NONE, None, 0, 0.0, None, 0,
                      dw, N, ws, size)
        else:
            fg.gemm16_weight_grad(self.type, t, self.experts, M, N, K, offsets, 1.0, x, ldx, g, ldg, 0.0, dw, N, K * N, ws, size)
        return dw

    def forward(self, x, offsets=None):
        """(Y, Saved) for tokens x (M x K)."""
        self._rows(x, self.K)
        offsets = self._offsets(offsets)
        M = x.shape[0]
        z, h = self._empty(M, self.N), self._empty(M, self.N)
        self._layer(x, self.w1, self.b1, self.act, z, None, h, offsets)
        y = self._layer(h, self.w2, self.b2, fg.ACT_NONE, None, x if self.residual else None, self._empty(M, self.K), offsets)
        return y, Saved(x, z, h, offsets, torch.cuda.current_stream(self.w1.device))

    def __call__(self, x, offsets=None):
        """Y for tokens x (M x K); nothing is kept."""
        self._rows(x, self.K)
        offsets = self._offsets(offsets)
        h = self._layer(x, self.w1, self.b1, self.act, None, None, self._empty(x.shape[0], self.N), offsets)
        return self._layer(h, self.w2, self.b2, fg.ACT_NONE, None, x if self.residual else None,
                           self._empty(x.shape[0], self.K), offsets)

    def backward(self, g, saved: Saved):
        """(dX, dW1, dW2, db1, db2) for the gradient g of Y; None for a bias that is not there."""
        ldg = self._rows(g, self.K)
        M, offsets, E = g.shape[0], self._offsets(saved.offsets), self.experts or 1
        if M != saved.x.shape[0]:
            raise ValueError("%d gradients for %d tokens" % (M, saved.x.shape[0]))
        self._rows(saved.x, self.K)
        for t in (saved.z, saved.h):
            if tuple(t.shape) != (M, self.N) or t.dtype != self.dtype or not t.is_contiguous():
                raise ValueError("saved: %s of %s, for %s" % (tuple(t.shape), t.dtype, (M, self.N)))
        lead = () if self.experts is None else (self.experts,)
        dev = self.w1.device
        saved.used_on(torch.cuda.current_stream(dev))
        db1 = torch.empty(*lead, self.N, device=dev) if self.b1 is not None else None
        db2 = None
        if self.b2 is not None:
            db2 = torch.empty(*lead, self.K, device=dev)
            ws, size = self._space(0, fg.gemm16_sums_workspace_size(E, M, self.K))
            fg.act16_grad(self.type, E, M, self.K, offsets, fg.ACT_NONE, g, ldg, None, 0, None, 0, db2, ws, size)
        dw2 = self._weight_grad(saved.h, g, offsets)
        dz = self._through(g, self.w2, self.act, saved.z, None, db1, offsets)
        dw1 = self._weight_grad(saved.x, dz, offsets)
        dx = self._through(dz, self.w1, fg.ACT_NONE, None, g if self.residual else None, None, offsets)
        return dx, dw1, dw2, db1, db2


def main(steps: int = 40, M: int = 512, K: int = 256, N: int = 512, E: int = 8) -> list[float]:
    """Fit a block of experts to another one's outputs; prints and returns the losses."""
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    make = lambda: [(rand(E, K, N) / K**0.5), (rand(E, N, K) / N**0.5), 0.1 * rand(E, N), torch.zeros(E, K, device="cuda")]  # noqa: E731
    target = make()
    teacher = FeedForward(target[0].bfloat16(), target[1].bfloat16(), target[2], target[3])
    params, losses = make(), []
    for step in range(steps):
        rows = torch.bincount(torch.randint(0, E, (M,), generator=g, device="cuda"), minlength=E)
        offsets = torch.cat((torch.zeros(1, device="cuda"), rows.cumsum(0))).int()
        x = rand(M, K).bfloat16()
        block = FeedForward(params[0].bfloat16(), params[1].bfloat16(), params[2], params[3])
        y, saved = block.forward(x, offsets)
        diff = y.float() - teacher(x, offsets).float()
        losses.append(float(diff.square().mean()))
        _, dw1, dw2, db1, db2 = block.backward((diff * (2.0 / M)).bfloat16(), saved)
        for p, d in zip(params, (dw1, dw2, db1, db2)):
            p -= 0.25 * d
        if step % 10 == 0 or step + 1 == steps:
            print("step %d: loss %.4f" % (step, losses[-1]))
    return losses


if __name__ == "__main__":
    main()
