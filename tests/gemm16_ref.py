"""The 16-bit layers in 64 bits on the CPU, with how far FP32 evaluation may be off.

Tolerances (u = 2^-23, one unit in the last place at most).  A product of two 16-bit values is
exact in FP32.  A sum of K of them (and the accumulator) rounds or cuts each addend and each sum
at most by u of the largest partial sum, which is at most mag = sum |a||b|: K + 2 of these with the
scaling by alpha.  Then
    Z is off by dz = |alpha| (K + 2) u mag + u (|alpha P| + |bias|),
    act(Z) by 1.13 dz (no activation here is steeper) and its own evaluation.  GELU, max(0, z) - a q: q is off by
        (6 + 1.2 z^2) u of itself (5e-7 the polynomial and t, 2 units the exponential, z^2 of its
        argument): (6 + 1.2 z^2) u a q + u |y|.  SiLU: the exponential 2 + 1.16 |z| units, sum and division
        4: (8 + 1.2 |z|) u |y|.  FP32's underflow (1e-30) for both.
    beta R by u (|beta R| + |y|) more.
    act'(Z) of a given Z:  GELU, Phi + z phi: Phi is 1/2 + z P, a sum that rounds by u/2, P with coefficients that
        add up to 0.4 off by u/2 of them a step and |z| times that, less than u in all (|z| P < 1/2): 1.5 u, and
        of z phi (at most 0.25) (4 + 1.2 z^2) units of it: 1.5 u + (4 + 1.2 z^2) u |z| phi;
        SiLU  s (1 + z (1 - s)): s off by (8 + 1.2 |z|) u, 1 - s by as much of s and a unit of 1:
        (12 + 3 |z|) u s (1 + |z|);  ReLU none.
Rounding to nearest is monotone, so an output lies between value - tol and value + tol, both
rounded to its type.
"""

import math

import torch

U = 2.0**-23
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ACTS = ("none", "relu", "gelu", "silu")


def phi(z):
    return torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)


def cdf(z):
    return 0.5 * torch.erfc(-z / math.sqrt(2))


def act(z, name):
    """(act(z), how far its evaluation may be off) in float64; limits at infinities."""
    if name == "relu":
        return torch.where(z > 0, z, torch.where(z.isnan(), z, 0 * z.nan_to_num(0, 0, 0))), torch.zeros_like(z)
    if name == "gelu":
        y = z.clamp(min=-50) * cdf(z)
        q = cdf(-z.abs())
        w = z.clamp(-30, 30)
        return y, (6 + 1.2 * w * w) * U * w.abs() * q + U * y.abs() + 1e-30
    if name == "silu":
        y = z.clamp(min=-800) * torch.sigmoid(z)
        return y, (8 + 1.2 * z.abs()).clamp(max=200) * U * y.abs() + 1e-30
    return z, torch.zeros_like(z)


def slope(z, name):
    """(act'(z), how far its evaluation may be off)."""
    a = z.abs().clamp(max=800)
    if name == "relu":
        return (z > 0).double(), torch.zeros_like(z)
    if name == "gelu":
        c, p = cdf(z), phi(z)
        w = z.clamp(-50, 50)
        return c + w * p, 1.5 * U + (4 + 1.2 * w * w) * U * w.abs() * p
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z.clamp(-800, 800) * torch.sigmoid(-z)), (12 + 3 * a) * U * s * (1 + a) + 1e-30
    return torch.ones_like(z), torch.zeros_like(z)


def layer(A, B, alpha=1.0, bias=None, name="none", beta=0.0, R=None):
    """A (M x K) and B (K x N) in float64 -> ((Y, tol), (Z, tol))."""
    K = A.shape[1]
    P, mag = A @ B, A.abs() @ B.abs()
    z, dz = alpha * P, abs(alpha) * (K + 2) * U * mag
    if bias is not None:
        dz = dz + U * (z.abs() + bias.abs())
        z = z + bias
    y, dy = act(z, name)
    dy = dy + 1.13 * dz
    if beta:
        dy = dy + U * ((beta * R).abs() + y.abs() + dy)
        y = y + beta * R
    return (y, dy), (z, dz)


def layer_grad(A, B, alpha=1.0, name="none", Z=None):
    """((Y, tol), (column sums, tol)) of the product through act'(Z)."""
    K = A.shape[1]
    P, mag = alpha * (A @ B), abs(alpha) * (A.abs() @ B.abs())
    if name == "none":
        y, dy = P, (K + 2) * U * mag
    else:
        s, ds = slope(Z, name)
        dp = (K + 2) * U * mag
        y, dy = P * s, dp * s.abs() + P.abs() * ds + dp * ds + U * (P * s).abs()
        if name == "relu":  # a closed gate hides anything
            y, dy = torch.where(Z > 0, P, torch.zeros_like(P)), torch.where(Z > 0, dp, torch.zeros_like(P))
    # (M additions in FP32 in some order, each off by a unit of at most the sum of magnitudes)
    sums, dsums = y.sum(0), dy.sum(0) + (y.shape[0] + 1) * U * (y.abs() + dy).sum(0)
    return (y, dy), (sums, dsums)


def outside(got, want, tol, dtype):
    """Which elements are not between want - tol and want + tol, rounded to the type (NaN for NaN)."""
    to = lambda x: x.to(dtype).double()  # noqa: E731
    got = got.double()
    inside = (got >= to(want - tol)) & (got <= to(want + tol))
    return ~(inside | (got.isnan() & want.isnan()) | (got == to(want)))


class Buffer:
    """A matrix inside a buffer: `pad` elements between rows, `offset` before the first one, all of them NaN
    (inputs: they must not count) or a sentinel (outputs: they must stay)."""

    SENTINEL = -77.0

    def __init__(self, values, pad=0, offset=0, fill=float("nan")):
        rows, cols = values.shape
        self.ld, self.shape, self.offset, self.fill = max(1, cols + pad), (rows, cols), offset, fill
        flat = torch.full((rows * self.ld + offset + 16,), fill, dtype=values.dtype)
        self.inside = torch.zeros_like(flat, dtype=torch.bool)
        flat[offset:offset + rows * self.ld].view(rows, self.ld)[:, :cols] = values
        self.inside[offset:offset + rows * self.ld].view(rows, self.ld)[:, :cols] = True
        self.data = flat.cuda()

    @property
    def ptr(self):
        return self.data.data_ptr() + self.offset * self.data.element_size()

    def result(self):
        got = self.data.cpu()
        rest = got[~self.inside]
        assert (rest == self.fill).all() if self.fill == self.fill else rest.isnan().all(), "written outside the matrix"
        rows, cols = self.shape
        return got[self.offset:self.offset + rows * self.ld].view(rows, self.ld)[:, :cols]


def output(rows, cols, dtype, pad=0, offset=0):
    return Buffer(torch.full((rows, cols), Buffer.SENTINEL, dtype=dtype), pad, offset, Buffer.SENTINEL)
