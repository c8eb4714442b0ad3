"""Plain 64-bit implementations of the 8-bit linear-layer operators, the
matrices their tests use, and the error bounds the tests allow.

Matrices are torch tensors of n rows (tokens or channels) of m elements, a row
stride `ld` apart and starting `offset` elements into their allocation, with a
sentinel everywhere outside the rows: the library's column-major storage with
one token a column.
"""
from __future__ import annotations

import torch

DTYPES = {"s": torch.float32, "h": torch.float16, "b": torch.bfloat16}
# unit roundoff of the result's type and of the arithmetic
UNIT = {"s": 2.0 ** -24, "h": 2.0 ** -11, "b": 2.0 ** -8}
U32 = 2.0 ** -24
SENTINEL = 77


class Matrix:
    """n rows of m elements on the device, the rest of the allocation a sentinel."""

    def __init__(self, n, m, dtype, ld=None, offset=0, values=None, device="cuda"):
        self.n, self.m, self.ld, self.offset = n, m, m if ld is None else ld, offset
        size = offset + (n - 1) * self.ld + m + 5
        self.flat = torch.full((size,), SENTINEL, dtype=dtype, device=device)
        self.rows = self.flat.as_strided((n, m), (self.ld, 1), offset)
        if values is not None:
            self.rows.copy_(values)

    @property
    def ptr(self):
        return self.flat.data_ptr() + self.offset * self.flat.element_size()

    def outside_untouched(self):
        f = self.flat.clone()
        f.as_strided((self.n, self.m), (self.ld, 1), self.offset).fill_(SENTINEL)
        return bool((f == SENTINEL).all())


def sum_depth(m):
    """Roundings on the way of one addend of a sum of m through the row kernels: a
    thread adds at most m / 128 of them (and 64 more), then the partial sums
    of lanes and warps are added."""
    return m / 128 + 64 + 40


def quantised(y):
    """(values in units of the scale, unrounded, and the scales) of rows of float64"""
    top = y.abs().amax(1)
    s = top / 127.0
    return torch.where(s[:, None] > 0, y / s[:, None], torch.zeros_like(y)), s


def rmsnorm(h, g, eps):
    rstd = 1.0 / torch.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * g, rstd


def rmsgrad(dy, h, g, rstd, dr):
    """(dX, dG, and the sums of magnitudes that their rounding errors go by)"""
    u = h * rstd[:, None]
    a = dy * g
    c = (a * u).mean(1, keepdim=True)
    dx = dr + rstd[:, None] * (a - u * c)
    dx_size = dr.abs() + rstd[:, None] * (a.abs() + u.abs() * (a * u).abs().mean(1, keepdim=True))
    return dx, (dy * u).sum(0), dx_size, (dy * u).abs().sum(0)


def gemmq(w, x, alpha, sw, sx, beta, y):
    """(Y, the magnitude its float rounding errors go by) from integer matrices
    w (m, k) and x (n, k); sums in float64 are exact (k < 2^39)."""
    acc = x.double() @ w.double().T
    scale = alpha * sx.double()[:, None] * sw.double()[None, :]
    out = acc * scale
    most = (x.double().abs() @ w.double().abs().T)
    # integer sums are exact below 2^24; beyond, each of the k/16 accumulations of
    # 16 products may lose 2^-23 of the running sum
    k = w.shape[1]
    lost = torch.where(most < 2.0 ** 24, torch.zeros_like(most), most * (k / 16 + 1) * 2.0 ** -23)
    size = out.abs() * 6 * U32 + lost * scale.abs()
    if beta != 0.0:
        out = out + beta * y.double()
        size = size + 2 * U32 * (beta * y.double()).abs()
    return out, size
