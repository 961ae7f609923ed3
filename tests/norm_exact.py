"""Rows for the residual + RMS norm of which no 16-byte vector can be left out unseen.

Every element lies between 0.5 and 1.5 in size, so a vector of V elements holds at least V / 4 of a row's sum of squares,
which is at most 2.25 d; without it the root mean square changes by V / (18 d) or more. The fp32 sum itself is off by at
most one rounding (2^-24) for each addition on the way from an element to the row's sum: up to 32 in a thread, 5 across a
warp, 31 across the warps. With the sum x + residual (once in r, twice in its square), the mean, eps, root, division and
two products: half of 68 + 2 + 2, then 1 + 1 + 1 + 2 roundings, 41 in all.
"""
import torch

F64 = torch.float64
REL = 41 * 2.0 ** -24 * (1 + 2.0 ** -10)  # of |y| in fp32
SHAPES = [(3, 64), (2, 2056), (5, 4096), (3, 8200), (2, 16384), (2, 32768)]


def inputs(gen, rows, d, dtype):
    """x, a residual of a quarter of it and the other sign, and a weight."""
    size = 0.5 + torch.rand(rows, d, generator=gen)
    sign = torch.randint(0, 2, (rows, d), generator=gen) * 2.0 - 1
    x = (size * sign).to(dtype)
    return x, (x.float() / -4).to(dtype), (0.75 + torch.rand(d, generator=gen) / 2).to(dtype)


def norm64(x, residual, weight, without=None):
    """In 64 bits; without: (first, end) columns that the sum of squares leaves out (a mistake for tests)."""
    r = x.to(F64) + (residual.to(F64) if residual is not None else 0)
    sq = r * r
    if without:
        sq[:, without[0]:without[1]] = 0
    return r / torch.sqrt(sq.mean(1, keepdim=True) + 1e-5) * weight.to(F64)
