"""4-bit expert products whose every sum is exact, for comparisons bit for bit.

Inputs are -1, 0 and 1, codes whole numbers and scales 1, 2 or 4, so both products are sums of whole numbers: exact in
fp32, in any order, while the terms' absolute values add up to less than 2^24 (asserted for the data at hand). The
hidden activation is ReLU's, rounded once to bf16, which the reference does too. A dropped or repeated chunk, group or
scale changes whole numbers and cannot hide in a tolerance.
"""
import torch

F64 = torch.float64


def inputs(gen, rows, d):
    """Rows of -1, 0 and 1 in bf16: one to four of every 32 columns are not 0."""
    x = torch.zeros(rows, d // 32, 32)
    for i in range(4):
        keep = 1.0 if i == 0 else 0.5
        at = torch.randint(0, 32, (rows, d // 32, 1), generator=gen)
        sign = torch.randint(0, 2, (rows, d // 32, 1), generator=gen) * 2.0 - 1
        x.scatter_(2, at, torch.where(torch.rand(sign.shape, generator=gen) < keep, sign, torch.zeros(())))
    return x.view(rows, d).to(torch.bfloat16)


def matrix(gen, n, rows, cols, group, long_scales=False):
    """Codes as whole numbers [n, rows, cols], scales [n, groups, rows] in bf16, values in 64 bits. long_scales: whole
    numbers of 7 bits, whose products with a code are rounded to bf16 once (whole numbers again)."""
    q = torch.randint(-8, 8, (n, rows, cols), generator=gen, dtype=torch.int32)
    shape = (n, -(-cols // group), rows)
    s = torch.randint(32, 64, shape, generator=gen) * 2.0 + 1 if long_scales else 2.0 ** torch.randint(0, 3, shape,
                                                                                                  generator=gen)
    value = q.to(F64) * s.to(F64).transpose(1, 2).repeat_interleave(group, 2)[:, :, :cols]
    return q, s.to(torch.bfloat16), value.to(torch.bfloat16).to(F64)


def ffn(x, gate, down):
    """Rows of x through one ReLU expert (values in 64 bits): what the kernels must give bit for bit."""
    g = x.to(F64) @ gate.t()
    assert (x.to(F64).abs() @ gate.abs().t()).max() < 2 ** 24
    h = g.clamp_min(0).to(torch.bfloat16).to(F64)
    assert (h @ down.abs().t()).max() < 2 ** 24
    return (h @ down.t()).float()


# lengths of the segments, d, f, group: long and odd K in either product, in every tile height, cut and whole tiles
CASES = [
    ([3], 4096, 6176, 128),
    ([1, 1], 14336, 64, 64),
    ([3, 0, 9], 96, 14336, 32),
    ([24, 20, 30], 4096, 1120, 32),
    ([16, 31], 288, 14336, 128),
    ([50, 49, 64, 0, 20], 4160, 1376, 32),
    ([60, 40], 160, 14336, 64),
    ([81, 64, 150, 0, 101], 4128, 544, 64),
    ([129, 128, 127, 100], 352, 8224, 128),
    ([400, 385, 193], 2080, 1312, 32),
    ([450, 0, 224, 225, 700], 4096, 160, 128),
    ([230, 449], 96, 8224, 32),
    ([500], 4160, 4096, 64),
    # more than a hundred pieces of work a block or pair
    ([4096], 64, 32768, 32),
    ([1] * 300, 32, 4096, 32),
]

# Relative 2-norm of a row's difference that SwiGLU products may show against a reference that rounds h to bf16 itself.
# What differs is the fp32 sums: were every step of a sum of 16 columns truncated (2^-23 of it, 2048 steps at most at
# these sizes, half of that on average as the sum grows), g and u would be off by 2^-13 of themselves. h is then rounded the other
# way where it lies within that of the middle of two bf16 numbers: at most 2 2^-13 2^8 = 2^-4 of its elements, each off by
# a step of at most 2^-7: together 2^-7 2^-2 = 2^-9 of the norm. Twice that; a lost group of 32 columns of 14336 is
# (32 / 14336)^1/2 = 0.047 of g.
FAR = 2.0 ** -8
SWIGLU = [(4096, 6176), (14336, 96), (352, 8224), (2080, 1376)]  # d, f


def ffn_swiglu(x, gate, up, down):
    g = x.to(F64) @ gate.t()
    h = (g * torch.sigmoid(g) * (x.to(F64) @ up.t())).to(torch.bfloat16).to(F64)
    return h @ down.t()


def far(got, want):
    """The largest relative 2-norm of a row's difference."""
    return ((got.to(F64) - want).norm(dim=1) / want.norm(dim=1)).max().item()
