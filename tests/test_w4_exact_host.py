"""The exact comparisons of the 4-bit products see a lost group of 32 columns, in either matrix, at every length of K
that the GPU tests use; and so do the relative norms of the SwiGLU cases. The mistakes are made in the reference."""
import pytest
import torch

import w4_exact as E


@pytest.mark.parametrize("case", sorted({(c[1], c[2], c[3]) for c in E.CASES}))
def test_a_lost_group_changes_the_exact_results(case):
    d, f, group = case
    gen = torch.Generator().manual_seed(d + f)
    d_few, f_few = min(d, 1024), min(f, 1024)  # the other matrix's side that K does not depend on
    x = E.inputs(gen, 5, d)
    gate, down = E.matrix(gen, 1, f_few, d, group)[2][0], E.matrix(gen, 1, d_few, f_few, group)[2][0]
    want = E.ffn(x, gate, down)
    for at in (0, d // 64 * 32, d - 32):  # the first, a middle and the last 32 columns of the first product
        lost = gate.clone()
        lost[:, at:at + 32] = 0
        assert not torch.equal(E.ffn(x, lost, down), want)
        scale = gate.clone()
        scale[:, at:at + 32] *= 2  # another group's scale
        assert not torch.equal(E.ffn(x, scale, down), want)
    x = E.inputs(gen, 5, 32)
    gate, down = E.matrix(gen, 1, f, 32, 32)[2][0], E.matrix(gen, 1, 64, f, group)[2][0]
    want = E.ffn(x, gate, down)
    for at in (0, f // 64 * 32, f - 32):  # and of the second
        lost = down.clone()
        lost[:, at:at + 32] = 0
        got = E.ffn(x, gate, lost)
        assert not torch.equal(got, want) and (got != want).float().mean() > 0.5


@pytest.mark.parametrize("d,f", E.SWIGLU)
def test_a_lost_group_is_far_outside_the_norms_of_swiglu(d, f):
    gen = torch.Generator().manual_seed(d * 3 + f)
    x = torch.randn(4, d, generator=gen).to(torch.bfloat16).to(E.F64)
    f_few = min(f, 512)
    gate, up, down = (torch.randn(*s, generator=gen).to(torch.bfloat16).to(E.F64) * s[1] ** -0.5
                      for s in ((f_few, d), (f_few, d), (64, f_few)))
    want = E.ffn_swiglu(x, gate, up, down)
    assert E.far(want, want) == 0
    for at in (0, d - 32):
        lost = gate.clone()
        lost[:, at:at + 32] = 0
        assert E.far(E.ffn_swiglu(x, lost, up, down), want) > 3 * E.FAR
        lost = up.clone()
        lost[:, at:at + 32] = 0
        assert E.far(E.ffn_swiglu(x, gate, lost, down), want) > 3 * E.FAR
    gate, up, down = (torch.randn(*s, generator=gen).to(torch.bfloat16).to(E.F64) * s[1] ** -0.5
                      for s in ((f, 64), (f, 64), (64, f)))
    x = x[:, :64]
    want = E.ffn_swiglu(x, gate, up, down)
    lost = down.clone()
    lost[:, f - 32:] = 0
    assert E.far(E.ffn_swiglu(x, gate, up, lost), want) > 3 * E.FAR
