"""4-bit expert products on the GPU where no tolerance can hide a lost chunk, group or scale.

ReLU experts on whole numbers, bit for bit (w4_exact.py), and SwiGLU experts by the relative 2-norm of each row. The
elementwise worst-case bounds of test_gpu_w4.py grow with K beyond what a lost chunk changes; these do not. Which
mistakes they see is tested in test_w4_exact_host.py.
"""
import pytest
import torch

import sparse_mixture_experts_08_b200 as moe
import w4_exact as E
from gpu_helpers import require_gpu
from test_gpu_w4 import _segments, encode, make_experts

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def _whole(gen, n, rows, cols, group, long_scales=False):
    q, s, value = E.matrix(gen, n, rows, cols, group, long_scales)
    return encode(q.cuda()), s.cuda(), value.cuda()


def _run(c, x, lengths, wq, ws=None):
    y = torch.full((len(x), c.d), float("nan"), device="cuda")
    ws = moe.w4_workspace(c) if ws is None else ws
    moe.moe_grouped_ffn_w4(c, x, _segments(lengths), wq, None, None, y, ws)
    assert moe.moe_read_device_status(ws) == moe.OK
    return y


def _check_exact(lengths, d, f, group, long_scales=False):
    gen = torch.Generator().manual_seed(sum(lengths) + d + f + group)
    m = len(lengths)
    n = min(m, 20)  # distinct experts (many small groups share them)
    gate, down = _whole(gen, n, f, d, group, long_scales), _whole(gen, n, d, f, group)
    pick = torch.arange(m) % n
    wq = {"group": group}
    for key, (codes, scales, _) in (("gate", gate), ("down", down)):
        wq[key], wq[key + "_scale"] = (t if m == n else t[pick].contiguous() for t in (codes, scales))
    x = E.inputs(gen, sum(lengths), d).cuda()
    y = _run(moe.make_config(len(x), d, f, m, 1, act=moe.RELU), x, lengths, wq)
    a = 0
    for e, rows in enumerate(lengths):
        if rows:
            want = E.ffn(x[a:a + rows], gate[2][e % n], down[2][e % n])
            assert torch.equal(y[a:a + rows], want), f"expert {e}: {int((y[a:a + rows] != want).sum())} elements differ"
        a += rows


@pytest.mark.parametrize("lengths,d,f,group", E.CASES)
def test_products_of_whole_numbers_are_exact(lengths, d, f, group):
    _check_exact(lengths, d, f, group)


@pytest.mark.parametrize("rows", [3, 24, 50, 100, 400])
def test_scales_that_are_rounded_with_their_codes(rows):
    _check_exact([rows, rows], 2080, 96, 64, long_scales=True)


@pytest.mark.parametrize("rows", [3, 24, 60, 130, 400])
@pytest.mark.parametrize("d,f", E.SWIGLU)
def test_swiglu_rows_by_their_norm(d, f, rows):
    gen = torch.Generator().manual_seed(d + f + rows)
    wq, val = make_experts(gen, 2, d, f, 32, moe.SWIGLU)
    x = torch.randn(2 * rows, d, generator=gen).to(torch.bfloat16).cuda()
    y = _run(moe.make_config(2 * rows, d, f, 2, 1), x, [rows, rows], wq)
    for e in range(2):
        part = slice(e * rows, (e + 1) * rows)
        want = E.ffn_swiglu(x[part], val["gate"][e], val["up"][e], val["down"][e])
        assert E.far(y[part], want) < E.FAR


@pytest.mark.parametrize("T,d,f,m,k,ns,fs,group", [(16, 4096, 1376, 8, 2, 1, 352, 128), (173, 2080, 5408, 12, 3, 0, 0, 32),
                                                   (40, 1056, 4128, 64, 6, 2, 4128, 64), (700, 4160, 416, 4, 2, 2, 2080, 64)])
def test_layers_of_whole_numbers(T, d, f, m, k, ns, fs, group):
    """The whole layer, routed and shared experts: each expert's rows are exact, what remains is their combination."""
    gen = torch.Generator().manual_seed(T + d)
    wq, val = {"group": group}, {}
    for key, n, rows, cols in (("gate", m, f, d), ("down", m, d, f), ("sh_gate", ns, fs, d), ("sh_down", ns, d, fs)):
        if n:
            wq[key], wq[key + "_scale"], val[key] = _whole(gen, n, rows, cols, group)
    x = E.inputs(gen, T, d).cuda()
    c = moe.make_config(T, d, f, m, k, n_shared=ns, f_shared=fs, act=moe.RELU, renormalize=True)
    wr = (torch.randn(m, d, generator=gen) * d ** -0.5).to(torch.bfloat16).cuda()
    ws, out = moe.w4_workspace(c), torch.empty_like(x)
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    moe.moe_layer_forward_w4(c, x, wr, None, wq, out, ws, topk_idx_out=idx, topk_w_out=w)
    assert moe.moe_read_device_status(ws) == moe.OK
    want = torch.zeros(T, d, dtype=E.F64, device="cuda")
    size = torch.zeros_like(want)
    for e in range(m):
        for s in range(k):
            t = torch.nonzero(idx[:, s] == e)[:, 0]
            if len(t):
                y = w[t, s].to(E.F64)[:, None] * E.ffn(x[t], val["gate"][e], val["down"][e]).to(E.F64)
                want[t] += y
                size[t] += y.abs()
    for e in range(ns):
        y = E.ffn(x, val["sh_gate"][e], val["sh_down"][e]).to(E.F64)
        want += y
        size += y.abs()
    # each of the k + ns rows is exact; then a product (2^-24 of it), k + ns additions (2^-24 of their sizes each) and
    # one rounding to bf16 (2^-8)
    assert ((out.to(E.F64) - want).abs() <= 2.0 ** -8 * want.abs() + (1 + k + ns) * 2.0 ** -24 * (1 + 2.0 ** -7) * size).all()
