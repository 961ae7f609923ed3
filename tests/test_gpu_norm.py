"""Residual + RMS norm with 8-bit output on the GPU against the formulas in 64 bits.

Bounds (relative, per element): the sum is one fp32 addition and one rounding to the
output type, so it is compared bit-exactly. y: fp32 squares and their sum over d terms
(any order: at most d 2^-24, half of it after the root), the sum x + residual (2^-24 each,
in r and, twice, in the mean), root, division and two products (4 x 2^-24), then half a
step of the output type. Codes: half a step of E4M3 (2^-4 of the value, or half the
smallest step) on top of the fp32 part.
"""
import pytest
import torch

import norm_exact as N
import sparse_mixture_experts_08_b200 as moe
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

F64 = torch.float64


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


def _inputs(rows, d, dtype, residual, seed=0):
    gen = torch.Generator().manual_seed(rows * 31 + d + seed)
    x = (torch.randn(rows, d, generator=gen) * torch.exp2(torch.randint(-8, 8, (rows, 1), generator=gen).float()))
    r = torch.randn(rows, d, generator=gen) * 3 if residual else None
    w = 1 + 0.3 * torch.randn(d, generator=gen)
    return x.to(dtype).cuda(), None if r is None else r.to(dtype).cuda(), w.to(dtype).cuda()


def norm64(x, residual, w, eps):
    r = x.to(F64) + (residual.to(F64) if residual is not None else 0)
    return r / torch.sqrt((r * r).mean(1, keepdim=True) + eps) * w.to(F64)


def fp32_part(d):
    return (0.5 * d + 8) * 2.0 ** -24


def check_codes(codes, scales, ref, d):
    rel = fp32_part(d) + 2.0 ** -22
    top = ref.abs().amax(1)
    want = torch.where(top > 0, top / 448, torch.ones_like(top))
    assert ((scales.to(F64) - want).abs() <= rel * want).all()
    val = codes.view(torch.float8_e4m3fn).to(F64) * scales.to(F64)[:, None]
    half = torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -10 * want[:, None])
    assert ((val - ref).abs() <= half * (1 + 2.0 ** -10) + rel * ref.abs()).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d", [(1, 8), (1, 4096), (3, 16), (5, 248), (16, 4096), (7, 264), (129, 512), (2, 520),
                                    (33, 1032), (4, 2048), (9, 2056), (5, 4104), (3, 8192), (2, 8200), (2, 16384),
                                    (3, 16392), (2, 32768), (1025, 64)])
def test_norm(rows, d, dtype):
    for residual in (False, True):
        x, r, w = _inputs(rows, d, dtype, residual)
        y = torch.full_like(x, float("nan"))
        total = torch.full_like(x, float("nan")) if residual else None
        with_codes = d % 16 == 0
        codes = torch.empty(rows, d, dtype=torch.uint8, device="cuda") if with_codes else None
        scales = torch.empty(rows, device="cuda") if with_codes else None
        moe.moe_add_rmsnorm(x, r, w, 1e-5, y, sum_out=total, codes=codes, scales=scales)
        ref = norm64(x, r, w, 1e-5)
        if residual:
            assert torch.equal(total, (x.float() + r.float()).to(dtype))
        half = torch.finfo(dtype).eps / 2
        assert ((y.to(F64) - ref).abs() <= (half + fp32_part(d)) * ref.abs() + 1e-38).all()
        if with_codes:
            check_codes(codes, scales, ref, d)
            only, osc = torch.empty_like(codes), torch.empty_like(scales)
            moe.moe_add_rmsnorm(x, r, w, 1e-5, None, codes=only, scales=osc)
            assert torch.equal(only, codes) and torch.equal(osc, scales)


def test_rows_of_zeros_and_extremes():
    d = 256
    x = torch.zeros(6, d, dtype=torch.bfloat16)
    x[1] = 1e-20
    x[2, 3] = 1e18
    x[3] = float("inf")
    x[4, 9] = float("nan")
    x = x.cuda()
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    y, codes, scales = torch.empty_like(x), torch.empty(6, d, dtype=torch.uint8, device="cuda"), torch.empty(6, device="cuda")
    moe.moe_add_rmsnorm(x, None, w, 1e-6, y, codes=codes, scales=scales)
    assert (y[0] == 0).all() and (y[5] == 0).all() and scales[0] == 1 and (codes[0] == 0).all()
    ref = norm64(x[1:3], None, w, 1e-6)
    assert ((y[1:3].to(F64) - ref).abs() <= (2.0 ** -8 + fp32_part(d)) * ref.abs() + 1e-38).all()
    assert torch.isnan(y[3]).all() and torch.isnan(y[4]).all()
    assert torch.isfinite(y[[0, 1, 2, 5]].float()).all()


@pytest.mark.parametrize("target", ["x", "residual"])
def test_in_place(target):
    x, r, w = _inputs(37, 1040, torch.bfloat16, True)
    y, total = torch.empty_like(x), torch.empty_like(x)
    moe.moe_add_rmsnorm(x, r, w, 1e-5, y, sum_out=total)
    a, b = x.clone(), r.clone()
    if target == "x":      # the sum over the residual, y over x
        moe.moe_add_rmsnorm(a, b, w, 1e-5, a, sum_out=b)
        assert torch.equal(a, y) and torch.equal(b, total)
    else:                  # the sum over x, y over the residual
        moe.moe_add_rmsnorm(a, b, w, 1e-5, b, sum_out=a)
        assert torch.equal(b, y) and torch.equal(a, total)


def test_rows_past_32_bit_offsets():
    rows, d = (1 << 31) // 4096 + 5, 4096
    x = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator().manual_seed(1)
    tail = torch.randn(7, d, generator=gen).to(torch.bfloat16).cuda()
    x[-7:] = tail
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    moe.moe_add_rmsnorm(x, None, w, 1e-5, y)
    want = torch.empty_like(tail)
    moe.moe_add_rmsnorm(tail, None, w, 1e-5, want)
    assert torch.equal(y[-7:], want) and (y[:3] == 0).all()


def test_captured_and_replayed():
    x, r, w = _inputs(16, 4096, torch.bfloat16, True)
    y, total = torch.empty_like(x), torch.empty_like(x)
    codes, scales = torch.empty(16, 4096, dtype=torch.uint8, device="cuda"), torch.empty(16, device="cuda")
    moe.moe_add_rmsnorm(x, r, w, 1e-5, y, sum_out=total, codes=codes, scales=scales)
    want = [t.clone() for t in (y, total, codes, scales)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_add_rmsnorm(x, r, w, 1e-5, y, sum_out=total, codes=codes, scales=scales)
    for t in (y, total, codes, scales):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((y, total, codes, scales), want))


# ------------------------------------------------------------------ into the layers

def _bf16(gen, *s):
    return (torch.randn(*s, generator=gen) * s[-1] ** -0.5).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("T,d,f,m,k,ns,fs,act", [(16, 256, 320, 8, 2, 0, 0, moe.SWIGLU), (3, 128, 64, 4, 4, 1, 96, moe.RELU),
                                                 (300, 256, 192, 6, 2, 2, 160, moe.SWIGLU),
                                                 (8200, 64, 64, 8, 1, 0, 0, moe.SWIGLU)])
def test_fp8_layer_on_given_codes(T, d, f, m, k, ns, fs, act):
    """With the codes that the 8-bit layer would make itself, the outputs are the same bits."""
    gen = torch.Generator().manual_seed(T + d)
    up = act == moe.SWIGLU
    w = [_bf16(gen, m, f, d), _bf16(gen, m, f, d) if up else None, _bf16(gen, m, d, f)]
    sh = [_bf16(gen, ns, fs, d), _bf16(gen, ns, fs, d) if up else None, _bf16(gen, ns, d, fs)] if ns else [None] * 3
    wq = moe.quantize_experts(*w, *sh)
    c = moe.make_config(T, d, f, m, k, n_shared=ns, f_shared=fs, act=act)
    x, wr = _bf16(gen, T, d) * 16, _bf16(gen, m, d)
    codes, scales = torch.empty(T, d, dtype=torch.uint8, device="cuda"), torch.empty(T, device="cuda")
    moe.moe_quantize_e4m3(x, codes, scales)
    a, b, ws = torch.empty_like(x), torch.empty_like(x), moe.fp8_workspace(c)
    moe.moe_layer_forward_fp8(c, x, wr, None, wq, a, ws)
    moe.moe_layer_forward_fp8_codes(c, x, codes, scales, wr, None, wq, b, ws)
    assert moe.moe_read_device_status(ws) == moe.OK
    assert torch.equal(a, b)


def test_block_norm_then_8_bit_and_4_bit_layers():
    """The block as a server runs it: sum and norm, then the layer, then the next block's sum and norm."""
    gen = torch.Generator().manual_seed(77)
    T, d, f, m, k = 24, 512, 640, 8, 2
    w = [_bf16(gen, m, f, d), _bf16(gen, m, f, d), _bf16(gen, m, d, f)]
    wr, weight = _bf16(gen, m, d), (1 + 0.1 * torch.randn(d, generator=gen)).to(torch.bfloat16).cuda()
    x, res = (torch.randn(T, d, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    c = moe.make_config(T, d, f, m, k, renormalize=True)
    y, codes, scales = torch.empty_like(x), torch.empty(T, d, dtype=torch.uint8, device="cuda"), torch.empty(T, device="cuda")
    stream = res.clone()
    moe.moe_add_rmsnorm(x, stream, weight, 1e-5, y, sum_out=stream, codes=codes, scales=scales)
    out = {}
    ref = torch.empty_like(x)
    moe.moe_layer_forward(c, y, wr, None, *w, None, None, None, ref, moe.workspace(c))
    q8, q4 = moe.quantize_experts(*w), moe.quantize_experts_w4(*w, group=32)
    for name in ("fp8", "w4"):
        out[name] = torch.empty_like(x)
    moe.moe_layer_forward_fp8_codes(c, y, codes, scales, wr, None, q8, out["fp8"], moe.fp8_workspace(c))
    moe.moe_layer_forward_w4(c, y, wr, None, q4, out["w4"], moe.w4_workspace(c))
    # the weights' own steps dominate: E4M3 rounds x, W and h by at most 2^-4 each, three
    # factors in each of two products; a 4-bit code is off by at most half a step of max/7
    # a group, 1/14 of the group's largest weight, which for 32 normal weights is below
    # 4 of their standard deviations: 0.29 of a typical weight at most, in three matrices.
    # As 2-norms over independent roundings (uniform: 1/sqrt(3) of the half step, and the
    # largest of 32 normals at 2.1 standard deviations): fp8 < sqrt(6) 2^-4 / sqrt(3),
    # w4 < sqrt(3) (2.1 / 14) / sqrt(3) with half as much again for the silu's slope.
    far = lambda a: ((a.float() - ref.float()).norm() / ref.float().norm()).item()  # noqa: E731
    assert far(out["fp8"]) < 0.09 and far(out["w4"]) < 0.23
    # the next block
    nxt = torch.empty_like(x)
    moe.moe_add_rmsnorm(out["w4"], stream, weight, 1e-5, nxt, sum_out=stream)
    s = (x.float() + res.float()).to(torch.bfloat16)
    assert torch.equal(stream, (out["w4"].float() + s.float()).to(torch.bfloat16))


def test_codes_of_tiny_rows():
    """Rows whose scale has no fp32 reciprocal: weights near the smallest normal number, and below it."""
    d = 512
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(5, d, generator=gen).cuda()
    for size in (1e-30, 1e-36, 3e-38, 1e-39):
        w = torch.full((d,), size, device="cuda")
        y, codes, scales = torch.empty_like(x), torch.empty(5, d, dtype=torch.uint8, device="cuda"), torch.empty(5, device="cuda")
        moe.moe_add_rmsnorm(x, None, w, 1e-6, y, codes=codes, scales=scales)
        ref = norm64(x, None, w, 1e-6)
        # below 2^-126 a number is off by up to 2^-150: y by one such rounding, and so the
        # scale, which then is off by that much of its own size
        step = 2.0 ** -150
        assert ((y.to(F64) - ref).abs() <= (2.0 ** -24 + fp32_part(d)) * ref.abs() + 2 * step).all()
        want = ref.abs().amax(1) / 448
        rel = fp32_part(d) + 2.0 ** -22
        assert ((scales.to(F64) - want).abs() <= rel * want + 2 * step).all()
        val = codes.view(torch.float8_e4m3fn).to(F64) * scales.to(F64)[:, None]
        off = 2 * step / want[:, None]  # the scale's own relative error
        half = torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -10 * want[:, None]) * (1 + 2.0 ** -10)
        assert ((val - ref).abs() <= half + (rel + 2 * off) * ref.abs() + 2 * step).all()


def test_codes_of_rows_too_small_for_a_scale():
    """amax / 448 rounds to zero in fp32: scale 1 and codes of zero (of either sign), no NaN code."""
    d = 512
    gen = torch.Generator().manual_seed(5)
    x = torch.randn(5, d, generator=gen).cuda()
    x[:, :9] = 0
    w = torch.full((d,), 1e-44, device="cuda")
    codes, scales = torch.empty(5, d, dtype=torch.uint8, device="cuda"), torch.empty(5, device="cuda")
    moe.moe_add_rmsnorm(x, None, w, 1e-6, None, codes=codes, scales=scales)
    assert (scales == 1).all() and (codes & 0x7F == 0).all()


def test_no_rows():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    moe.moe_add_rmsnorm(x, None, w, 1e-6, torch.empty_like(x))


def test_binding_refuses_strided_and_host_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    wide = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    for a in ((wide[:, ::2], None, w, x), (x, wide[:, :64], w, x), (x, None, w.cpu(), x), (x.cpu(), None, w, x)):
        with pytest.raises(moe.MoEError):
            moe.moe_add_rmsnorm(a[0], a[1], a[2], 1e-6, a[3])


def test_binding_refuses_other_types_and_sizes():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    codes, scales = torch.empty(4, 64, dtype=torch.uint8, device="cuda"), torch.empty(4, device="cuda")
    for bad in (dict(weight=w.float()), dict(weight=w[:56]), dict(residual=x[:3]), dict(y=x.float()), dict(y=x[:2]),
                dict(sum_out=x[:1]), dict(codes=codes[:3]), dict(codes=x), dict(scales=scales[:3]),
                dict(scales=scales.half())):
        a = dict(dict(residual=None, weight=w, y=torch.empty_like(x), sum_out=None, codes=codes, scales=scales), **bad)
        with pytest.raises(moe.MoEError):
            moe.moe_add_rmsnorm(x, a["residual"], a["weight"], 1e-6, a["y"], sum_out=a["sum_out"], codes=a["codes"],
                                scales=a["scales"])


def _e4m3_ties():
    """The numbers halfway between two neighbouring E4M3 numbers."""
    v = torch.arange(0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    return (v[1:] + v[:-1]) / 2


@pytest.mark.parametrize("size", [1.0, 1e4, 3e-5, 1e30, 1e-35])
def test_codes_are_those_of_the_rounded_quotient(size):
    """Rows of one and minus one have a root mean square of exactly 1, so y is the weight, bit for bit: values around
    every tie between two codes, whose quotients by the scale decide which of them it is."""
    gen = torch.Generator().manual_seed(8)
    ties = _e4m3_ties()
    steps = torch.arange(-2, 3)
    d = len(ties) * len(steps) + 10
    assert d % 16 == 0
    sign = torch.where(torch.rand(2, d, generator=gen) < 0.5, -1.0, 1.0).cuda()
    for _ in range(200):
        top = (1 + torch.rand(1, generator=gen)) * size
        scale = top / 448
        v = (ties * scale.double()).float()
        w = (v[:, None].view(torch.int32) + steps).to(torch.int32).view(torch.float32).reshape(-1)
        w = torch.cat([w, top.expand(10)]).minimum(top).cuda()
        y, codes, scales = torch.empty_like(sign), torch.empty(2, d, dtype=torch.uint8, device="cuda"), torch.empty(2, device="cuda")
        moe.moe_add_rmsnorm(sign, None, w, 0.0, y, codes=codes, scales=scales)
        assert torch.equal(y, sign * w) and (scales.cpu() == scale).all()
        want = (y.cpu() / scale).to(torch.float8_e4m3fn)
        assert torch.equal(codes.cpu(), want.view(torch.uint8))


@pytest.mark.parametrize("d", [256, 512, 4096, 16384])
def test_codes_of_bf16_rows_are_the_quantizers(d):
    """The same bf16 rows through the norm and through moe_quantize_e4m3: one format."""
    gen = torch.Generator().manual_seed(d)
    x = torch.where(torch.rand(3, d, generator=gen) < 0.5, -1.0, 1.0).to(torch.bfloat16).cuda()
    codes, want = (torch.empty(3, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    scales, want_scales = (torch.empty(3, device="cuda") for _ in range(2))
    y = torch.empty_like(x)
    for i in range(50):
        w = (torch.randn(d, generator=gen) * 2.0 ** torch.randint(-60, 60, (1,), generator=gen)).to(torch.bfloat16).cuda()
        w[7] = (-0.0, 1.0, float("inf"), float("nan"))[i % 4]
        moe.moe_add_rmsnorm(x, None, w, 0.0, y, codes=codes, scales=scales)
        moe.moe_quantize_e4m3(y, want, want_scales)
        nan = torch.isnan(y)  # (which has two codes)
        assert torch.equal(y[~nan], (x * w)[~nan]) and torch.equal(nan, torch.isnan(w).expand(3, d))
        assert torch.equal(scales, want_scales) and torch.equal(codes & 0x7F, want & 0x7F)
        assert torch.equal(codes[~nan], want[~nan])


@pytest.mark.parametrize("T", [300, 8200])  # three routing launches, and the fused router with its scatter
def test_given_codes_are_moved_in_place_of_the_rows(T):
    """The 8-bit layer on given codes writes no bf16 rows in segment order: on a zeroed workspace it leaves as many
    bytes untouched as those rows have (less what random rows hold in zero bytes)."""
    gen = torch.Generator().manual_seed(T)
    d, f, m, k = 64, 64, 8, 2
    wq = moe.quantize_experts(_bf16(gen, m, f, d), _bf16(gen, m, f, d), _bf16(gen, m, d, f))
    c = moe.make_config(T, d, f, m, k)
    x, wr = _bf16(gen, T, d) * 16, _bf16(gen, m, d)
    codes, scales = torch.empty(T, d, dtype=torch.uint8, device="cuda"), torch.empty(T, device="cuda")
    moe.moe_quantize_e4m3(x, codes, scales)
    a, b, wa, wb = torch.empty_like(x), torch.empty_like(x), moe.fp8_workspace(c), moe.fp8_workspace(c)
    moe.moe_layer_forward_fp8(c, x, wr, None, wq, a, wa)
    moe.moe_layer_forward_fp8_codes(c, x, codes, scales, wr, None, wq, b, wb)
    assert torch.equal(a, b)
    assert int((wa != 0).sum()) - int((wb != 0).sum()) > 0.95 * T * k * d * 2


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,d", N.SHAPES)
def test_no_vector_is_left_out_of_the_sum(rows, d, dtype):
    """Within the roundings that the sum of squares has on its way, not one for each of its terms: y of fp32 rows, and
    the fp32 scale of the codes of either type."""
    gen = torch.Generator().manual_seed(rows + d)
    x, r, w = (t.cuda() for t in N.inputs(gen, rows, d, dtype))
    for residual in (None, r):
        y, with_codes = torch.empty_like(x), d % 16 == 0
        codes = torch.empty(rows, d, dtype=torch.uint8, device="cuda") if with_codes else None
        scales = torch.empty(rows, device="cuda") if with_codes else None
        moe.moe_add_rmsnorm(x, residual, w, 1e-5, y, codes=codes, scales=scales)
        ref = N.norm64(x, residual, w)
        rel = N.REL + (torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 2.0 ** -24)
        assert ((y.to(F64) - ref).abs() <= rel * ref.abs()).all()
        if with_codes:
            want = ref.abs().amax(1) / 448
            assert ((scales.to(F64) - want).abs() <= (N.REL + 2 * 2.0 ** -24) * want).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 256, 512, 2048, 4096, 16384, 32768])
def test_rows_whose_squares_leave_the_range(d, dtype):
    """Rows near the largest and the smallest numbers, whose squares fp32 cannot hold: the formula's values, for every
    number of threads a row takes; ordinary rows between them are not touched by that."""
    gen = torch.Generator().manual_seed(d)
    sizes = [2.0 ** e for e in (125, 100, 64, 0, -40, -62, -64, -75, -100, -120)]
    x = (0.5 + torch.rand(len(sizes), d, generator=gen)) * torch.tensor(sizes)[:, None]
    x = (x * (torch.randint(0, 2, x.shape, generator=gen) * 2 - 1)).to(dtype).cuda()
    w = (0.5 + torch.rand(d, generator=gen)).to(dtype).cuda()
    half = torch.finfo(dtype).eps / 2
    for eps in (0.0, 1e-38, 1e-30, 1e-20, 1e-12, 1e-5):
        y = torch.empty_like(x)
        codes, scales = torch.empty(x.shape, dtype=torch.uint8, device="cuda"), torch.empty(len(sizes), device="cuda")
        moe.moe_add_rmsnorm(x, None, w, eps, y, codes=codes, scales=scales)
        eps32 = torch.tensor(eps, dtype=torch.float32).item()
        ref = norm64(x, None, w, eps32)
        # below 2^-126 y is off by up to 2^-150, or half a step of bf16's there, 2^-134
        tiny = 2.0 ** -149 if dtype == torch.float32 else 2.0 ** -133
        assert ((y.to(F64) - ref).abs() <= (half + N.REL) * ref.abs() + tiny).all(), eps
        top = ref.abs().amax(1)
        ok = top > 2.0 ** -100
        assert ((scales.to(F64) - top / 448).abs()[ok] <= (N.REL + 2.0 ** -23) * top[ok] / 448).all()
        assert not torch.isnan(codes.view(torch.float8_e4m3fn).float()).any()
        lone = torch.empty(1, d, dtype=dtype, device="cuda")
        moe.moe_add_rmsnorm(x[3:4].contiguous(), None, w, eps, lone)
        assert torch.equal(lone[0], y[3])


def test_infinities_zeros_and_nan_beside_large_and_small_rows():
    d = 1024
    x = torch.ones(6, d)
    x[0, 5], x[1, 7], x[2], x[3], x[4], x[5, 1:] = float("inf"), float("nan"), 0.0, 1e30, 1e-30, 0.0
    x[4, 3], x[5, 0] = 1e-45, 3e38
    w = torch.ones(d, device="cuda")
    y = torch.empty(6, d, device="cuda")
    moe.moe_add_rmsnorm(x.cuda(), None, w, 0.0, y)
    assert torch.isnan(y[0, 5]) and (y[0, :5] == 0).all() and (y[0, 6:] == 0).all()  # inf / inf, and 1 / inf
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all()  # 0 / 0
    ref = norm64(x[3:].cuda(), None, w, 0.0)
    assert ((y[3:].to(F64) - ref).abs() <= (N.REL + 2.0 ** -24) * ref.abs() + 2.0 ** -149).all()
