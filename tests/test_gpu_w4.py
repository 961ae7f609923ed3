"""4-bit expert weights on the GPU against plain formulas in 64 bits.

- Quantizer: codes and scales bit-exact (one IEEE fp32 division each, then roundings).
- Dequantizer: bit-exact.
- Expert products: every output element within a bound built from what the kernels may
  round, elementwise and without statistics (u = 2^-8, bf16's half step):
    out   is rounded to bf16 once:                       u |out|
    h     is rounded to bf16 once:                       u sum_j |h_j| |W_down j|
    sums  are fp32 over K terms, any order, at most one rounding a term and one for each
          group's scale: 2 K 2^-24 times the sum of the absolute terms; for h through
          |d silu| <= 1.1, and 2^-18 relative for the exponential and the division.
  Scales with more than 5 significant bits are a weight of 8 more bits that may be
  rounded to bf16: u sum |x| |W| more in each sum.
"""
import numpy as np
import pytest
import torch

import sparse_mixture_experts_08_b200 as moe
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
F64 = torch.float64


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    require_gpu()


# ------------------------------------------------------------------ the format, in torch

def pack_ref(v, group):
    """Codes (as whole numbers [n, rows, cols]) and scales [n, ng, rows] of v (bf16) by the format's rules."""
    n, rows, cols = v.shape
    ng = -(-cols // group)
    f = torch.nn.functional.pad(v.float(), (0, ng * group - cols)).view(n, rows, ng, group)
    mant, ex = torch.frexp(f.abs().amax(3) / 7)
    scale = torch.ldexp(torch.round(mant * 32) / 32, ex)
    scale = torch.where(scale >= 2.0 ** -126, scale, torch.ones_like(scale))
    q = torch.round(f / scale[..., None]).view(n, rows, ng * group)[:, :, :cols]
    return q.to(torch.int32), scale.to(torch.bfloat16).transpose(1, 2).contiguous()


def encode(q):
    """Whole numbers [n, rows, cols] -> codes [n, rows, cols / 2]."""
    n, rows, cols = q.shape
    w = (q + 8).view(n, rows, cols // 8, 8)
    word = torch.zeros(n, rows, cols // 8, dtype=torch.int32, device=q.device)
    for c in range(8):
        word |= w[..., c] << ((16 if c & 1 else 0) + 4 * (c >> 1))
    return word.view(torch.uint8)


def values64(q, scales, group):
    cols = q.shape[2]
    return q.to(F64) * scales.to(F64).transpose(1, 2).repeat_interleave(group, 2)[:, :, :cols]


def make_matrix(gen, n, rows, cols, group, five_bits=True):
    v = (torch.randn(n, rows, cols, generator=gen) * cols ** -0.5).to(torch.bfloat16).cuda()
    q, s = pack_ref(v, group)
    if not five_bits:  # scales of another origin: all 8 bits of a bf16, and code -8
        s = (s.float() * (1 + torch.rand(s.shape, generator=gen).cuda() / 16)).to(torch.bfloat16)
        q[:, ::3, ::5] = -8
    return encode(q), s, values64(q, s, group)


def make_experts(gen, m, d, f, group, act, ns=0, fs=0, five_bits=True):
    wq, val = {"group": group}, {}
    for key, n, rows, cols in (("gate", m, f, d), ("up", m, f, d), ("down", m, d, f), ("sh_gate", ns, fs, d),
                               ("sh_up", ns, fs, d), ("sh_down", ns, d, fs)):
        if n and not (key.endswith("up") and act == moe.RELU):
            wq[key], wq[key + "_scale"], val[key] = make_matrix(gen, n, rows, cols, group, five_bits)
    return wq, val


def ffn64(x, val, pre, e, act, extra=0.0):
    """(y, bound of |kernel - y|) of expert e for rows x (fp64 of bf16 values)."""
    wg, wd = val[pre + "gate"][e], val[pre + "down"][e]
    d, f = wg.shape[1], wd.shape[1]
    eps = 2 * d * 2.0 ** -24 + extra
    g, ga = x @ wg.t(), (x.abs() @ wg.abs().t()) * eps
    if act == moe.SWIGLU:
        wu = val[pre + "up"][e]
        u, ua = x @ wu.t(), (x.abs() @ wu.abs().t()) * eps
        sg = torch.sigmoid(g)
        h = g * sg * u
        eh = (1.1 * ga) * (u.abs() + ua) + (g * sg).abs() * ua + 2.0 ** -18 * h.abs()
    else:
        h, eh = g.clamp_min(0), ga
    eh = eh + U * (h.abs() + eh)
    y = h @ wd.t()
    return y, eh @ wd.abs().t() + (2 * f * 2.0 ** -24 + extra) * ((h.abs() + eh) @ wd.abs().t())


def check(got, ref, bound, what=""):
    over = ((got.to(F64) - ref).abs() - bound).max().item()
    assert torch.isfinite(got.float()).all(), what
    assert over <= 0, f"{what}: an element is {over:.3e} over its bound"


# ------------------------------------------------------------------ quantizer

@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("shape", [(1, 8, 32), (3, 40, 96), (2, 264, 1376), (1, 72, 4096), (5, 16, 544)])
def test_quantizer_and_dequantizer_are_bit_exact(shape, group):
    gen = torch.Generator().manual_seed(shape[1] * 131 + shape[2] + group)
    v = torch.randn(shape, generator=gen) * torch.exp2(torch.randint(-30, 30, shape[:2] + (1,), generator=gen).float())
    v[0, 0] = 0.0                                              # scale 1
    v[0, 1] = -0.0
    v[0, 2] = torch.randint(-3, 4, shape[2:], generator=gen) * 2.0 ** -130   # below the smallest scale
    v[0, 3] = torch.randint(-14, 15, shape[2:], generator=gen) * 0.5         # ties between codes
    v[0, 4, :] = 3.0e38                                        # the largest scale
    v[0, 5, 0] = 1.0e30                                        # one large value
    v = v.to(torch.bfloat16).cuda()
    n, rows, cols = shape
    codes = torch.full((n, rows, cols // 2), 0x5A, dtype=torch.uint8, device="cuda")
    scales = torch.full((n, -(-cols // group), rows), -1.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_quantize_w4(v, group, codes, scales)
    q, s = pack_ref(v, group)
    assert torch.equal(scales.view(torch.int16), s.view(torch.int16))
    assert torch.equal(codes, encode(q))
    back = torch.empty_like(v)
    moe.moe_dequantize_w4(codes, scales, group, back)
    ref = values64(q, s, group)
    assert torch.equal(back.to(F64), ref)  # code x scale is a bf16 number: no rounding
    # and within half a step of the weight
    step = s.to(F64).transpose(1, 2).repeat_interleave(group, 2)[:, :, :cols]
    assert ((ref - v.to(F64)).abs() <= step / 2 * (1 + 2.0 ** -20)).all()


def test_dequantizer_rounds_scales_of_another_origin_once():
    gen = torch.Generator().manual_seed(5)
    codes, scales, ref = make_matrix(gen, 2, 24, 160, 64, five_bits=False)
    out = torch.empty(2, 24, 160, dtype=torch.bfloat16, device="cuda")
    moe.moe_dequantize_w4(codes, scales, 64, out)
    assert torch.equal(out, ref.float().to(torch.bfloat16))  # a product of 4 and 8 bits is exact in fp32


def test_quantizer_takes_infinities_and_nan_without_writing_elsewhere():
    v = torch.randn(1, 16, 128).to(torch.bfloat16)
    v[0, 3, 7], v[0, 5, 64] = float("inf"), float("nan")
    v = v.cuda()
    codes = torch.empty(1, 16, 64, dtype=torch.uint8, device="cuda")
    scales = torch.empty(1, 4, 16, dtype=torch.bfloat16, device="cuda")
    moe.moe_quantize_w4(v, 32, codes, scales)
    q, s = pack_ref(v[:, [0, 1, 2, 4, 6, 7]], 32)
    keep = torch.tensor([0, 1, 2, 4, 6, 7], device="cuda")
    assert torch.equal(codes[:, keep], encode(q)) and torch.equal(scales[:, :, keep], s)


# ------------------------------------------------------------------ grouped products

def _segments(lengths):
    return torch.tensor([0] + np.cumsum(lengths).tolist(), dtype=torch.int32, device="cuda")


GROUPED = [
    # lengths of the segments, d, f, group, act
    ([1], 32, 32, 32, moe.SWIGLU),
    ([0, 1, 0, 3], 64, 96, 64, moe.SWIGLU),
    ([8, 9, 0, 16, 17, 7], 160, 224, 32, moe.SWIGLU),
    ([5, 0, 2], 4096, 512, 128, moe.SWIGLU),
    ([33, 0, 31, 64, 65, 1], 288, 416, 64, moe.SWIGLU),
    ([2, 130, 0, 257, 15], 512, 1408, 128, moe.SWIGLU),
    ([40, 3, 12], 2080, 1376, 32, moe.RELU),
    ([0, 0, 19], 96, 2080, 128, moe.RELU),
    ([300, 1, 0, 513], 224, 352, 64, moe.RELU),
    ([129, 128, 127, 256], 1056, 544, 128, moe.SWIGLU),
    # segments around 12 rows (tiles of 32), K that ends inside 64 and inside 256 columns
    ([13, 30, 0, 9, 17, 3, 1, 24], 352, 1120, 32, moe.SWIGLU),
    ([32, 31, 33, 1], 1056, 96, 64, moe.RELU),
    # few long tiles, each cut between many blocks; both products in one launch
    ([3], 4096, 6176, 128, moe.SWIGLU),
    ([1, 1], 14336, 64, 64, moe.RELU),
    # around 50, 80 and 400 rows (tiles of 64, 128 and 192 over two blocks), rows of weights
    # that end inside a pair's tile, one tile of the second block empty
    ([50, 49, 64, 0, 20], 640, 1376, 32, moe.SWIGLU),
    ([81, 64, 192, 0, 1], 1376, 544, 64, moe.RELU),
    ([400, 17, 385, 193], 288, 1312, 32, moe.SWIGLU),
    ([577], 2080, 160, 128, moe.SWIGLU),
    # tiles of 224 rows, for the first product, the second and both
    ([450, 0, 224, 225, 1, 700], 4096, 160, 128, moe.SWIGLU),
    ([230, 449], 96, 4128, 32, moe.RELU),
    ([800], 4160, 4096, 64, moe.SWIGLU),
    # more than a hundred pieces of work a block or pair (those past the listed ones are worked out on the way)
    ([12288], 64, 32768, 32, moe.RELU),
    ([1] * 600, 32, 4096, 32, moe.RELU),
    # more groups than a warp has lanes
    ([(7 * i) % 5 for i in range(150)], 64, 96, 32, moe.SWIGLU),
    ([(11 * i) % 190 for i in range(40)], 96, 160, 64, moe.RELU),
]


@pytest.mark.parametrize("lengths,d,f,group,act", GROUPED)
def test_grouped_ffn(lengths, d, f, group, act):
    gen = torch.Generator().manual_seed(sum(lengths) * 7 + d + f + group)
    m, rows = len(lengths), sum(lengths)
    wq, val = make_experts(gen, m, d, f, group, act)
    x = torch.randn(rows, d, generator=gen).to(torch.bfloat16).cuda()
    offsets = _segments(lengths)
    # two tasks more than the segments hold: rows behind the last segment stay as they were
    c = moe.make_config(rows + 2, d, f, m, 1, act=act)
    xp = torch.cat([x, torch.full((2, d), float("nan"), dtype=torch.bfloat16, device="cuda")])
    ws = moe.w4_workspace(c)
    y = torch.full((rows + 2, d), -7.0, dtype=torch.float32, device="cuda")
    moe.moe_grouped_ffn_w4(c, xp, offsets, wq, None, None, y, ws)
    assert moe.moe_read_device_status(ws) == moe.OK
    assert (y[rows:] == -7.0).all()
    # and with task weights, in another row order
    perm = torch.randperm(rows + 2, generator=gen).to(torch.int32).cuda()
    task_w = torch.rand(rows + 2, generator=gen).cuda()
    yw = torch.empty_like(y)
    moe.moe_grouped_ffn_w4(c, xp, offsets, wq, task_w, perm, yw, ws)
    a = 0
    for e, n in enumerate(lengths):
        if n:
            ref, bound = ffn64(x[a:a + n].to(F64), val, "", e, act)
            check(y[a:a + n], ref, bound, f"expert {e}")
            w = task_w[perm[a:a + n].long()].to(F64)[:, None]
            check(yw[a:a + n], ref * w, bound * w * (1 + 2.0 ** -20) + 2.0 ** -23 * (ref * w).abs(), f"weighted {e}")
        a += n


@pytest.mark.parametrize("rows", [3, 300])
def test_scales_of_another_origin(rows):
    gen = torch.Generator().manual_seed(rows)
    d, f, group = 320, 256, 64
    wq, val = make_experts(gen, 2, d, f, group, moe.SWIGLU, five_bits=False)
    x = torch.randn(2 * rows, d, generator=gen).to(torch.bfloat16).cuda()
    c = moe.make_config(2 * rows, d, f, 2, 1)
    y = torch.empty(2 * rows, d, dtype=torch.float32, device="cuda")
    moe.moe_grouped_ffn_w4(c, x, _segments([rows, rows]), wq, None, None, y, moe.w4_workspace(c))
    for e in range(2):
        ref, bound = ffn64(x[e * rows:(e + 1) * rows].to(F64), val, "", e, moe.SWIGLU, extra=U)
        check(y[e * rows:(e + 1) * rows], ref, bound)


@pytest.mark.parametrize("rows", [6, 200])
def test_infinities_and_nan_stay_in_their_rows(rows):
    gen = torch.Generator().manual_seed(rows + 1)
    d, f = 256, 320
    wq, _ = make_experts(gen, 2, d, f, 64, moe.SWIGLU)
    x = torch.randn(2 * rows, d, generator=gen).to(torch.bfloat16).cuda()
    bad = x.clone()
    bad[2, 5], bad[rows + 1, 17] = float("nan"), float("inf")
    c = moe.make_config(2 * rows, d, f, 2, 1)
    y, yb = (torch.empty(2 * rows, d, dtype=torch.float32, device="cuda") for _ in range(2))
    ws = moe.w4_workspace(c)
    moe.moe_grouped_ffn_w4(c, x, _segments([rows, rows]), wq, None, None, y, ws)
    moe.moe_grouped_ffn_w4(c, bad, _segments([rows, rows]), wq, None, None, yb, ws)
    keep = torch.ones(2 * rows, dtype=torch.bool, device="cuda")
    keep[2] = keep[rows + 1] = False
    assert torch.equal(y[keep], yb[keep])
    assert torch.isnan(yb[2]).all() and not torch.isfinite(yb[rows + 1]).all()


def test_bad_offsets_are_reported_and_nothing_is_written():
    gen = torch.Generator().manual_seed(3)
    wq, _ = make_experts(gen, 3, 64, 96, 32, moe.RELU)
    c = moe.make_config(4, 64, 96, 3, 1, act=moe.RELU)
    x = torch.randn(4, 64, generator=gen).to(torch.bfloat16).cuda()
    for offsets in ([0, 2, 5, 5], [0, 3, 2, 4], [-1, 1, 2, 3]):
        ws = moe.w4_workspace(c)
        y = torch.full((4, 64), -7.0, device="cuda")
        moe.moe_grouped_ffn_w4(c, x, torch.tensor(offsets, dtype=torch.int32, device="cuda"), wq, None, None, y, ws)
        assert moe.moe_read_device_status(ws) == moe.ERR_DEVICE_INDEX
        assert torch.isfinite(y).all()
        # the same workspace works again afterwards
        moe.moe_grouped_ffn_w4(c, x, _segments([1, 2, 1]), wq, None, None, y, ws)
        assert moe.moe_read_device_status(ws) == moe.OK


def test_codes_past_4_gib():
    """The last expert's codes lie behind the 32-bit range of bytes."""
    m, d, f, group = 70, 8192, 15360, 128
    assert m * f * d // 2 > 1 << 32
    gen = torch.Generator().manual_seed(9)
    wq = {"group": group}
    val = {}
    for key, rows, cols in (("gate", f, d), ("down", d, f)):
        codes = torch.zeros(m, rows, cols // 2, dtype=torch.uint8, device="cuda")
        scales = torch.zeros(m, cols // group, rows, dtype=torch.bfloat16, device="cuda")
        codes[-1:], scales[-1:], val[key] = make_matrix(gen, 1, rows, cols, group)
        wq[key], wq[key + "_scale"] = codes, scales
    for n in (3, 150):
        x = torch.randn(n, d, generator=gen).to(torch.bfloat16).cuda()
        c = moe.make_config(n, d, f, m, 1, act=moe.RELU)
        y = torch.empty(n, d, dtype=torch.float32, device="cuda")
        moe.moe_grouped_ffn_w4(c, x, _segments([0] * (m - 1) + [n]), wq, None, None, y, moe.w4_workspace(c))
        ref, bound = ffn64(x.to(F64), val, "", 0, moe.RELU)
        check(y, ref, bound)


# ------------------------------------------------------------------ the layer

def layer_ref(x, idx, w, val, c, act):
    """(out, bound) in 64 bits from the routing that the call reports."""
    x64 = x.to(F64)
    ref = torch.zeros_like(x64)
    bound = torch.zeros_like(x64)
    for e in range(c.m):
        for s in range(c.k):
            t = torch.nonzero(idx[:, s] == e)[:, 0]
            if len(t):
                y, b = ffn64(x64[t], val, "", e, act)
                g = w[t, s].to(F64)[:, None]
                ref[t] += g * y
                bound[t] += g * b + 2.0 ** -22 * (g * y).abs()
    for e in range(c.n_shared):
        y, b = ffn64(x64, val, "sh_", e, act)
        ref += y
        bound += b + 2.0 ** -22 * y.abs()
    return ref, bound + U * (ref.abs() + bound)


def run_layer(c, x, wr, bias, wq, ws=None, stream=None):
    ws = moe.w4_workspace(c) if ws is None else ws
    out = torch.empty_like(x)
    r = {"logits": torch.empty(c.T, c.m, device="cuda"),
         "idx": torch.empty(c.T, c.k, dtype=torch.int32, device="cuda"), "w": torch.empty(c.T, c.k, device="cuda"),
         "counts": torch.empty(c.m, dtype=torch.int32, device="cuda"), "lis": moe.lis_buffer(), "out": out, "ws": ws}
    moe.moe_layer_forward_w4(c, x, wr, bias, wq, out, ws, logits_out=r["logits"], topk_idx_out=r["idx"],
                             topk_w_out=r["w"], counts_out=r["counts"], lis_out=r["lis"], stream=stream)
    return r


LAYERS = [
    # T, d, f, m, k, n_shared, f_shared, group, act, renormalize
    (1, 256, 352, 8, 2, 0, 0, 128, moe.SWIGLU, True),
    (1, 64, 64, 1, 1, 0, 0, 32, moe.RELU, False),
    (16, 512, 1408, 64, 6, 2, 1408, 64, moe.SWIGLU, False),
    (7, 160, 224, 5, 5, 1, 96, 32, moe.SWIGLU, True),
    (61, 288, 544, 12, 1, 0, 0, 64, moe.RELU, False),
    (173, 416, 352, 12, 3, 0, 0, 32, moe.RELU, False),
    (500, 256, 224, 4, 2, 2, 160, 128, moe.SWIGLU, True),
    (2048, 128, 160, 16, 4, 0, 0, 64, moe.SWIGLU, False),
    (8300, 64, 96, 8, 2, 1, 64, 32, moe.SWIGLU, True),
    (33, 128, 128, 700, 8, 0, 0, 128, moe.SWIGLU, False),
    (64, 96, 64, 24, 8, 0, 0, 32, moe.SWIGLU, True),
    (57, 96, 64, 24, 9, 1, 32, 32, moe.RELU, False),
    # 1024 tasks and 1026: the last batch whose dispatch is one launch, the first with three
    (128, 96, 64, 24, 8, 0, 0, 32, moe.SWIGLU, True),
    (114, 96, 64, 24, 9, 1, 32, 32, moe.RELU, False),
    (1, 64, 64, 1024, 32, 0, 0, 32, moe.SWIGLU, True),
    (3, 2080, 1376, 6, 2, 1, 1376, 64, moe.SWIGLU, True),
]


def _layer_case(case, seed=0):
    T, d, f, m, k, ns, fs, group, act, renorm = case
    gen = torch.Generator().manual_seed(T + d + m + seed)
    c = moe.make_config(T, d, f, m, k, n_shared=ns, f_shared=fs, act=act, renormalize=renorm)
    wq, val = make_experts(gen, m, d, f, group, act, ns, fs)
    x = torch.randn(T, d, generator=gen).to(torch.bfloat16).cuda()
    wr = (torch.randn(m, d, generator=gen) * d ** -0.5).to(torch.bfloat16).cuda()
    bias = (-0.5 * torch.log(1 + torch.arange(m).float())).cuda()
    return c, wq, val, x, wr, bias, act


@pytest.mark.parametrize("case", LAYERS)
def test_layer(case):
    c, wq, val, x, wr, bias, act = _layer_case(case)
    r = run_layer(c, x, wr, bias, wq)
    assert moe.moe_read_device_status(r["ws"]) == moe.OK
    # the router is the bf16 layer's
    idx, w = torch.empty_like(r["idx"]), torch.empty_like(r["w"])
    moe.moe_route(c, x, wr, bias, None, None, idx, w, moe.workspace(c))
    assert torch.equal(idx, r["idx"]) and torch.equal(w, r["w"])
    assert torch.equal(r["counts"].long(), torch.bincount(r["idx"].flatten().long(), minlength=c.m))
    assert moe.unpack_lis(r["lis"])[0] == int(r["counts"].max())
    ref, bound = layer_ref(x, r["idx"], r["w"], val, c, act)
    check(r["out"], ref, bound)
    # the same call again gives the same bits
    assert torch.equal(run_layer(c, x, wr, bias, wq, ws=r["ws"])["out"], r["out"])


def test_quantized_weights_of_a_bf16_layer():
    """quantize_experts_w4 and the layer: against the bf16 layer run on the values that the codes stand for."""
    gen = torch.Generator().manual_seed(21)
    T, d, f, m, k, ns, fs = 40, 256, 384, 6, 2, 1, 192
    dev = lambda *s: (torch.randn(*s, generator=gen) * s[-1] ** -0.5).to(torch.bfloat16).cuda()  # noqa: E731
    w = {"gate": dev(m, f, d), "up": dev(m, f, d), "down": dev(m, d, f), "sh_gate": dev(ns, fs, d),
         "sh_up": dev(ns, fs, d), "sh_down": dev(ns, d, fs)}
    wq = moe.quantize_experts_w4(*w.values(), group=64)
    val = {}
    for key in w:
        back = torch.empty_like(w[key])
        moe.moe_dequantize_w4(wq[key], wq[key + "_scale"], 64, back)
        val[key] = back
    c = moe.make_config(T, d, f, m, k, n_shared=ns, f_shared=fs)
    x, wr = torch.randn(T, d, generator=gen).to(torch.bfloat16).cuda(), dev(m, d)
    r = run_layer(c, x, wr, None, wq)
    ref, bound = layer_ref(x, r["idx"], r["w"], {key: v.to(F64) for key, v in val.items()}, c, moe.SWIGLU)
    check(r["out"], ref, bound)
    out = torch.empty_like(x)
    moe.moe_layer_forward(c, x, wr, None, *(val[key] for key in ("gate", "up", "down", "sh_gate", "sh_up", "sh_down")),
                          out, moe.workspace(c))
    check(out, ref, bound)


@pytest.mark.parametrize("case", [LAYERS[2], LAYERS[6]])
def test_captured_on_a_side_stream_and_replayed(case):
    c, wq, _, x, wr, bias, _ = _layer_case(case)
    want = run_layer(c, x, wr, bias, wq)["out"]
    x2 = torch.flip(x, [0]).contiguous()
    want2 = run_layer(c, x2, wr, bias, wq)["out"]
    xs, ws, out = x.clone(), moe.w4_workspace(c), torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        moe.moe_layer_forward_w4(c, xs, wr, bias, wq, out, ws)
    for src, ref in ((x, want), (x2, want2), (x, want)):
        xs.copy_(src)
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    assert moe.moe_read_device_status(ws) == moe.OK


def test_two_streams_with_workspaces_of_their_own():
    c, wq, _, x, wr, bias, _ = _layer_case(LAYERS[2])
    want = run_layer(c, x, wr, bias, wq)["out"]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [moe.w4_workspace(c) for _ in range(2)]
    outs = [torch.empty_like(x) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, ws, out in zip(streams, spaces, outs):
            moe.moe_layer_forward_w4(c, x, wr, bias, wq, out, ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for out in outs)


def test_fp8_refuses_and_w4_accepts_the_same_widths():
    """d, f multiples of 32; anything else is refused before a launch."""
    ok = moe.make_config(4, 96, 160, 3, 1)
    assert moe.moe_w4_workspace_size(ok) > 0
    with pytest.raises(moe.MoEError):
        moe.moe_w4_workspace_size(moe.make_config(4, 48, 160, 3, 1))


def _outputs(case, ws, seed=0):
    c, wq, _, x, wr, bias, _ = _layer_case(case, seed)
    return lambda: run_layer(c, x, wr, bias, wq, ws=ws)["out"]


def test_one_workspace_for_batches_of_all_sizes():
    """A server allocates for its largest batch: batches that take both products in one launch, in two, cut tiles
    and whole ones, in turn on the same memory, give what each gives on a workspace of its own."""
    cases = [(T, 288, 2080, 8, 2, 1, 160, 32, moe.SWIGLU, True) for T in (1, 700, 16, 90, 33, 2, 1500, 5)]
    big = max((_layer_case(case)[0] for case in cases), key=moe.moe_w4_workspace_size)
    shared = moe.w4_workspace(big)
    calls = [(_outputs(case, shared), _outputs(case, None)()) for case in cases]
    for _ in range(3):
        for call, want in calls:
            assert torch.equal(call(), want)
    assert moe.moe_read_device_status(shared) == moe.OK


@pytest.mark.parametrize("T", [2, 28, 60, 200, 640])
def test_many_calls_give_the_same_bits(T):
    """Sums that are cut between blocks are joined by whichever block is last: the order of the additions is fixed."""
    c, wq, _, x, wr, bias, _ = _layer_case((T, 512, 4128, 4, 2, 0, 0, 64, moe.SWIGLU, False))
    ws, want, out = moe.w4_workspace(c), torch.empty_like(x), torch.empty_like(x)
    moe.moe_layer_forward_w4(c, x, wr, bias, wq, want, ws)
    for _ in range(100):
        moe.moe_layer_forward_w4(c, x, wr, bias, wq, out, ws)
        assert torch.equal(out, want)
    assert moe.moe_read_device_status(ws) == moe.OK


@pytest.mark.parametrize("T", [4, 30, 70, 300, 900])
def test_waits_that_run_out_are_reported_and_the_next_call_is_right(T):
    """With a time limit of 1 ns the kernels give up at a wait that outlasts one poll of its barrier and return; the
    workspace works again afterwards (the counters of cut tiles do not keep what the broken call left). A poll blocks
    for a while by itself, so a call whose waits are all shorter than that completes, and must be right then."""
    case = (T, 256, 1120, 4, 2, 1, 96, 64, moe.SWIGLU, True)
    c, wq, _, x, wr, bias, _ = _layer_case(case)
    ws = moe.w4_workspace(c)
    want = run_layer(c, x, wr, bias, wq, ws=ws)["out"]
    try:
        moe.moe_debug_set_wait_limit_ns(1)
        got = run_layer(c, x, wr, bias, wq, ws=ws)["out"]
        status = moe.moe_read_device_status(ws)  # synchronises: the kernels returned
    finally:
        moe.moe_debug_set_wait_limit_ns(0)
    assert status == moe.ERR_TIMEOUT or (status == moe.OK and torch.equal(got, want))
    for _ in range(3):
        assert torch.equal(run_layer(c, x, wr, bias, wq, ws=ws)["out"], want)
    assert moe.moe_read_device_status(ws) == moe.OK


def test_two_graphs_in_turn_on_one_workspace():
    """A prompt's graph and a decode step's graph replayed in turn, as a server does, with one workspace."""
    cases = [(T, 256, 1408, 8, 2, 1, 352, 64, moe.SWIGLU, True) for T in (300, 8)]
    parts = [_layer_case(case) for case in cases]
    ws = moe.w4_workspace(parts[0][0])
    graphs = []
    for c, wq, _, x, wr, bias, _ in parts:
        want = run_layer(c, x, wr, bias, wq)["out"]
        out, graph = torch.empty_like(x), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            moe.moe_layer_forward_w4(c, x, wr, bias, wq, out, ws)
        graphs.append((graph, out, want))
    for i in (0, 1, 1, 0, 1, 0, 0):
        graph, out, want = graphs[i]
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_all_tokens_on_one_expert():
    """Routing that leaves all experts but one empty."""
    c, wq, val, x, wr, _, act = _layer_case((48, 160, 224, 6, 1, 0, 0, 32, moe.SWIGLU, True))
    bias = torch.tensor([0.0, 0, 1e4, 0, 0, 0], device="cuda")
    r = run_layer(c, x, wr, bias, wq)
    assert (r["idx"] == 2).all() and r["counts"].tolist() == [0, 0, 48, 0, 0, 0]
    ref, bound = layer_ref(x, r["idx"], r["w"], val, c, act)
    check(r["out"], ref, bound)


def test_binding_refuses_strided_and_host_tensors():
    c, wq, _, x, wr, bias, _ = _layer_case(LAYERS[0])
    ws, out = moe.w4_workspace(c), torch.empty_like(x)
    wide = torch.empty(c.T, 2 * c.d, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(x=wide[:, ::2]), dict(x=x.cpu()), dict(out=wide[:, ::2]), dict(wr=wr.cpu()),
                dict(wq=dict(wq, up=wq["up"].cpu())), dict(wq=dict(wq, gate=wq["gate"].transpose(1, 2)))):
        a = dict(dict(x=x, wr=wr, wq=wq, out=out), **bad)
        with pytest.raises(moe.MoEError):
            moe.moe_layer_forward_w4(c, a["x"], a["wr"], bias, a["wq"], a["out"], ws)
    v = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    codes = torch.empty(8, 32, dtype=torch.uint8, device="cuda")
    scales = torch.empty(2, 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(moe.MoEError):
        moe.moe_quantize_w4(v.t(), 32, codes, scales)
    with pytest.raises(moe.MoEError):
        moe.moe_dequantize_w4(codes, scales.cpu(), 32, v)


def test_binding_refuses_other_types_and_sizes():
    c, wq, _, x, wr, bias, _ = _layer_case(LAYERS[0])
    ws, out = moe.w4_workspace(c), torch.empty_like(x)
    for bad in (dict(x=x.float()), dict(out=out.float()), dict(wr=wr[:-1]), dict(wr=wr.float()),
                dict(bias=bias.to(torch.bfloat16)), dict(counts_out=torch.empty(c.m - 1, dtype=torch.int32, device="cuda")),
                dict(wq=dict(wq, up=wq["up"][:-1])), dict(wq=dict(wq, group=32)),
                dict(wq=dict(wq, down_scale=wq["down_scale"].float()))):
        a = dict(dict(x=x, wr=wr, bias=bias, wq=wq, out=out, counts_out=None), **bad)
        with pytest.raises(moe.MoEError):
            moe.moe_layer_forward_w4(c, a["x"], a["wr"], a["bias"], a["wq"], a["out"], ws, counts_out=a["counts_out"])
    v = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    codes = torch.empty(8, 32, dtype=torch.uint8, device="cuda")
    scales = torch.empty(2, 8, dtype=torch.bfloat16, device="cuda")
    for bad in ((v.float(), codes, scales), (v, codes[:7], scales), (v, codes, scales[:1]), (v, codes, scales.half())):
        with pytest.raises(moe.MoEError):
            moe.moe_quantize_w4(bad[0], 32, bad[1], bad[2])
        with pytest.raises(moe.MoEError):
            moe.moe_dequantize_w4(bad[1], bad[2], 32, bad[0])
    with pytest.raises(moe.MoEError):
        moe.moe_quantize_w4(v, 0, codes, scales)
    # bf16 as its bits is no other type
    a, b = torch.empty_like(x), torch.empty_like(x)
    moe.moe_layer_forward_w4(c, x, wr, bias, wq, a, ws)
    moe.moe_layer_forward_w4(c, x.view(torch.int16), wr.view(torch.int16), bias, wq, b.view(torch.int16), ws)
    assert torch.equal(a, b)


def _huge_last_group(gen, m, rows, cols, group):
    """Weights whose last group, shorter than the others, reaches 3.3e38: eight times its scale is no bf16 number."""
    v = torch.randn(m, rows, cols, generator=gen) * cols ** -0.5
    last = v[:, :, cols // group * group:]
    last /= last.abs().amax(2, keepdim=True)
    last *= 3.3e38
    q, s = pack_ref(v.to(torch.bfloat16).cuda(), group)
    assert cols % group and torch.isfinite(values64(q, s, group).to(torch.bfloat16)).all() and torch.isinf(s * 8).any()
    return encode(q), s, values64(q, s, group)


@pytest.mark.parametrize("rows", [3, 24, 50, 100, 400])
@pytest.mark.parametrize("key", ["gate", "down"])
def test_scales_near_the_top_of_the_range_in_a_short_last_group(key, rows):
    """Codes behind K stand for no weight: rows of zeros give zeros, rows of tiny inputs what the formula gives."""
    gen = torch.Generator().manual_seed(rows)
    d, f, group = 96, 352, 64
    wq, val = make_experts(gen, 2, d, f, group, moe.RELU)
    wq[key], wq[key + "_scale"], val[key] = _huge_last_group(gen, 2, *((f, d) if key == "gate" else (d, f)), group)
    x = (torch.randn(2 * rows, d, generator=gen) * 2.0 ** -110).to(torch.bfloat16).cuda()
    x[0] = x[rows] = 0
    c = moe.make_config(2 * rows, d, f, 2, 1, act=moe.RELU)
    ws, y = moe.w4_workspace(c), torch.empty(2 * rows, d, dtype=torch.float32, device="cuda")
    moe.moe_grouped_ffn_w4(c, x, _segments([rows, rows]), wq, None, None, y, ws)
    assert (y[0] == 0).all() and (y[rows] == 0).all()
    for e in range(2):
        ref, bound = ffn64(x[e * rows:(e + 1) * rows].to(F64), val, "", e, moe.RELU)
        check(y[e * rows:(e + 1) * rows], ref, bound)
