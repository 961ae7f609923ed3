"""The 4-bit and norm entry points without a GPU: sizes, and every refusal that the host
makes before it touches the device."""
import ctypes

import pytest

import norm_exact as N
import sparse_mixture_experts_08_b200 as moe
from sparse_mixture_experts_08_b200.moe import MoEConfig, MoEW4Experts

A = ctypes.c_void_p(1 << 24)
ODD = ctypes.c_void_p((1 << 24) + 8)


def test_struct_layout():
    # int32 group, padded to the pointers' alignment, then 12 pointers
    assert ctypes.sizeof(MoEW4Experts) == 8 + 12 * 8


@pytest.mark.parametrize("args,code", [
    ((-1, 8, 64, 32), moe.ERR_INVALID_ARG),
    ((1, -8, 64, 32), moe.ERR_INVALID_ARG),
    ((1, 8, 0, 32), moe.ERR_INVALID_ARG),
    ((1, 8, 64, 48), moe.ERR_UNSUPPORTED),       # groups of 32, 64, 128
    ((1, 8, 64, 0), moe.ERR_UNSUPPORTED),
    ((1, 12, 64, 32), moe.ERR_UNSUPPORTED),      # rows % 8
    ((1, 8, 48, 32), moe.ERR_UNSUPPORTED),       # cols % 32
    ((65536, 8, 64, 32), moe.ERR_UNSUPPORTED),
    ((1, 1 << 21, 64, 32), moe.ERR_UNSUPPORTED),
    ((0, 8, 64, 32), moe.OK),                    # nothing to do
    ((3, 0, 64, 32), moe.OK),
])
def test_quantizer_sizes(args, code):
    lib = moe.moe.lib()
    assert lib.moe_quantize_w4(*args, A if code else None, A, A, None) == code
    assert lib.moe_dequantize_w4(*args, A if code else None, A, A, None) == code


def test_quantizer_pointers():
    lib = moe.moe.lib()
    for bad in range(3):
        for p in (None, ODD):
            args = [A, A, A]
            args[bad] = p
            assert lib.moe_quantize_w4(1, 8, 64, 32, *args, None) == moe.ERR_INVALID_ARG
            assert lib.moe_dequantize_w4(1, 8, 64, 32, *args, None) == moe.ERR_INVALID_ARG


def _norm(rows=4, d=64, dtype=moe.BF16, eps=1e-5, x=A, residual=None, weight=A, total=None, y=A, codes=None,
          scales=None):
    return moe.moe.lib().moe_add_rmsnorm(rows, d, dtype, eps, x, residual, weight, total, y, codes, scales, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), moe.ERR_INVALID_ARG),
    (dict(d=0), moe.ERR_INVALID_ARG),
    (dict(dtype=2), moe.ERR_INVALID_ARG),
    (dict(dtype=-1), moe.ERR_INVALID_ARG),
    (dict(eps=-1e-5), moe.ERR_INVALID_ARG),
    (dict(eps=float("nan")), moe.ERR_INVALID_ARG),
    (dict(eps=float("inf")), moe.ERR_INVALID_ARG),
    (dict(y=None), moe.ERR_INVALID_ARG),                              # no output
    (dict(codes=A), moe.ERR_INVALID_ARG),                             # codes without scales
    (dict(scales=A), moe.ERR_INVALID_ARG),
    (dict(x=None), moe.ERR_INVALID_ARG),
    (dict(weight=None), moe.ERR_INVALID_ARG),
    (dict(x=ODD), moe.ERR_INVALID_ARG),
    (dict(residual=ODD), moe.ERR_INVALID_ARG),
    (dict(weight=ODD), moe.ERR_INVALID_ARG),
    (dict(total=ODD), moe.ERR_INVALID_ARG),
    (dict(y=ODD), moe.ERR_INVALID_ARG),
    (dict(codes=ODD, scales=A), moe.ERR_INVALID_ARG),
    (dict(codes=A, scales=ctypes.c_void_p((1 << 24) + 2)), moe.ERR_INVALID_ARG),
    (dict(total=ctypes.c_void_p(1 << 25), y=ctypes.c_void_p(1 << 25)), moe.ERR_INVALID_ARG),
    (dict(d=68), moe.ERR_UNSUPPORTED),
    (dict(d=72, codes=A, scales=A), moe.ERR_UNSUPPORTED),             # 16-byte code rows
    (dict(d=32776), moe.ERR_UNSUPPORTED),
    (dict(rows=0, x=None), moe.OK),
])
def test_norm_refusals(kw, code):
    assert _norm(**kw) == code


OK_CFG = (16, 256, 320, 4, 2, 1, 64, moe.BF16, moe.SWIGLU, 0)


def test_workspace_size_and_widths():
    lib = moe.moe.lib()
    n = ctypes.c_size_t(0)
    assert lib.moe_w4_workspace_size(ctypes.byref(MoEConfig(*OK_CFG)), ctypes.byref(n)) == moe.OK and n.value > 0
    assert lib.moe_w4_workspace_size(ctypes.byref(MoEConfig(*OK_CFG)), None) == moe.ERR_INVALID_ARG
    assert lib.moe_w4_workspace_size(None, ctypes.byref(n)) == moe.ERR_INVALID_ARG
    for at, value, code in ((7, moe.F32, moe.ERR_UNSUPPORTED), (1, 272, moe.ERR_UNSUPPORTED),
                            (2, 336, moe.ERR_UNSUPPORTED), (6, 80, moe.ERR_UNSUPPORTED), (0, 0, moe.ERR_INVALID_ARG),
                            (4, 5, moe.ERR_INVALID_ARG)):
        bad = list(OK_CFG)
        bad[at] = value
        assert lib.moe_w4_workspace_size(ctypes.byref(MoEConfig(*bad)), ctypes.byref(n)) == code, (at, value)


def _experts(group=64, **kw):
    full = {name: 1 << 24 for name, _ in MoEW4Experts._fields_[1:]}
    full.update(kw)
    return MoEW4Experts(group=group, **full)


def test_layer_and_grouped_refusals():
    lib = moe.moe.lib()
    c = MoEConfig(*OK_CFG)
    n = ctypes.c_size_t(0)
    lib.moe_w4_workspace_size(ctypes.byref(c), ctypes.byref(n))

    def layer(cfg=c, x=A, wr=A, w=None, out=A, ws=A, size=None):
        w = _experts() if w is None else w
        return lib.moe_layer_forward_w4(ctypes.byref(cfg), x, wr, None, ctypes.byref(w), out, None, None, None, None,
                                        None, ws, n.value if size is None else size, None)

    def grouped(cfg=c, x=A, off=A, w=None, task_w=None, perm=None, y=A, ws=A, size=1 << 30):
        w = _experts() if w is None else w
        return lib.moe_grouped_ffn_w4(ctypes.byref(cfg), x, off, ctypes.byref(w), task_w, perm, y, ws, size, None)

    for kw in (dict(x=None), dict(wr=None), dict(out=None), dict(x=ODD), dict(wr=ODD), dict(out=ODD), dict(ws=None),
               dict(ws=ctypes.c_void_p((1 << 24) + 16))):
        assert layer(**kw) == moe.ERR_INVALID_ARG, kw
    assert layer(size=n.value - 256) == moe.ERR_WORKSPACE
    for kw in (dict(x=None), dict(off=None), dict(y=None), dict(task_w=A), dict(x=ODD), dict(off=ODD), dict(y=ODD),
               dict(ws=None)):
        assert grouped(**kw) == moe.ERR_INVALID_ARG, kw
    assert grouped(size=1024) == moe.ERR_WORKSPACE
    for name, _ in MoEW4Experts._fields_[1:]:
        assert layer(w=_experts(**{name: None})) == moe.ERR_INVALID_ARG, name
        assert layer(w=_experts(**{name: (1 << 24) + 8})) == moe.ERR_INVALID_ARG, name
        if not name.startswith("sh_"):
            assert grouped(w=_experts(**{name: None})) == moe.ERR_INVALID_ARG, name
    for group in (0, 16, 96, 256, -32):
        assert layer(w=_experts(group=group)) == moe.ERR_UNSUPPORTED
        assert grouped(w=_experts(group=group)) == moe.ERR_UNSUPPORTED
    assert lib.moe_layer_forward_w4(ctypes.byref(c), A, A, None, None, A, None, None, None, None, None, A, n.value,
                                    None) == moe.ERR_INVALID_ARG
    # ReLU experts have no up matrix, a layer without shared experts no sh_ ones: the
    # pointers are complete, and what is refused is the workspace
    relu = MoEConfig(16, 256, 320, 4, 2, 0, 0, moe.BF16, moe.RELU, 0)
    bare = _experts(up=None, up_scale=None, **{k: None for k, _ in MoEW4Experts._fields_[1:] if k.startswith("sh_")})
    assert layer(cfg=relu, w=bare, size=256) == moe.ERR_WORKSPACE


def test_fp8_codes_refusals():
    lib = moe.moe.lib()
    c = MoEConfig(*OK_CFG)
    full = moe.moe.MoEFp8Experts(**{f: 1 << 24 for f, _ in moe.moe.MoEFp8Experts._fields_})

    def call(codes=A, scales=A, x=A, size=1 << 30):
        return lib.moe_layer_forward_fp8_codes(ctypes.byref(c), x, codes, scales, A, None, ctypes.byref(full), A, None,
                                               None, None, None, None, None, None, None, A, size, None)

    for kw in (dict(codes=None), dict(scales=None), dict(codes=ODD), dict(scales=ctypes.c_void_p((1 << 24) + 2)),
               dict(x=None)):
        assert call(**kw) == moe.ERR_INVALID_ARG, kw
    assert call(size=256) == moe.ERR_WORKSPACE


def test_binding_refuses_other_types():
    import torch
    x = torch.zeros(2, 16, dtype=torch.float16)
    with pytest.raises(moe.MoEError):
        moe.moe_add_rmsnorm(x, None, x, 1e-5, x, stream=0)


def test_binding_checks_types_and_sizes(monkeypatch):
    import torch
    from sparse_mixture_experts_08_b200 import moe as binding

    class Fake:  # a tensor that says it is on the device
        def __init__(self, *shape, dtype):
            self.t, self.dtype = torch.zeros(shape, dtype=dtype), dtype
            self.numel, self.is_contiguous, self.data_ptr = self.t.numel, self.t.is_contiguous, self.t.data_ptr

        def get_device(self):
            return 0

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    t = Fake(4, 8, dtype=torch.bfloat16)
    got = binding._pointers("f", ((t, torch.bfloat16, 32), (None, torch.float32, 9), (1 << 20, torch.float32, 9),
                                  (t, None, 1)))
    assert got == [t.data_ptr(), None, 1 << 20, t.data_ptr()]
    bits, e4m3 = Fake(32, dtype=torch.int16), Fake(32, dtype=torch.float8_e4m3fn)
    binding._pointers("f", ((bits, torch.bfloat16, 32), (e4m3, torch.uint8, 32)))
    for spec in ((bits, torch.float32, 16), (Fake(32, dtype=torch.float16), torch.bfloat16, 32), (bits, torch.uint8, 32),
                 (t, torch.float32, 32), (t, torch.bfloat16, 33), (torch.zeros(4), torch.float32, 4)):
        with pytest.raises(moe.MoEError):
            binding._pointers("f", ((t, torch.bfloat16, 32), spec))

    def experts(act, **kw):
        m, d, f, g = 3, 96, 160, 64
        wq = {"group": g}
        for key, rows, cols in (("gate", f, d), ("up", f, d), ("down", d, f)):
            wq[key] = Fake(m, rows, cols // 2, dtype=torch.uint8)
            wq[key + "_scale"] = Fake(m, -(-cols // g), rows, dtype=torch.bfloat16)
        wq.update(kw)
        st, ptrs = binding._w4_experts("f", moe.make_config(4, d, f, m, 1, act=act), wq, ((t, torch.bfloat16, 32),))
        assert ptrs == [t.data_ptr()] and (st.gate, st.down_scale) == (wq["gate"].data_ptr(), wq["down_scale"].data_ptr())
        assert st.sh_gate is None and st.group == wq["group"]

    experts(moe.SWIGLU)
    experts(moe.RELU, up=Fake(1, dtype=torch.float32), up_scale=None)  # not used
    experts(moe.SWIGLU, group=0)  # the library refuses it
    for kw in (dict(up=Fake(3, 160, 47, dtype=torch.uint8)), dict(down=Fake(3, 96, 80, dtype=torch.float32)),
               dict(gate_scale=Fake(3, 1, 160, dtype=torch.bfloat16)),
               dict(down_scale=Fake(3, 3, 96, dtype=torch.float16)), dict(group=32)):
        with pytest.raises(moe.MoEError):
            experts(moe.SWIGLU, **kw)


@pytest.mark.parametrize("act,n_shared", [(moe.SWIGLU, 2), (moe.RELU, 0)])
def test_binding_checks_every_tensor_of_the_8_bit_layer_on_codes(monkeypatch, act, n_shared):
    """Weights, scales and optional outputs of another type, too small, strided or on the host are refused before the
    library is called; entries that the layer does not use are not looked at."""
    import torch
    from sparse_mixture_experts_08_b200 import moe as binding

    class Fake:  # a tensor that says it is on the device
        def __init__(self, *shape, dtype):
            self.t, self.dtype, self.shape, self.is_cuda = torch.zeros(shape, dtype=dtype), dtype, shape, True
            self.numel, self.is_contiguous, self.data_ptr = self.t.numel, self.t.is_contiguous, self.t.data_ptr

        def get_device(self):
            return 0

    calls = []

    class Library:
        @staticmethod
        def moe_layer_forward_fp8_codes(*args):
            calls.append(args)
            return moe.OK

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(binding, "lib", lambda: Library)
    T, d, f, m, k, fs = 4, 32, 48, 3, 2, 64
    u8, bf16, f32, i32 = torch.uint8, torch.bfloat16, torch.float32, torch.int32
    up = act == moe.SWIGLU
    c = moe.make_config(T, d, f, m, k, n_shared=n_shared, f_shared=fs if n_shared else 0, act=act)
    shapes = {"gate": (m, f, d), "down": (m, d, f)}
    if up:
        shapes["up"] = (m, f, d)
    if n_shared:
        shapes.update({"sh_gate": (n_shared, fs, d), "sh_up": (n_shared, fs, d), "sh_down": (n_shared, d, fs)})
    wq = {}
    for key, shape in shapes.items():
        wq[key], wq[key + "_scale"] = Fake(*shape, dtype=u8), Fake(*shape[:2], dtype=f32)
    good = {"x": Fake(T, d, dtype=bf16), "x_codes": Fake(T, d, dtype=u8), "x_scales": Fake(T, dtype=f32),
            "w_router": Fake(m, d, dtype=bf16), "bias": Fake(m, dtype=f32), "out": Fake(T, d, dtype=bf16),
            "logits_out": Fake(T, m, dtype=f32), "topk_idx_out": Fake(T, k, dtype=i32),
            "topk_w_out": Fake(T, k, dtype=f32), "counts_out": Fake(m, dtype=i32),
            "lis_out": Fake(binding.LIS_BYTES, dtype=u8), "h_out": Fake(T * k, f, dtype=bf16),
            "perm_out": Fake(T * k, dtype=i32)}
    if n_shared:
        good["h_shared_out"] = Fake(n_shared * T, fs, dtype=bf16)

    def call(wq=wq, **kw):
        a = dict(good, **kw)
        binding.moe_layer_forward_fp8_codes(c, wq=wq, ws=Fake(1 << 16, dtype=u8), stream=0, **a)

    call()
    call(wq=dict(wq, **({} if up else {"up": Fake(1, dtype=f32)}), **({} if n_shared else {"sh_down": Fake(1, dtype=f32)})))
    assert len(calls) == 2
    # the library's arguments in its order
    st = calls[0][6]._obj
    assert calls[0][1:6] == tuple(good[key].data_ptr() for key in ("x", "x_codes", "x_scales", "w_router", "bias"))
    assert calls[0][7:15] == tuple(good[key].data_ptr() for key in (
        "out", "logits_out", "topk_idx_out", "topk_w_out", "counts_out", "lis_out", "h_out")) + (
        good["h_shared_out"].data_ptr() if n_shared else None,)
    assert calls[0][15] == good["perm_out"].data_ptr()
    for name, _ in binding.MoEFp8Experts._fields_:
        assert getattr(st, name) == (wq[name].data_ptr() if name in wq else None), name
    double = torch.float64
    for where in (good, wq):
        for name, t in where.items():
            strided = Fake(*t.shape, dtype=t.dtype)
            strided.is_contiguous = lambda: False
            for bad in (Fake(t.numel() - 1, dtype=t.dtype), Fake(*t.shape, dtype=double), strided,
                        torch.zeros(t.shape, dtype=t.dtype)):
                with pytest.raises(moe.MoEError) as e:
                    call(**{name: bad}) if where is good else call(wq=dict(wq, **{name: bad}))
                assert e.value.status == moe.ERR_INVALID_ARG, name
    assert len(calls) == 2


@pytest.mark.parametrize("rows,d", N.SHAPES)
def test_a_vector_left_out_of_the_norm_is_seen(rows, d):
    """The bound of test_gpu_norm.py's comparison, with the mistake in the reference: any one 16-byte vector of a row
    missing from the sum of squares moves y, and the codes' scale, by several times that."""
    import torch
    gen = torch.Generator().manual_seed(rows + d)
    for dtype, vec in ((torch.float32, 4), (torch.bfloat16, 8)):
        x, r, w = N.inputs(gen, rows, d, dtype)
        for residual in (None, r):
            ref = N.norm64(x, residual, w)
            s = x.to(N.F64) + (0 if residual is None else residual.to(N.F64))
            least = int((s * s).view(rows, d // vec, vec).sum(2).amax(0).argmin())  # the vector that matters least
            bad = N.norm64(x, residual, w, without=(vec * least, vec * least + vec))
            assert ((bad - ref).abs() > 3 * N.REL * ref.abs()).all(1).any()
            top, want = bad.abs().amax(1), ref.abs().amax(1)
            assert ((top - want).abs() > 3 * (N.REL + 2 * 2.0 ** -24) * want).any()
