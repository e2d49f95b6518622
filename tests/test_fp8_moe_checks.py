"""Refusals of the FP8, norm and mixture-of-experts entry points (CPU only):
the C entry points' argument errors, which come before any HIP call, and the
binding's shape and layout checks, which come before the library is called."""

import ctypes
import os

import pytest
import torch

import bit_quantized_linear_int4_amd as wq

OK, NULL, SHAPE, ALIGN, UNSUP, WS = 0, 1, 2, 3, 4, 5
# fake device addresses: never dereferenced, because validation fails first
P, ODD = 0x10000, 0x10001

needs_lib = pytest.mark.skipif(not os.path.exists(wq.library_path()), reason="libwq.so not built")


def caller(fn, **base):
    def call(**kw):
        assert not set(kw) - set(base), "unknown argument"
        return fn(*{**base, **kw}.values())
    return call


def desc(fmt=wq.FMT_FP8_BLOCK, n=256, k=256, group=128, codes=P, scales=P, zeros=None, perm=None):
    d = wq._Weight()
    d.fmt, d.group, d.n, d.k, d.codes, d.scales, d.zeros, d.perm = (fmt, group, n, k, codes,
                                                                   scales, zeros, perm)
    return d


def i4(**kw):
    return desc(**{**dict(fmt=wq.FMT_INT4_ASYM, zeros=P), **kw})


@needs_lib
def test_norm_errors():
    call = caller(wq._load().wq_add_rmsnorm, x=P, dt=wq.F16, m=4, k=256, ldx=256, res=P, out=P,
                  ldr=256, gain=P, eps=1e-5, y=P, q=P, scales=P, stream=None)
    assert call(x=None) == NULL and call(gain=None) == NULL
    assert call(res=None) == NULL and call(out=None) == NULL
    assert call(scales=None) == NULL and call(q=None) == NULL
    assert call(y=None, q=None, scales=None) == NULL
    assert call(dt=wq.F32) == UNSUP
    assert call(m=0) == SHAPE and call(k=0) == SHAPE and call(k=260) == SHAPE
    assert call(m=1 << 23) == SHAPE and call(k=1 << 23, ldx=1 << 23, ldr=1 << 23) == SHAPE
    assert call(ldx=248) == SHAPE and call(ldx=260) == SHAPE and call(ldx=1 << 23) == SHAPE
    assert call(ldr=248) == SHAPE and call(ldr=260) == SHAPE
    assert call(eps=-1.0) == SHAPE and call(eps=float("nan")) == SHAPE
    for p in ("x", "res", "out", "gain", "y"):
        assert call(**{p: P + 8}) == ALIGN
    assert call(q=P + 4) == ALIGN and call(scales=P + 2) == ALIGN


@needs_lib
def test_quantizer_errors():
    lib = wq._load()
    call = caller(lib.wq_quantize_fp8_rows, x=P, up=P, dt=wq.F16, m=4, k=256, q=P, scales=P,
                  stream=None)
    assert call(x=None) == NULL and call(q=None) == NULL and call(scales=None) == NULL
    assert call(dt=wq.F32) == UNSUP and call(m=0) == SHAPE and call(k=252) == SHAPE
    assert call(x=P + 8) == ALIGN and call(up=P + 8) == ALIGN
    assert call(q=P + 4) == ALIGN and call(scales=ODD) == ALIGN
    call = caller(lib.wq_quantize_fp8_block, w=P, dt=wq.F16, n=4, k=256, codes=P, scales=P,
                  stream=None)
    assert call(w=None) == NULL and call(codes=None) == NULL and call(scales=None) == NULL
    assert call(dt=wq.F32) == UNSUP and call(n=0) == SHAPE and call(k=264) == SHAPE
    assert call(w=P + 8) == ALIGN and call(codes=P + 8) == ALIGN and call(scales=ODD) == ALIGN


@needs_lib
def test_linear_fp8_errors():
    call = caller(wq._load().wq_linear_fp8, q=P, scales=P, m=4, w=ctypes.byref(desc()), y=P,
                  ydt=wq.F16, ws=None, ws_bytes=0, stream=None)

    def w(**kw):
        return {"w": ctypes.byref(desc(**kw))}

    assert call(q=None) == NULL and call(scales=None) == NULL and call(y=None) == NULL
    assert call(w=None) == NULL and call(**w(codes=None)) == NULL and call(**w(scales=None)) == NULL
    assert call(m=0) == SHAPE and call(m=1 << 23) == SHAPE
    assert call(**w(k=264)) == SHAPE and call(**w(n=0)) == SHAPE
    assert call(**w(group=64)) == UNSUP and call(ydt=7) == UNSUP
    assert call(w=ctypes.byref(i4())) == UNSUP and call(**w(perm=P)) == UNSUP
    assert call(q=P + 8) == ALIGN and call(y=P + 8) == ALIGN and call(scales=ODD) == ALIGN
    assert call(**w(codes=P + 8)) == ALIGN and call(**w(scales=ODD)) == ALIGN
    # a split product needs its workspace
    big = desc(n=512, k=8192)
    need = wq._load().wq_linear_fp8_workspace(100, ctypes.byref(big))
    assert 0 < need <= 64 << 20
    split = dict(m=100, w=ctypes.byref(big))
    assert call(**split) == WS and call(**split, ws=P, ws_bytes=need - 1) == WS
    assert call(**split, ws=P + 128, ws_bytes=need) == ALIGN
    assert wq._load().wq_linear_fp8_workspace(0, ctypes.byref(big)) == 0
    assert wq._load().wq_linear_fp8_workspace(64, ctypes.byref(i4())) == 0


@needs_lib
@pytest.mark.parametrize("m,n,k", [(17, 128, 16), (333, 5000, 4112), (128, 14336, 16384),
                                   (4096, 4096, 4096), (2048, 28672, 8192)])
def test_linear_fp8_workspace_is_bounded(m, n, k):
    assert wq._load().wq_linear_fp8_workspace(m, ctypes.byref(desc(n=n, k=k))) <= 64 << 20


@needs_lib
def test_other_products_refuse_fp8():
    lib = wq._load()
    w = ctypes.byref(desc())
    assert lib.wq_linear_w4a16(P, wq.F16, 4, w, P, wq.F16, None, 0, None) == UNSUP
    assert lib.wq_linear_w4a16_gate_up(P, wq.F16, 4, w, w, 0, P, P, wq.F16, None) == UNSUP
    assert lib.wq_linear_int8_decomp(P, 4, w, 6.0, P, wq.F16, P, 1 << 30, None, None, None) == UNSUP


@needs_lib
def test_moe_errors():
    lib = wq._load()
    # 4 experts, h = 256, i = 128
    g = dict(n=512, k=256)
    base = dict(x=P, xdt=wq.BF16, m=4, router=P, logits=None, experts=4, top_k=2, renorm=1,
                gate=i4(**g), up=i4(**g), down=i4(n=1024, k=128), y=P, ydt=wq.BF16, ids=P,
                probs=P, ws=P, ws_bytes=1 << 30, stream=None)

    def call(**kw):
        a = {**base, **kw}
        for n in ("gate", "up", "down"):
            a[n] = None if a[n] is None else ctypes.byref(a[n])
        return lib.wq_moe(*a.values())

    assert call(x=None) == NULL and call(y=None) == NULL
    assert call(router=None) == NULL and call(logits=P) == NULL
    for n in ("gate", "up", "down"):
        assert call(**{n: None}) == NULL
    assert call(gate=i4(**g, zeros=None)) == NULL
    assert call(m=0) == SHAPE and call(top_k=0) == SHAPE and call(top_k=5) == SHAPE
    assert call(m=65) == UNSUP and call(xdt=wq.F32) == UNSUP and call(ydt=9) == UNSUP
    assert call(experts=513) == UNSUP
    assert call(experts=17, top_k=17) == UNSUP
    assert call(up=desc(**g)) == UNSUP and call(gate=desc(**g)) == UNSUP    # mixed formats
    assert call(gate=i4(**g, perm=P)) == UNSUP
    i8 = dict(fmt=wq.FMT_INT8_SYM_ROW, zeros=None)
    assert call(gate=i4(**i8, n=512, k=256, group=256)) == UNSUP
    nf4 = dict(fmt=wq.FMT_NF4, zeros=None, group=64)
    assert call(gate=i4(**g, **nf4), up=i4(**g, **nf4), down=i4(n=1024, k=128, **nf4)) == UNSUP
    assert call(up=i4(**g, group=64)) == SHAPE
    assert call(up=i4(n=256, k=256)) == SHAPE and call(up=i4(n=512, k=128)) == SHAPE
    assert call(down=i4(n=512, k=128)) == SHAPE and call(experts=2) == SHAPE
    # h, i not multiples of 128
    s = dict(group=64)
    assert call(gate=i4(n=512, k=192, **s), up=i4(n=512, k=192, **s),
                down=i4(n=768, k=128, **s)) == SHAPE
    assert call(x=P + 8) == ALIGN and call(router=P + 8) == ALIGN and call(y=ODD) == ALIGN
    assert call(ids=P + 2) == ALIGN and call(probs=P + 2) == ALIGN
    assert call(gate=i4(**g, scales=P + 4)) == ALIGN and call(gate=i4(**g, zeros=ODD)) == ALIGN
    gate = i4(**g)
    need = lib.wq_moe_workspace(4, 2, ctypes.byref(gate), 4)
    assert need > 0
    assert call(ws=None) == WS and call(ws_bytes=need - 1) == WS and call(ws=P + 128) == ALIGN
    assert lib.wq_moe_workspace(65, 2, ctypes.byref(gate), 4) == 0
    assert lib.wq_moe_workspace(4, 2, ctypes.byref(gate), 3) == 0


# ------------------------------------------------------------ binding, CPU tensors
def status(fn, *a, **kw):
    with pytest.raises(wq.WqError) as e:
        fn(*a, **kw)
    return e.value.status


H = torch.float16


def test_norm_binding():
    x, g, y = torch.zeros((4, 256), dtype=H), torch.zeros(256, dtype=H), torch.zeros((4, 256), dtype=H)
    q, s = wq.alloc_fp8_rows(4, 256, device="cpu")
    f = wq.wq_add_rmsnorm
    assert status(f, x, g, 1e-5, y=y, q=q, scales=s) == UNSUP          # well formed, not on a GPU
    wide = torch.zeros((4, 512), dtype=H)
    assert status(f, wide[:, :256], g, 1e-5, y=y) == UNSUP             # strided rows are fine
    assert status(f, wide[:, ::2], g, 1e-5, y=y) == SHAPE
    assert status(f, x.t(), g, 1e-5, y=y) == SHAPE
    assert status(f, x, g[:128], 1e-5, y=y) == SHAPE
    assert status(f, x, g.float(), 1e-5, y=y) == UNSUP
    assert status(f, x, g, 1e-5) == SHAPE
    assert status(f, x, g, 1e-5, y=y[:3]) == SHAPE
    assert status(f, x, g, 1e-5, q=q) == SHAPE
    assert status(f, x, g, 1e-5, q=q, scales=s.t().contiguous()) == SHAPE
    assert status(f, x, g, 1e-5, residual=x, y=y) == SHAPE
    assert status(f, x, g, 1e-5, residual=wide[:, :256], residual_out=x, y=y) == SHAPE
    assert status(f, x, g, 1e-5, residual=x[:3], residual_out=x[:3], y=y) == SHAPE


def test_fp8_binding():
    x = torch.zeros((4, 256), dtype=H)
    q, s = wq.alloc_fp8_rows(4, 256, device="cpu")
    assert status(wq.wq_quantize_fp8_rows, x, q, s) == UNSUP
    assert status(wq.wq_quantize_fp8_rows, x, q[:3], s) == SHAPE
    assert status(wq.wq_quantize_fp8_rows, x, q, s, up=x[:3]) == SHAPE
    assert status(wq.wq_quantize_fp8_rows, x, q, s, up=x.float()) == UNSUP
    w = wq.alloc_fp8(300, 256, device="cpu")
    assert w.scales.shape == (3, 2)
    assert status(wq.wq_quantize_fp8_block, torch.zeros((300, 256), dtype=H), w.codes,
                  w.scales[:2]) == SHAPE
    y = torch.zeros((4, 300), dtype=H)
    f = wq.wq_linear_fp8
    assert status(f, q, s, w, y) == UNSUP
    assert status(f, q[:, :128], s, w, y) == SHAPE
    assert status(f, q, s[:1], w, y) == SHAPE
    assert status(f, q, s, w, y[:, :299]) == SHAPE
    assert status(f, x, s, w, y) == SHAPE                              # 16-bit activations
    bad = wq.alloc_fp8(300, 256, device="cpu")
    bad.scales = bad.scales[:2]
    assert status(f, q, s, bad, y) == SHAPE


def test_moe_binding():
    x, r = torch.zeros((3, 256), dtype=H), torch.zeros((4, 256), dtype=H)
    g, u, d = (wq.alloc_int4(n, k, device="cpu") for n, k in ((512, 256), (512, 256), (1024, 128)))
    ws = torch.zeros(1024, dtype=torch.uint8)
    y = torch.zeros((3, 256), dtype=H)
    f = wq.wq_moe
    assert status(f, x, r, 2, g, u, d, y, ws) == UNSUP
    assert status(f, x, None, 2, g, u, d, y, ws) == SHAPE
    assert status(f, x, r.bfloat16(), 2, g, u, d, y, ws) == SHAPE
    assert status(f, x, r[:, :128], 2, g, u, d, y, ws) == SHAPE
    assert status(f, x, r[:3], 2, g, u, d, y, ws) == SHAPE
    assert status(f, x, r, 2, g, u, g, y, ws) == SHAPE
    assert status(f, x, r, 2, g, u, d, y[:2], ws) == SHAPE
    assert status(f, x, r, 2, g, u, d, y, None) == SHAPE
    assert status(f, x, r, 2, g, u, d, y, ws, ids=torch.zeros((3, 3), dtype=torch.int32)) == SHAPE
    assert status(f, x, None, 2, g, u, d, y, ws, logits=torch.zeros((2, 4))) == SHAPE
    assert status(f, x, None, 2, g, u, d, y, ws, logits=torch.zeros((3, 4)).double()) == UNSUP


# ------------------------------------------- types of the same size, on CPU tensors
def refusal(fn, *a, **kw):
    with pytest.raises(wq.WqError) as e:
        fn(*a, **kw)
    return e.value.status, str(e.value)


def refused_type(fn, *a, **kw):
    st, msg = refusal(fn, *a, **kw)
    return st == UNSUP and "dtype" in msg


def well_formed(fn, *a, **kw):
    st, msg = refusal(fn, *a, **kw)
    return st == UNSUP and "GPU" in msg


OTHER8 = (torch.float8_e5m2, torch.float8_e4m3fnuz, torch.int8)


def test_rows_of_other_types():
    x, g = torch.zeros((4, 256), dtype=H), torch.zeros(256, dtype=H)
    q, s = wq.alloc_fp8_rows(4, 256, device="cpu")
    for call in (lambda q, s: (wq.wq_add_rmsnorm, x, g, 1e-5, None, None, None, q, s),
                 lambda q, s: (wq.wq_quantize_fp8_rows, x, q, s)):
        assert well_formed(*call(q, s)) and well_formed(*call(q.view(torch.uint8), s))
        for dt in OTHER8:
            assert refused_type(*call(q.view(dt), s))
        assert refused_type(*call(q, s.view(torch.int32)))


def test_fp8_weights_of_other_types():
    w = wq.alloc_fp8(300, 256, device="cpu")
    w16, y = torch.zeros((300, 256), dtype=H), torch.zeros((4, 300), dtype=H)
    q, s = wq.alloc_fp8_rows(4, 256, device="cpu")
    f, pack = wq.wq_linear_fp8, wq.wq_quantize_fp8_block
    raw = wq.QuantizedWeight(wq.FMT_FP8_BLOCK, 300, 256, 128, w.codes.view(torch.uint8), w.scales)
    assert well_formed(f, q, s, w, y) and well_formed(f, q.view(torch.uint8), s, raw, y)
    assert well_formed(pack, w16, w.codes, w.scales) and well_formed(pack, w16, raw.codes, w.scales)
    assert well_formed(wq.wq_dequantize, w, w16)
    for dt in OTHER8:
        assert refused_type(f, q.view(dt), s, w, y)
        bad = wq.QuantizedWeight(wq.FMT_FP8_BLOCK, 300, 256, 128, w.codes.view(dt), w.scales)
        assert refused_type(f, q, s, bad, y) and refused_type(wq.wq_dequantize, bad, w16)
        assert refused_type(pack, w16, bad.codes, w.scales)
    bad = wq.QuantizedWeight(wq.FMT_FP8_BLOCK, 300, 256, 128, w.codes, w.scales.view(torch.int32))
    assert refused_type(f, q, s, bad, y) and refused_type(pack, w16, w.codes, bad.scales)
    assert refused_type(f, q, s.view(torch.int32), w, y)
    assert refused_type(f, q, s, w, y.view(torch.int16))
    assert status(f, q, s, w, None) == SHAPE


@pytest.mark.parametrize("fmt", ["int4", "fp8"])
def test_experts_of_other_types(fmt):
    x, r = torch.zeros((3, 256), dtype=H), torch.zeros((4, 256), dtype=H)
    alloc = wq.alloc_int4 if fmt == "int4" else wq.alloc_fp8
    g, u, d = (alloc(n, k, device="cpu") for n, k in ((512, 256), (512, 256), (1024, 128)))
    ws, y = torch.zeros(1024, dtype=torch.uint8), torch.zeros((3, 256), dtype=H)
    ids, probs = torch.zeros((3, 2), dtype=torch.int32), torch.zeros((3, 2))

    def call(**kw):
        a = dict(x=x, router=r, top_k=2, gate=g, up=u, down=d, y=y, workspace=ws, ids=ids,
                 probs=probs)
        return (lambda: wq.wq_moe(**{**a, **kw}),)

    assert well_formed(*call())
    assert refused_type(*call(ids=probs)) and refused_type(*call(probs=ids))
    for name, w in (("gate", g), ("up", u), ("down", d)):
        bad = w.clone()
        bad.scales = w.scales.view(torch.bfloat16 if fmt == "int4" else torch.int32)
        assert refused_type(*call(**{name: bad}))
        if fmt == "fp8":
            bad = w.clone()
            bad.codes = w.codes.view(torch.float8_e5m2)
            assert refused_type(*call(**{name: bad}))


@needs_lib
def test_moe_workspace_of_weights_it_does_not_take():
    """0, as the other workspace queries say for arguments that the call refuses."""
    ask = wq._load().wq_moe_workspace
    assert ask(4, 2, ctypes.byref(i4(n=512, k=256)), 4) > 0
    assert ask(4, 2, ctypes.byref(desc(n=512, k=256)), 4) > 0
    for bad in (i4(n=512, k=256, fmt=wq.FMT_NF4, zeros=None, group=64), i4(n=512, k=256, perm=P),
                i4(n=512, k=192, group=64), desc(n=512, k=272), i4(n=256, k=256)):
        assert ask(4, 2, ctypes.byref(bad), 4) == 0
