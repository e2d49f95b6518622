"""Refusals of the cache and attention entry points (CPU only): the C entry
points' argument errors, which come before any HIP call, and the binding's
shape, type and layout checks, which come before the library is called."""

import ctypes
import os
import subprocess
import sys

import pytest
import torch

import bit_quantized_linear_int4_amd as wq
from test_abi_sanitized import _build, _have_hipcc, ROOT
from test_fp8_moe_checks import ALIGN, NULL, ODD, P, SHAPE, UNSUP, WS, caller, needs_lib, status

H, BF, F8 = torch.float16, torch.bfloat16, torch.float8_e4m3fn
BIG = 1 << 34


def cache(dt=wq.F16, kv=2, d=128, page=16, pages=10, ps=16 * 2 * 128, hs=16 * 128, ts=128, k=P,
          v=P, ks=None, vs=None):
    return wq._Cache(dt, kv, d, page, pages, ps, hs, ts, k, v, ks, vs)


# every call's cache argument is checked the same way
BAD_CACHES = [
    (NULL, dict(k=None)), (NULL, dict(v=None)), (NULL, dict(dt=wq.E4M3)),
    (NULL, dict(dt=wq.E4M3, ks=P)), (UNSUP, dict(ks=P, vs=P)), (UNSUP, dict(vs=P)),
    (UNSUP, dict(dt=wq.F32)), (UNSUP, dict(dt=9)), (UNSUP, dict(d=96)), (UNSUP, dict(d=256)),
    (SHAPE, dict(kv=0)), (SHAPE, dict(kv=2000, hs=16 * 128, ps=1 << 23)), (SHAPE, dict(pages=0)),
    (SHAPE, dict(page=0)), (SHAPE, dict(page=24)), (SHAPE, dict(page=1 << 17)),
    (SHAPE, dict(pages=1 << 27)), (SHAPE, dict(pages=1 << 40)),
    (SHAPE, dict(ts=127)), (SHAPE, dict(ts=132)), (SHAPE, dict(hs=15 * 128)),
    (SHAPE, dict(ps=31 * 128)), (SHAPE, dict(ps=0)), (SHAPE, dict(hs=-128)),
    (SHAPE, dict(ps=1 << 62)), (SHAPE, dict(ps=BIG // 9 + 8 - BIG // 9 % 8)),
    (SHAPE, dict(dt=wq.E4M3, ks=P, vs=P, ts=136, hs=16 * 136, ps=32 * 136)),
    (ALIGN, dict(k=P + 8)), (ALIGN, dict(v=P + 8)), (ALIGN, dict(dt=wq.E4M3, ks=ODD, vs=P)),
    (ALIGN, dict(dt=wq.E4M3, ks=P, vs=P + 2)),
]


def append():
    return caller(wq._load().wq_append_kv, q=P, k=P, v=P, dt=wq.F16, m=4, heads=4, ldq=512,
                  ldk=256, ldv=256, positions=P, cos_sin=P, max_pos=100, rot=128, interleaved=0,
                  q_out=P, ldo=512, slots=P, cache=ctypes.byref(cache()), stream=None)


def decode(**more):
    return caller(wq._load().wq_attention_decode, **{**dict(
        q=P, dt=wq.F16, m=4, heads=4, ldq=512, cache=ctypes.byref(cache()), pages=P, max_pages=3,
        ldp=3, lens=P, scale=0.1, window=0, sinks=0, y=P, lse=P, ws=P, ws_bytes=1 << 40,
        stream=None), **more})


def prompt(**more):
    return caller(wq._load().wq_attention_prompt, **{**dict(
        q=P, dt=wq.F16, m=40, heads=4, ldq=512, starts=P, batch=4, cache=ctypes.byref(cache()),
        pages=P, max_pages=3, ldp=3, lens=P, scale=0.1, window=0, sinks=0, y=P, lse=P, ws=P,
        ws_bytes=1 << 40, stream=None), **more})


@needs_lib
@pytest.mark.parametrize("i", range(len(BAD_CACHES)))
def test_bad_caches(i):
    want, kw = BAD_CACHES[i]
    for call in (append(), decode(), prompt()):
        assert call(cache=ctypes.byref(cache(**kw))) == want
    lib = wq._load()
    assert lib.wq_attention_decode_workspace(4, 4, ctypes.byref(cache(**kw))) == 0
    assert lib.wq_attention_prompt_workspace(4, 4, 2, ctypes.byref(cache(**kw))) == 0


@needs_lib
def test_append_errors():
    call = append()
    assert call(k=None) == NULL and call(v=None) == NULL and call(slots=None) == NULL
    assert call(q=None) == NULL and call(q_out=None) == NULL and call(cache=None) == NULL
    assert call(positions=None) == NULL and call(cos_sin=None) == NULL
    assert call(dt=wq.F32) == UNSUP and call(dt=wq.E4M3) == UNSUP and call(dt=wq.BF16) == UNSUP
    assert call(interleaved=2) == UNSUP
    assert call(rot=-16) == SHAPE and call(rot=8) == SHAPE and call(rot=144) == SHAPE
    assert call(max_pos=0) == SHAPE and call(max_pos=1 << 31) == SHAPE
    assert call(m=0) == SHAPE and call(m=1 << 23) == SHAPE
    assert call(heads=0) == SHAPE and call(heads=1025, ldq=1025 * 128, ldo=1025 * 128) == SHAPE
    for ld in ("ldq", "ldo"):
        assert call(**{ld: 504}) == SHAPE and call(**{ld: 516}) == SHAPE
        assert call(**{ld: 1 << 23}) == SHAPE
    for ld in ("ldk", "ldv"):
        assert call(**{ld: 248}) == SHAPE and call(**{ld: 260}) == SHAPE
    for p in ("q", "k", "v", "q_out", "cos_sin"):
        assert call(**{p: P + 8}) == ALIGN
    assert call(positions=P + 2) == ALIGN and call(slots=ODD) == ALIGN


@needs_lib
@pytest.mark.parametrize("make", [decode, prompt])
def test_attention_errors(make):
    call = make()
    for p in ("q", "cache", "pages", "lens", "y"):
        assert call(**{p: None}) == NULL
    assert call(dt=wq.F32) == UNSUP and call(dt=wq.E4M3) == UNSUP and call(dt=wq.BF16) == UNSUP
    assert call(heads=0) == SHAPE and call(heads=5, ldq=640) == SHAPE
    assert call(heads=1026, ldq=1026 * 128) == SHAPE
    assert call(m=0) == SHAPE and call(m=1 << 23) == SHAPE
    assert call(ldq=504) == SHAPE and call(ldq=516) == SHAPE and call(ldq=1 << 23) == SHAPE
    assert call(max_pages=0) == SHAPE and call(max_pages=4) == SHAPE
    assert call(max_pages=1 << 23, ldp=1 << 23) == SHAPE and call(ldp=1 << 23) == SHAPE
    wide = dict(cache=ctypes.byref(cache(page=1024, ps=1024 * 256, hs=1024 * 128)))
    assert call(**wide, max_pages=(1 << 20) + 1, ldp=(1 << 20) + 1) == SHAPE
    for s in (0.0, -0.1, float("nan"), float("inf")):
        assert call(scale=s) == SHAPE
    assert call(window=-1) == SHAPE and call(sinks=-1) == SHAPE
    assert call(q=P + 8) == ALIGN and call(y=P + 8) == ALIGN
    assert call(pages=P + 2) == ALIGN and call(lens=ODD) == ALIGN and call(lse=P + 2) == ALIGN


@needs_lib
def test_prompt_errors():
    call = prompt()
    assert call(starts=None) == NULL and call(starts=P + 2) == ALIGN
    assert call(batch=0) == SHAPE and call(batch=1 << 23) == SHAPE
    many = dict(m=1 << 22, batch=1 << 22)
    assert call(**many) == SHAPE
    assert wq._load().wq_attention_prompt_workspace(1 << 22, 4, 1 << 22, ctypes.byref(cache())) == 0


@needs_lib
@pytest.mark.parametrize("d,kv,heads", [(128, 8, 32), (64, 1, 71), (128, 32, 32)])
@pytest.mark.parametrize("m", [1, 7, 300])
def test_workspaces(d, kv, heads, m):
    lib = wq._load()
    c = ctypes.byref(cache(d=d, kv=kv, ts=d, hs=16 * d, ps=16 * kv * d))
    big = dict(m=m, heads=heads, ldq=heads * d, cache=c)
    for make, need in ((decode, lib.wq_attention_decode_workspace(m, heads, c)),
                       (prompt, lib.wq_attention_prompt_workspace(m, heads, 1, c))):
        assert need <= 128 << 20
        if need:
            call = make(**big)
            assert call(ws=None) == WS and call(ws_bytes=need - 1) == WS
            assert call(ws=P + 128, ws_bytes=need) == ALIGN
    assert lib.wq_attention_decode_workspace(0, heads, c) == 0
    assert lib.wq_attention_decode_workspace(m, kv * 1025, c) == 0
    assert lib.wq_attention_prompt_workspace(m, heads, 0, c) == 0


@needs_lib
@pytest.mark.parametrize("d,kv,heads", [(128, 8, 32), (64, 1, 71), (128, 32, 32), (64, 200, 200)])
def test_workspaces_suffice_for_fewer_rows(d, kv, heads):
    lib = wq._load()
    c = ctypes.byref(cache(d=d, kv=kv, ts=d, hs=16 * d, ps=16 * kv * d))
    for need in (lambda m, b: lib.wq_attention_decode_workspace(m, heads, c),
                 lambda m, b: lib.wq_attention_prompt_workspace(m, heads, b, c)):
        last = 0
        for m in list(range(1, 130)) + [300, 1000, 4096, 20000]:
            assert need(m, 1) == need(m, 3) == need(m, 1000) >= last
            last = need(m, 1)


# ------------------------------------------------------------ binding, CPU tensors
def refused_type(fn, *a, **kw):
    with pytest.raises(wq.WqError) as e:
        fn(*a, **kw)
    return e.value.status == UNSUP and "dtype" in str(e.value)


def test_cache_binding():
    k = torch.zeros((3, 2, 16, 64), dtype=H)
    s = torch.zeros((3, 2, 16))
    c = wq.KVCache(k, k.clone())
    assert c.shape == (3, 2, 16, 64) and c.nbytes() == 2 * k.nbytes
    t = torch.zeros((3, 16, 2, 64), dtype=H).transpose(1, 2)             # tokens outermost
    c = wq.KVCache(t, torch.zeros((3, 16, 2, 64), dtype=H).transpose(1, 2))
    assert (c._desc.head_stride, c._desc.token_stride) == (64, 128)
    both = torch.zeros((3, 2, 2, 16, 64), dtype=H)                       # k and v in one tensor
    assert wq.KVCache(both[:, 0], both[:, 1])._desc.page_stride == 2 * 2 * 16 * 64
    assert status(wq.KVCache, k, t) == SHAPE                             # strides differ
    assert status(wq.KVCache, k, k[:2]) == SHAPE and status(wq.KVCache, k, None) == SHAPE
    assert status(wq.KVCache, None, k) == SHAPE and status(wq.KVCache, k[0], k[0]) == SHAPE
    assert status(wq.KVCache, k, k.bfloat16()) == SHAPE
    assert refused_type(wq.KVCache, k.float(), k.float())
    assert status(wq.KVCache, k[..., ::2], k[..., ::2]) == SHAPE
    assert status(wq.KVCache, k, k, s, s) == UNSUP
    f = k.to(F8)
    assert wq.KVCache(f, f, s, s).shape == k.shape
    assert wq.KVCache(f.view(torch.uint8), f.view(torch.uint8), s, s)._desc.dt == wq.E4M3
    assert status(wq.KVCache, f, f) == SHAPE and status(wq.KVCache, f, f, s, s[:2]) == SHAPE
    assert refused_type(wq.KVCache, f, f, s, s.int())
    assert refused_type(wq.KVCache, f.view(torch.float8_e5m2), f.view(torch.float8_e5m2), s, s)
    a = wq.alloc_kv_cache(5, 2, 32, 64, F8, "cpu")
    assert a.shape == (5, 2, 32, 64) and a.k_scales.shape == (5, 2, 32)
    assert wq.alloc_kv_cache(5, 2, 32, 64, BF, "cpu").k_scales is None


def test_append_binding():
    c = wq.alloc_kv_cache(5, 2, 16, 64, H, "cpu")
    qkv = torch.zeros((7, 8, 64), dtype=H)
    q, k, v, out = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], torch.zeros((7, 4, 64), dtype=H)
    slots, pos, t = torch.zeros(7, dtype=torch.int32), torch.zeros(7, dtype=torch.int32), torch.zeros((9, 64))

    def st(**kw):
        a = dict(q=q, k=k, v=v, cache=c, slots=slots, positions=pos, cos_sin=t, q_out=out)
        return status(lambda: wq.wq_append_kv(**{**a, **kw}))

    def bad_type(**kw):
        a = dict(q=q, k=k, v=v, cache=c, slots=slots, positions=pos, cos_sin=t, q_out=out)
        return refused_type(lambda: wq.wq_append_kv(**{**a, **kw}))

    assert st() == UNSUP and st(q=None, q_out=None) == UNSUP             # well formed, not on a GPU
    assert st(positions=None, cos_sin=None) == UNSUP and st(q_out=q) == UNSUP
    assert st(k=None) == SHAPE and st(v=None) == SHAPE and st(q=None) == SHAPE
    assert st(q_out=None) == SHAPE and st(slots=None) == SHAPE
    assert st(cos_sin=None) == SHAPE and st(positions=None) == SHAPE
    assert st(k=k[:6]) == SHAPE and st(v=v[:, :1]) == SHAPE and st(k=q) == SHAPE
    assert st(q=q[:6]) == SHAPE and st(q_out=out[:, :3]) == SHAPE and st(slots=slots[:6]) == SHAPE
    assert st(positions=pos[:6]) == SHAPE and st(cos_sin=t[0]) == SHAPE
    assert st(cos_sin=t.t()) == SHAPE and st(k=k[..., :32]) == SHAPE
    assert st(k=qkv[:, 0:4:2]) == SHAPE and st(k=qkv.flatten(1)) == SHAPE
    assert st(k=k.transpose(0, 1).contiguous().transpose(0, 1)) == SHAPE
    # another size of integer is refused for its bytes, another type of that size for itself
    assert st(slots=slots.long()) == SHAPE and bad_type(slots=slots.float())
    assert st(positions=pos.long()) == SHAPE and bad_type(positions=pos.float())
    assert st(cos_sin=t.double()) == SHAPE and bad_type(cos_sin=t.int())
    assert bad_type(v=v.bfloat16()) and bad_type(q=q.bfloat16())
    assert bad_type(q_out=out.float())


@pytest.mark.parametrize("fn", ["decode", "prompt"])
def test_attention_binding(fn):
    c = wq.alloc_kv_cache(5, 2, 16, 64, H, "cpu")
    q, y = torch.zeros((3, 4, 64), dtype=H), torch.zeros((3, 4, 64), dtype=H)
    pages, lens = torch.zeros((3, 6), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    starts = torch.arange(4, dtype=torch.int32)
    base = dict(q=q, cache=c, pages=pages, lens=lens, y=y, workspace=torch.zeros(8))
    if fn == "prompt":
        base["starts"] = starts
    call = {"decode": wq.wq_attention_decode, "prompt": wq.wq_attention_prompt}[fn]

    def st(**kw):
        return status(lambda: call(**{**base, **kw}))

    def bad_type(**kw):
        return refused_type(lambda: call(**{**base, **kw}))

    assert st() == UNSUP and st(workspace=None) == UNSUP and st(lse=torch.zeros((3, 4))) == UNSUP
    wide = torch.zeros((3, 9), dtype=torch.int32)
    assert st(pages=wide[:, :6]) == UNSUP                                # rows apart are fine
    qkv = torch.zeros((3, 8, 64), dtype=H)
    assert st(q=qkv[:, :4]) == UNSUP
    assert st(q=None) == SHAPE and st(y=None) == SHAPE and st(pages=None) == SHAPE
    assert st(lens=None) == SHAPE and st(pages=pages[0]) == SHAPE and st(pages=pages[:2]) == SHAPE
    assert st(pages=wide[:, ::2]) == SHAPE and st(lens=lens[:2]) == SHAPE
    assert st(y=y[:2]) == SHAPE and st(y=qkv[:, :4]) == SHAPE and st(q=q[..., :32]) == SHAPE
    assert st(q=q.flatten(1)) == SHAPE and st(lse=torch.zeros((3, 3))) == SHAPE
    assert bad_type(pages=pages.long()) and st(lens=lens.long()) == SHAPE
    assert bad_type(lens=lens.float())
    assert bad_type(y=y.bfloat16()) and bad_type(lse=torch.zeros((3, 4), dtype=torch.int32))
    assert st(q=q.float(), y=y.float()) == UNSUP
    if fn == "prompt":
        assert st(starts=None) == SHAPE and st(starts=starts[:1]) == SHAPE
        assert st(starts=starts[:3]) == SHAPE and bad_type(starts=starts.float())
        # sequences and rows need not be equal in number
        assert st(starts=starts[:3], pages=pages[:2], lens=lens[:2]) == UNSUP


@pytest.mark.skipif(not _have_hipcc(), reason="hipcc not available")
def test_checks_clean_under_asan_and_ubsan():
    if "WQ_LIBRARY" in os.environ:
        pytest.skip("already under the sanitizers")
    env = dict(os.environ)
    env.update({
        "WQ_LIBRARY": _build.build_host_sanitized(),
        "LD_PRELOAD": _build.sanitizer_runtime(),
        "ASAN_OPTIONS": "detect_leaks=0:halt_on_error=1",
        "UBSAN_OPTIONS": "halt_on_error=1:print_stacktrace=1",
    })
    r = subprocess.run(
        [sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "not gpu",
         os.path.join(ROOT, "tests", "test_attention_checks.py"), "-k", "not asan"],
        cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert " passed" in out and "skipped" not in out
