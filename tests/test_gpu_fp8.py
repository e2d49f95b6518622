"""RMS norm, FP8 packers and FP8 linear on the GPU against the fp64 oracle.

Tolerances, from the number formats and the order of the fp32 sums:
  * scales and codes of given values: equal to the oracle's bit for bit;
  * norm: a thread adds ceil(k / 256) squares in turn, then a tree of at most
    about 10 levels; with the square root halving the relative error and four
    more roundings, |dv| <= (k / 256 + 40) 2^-24 |v|;
  * silu: the hardware exponential's argument x * log2(e) is rounded, which
    costs |x| 2^-24 of the result, and a few roundings: for |x| <= 16 below
    2^-19 |v|;
  * a code of a value known to d: half an E4M3 step (|v| / 16, or 2^-10 of
    the scale for small values) plus d;
  * linear, fp32 y: every product is exact, an instruction chain adds 128 of
    them and the blocks are added in turn, so |dy| <= (kb + 16) 2^-23 S with S
    the sum of the magnitudes; 16-bit y: the FP8 instruction keeps 2^-16 of the
    largest product over at most 16 partial sums, |dy| <= 2^-12 S, plus the
    rounding of y.
"""

import numpy as np
import pytest
import torch

import bit_quantized_linear_int4_amd as wq
from gpu_util import say
from oracle import fp8

pytestmark = pytest.mark.gpu

TD = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ULP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -25, "bf16": 0.0, "f32": 0.0}      # half a subnormal step


def rand(shape, seed, dtype, scale=1.0, outliers=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * scale
    if outliers:
        at = torch.randperm(shape[-1], generator=g)[:outliers]
        x[..., at] *= 30
    return x.to(TD[dtype])


def bits(t):
    return t.detach().cpu().view(torch.uint8).numpy()


def check_codes(q, s, v, tol):
    """Codes and scales of values known to a relative `tol` each."""
    m, k = v.shape
    kb = -(-k // 128)
    s, code = s.cpu().numpy().astype(np.float64), fp8.decode(bits(q))
    pad = np.zeros((m, kb * 128))
    pad[:, :k] = np.abs(v)
    ref = pad.reshape(m, kb, 128).max(-1).T / 448
    ref = np.where(ref == 0, 1.0, np.maximum(ref, 2.0 ** -126))
    assert np.all(np.abs(s - ref) <= (tol + 2.0 ** -23) * ref)
    full = np.repeat(s.T, 128, axis=1)[:, :k]
    half = np.maximum(np.abs(v) / 16, full * 2.0 ** -10) * (1 + 1e-4)
    assert np.all(np.abs(code * full - v) <= half + 2 * tol * np.abs(v))


# ------------------------------------------------------------------- norm
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,k", [(1, 8), (1, 4096), (3, 136), (5, 2056), (16, 128), (7, 5008),
                                 (2, 8200), (3, 16392), (2, 40000), (2055, 264), (4100, 1024)])
def test_norm(m, k, dtype):
    say(f"norm m={m} k={k} {dtype}")
    x, r = rand((m, k), 1, dtype, outliers=2).cuda(), rand((m, k), 2, dtype, 3.0).cuda()
    g = (1 + 0.2 * rand((k,), 3, "f32")).to(TD[dtype]).cuda()
    tol = (k / 256 + 40) * 2.0 ** -24
    for res in (None, r):
        out = torch.full_like(x, float("nan")) if res is not None else None
        y = torch.full_like(x, float("nan"))
        q, s = wq.alloc_fp8_rows(m, k)
        wq.wq_add_rmsnorm(x, g, 1e-5, residual=res, residual_out=out, y=y, q=q, scales=s)
        torch.cuda.synchronize()
        _, v = fp8.add_rmsnorm(x.double().cpu().numpy(), g.double().cpu().numpy(), 1e-5,
                               None if res is None else res.double().cpu().numpy())
        if res is not None:
            assert torch.equal(out, (x.float() + res.float()).to(x.dtype))
        err = np.abs(y.double().cpu().numpy() - v)
        assert np.all(err <= (ULP[dtype] * (1 + 1e-3) + tol) * np.abs(v) + TINY[dtype])
        check_codes(q, s, v, tol)
        # each output alone gives the same bits
        y2 = torch.empty_like(x)
        wq.wq_add_rmsnorm(x, g, 1e-5, residual=res,
                          residual_out=None if res is None else torch.empty_like(x), y=y2)
        q2, s2 = wq.alloc_fp8_rows(m, k)
        wq.wq_add_rmsnorm(x, g, 1e-5, residual=res,
                          residual_out=None if res is None else torch.empty_like(x), q=q2,
                          scales=s2)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(s, s2) and np.array_equal(bits(q), bits(q2))


@pytest.mark.parametrize("k", [512, 40000])
def test_norm_strides_and_in_place(k):
    m, dtype = 6, "bf16"
    big, rbig = rand((m, k + 24), 4, dtype).cuda(), rand((m, 2 * k), 5, dtype).cuda()
    g = rand((k,), 6, dtype).cuda()
    x, r = big[:, 8:8 + k], rbig[:, k:]
    ref_y, ref_out = torch.empty((m, k), dtype=TD[dtype], device="cuda"), torch.empty(
        (m, k), dtype=TD[dtype], device="cuda")
    wq.wq_add_rmsnorm(x.contiguous(), g, 1e-6, residual=r.contiguous(), residual_out=ref_out,
                      y=ref_y)
    y = torch.empty_like(ref_y)
    left, rest = rbig[:, :k].clone(), torch.cat((big[:, :8], big[:, 8 + k:]), 1)
    wq.wq_add_rmsnorm(x, g, 1e-6, residual=r, residual_out=r, y=y)           # in place, strided
    torch.cuda.synchronize()
    assert torch.equal(y, ref_y) and torch.equal(r, ref_out) and torch.equal(rbig[:, :k], left)
    assert torch.equal(torch.cat((big[:, :8], big[:, 8 + k:]), 1), rest)
    # into x
    xc, rc = big[:, 8:8 + k].contiguous(), rand((m, 2 * k), 5, dtype).cuda()[:, k:].contiguous()
    wq.wq_add_rmsnorm(xc, g, 1e-6, residual=rc, residual_out=xc, y=y)
    torch.cuda.synchronize()
    assert torch.equal(xc, ref_out) and torch.equal(y, ref_y)


def test_norm_zeros_and_non_finite_rows():
    m, k = 8, 512
    x = rand((m, k), 7, "bf16").cuda()
    g = torch.ones(k, dtype=torch.bfloat16, device="cuda")
    y0, (q0, s0) = torch.empty_like(x), wq.alloc_fp8_rows(m, k)
    wq.wq_add_rmsnorm(x, g, 1e-5, y=y0, q=q0, scales=s0)
    x[1] = 0
    x[3, 130] = float("nan")
    x[5, 7] = float("inf")
    y, (q, s) = torch.empty_like(x), wq.alloc_fp8_rows(m, k)
    wq.wq_add_rmsnorm(x, g, 1e-5, y=y, q=q, scales=s)
    torch.cuda.synchronize()
    assert not y[1].any() and not bits(q)[1].any() and bool((s[:, 1] == 1).all())
    assert bool(y[3].isnan().all()) and bool(s[:, 3].isnan().all())
    assert bool(y[5, 7].isnan()) and int(y[5].isnan().sum()) == 1 and bool(s[0, 5].isnan())
    keep = [0, 2, 4, 6, 7]
    assert torch.equal(y[keep], y0[keep]) and torch.equal(s[:, keep], s0[:, keep])
    assert np.array_equal(bits(q)[keep], bits(q0)[keep])


# ---------------------------------------------------------------- packers
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,k", [(1, 8), (1, 4096), (2, 24), (3, 1032), (4, 512), (15, 264),
                                 (16, 2048), (33, 5000), (250, 136)])
def test_rows(m, k, dtype):
    say(f"rows m={m} k={k} {dtype}")
    x = rand((m, k), 11, dtype, outliers=1)
    x[0, :8] = 0
    x[-1] *= 1e-6
    if k > 256:
        x[m // 2, 128:256] = 0
    q, s = wq.alloc_fp8_rows(m, k)
    wq.wq_quantize_fp8_rows(x.cuda(), q, s)
    torch.cuda.synchronize()
    codes, scales = fp8.quantize_rows(x.float().numpy())
    assert np.array_equal(s.cpu().numpy(), scales) and np.array_equal(bits(q), codes)
    up = rand((m, k), 12, dtype)
    x = (rand((m, k), 13, dtype) * 3).clamp(-16, 16)
    wq.wq_quantize_fp8_rows(x.cuda(), q, s, up=up.cuda())
    torch.cuda.synchronize()
    check_codes(q, s, fp8.silu_product(x.double().numpy(), up.double().numpy()), 2.0 ** -19)


def test_rows_extremes():
    """Subnormal blocks, exact halves, silu limits, values that are not finite."""
    x = torch.zeros((2, 640), dtype=torch.bfloat16)
    x[0, 0], x[0, 1] = 1e-38, -1e-40                          # scale held at 2^-126
    x[0, 128:131] = torch.tensor([448.0, 26.0, 27.0])         # scale 1; 27 is half-way
    x[0, 256] = float("inf")
    x[0, 384], x[0, 385] = float("nan"), 1.0
    x[1, :3] = torch.tensor([3e38, -3e38, 1.0])
    q, s = wq.alloc_fp8_rows(2, 640)
    wq.wq_quantize_fp8_rows(x.cuda(), q, s)
    torch.cuda.synchronize()
    sc, c = s.cpu(), fp8.decode(bits(q))
    fin = x.clone()
    fin[0, 256:512] = 0
    codes, scales = fp8.quantize_rows(fin.float().numpy())
    at = [0, 1, 4]
    assert np.array_equal(sc.numpy()[at], scales[at])
    assert np.array_equal(bits(q)[:, :256], codes[:, :256])
    assert np.isinf(sc[2, 0].item()) and np.isnan(c[0, 256]) and c[0, 257] == 0
    assert np.isnan(sc[3, 0].item()) and np.isnan(c[0, 384:512]).all()
    x = torch.tensor([[-30000.0, -100.0, 0.0, 100.0, 30000.0, -0.5, 0.5, 1.0]], dtype=torch.float16)
    up = torch.full((1, 8), 0.5, dtype=torch.float16)
    q, s = wq.alloc_fp8_rows(1, 8)
    wq.wq_quantize_fp8_rows(x.cuda(), q, s, up=up.cuda())
    torch.cuda.synchronize()
    got = fp8.decode(bits(q)) * s.cpu().numpy()[0, 0]
    # the scale 15000 / 448 is rounded once
    assert abs(got[0, 4] - 15000) <= 15000 * 2.0 ** -23 and not got[0, :3].any()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n,k", [(1, 16), (128, 128), (200, 144), (384, 272), (130, 4096)])
def test_block(n, k, dtype):
    w = rand((n, k), 21, dtype, 0.02)
    w[0, 0] = 3
    if n > 128:
        w[128:] = 0
    qw = wq.alloc_fp8(n, k)
    wq.wq_quantize_fp8_block(w.cuda(), qw.codes, qw.scales)
    out = torch.empty((n, k), dtype=TD[dtype], device="cuda")
    wq.wq_dequantize(qw, out)
    torch.cuda.synchronize()
    codes, scales = fp8.quantize_block(w.float().numpy())
    assert np.array_equal(qw.scales.cpu().numpy(), scales) and np.array_equal(bits(qw.codes), codes)
    prod = (fp8.decode(codes).astype(np.float32)
            * np.repeat(np.repeat(scales, 128, 0)[:n], 128, 1)[:, :k])
    assert torch.equal(out.cpu(), torch.from_numpy(prod).to(TD[dtype]))


# ----------------------------------------------------------------- linear
def make_linear(m, n, k, seed):
    q, s = wq.alloc_fp8_rows(m, k)
    wq.wq_quantize_fp8_rows(rand((m, k), seed, "bf16", outliers=min(3, k)).cuda(), q, s)
    w = wq.alloc_fp8(n, k)
    wq.wq_quantize_fp8_block(rand((n, k), seed + 1, "bf16", 0.02).cuda(), w.codes, w.scales)
    return q, s, w


def reference(q, s, w):
    """fp64 y and the sums of magnitudes."""
    n, k = w.n, w.k
    x = q.double() * s.double().t().repeat_interleave(128, 1)[:, :k]
    e = w.scales.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    wd = w.codes.double() * e
    return x @ wd.t().contiguous(), x.abs() @ wd.abs().t().contiguous()


def linear(q, s, w, ydt, stream=None):
    y = torch.full((q.shape[0], w.n), float("nan"), dtype=TD[ydt], device="cuda")
    need = wq.wq_linear_fp8_workspace(q.shape[0], w)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") if need else None
    wq.wq_linear_fp8(q, s, w, y, ws, stream=stream)
    return y


def check_linear(y, q, s, w, ydt):
    ref, mag = reference(q, s, w)
    kb = -(-w.k // 128)
    tol = ((kb + 16) * 2.0 ** -23 if ydt == "f32" else 2.0 ** -12) * mag
    err = (y.double() - ref).abs()
    assert bool((err <= tol + ULP[ydt] * (1 + 1e-3) * (ref.abs() + tol) + TINY[ydt]).all()), (
        f"worst {float((err / (tol + 1e-300)).max()):.3g} of the bound")


SHAPES = [(1, 128, 16), (1, 16, 128), (1, 4096, 4096), (2, 300, 144), (5, 1, 400), (16, 515, 2064),
          (16, 100, 128), (17, 129, 272), (31, 4096, 1024), (64, 200, 8192), (65, 257, 16),
          (129, 256, 400), (300, 513, 1040), (333, 640, 4112), (512, 1030, 256)]


@pytest.mark.parametrize("ydt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_linear(m, n, k, ydt):
    say(f"fp8 linear m={m} n={n} k={k} y={ydt}")
    q, s, w = make_linear(m, n, k, 31)
    y = linear(q, s, w, ydt)
    torch.cuda.synchronize()
    check_linear(y, q, s, w, ydt)
    again = linear(q, s, w, ydt)
    torch.cuda.synchronize()
    assert torch.equal(y, again)


@pytest.mark.parametrize("ydt", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(3200, 4100, 272), (4095, 4097, 144), (2304, 6400, 1152)])
def test_linear_large_tiles(m, n, k, ydt):
    say(f"fp8 linear m={m} n={n} k={k} y={ydt}")
    q, s, w = make_linear(m, n, k, 33)
    y = linear(q, s, w, ydt)
    torch.cuda.synchronize()
    check_linear(y, q, s, w, ydt)


@pytest.mark.parametrize("m", [4, 40, 200])
def test_linear_nan_stays_in_its_row(m):
    q, s, w = make_linear(m, 300, 272, 35)
    y0 = linear(q, s, w, "bf16")
    q.view(torch.uint8)[m // 2, 270] = 0x7F
    w.codes.view(torch.uint8)[299, 5] = 0xFF
    y = linear(q, s, w, "bf16")
    torch.cuda.synchronize()
    bad = y.isnan()
    assert bool(bad[m // 2].all()) and bool(bad[:, 299].all())
    assert int(bad.sum()) == 300 + m - 1
    assert torch.equal(y[~bad], y0[~bad])


def test_streams_and_graph():
    """The norm, packer and products on a stream of their own and replayed from
    a graph, with other work between the replays."""
    say("fp8: stream and graph replay")
    m, n, k = 100, 512, 4096
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        x, r = rand((m, k), 41, "bf16").cuda(), rand((m, k), 42, "bf16").cuda()
        g = rand((k,), 43, "bf16").cuda()
        _, _, w = make_linear(1, n, k, 44)
        _, _, w2 = make_linear(1, 256, n, 46)
        q, s = wq.alloc_fp8_rows(m, k)
        q2, s2 = wq.alloc_fp8_rows(m, n)
        out = torch.empty_like(x)
        y = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
        z = torch.empty((m, 256), dtype=torch.float32, device="cuda")
        need = max(wq.wq_linear_fp8_workspace(m, w), wq.wq_linear_fp8_workspace(m, w2))
        assert need > 0
        ws = torch.empty((need,), dtype=torch.uint8, device="cuda")

        def calls():
            wq.wq_add_rmsnorm(x, g, 1e-5, residual=r, residual_out=out, q=q, scales=s)
            wq.wq_linear_fp8(q, s, w, y, ws)
            wq.wq_quantize_fp8_rows(y, q2, s2, up=y)
            wq.wq_linear_fp8(q2, s2, w2, z, ws)

        calls()
        st.synchronize()
        ref = [t.clone() for t in (out, y, z, s, s2)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            calls()
        for _ in range(3):
            for t in (out, y, z, s, s2, ws):
                t.zero_()
            st.synchronize()
            graph.replay()
            st.synchronize()
            assert all(torch.equal(a, b) for a, b in zip((out, y, z, s, s2), ref))
            linear(q, s, w, "f32")
            st.synchronize()


# more tiles than CUs, whole and cut tiles, one block of k, tiles of 128 tokens
# after the last whole round and without one
@pytest.mark.parametrize("m,n,k", [(4096, 5120, 256), (4100, 8196, 128), (2048, 4096, 400),
                                   (8192, 4224, 384)])
def test_linear_many_tiles(m, n, k):
    say(f"fp8 linear m={m} n={n} k={k}")
    q, s, w = make_linear(m, n, k, 37)
    # a tile whose results are not finite leaves the next one of its workgroup alone
    q.view(torch.uint8)[3, k - 1] = 0x7F
    y = linear(q, s, w, "bf16")
    torch.cuda.synchronize()
    assert bool(y[3].isnan().all())
    q.view(torch.uint8)[3, k - 1] = 0
    y[3] = linear(q, s, w, "bf16")[3]
    torch.cuda.synchronize()
    check_linear(y, q, s, w, "bf16")


# tiles of 64 and of 128 tokens, whole and split over k, cut at every side
@pytest.mark.parametrize("ydt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(40, 12301, 400), (64, 8201, 272), (33, 515, 1040),
                                   (49, 4200, 656), (65, 130, 2048),
                                   (150, 1000, 4112), (300, 8000, 208), (1000, 4000, 1296)])
def test_linear_tiles(m, n, k, ydt):
    say(f"fp8 linear m={m} n={n} k={k} y={ydt}")
    q, s, w = make_linear(m, n, k, 39)
    y = linear(q, s, w, ydt)
    torch.cuda.synchronize()
    check_linear(y, q, s, w, ydt)
    assert torch.equal(y, linear(q, s, w, ydt))


def test_linear_more_blocks_than_a_wave_has_lanes():
    """k of 70 blocks: the weight scales come 64 at a time."""
    for m, ydt in ((100, "bf16"), (200, "f32"), (1, "f32"), (4100, "f16")):
        q, s, w = make_linear(m, 4200 if m > 1000 else 136, 8832, 47)
        y = linear(q, s, w, ydt)
        torch.cuda.synchronize()
        check_linear(y, q, s, w, ydt)


# rows of every workgroup size, few and many of them
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,k", [(3, 512), (3, 1544), (600, 1544), (513, 2600), (515, 8000),
                                 (514, 4104), (512, 4096), (2, 8192), (520, 9000)])
def test_norm_sizes(m, k, dtype):
    say(f"norm m={m} k={k} {dtype}")
    x, r = rand((m, k), 51, dtype, outliers=2).cuda(), rand((m, k), 52, dtype, 3.0).cuda()
    g = (1 + 0.2 * rand((k,), 53, "f32")).to(TD[dtype]).cuda()
    tol = (k / 256 + 40) * 2.0 ** -24
    out, y = torch.empty_like(x), torch.empty_like(x)
    q, s = wq.alloc_fp8_rows(m, k)
    wq.wq_add_rmsnorm(x, g, 1e-5, residual=r, residual_out=out, y=y, q=q, scales=s)
    torch.cuda.synchronize()
    _, v = fp8.add_rmsnorm(x.double().cpu().numpy(), g.double().cpu().numpy(), 1e-5,
                           r.double().cpu().numpy())
    assert torch.equal(out, (x.float() + r.float()).to(x.dtype))
    err = np.abs(y.double().cpu().numpy() - v)
    assert np.all(err <= (ULP[dtype] * (1 + 1e-3) + tol) * np.abs(v) + TINY[dtype])
    check_codes(q, s, v, tol)


def quotient_rows(dtype, seed):
    """A row of 128 for each 16-bit mantissa of the largest value, with values
    whose quotient by the scale is next to a midpoint of two codes in front, at
    many magnitudes of the whole row."""
    mant, exps = {"f16": (1024, (-12, -3, 0, 7)), "bf16": (128, (-130, -122, -80, -64, 0, 60, 119))}[
        dtype]
    lat = np.concatenate([(1 + np.arange(mant) / mant) * 2.0 ** -e for e in range(10)])
    lat = lat.astype(np.float32)
    r = np.random.default_rng(seed)
    rows = []
    for a in (1 + np.arange(mant) / mant).astype(np.float32):
        s = np.float32(a / np.float32(448))
        v = lat[lat <= a]
        hard = v[fp8.encode(v * (np.float32(1) / s)) != fp8.encode(v / s)][:60]
        row = np.concatenate([[a], hard, -hard, r.choice(v, 128)])[:128]
        rows += [row * np.float32(2.0 ** e) for e in exps]
    return torch.from_numpy(np.array(rows, np.float32)).to(TD[dtype])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_codes_are_of_the_quotient(dtype):
    say(f"codes of the fp32 quotient, {dtype}")
    x = quotient_rows(dtype, 14)
    m, k = x.shape
    codes, scales = fp8.quantize_rows(x.float().numpy())
    # the values do tell a product with the reciprocal from the quotient
    inv = (np.float32(1) / scales[0])[:, None]
    with np.errstate(over="ignore"):
        assert (fp8.encode(x.float().numpy() * inv) != codes).sum() > 100
    q, s = wq.alloc_fp8_rows(m, k)
    wq.wq_quantize_fp8_rows(x.cuda(), q, s)
    torch.cuda.synchronize()
    assert np.array_equal(s.cpu().numpy(), scales) and np.array_equal(bits(q), codes)
    # the norm of rows of ones is 1: it leaves the gains, in fp32 as they are
    for row in x[x.abs().max(1).values < 1e4][::97]:
        one = torch.ones((3, k), dtype=x.dtype)
        one[1] = -1
        q3, s3 = wq.alloc_fp8_rows(3, k)
        wq.wq_add_rmsnorm(one.cuda(), row.cuda(), 0.0, q=q3, scales=s3)
        torch.cuda.synchronize()
        codes, scales = fp8.quantize_rows(one.float().numpy() * row.float().numpy())
        assert np.array_equal(s3.cpu().numpy(), scales) and np.array_equal(bits(q3), codes)
    # and one row of a weight block, zeros below
    for row in x[::53]:
        w16 = torch.zeros((2, k), dtype=x.dtype)
        w16[1] = row
        w = wq.alloc_fp8(2, k)
        wq.wq_quantize_fp8_block(w16.cuda(), w.codes, w.scales)
        torch.cuda.synchronize()
        codes, scales = fp8.quantize_block(w16.float().numpy())
        assert np.array_equal(w.scales.cpu().numpy(), scales)
        assert np.array_equal(bits(w.codes), codes)


# ------------------------------------------------- products without a tolerance
def integer_linear(m, n, k, seed, pairs=False):
    """Codes that are integers up to 4 and scales that are powers of two: every
    product, and every sum of them in any order, is exact in fp32, so one lost,
    doubled or misplaced code shows.  With `pairs`, each whole block also holds
    448 * 448 and its negative."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(-4, 5, (m, k), generator=g).float()
    w = torch.randint(-4, 5, (n, k), generator=g).float()
    if pairs:
        for b in range(k // 128):
            i, j = (b * 128 + torch.randperm(128, generator=g)[:2]).tolist()
            x[:, i], x[:, j], w[:, i], w[:, j] = 448.0, 448.0, 448.0, -448.0
    kb, nb = -(-k // 128), -(-n // 128)
    s = torch.exp2(torch.randint(-2, 3, (kb, m), generator=g).float())
    e = torch.exp2(torch.randint(-2, 3, (nb, kb), generator=g).float())
    f8 = torch.float8_e4m3fn
    return (x.to(f8).cuda(), s.cuda(),
            wq.QuantizedWeight(wq.FMT_FP8_BLOCK, n, k, 128, w.to(f8).cuda(), e.cuda()))


# every schedule: one token, 1 to 4 tiles of 16 tokens with few and many features,
# tiles of 64 and 128 tokens whole and split, 256 x 256 tiles with and without
# tiles of 128 tokens after them
EXACT = [(1, 300, 400), (1, 4500, 144), (7, 515, 2064), (16, 4200, 272), (31, 200, 1024),
         (40, 5000, 400), (48, 12301, 400), (64, 200, 2064), (64, 8201, 272), (65, 257, 16),
         (100, 136, 8832), (150, 1000, 4112), (300, 513, 1040), (512, 1030, 272),
         (1000, 4000, 1296), (2049, 4100, 400), (4096, 5120, 272)]


@pytest.mark.parametrize("ydt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,n,k", EXACT)
def test_linear_of_integers_is_exact(m, n, k, ydt):
    say(f"fp8 linear of integers m={m} n={n} k={k} y={ydt}")
    q, s, w = integer_linear(m, n, k, 61)
    ref = reference(q, s, w)[0]
    assert float(ref.abs().max()) < 2.0 ** 15
    y = linear(q, s, w, ydt)
    torch.cuda.synchronize()
    assert torch.equal(y, ref.float().to(TD[ydt]))


@pytest.mark.parametrize("m,n,k", [c for c in EXACT if c[0] <= 1000])
def test_linear_fp32_products_are_exact(m, n, k):
    """What the FP8 matrix instructions drop beside 448 * 448 (products below 2)."""
    say(f"fp8 linear, large pairs, m={m} n={n} k={k}")
    q, s, w = integer_linear(m, n, k, 62, pairs=True)
    ref = reference(q, s, w)[0]
    y = linear(q, s, w, "f32")
    torch.cuda.synchronize()
    assert torch.equal(y, ref.float())


def power(t):
    """The power of two of a code, 2^-6 for smaller ones."""
    return torch.exp2(torch.floor(torch.log2(t.double().abs().clamp(min=2.0 ** -6))))


@pytest.mark.parametrize("ydt", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["one large", "all codes", "normal"])
@pytest.mark.parametrize("m,n,k", [(1, 130, 400), (16, 300, 1040), (64, 200, 528), (150, 140, 656),
                                   (300, 1000, 272), (2049, 4100, 144)])
def test_linear_16_bit_bound(m, n, k, kind, ydt):
    """Each product of a block is cut at 2^-17 of the largest power of two among the
    block's products: 128 of them lose at most 2^-10 of it.  Then fp32 sums, and the
    rounding of y."""
    say(f"fp8 linear bound m={m} n={n} k={k} {kind} y={ydt}")
    f8 = torch.float8_e4m3fn
    g = torch.Generator().manual_seed(63)
    if kind == "normal":
        x, w = (torch.randn(r, k, generator=g).mul(100).clamp(-448, 448).to(f8) for r in (m, n))
    else:
        x, w = (torch.randint(0, 127, (r, k), generator=g, dtype=torch.uint8) for r in (m, n))
        if kind == "one large":
            # 256 * 256 beside products that are alike within a row and column
            x[:], w[:] = x[:, :1], w[:, :1]
            x[:, 5::128], w[:, 5::128] = 0x78, 0x78
        else:
            x |= torch.randint(0, 2, (m, k), generator=g, dtype=torch.uint8) << 7
        x, w = x.view(f8), w.view(f8)
    kb, nb = -(-k // 128), -(-n // 128)
    q = x.cuda()
    # y of every kind within 16 bits' range
    s = (torch.rand((kb, m), generator=g) + 0.5).mul(2.0 ** -8).cuda()
    w = wq.QuantizedWeight(wq.FMT_FP8_BLOCK, n, k, 128, w.cuda(),
                           (torch.rand((nb, kb), generator=g) + 0.5).mul(2.0 ** -8).cuda())
    ref, mag = reference(q, s, w)
    tol = (kb + 16) * 2.0 ** -23 * mag
    for b in range(kb):
        c = slice(b * 128, (b + 1) * 128)
        px, pw = power(q[:, c].float()), power(w.codes[:, c].float())
        e = (s[b].double()[:, None] * w.scales[:, b].double().repeat_interleave(128)[:n]) * 2.0 ** -10
        for r in range(0, m, 64):
            u = torch.zeros((min(64, m - r), n), dtype=torch.float64, device="cuda")
            for i in range(px.shape[1]):
                u = torch.maximum(u, px[r:r + 64, i:i + 1] * pw[:, i])
            tol[r:r + 64] += e[r:r + 64] * u
    y = linear(q, s, w, ydt)
    torch.cuda.synchronize()
    err = (y.double() - ref).abs()
    assert bool((err <= tol + ULP[ydt] * (1 + 1e-3) * (ref.abs() + tol) + TINY[ydt]).all()), (
        f"worst {float((err / (tol + 1e-300)).max()):.3g} of the bound")
