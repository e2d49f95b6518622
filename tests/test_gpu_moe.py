"""The mixture-of-experts layer on the GPU against the fp64 oracle.

Tolerance, element by element in fp64: gate and up are fp32 sums whose INT4
form adds x * (16 + q) and takes (16 + z) * sum x away, so each is off by at
most d = (32 + h / 128) 2^-24 S with S = sum |x| s (31 + 31) (FP8: sum |x w|);
the intermediate p silu(g) u moves by p (1.1 |u| dg + |silu(g)| du) and a few
roundings, and is rounded once to 16 bits; the down product sums that with the
same kind of error; y is rounded once.
"""

import numpy as np
import pytest
import torch

import bit_quantized_linear_int4_amd as wq
from gpu_util import say
from oracle import fp8, int4, moe

pytestmark = pytest.mark.gpu

TD = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ULP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def rand(shape, seed, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(TD[dtype])


class Experts:
    """Packed experts, their fp64 values and what bounds a sum over them."""

    def __init__(self, e, h, i, fmt, group, seed):
        self.e, self.h, self.i = e, h, i
        self.w, self.val, self.mag = [], [], []
        for j, (rows, k) in enumerate(((i, h), (i, h), (h, i))):
            n = e * rows
            w16 = rand((n, k), seed + j, "f16", 0.05)
            if fmt == "fp8":
                q = wq.alloc_fp8(n, k)
                wq.wq_quantize_fp8_block(w16.cuda(), q.codes, q.scales)
                torch.cuda.synchronize()
                val = fp8.dequantize_block(q.codes.cpu().view(torch.uint8).numpy(),
                                           q.scales.cpu().numpy())
                mag = np.abs(val)
            else:
                q = wq.alloc_int4(n, k, group)
                wq.wq_quantize_groupwise(w16.cuda(), 4, group, 0, q.codes, q.scales, q.zeros)
                torch.cuda.synchronize()
                s = np.repeat(q.scales.cpu().numpy().astype(np.float64), group, 1)
                words = q.codes.cpu().numpy().view(np.uint32)
                c = ((words[..., None] >> (4 * np.arange(8, dtype=np.uint32))) & 15).reshape(n, k)
                zb = q.zeros.cpu().numpy()
                z = np.stack((zb & 15, zb >> 4), -1).reshape(n, -1)[:, :k // group]
                val = (c - np.repeat(z.astype(np.float64), group, 1)) * s
                mag = 62 * s
            self.w.append(q)
            self.val.append(val.reshape(e, rows, k))
            self.mag.append(mag.reshape(e, rows, k))


def bound(x, ids, probs, ex, xdt):
    """How far y may be off before its own rounding."""
    x = np.abs(x.double().cpu().numpy()), x.double().cpu().numpy()
    out = np.zeros((x[0].shape[0], ex.h))
    cg, cd = (32 + ex.h / 128) * 2.0 ** -24, (32 + 16 * ex.i / 128) * 2.0 ** -24
    for t in range(out.shape[0]):
        for e, p in zip(ids[t], probs[t]):
            if p == 0:
                continue
            g, u = ex.val[0][e] @ x[1][t], ex.val[1][e] @ x[1][t]
            dg, du = cg * (ex.mag[0][e] @ x[0][t]), cg * (ex.mag[1][e] @ x[0][t])
            sl = g / (1 + np.exp(-g))
            a = np.abs(p * sl * u)
            da = p * (1.1 * np.abs(u) * dg + np.abs(sl) * du + dg * du) + 2.0 ** -18 * a
            da += ULP[xdt] * (a + da) + (2.0 ** -25 if xdt == "f16" else 0)
            out[t] += np.abs(ex.val[2][e]) @ da + cd * (ex.mag[2][e] @ (a + da))
    return out


def run(x, ex, top_k, router=None, logits=None, renorm=True, ydt="f32", stream=None):
    t = x.shape[0]
    y = torch.full((t, ex.h), float("nan"), dtype=TD[ydt], device="cuda")
    ids = torch.full((t, top_k), -1, dtype=torch.int32, device="cuda")
    probs = torch.full((t, top_k), float("nan"), device="cuda")
    ws = torch.full((wq.wq_moe_workspace(t, top_k, ex.w[0], ex.e),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    wq.wq_moe(x, router, top_k, *ex.w, y, ws, renormalize=renorm, logits=logits, ids=ids,
              probs=probs, stream=stream)
    torch.cuda.synchronize()
    return y, ids.cpu().numpy(), probs.cpu().numpy()


def check(x, ex, logits64, top_k, xdt, got, renorm, ydt, logit_err=0.0):
    y, ids, probs = got
    rid, rp = moe.route(logits64, top_k, renorm)
    # the fp32 softmax: exponent rounding, sums, the logits' own error
    assert np.all(np.abs(probs - rp) <= (2.0 ** -18 + 4 * logit_err) * rp + 1e-38)
    assert np.array_equal(ids, rid)
    ref = moe.experts(x.double().cpu().numpy(), rid, rp, *ex.val)
    # y is linear in the probabilities
    tol = bound(x, rid, rp, ex, xdt) * (1 + 1e-3)
    if logit_err:
        big = np.zeros_like(ref)
        for j in range(top_k):
            part = np.zeros_like(rp)
            part[:, j] = rp[:, j]
            big += np.abs(moe.experts(x.double().cpu().numpy(), rid, part, *ex.val))
        tol += (4 * logit_err + 2.0 ** -18) * big
    err = np.abs(y.double().cpu().numpy() - ref)
    lim = tol + ULP[ydt] * (np.abs(ref) + tol) * (1 + 1e-3) + (2.0 ** -25 if ydt == "f16" else 0)
    assert np.all(err <= lim), f"worst {np.max(err / (lim + 1e-300)):.3g} of the bound"


FORMATS = [("int4", 128), ("int4", 64), ("int4", 32), ("fp8", 128)]


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("xdt", ["f16", "bf16"])
@pytest.mark.parametrize("t,e,top_k,h,i", [(1, 4, 2, 256, 128), (3, 8, 3, 384, 256),
                                           (17, 70, 4, 128, 128), (33, 5, 2, 256, 384),
                                           (64, 6, 6, 128, 256)])
def test_layer(t, e, top_k, h, i, xdt, fmt, group):
    say(f"moe t={t} e={e} k={top_k} h={h} i={i} {xdt} {fmt} g{group}")
    ex = Experts(e, h, i, fmt, group, 50)
    x = rand((t, h), 60, xdt).cuda()
    logits = rand((t, e), 61, "f32", 2.0)
    for renorm, ydt in ((True, xdt), (False, "f32")):
        got = run(x, ex, top_k, logits=logits.cuda(), renorm=renorm, ydt=ydt)
        check(x, ex, logits.double().numpy(), top_k, xdt, got, renorm, ydt)
        again = run(x, ex, top_k, logits=logits.cuda(), renorm=renorm, ydt=ydt)
        assert torch.equal(got[0], again[0])


@pytest.mark.parametrize("xdt", ["f16", "bf16"])
@pytest.mark.parametrize("t,e,h", [(1, 3, 128), (6, 64, 640), (64, 130, 1152), (2, 512, 256)])
def test_router(t, e, h, xdt):
    say(f"moe router t={t} e={e} h={h} {xdt}")
    ex = Experts(e, h, 128, "int4", 128, 70)
    x, wr = rand((t, h), 80, xdt).cuda(), rand((e, h), 81, xdt, 0.05).cuda()
    l64 = (x.double() @ wr.double().t()).cpu().numpy()
    # fp32 sums of h products, over 64 lanes
    err = (h / 64 + 16) * 2.0 ** -24 * float((x.double().abs() @ wr.double().abs().t()).max())
    top_k = min(3, e)
    y, ids, probs = run(x, ex, top_k, router=wr, ydt=xdt)
    # tokens whose choice no rounding can change
    gap = np.diff(np.sort(-l64, axis=1)[:, :top_k + 1], axis=1)
    sure = (gap > 2 * err).all(axis=1)
    assert sure.mean() > 0.5
    check(x[torch.from_numpy(sure).cuda()], ex, l64[sure], top_k, xdt,
          (y[torch.from_numpy(sure).cuda()], ids[sure], probs[sure]), True, xdt, logit_err=err)


def test_all_tokens_to_one_expert_and_none_to_others():
    t, e = 64, 9
    ex = Experts(e, 256, 128, "int4", 128, 90)
    x = rand((t, 256), 91, "bf16").cuda()
    logits = torch.full((t, e), -5.0)
    logits[:, 7] = 5.0
    logits[:, 2] = torch.linspace(-4, 4, t)
    got = run(x, ex, 2, logits=logits.cuda())
    check(x, ex, logits.double().numpy(), 2, "bf16", got, True, "f32")
    assert (got[1] == [7, 2]).all()


def test_ties_go_to_the_lowest_index():
    ex = Experts(130, 128, 128, "int4", 128, 95)
    x = rand((3, 128), 96, "f16").cuda()
    logits = torch.zeros((3, 130))
    logits[1, 64:] = 1.0
    logits[2, 1::2] = -0.0
    got = run(x, ex, 4, logits=logits.cuda(), renorm=False)
    check(x, ex, logits.double().numpy(), 4, "f16", got, False, "f32")
    assert got[1].tolist() == [[0, 1, 2, 3], [64, 65, 66, 67], [0, 1, 2, 3]]


@pytest.mark.parametrize("renorm", [True, False])
def test_masked_experts_and_rows_that_are_not_finite(renorm):
    inf = float("inf")
    t, e, top_k = 6, 5, 3
    ex = Experts(e, 128, 128, "fp8", 128, 97)
    x = rand((t, 128), 98, "bf16").cuda()
    logits = rand((t, e), 99, "f32")
    ref = run(x, ex, top_k, logits=logits.cuda(), renorm=renorm)
    logits[1] = -inf                              # everything masked
    logits[2] = torch.tensor([-inf, 0.5, -inf, -inf, -inf])
    low = torch.finfo(torch.float32).min
    logits[3] = torch.tensor([low, 1.0, low, 2.0, low])      # the type's lowest value as mask
    logits[4, 3] = float("nan")
    logits[5, 0] = inf
    got = run(x, ex, top_k, logits=logits.cuda(), renorm=renorm)
    y, ids, probs = got
    assert not y[1].any() and not probs[1].any() and ids[1].tolist() == [0, 1, 2]
    assert ids[2].tolist() == [1, 0, 2] and probs[2].tolist() == [1.0, 0.0, 0.0]
    assert ids[3].tolist() == [3, 1, 0] and probs[3, 2] == 0
    fine = [0, 1, 2, 3]
    check(x[fine], ex, logits[fine].double().numpy(), top_k, "bf16",
          (y[fine], ids[fine], probs[fine]), renorm, "f32")
    assert torch.equal(y[0], ref[0][0])
    for row in (4, 5):
        assert bool(y[row].isnan().all()) and np.isnan(probs[row]).any()
        assert ((ids[row] >= 0) & (ids[row] < e)).all() and len(set(ids[row])) == top_k


def test_nan_token_stays_alone():
    ex = Experts(3, 256, 128, "int4", 64, 100)
    x = rand((20, 256), 101, "f16").cuda()
    logits = rand((20, 3), 102, "f32").cuda()
    ref = run(x, ex, 2, logits=logits)[0]
    x[11, 200] = float("nan")
    y = run(x, ex, 2, logits=logits)[0]
    keep = [i for i in range(20) if i != 11]
    assert bool(y[11].isnan().all()) and torch.equal(y[keep], ref[keep])


def test_stream_and_graph():
    say("moe: stream and graph replay")
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        ex = Experts(6, 256, 256, "int4", 128, 103)
        x, wr = rand((9, 256), 104, "bf16").cuda(), rand((6, 256), 105, "bf16", 0.1).cuda()
        y = torch.empty((9, 256), dtype=torch.bfloat16, device="cuda")
        ws = torch.empty((wq.wq_moe_workspace(9, 2, ex.w[0], 6),), dtype=torch.uint8, device="cuda")
        wq.wq_moe(x, wr, 2, *ex.w, y, ws)
        st.synchronize()
        ref = y.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            wq.wq_moe(x, wr, 2, *ex.w, y, ws)
        for _ in range(3):
            y.zero_()
            ws.zero_()
            st.synchronize()
            g.replay()
            st.synchronize()
            assert torch.equal(y, ref)
            x2 = x * 2
            st.synchronize()


# k past what 8 waves, and past what 16 waves, hold in one pass; a long k of the
# down product; one token, some and more than a chunk of an expert
@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("t,e,top_k,h,i", [(1, 3, 2, 2304, 128), (20, 2, 1, 2176, 256),
                                           (1, 2, 2, 4224, 128), (5, 3, 2, 8320, 128),
                                           (40, 2, 2, 128, 4224)])
def test_long_k(t, e, top_k, h, i, fmt, group):
    say(f"moe t={t} e={e} k={top_k} h={h} i={i} {fmt} g{group}")
    ex = Experts(e, h, i, fmt, group, 90)
    x = rand((t, h), 91, "bf16", 0.5).cuda()
    logits = rand((t, e), 92, "f32", 2.0)
    got = run(x, ex, top_k, logits=logits.cuda(), ydt="f32")
    check(x, ex, logits.double().numpy(), top_k, "bf16", got, True, "f32")


def spread_bound(x, ids, probs, ex, xdt):
    """How far y may be off before its own rounding when the gated product is
    rounded by itself and its share multiplies the sums: every term, the half
    subnormal step of the intermediate too, comes times p."""
    x64 = x.double().cpu().numpy()
    out = np.zeros((x64.shape[0], ex.h))
    cg, cd = (32 + ex.h / 128) * 2.0 ** -24, (32 + 16 * ex.i / 128) * 2.0 ** -24
    for t in range(out.shape[0]):
        for e, p in zip(ids[t], probs[t]):
            if p == 0:
                continue
            g, u = ex.val[0][e] @ x64[t], ex.val[1][e] @ x64[t]
            dg, du = (cg * (ex.mag[j][e] @ np.abs(x64[t])) for j in (0, 1))
            sl = g / (1 + np.exp(-g))
            a = np.abs(sl * u)
            da = 1.1 * np.abs(u) * dg + np.abs(sl) * du + dg * du + 2.0 ** -18 * a
            da += ULP[xdt] * (a + da) + (2.0 ** -25 if xdt == "f16" else 0)
            out[t] += p * (np.abs(ex.val[2][e]) @ da + cd * (ex.mag[2][e] @ (a + da)))
    return out


# Small shares of small values: the gated product is near fp16's smallest normal
# value, and a share multiplied in before it is rounded to fp16 leaves three bits
# of it.  The most experts and choices there are.
@pytest.mark.parametrize("fmt,group", [("int4", 128), ("fp8", 128)])
@pytest.mark.parametrize("t", [1, 5, 64])
def test_small_shares_of_small_values(t, fmt, group):
    say(f"moe small shares t={t} {fmt}")
    e, top_k, h, i = 512, 16, 128, 128
    ex = Experts(e, h, i, fmt, group, 110)
    x = rand((t, h), 111, "f16", 0.02).cuda()
    logits = rand((t, e), 112, "f32", 0.1)
    y, ids, probs = run(x, ex, top_k, logits=logits.cuda(), renorm=False)
    rid, rp = moe.route(logits.double().numpy(), top_k, False)
    assert np.array_equal(ids, rid) and rp.max() < 4 / e
    assert np.all(np.abs(probs - rp) <= 2.0 ** -18 * rp)
    ref = moe.experts(x.double().cpu().numpy(), rid, rp, *ex.val)
    # the shares' own error, 2^-18, of sums no larger than those of magnitudes
    tol = spread_bound(x, rid, rp, ex, "f16")
    big = np.zeros_like(ref)
    for j in range(top_k):
        part = np.zeros_like(rp)
        part[:, j] = rp[:, j]
        big += np.abs(moe.experts(x.double().cpu().numpy(), rid, part, *ex.val))
    err = np.abs(y.double().cpu().numpy() - ref)
    lim = (tol + 2.0 ** -18 * big) * (1 + 1e-3) + ULP["f32"] * np.abs(ref)
    assert np.all(err <= lim), f"worst {np.max(err / lim):.3g} of the bound"


def spread(t, top_k, counts, seed):
    """Logits fp32 [t][e] that route counts[e] tokens to expert e."""
    left = np.array(counts)
    assert left.sum() == t * top_k and left.max() <= t
    r = np.random.default_rng(seed)
    logits = r.uniform(-2, -1, (t, len(counts)))
    for i in range(t):
        pick = np.argsort(-left, kind="stable")[:top_k]
        left[pick] -= 1
        logits[i, pick] = r.uniform(1, 2, top_k)
    assert not left.any()
    return torch.from_numpy(logits.astype(np.float32))


# The walk over the gate/up steps: from tile to tile, chunk (16 tokens) to chunk and
# expert to expert within a workgroup, with a last block of tiles that is shorter than
# the others; 8 and 16 waves, k in one pass and in two, grids as large as the tiles and
# as large as the GPU holds.
@pytest.mark.parametrize("xdt", ["f16", "bf16"])
@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("t,top_k,counts,h,i,per", [
    (50, 2, (20, 50, 30), 384, 128, 3), (50, 2, (20, 50, 30), 2176, 128, 3),
    (50, 2, (20, 50, 30), 4224, 128, 3), (37, 1, (37,), 256, 128, 3), (33, 1, (33,), 2304, 128, 3),
    (64, 3, (64, 40, 1, 33, 17, 16, 17, 4), 256, 1280, 3)])
def test_steps(t, top_k, counts, h, i, per, fmt, group, xdt):
    steps_case(t, top_k, counts, h, i, per, fmt, group, xdt)


@pytest.mark.parametrize("fmt,group", [("int4", 128), ("int4", 32), ("fp8", 128)])
def test_steps_of_large_experts(fmt, group):
    steps_case(64, 2, (17, 64, 14, 33), 2176, 1664, 5, fmt, group, "bf16")


def steps_case(t, top_k, counts, h, i, per, fmt, group, xdt):
    say(f"moe steps t={t} {counts} h={h} i={i} {fmt} g{group} {xdt}")
    e, tiles = len(counts), i // 16
    chunks = sum((c + 15) // 16 for c in counts)
    # as launched: workgroups, steps of each, and a block of tiles that is cut short
    grid = min(min(e, t * top_k) * tiles, 512 if h <= 2048 else 256)
    assert -(-tiles * chunks // grid) == per and per > 1 and tiles % per != 0
    ex = Experts(e, h, i, fmt, group, 120)
    x = rand((t, h), 121, xdt, 0.5).cuda()
    logits = spread(t, top_k, counts, 122)
    got = run(x, ex, top_k, logits=logits.cuda(), ydt="f32")
    assert np.bincount(got[1].ravel(), minlength=e).tolist() == list(counts)
    check(x, ex, logits.double().numpy(), top_k, xdt, got, True, "f32")
