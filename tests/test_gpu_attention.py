"""Append to a paged cache and attention over it on the GPU against the fp64 oracle.

Append: a rotated element is a c + b s in fp32, off by at most 3 * 2^-24 (|a c| +
|b s|), then rounded once: to 16 bits (half a step), or to E4M3 of its quotient
with the scale (half a step: 2^-4 of the value, 2^-10 of the scale below 2^-6 of it),
where the scale is max / 448 of the fp32 values.  Values are not rotated: codes and
scales are the oracle's bits.

Attention, element by element: z is an fp32 sum over d products and a few
roundings, off by dz = (d + 12) 2^-24 scale sum |q k| (the same for the maximum it is
measured from); a weight exp(z) then by 2 dz + 2^-21 of itself, and its rounding to
16 bits r (decode two parts of bf16, 2^-16; prompt 2^-8 for bf16, 2^-11 and the
subnormal 2^-25 of the largest weight for f16).  Sums over n tokens add (n + 64)
2^-23.  So y is off by at most
  sum_j w_j |v_j| (2 max dz + r + 2^-20 + (n + 64) 2^-22),
then half a step of its own type, and lse by max dz + (n + 64) 2^-23 + 2^-21 |lse|.
"""

import numpy as np
import pytest
import torch

import bit_quantized_linear_int4_amd as wq
from gpu_util import say
from oracle import attention as oracle
from oracle import fp8

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
TD = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": F8}
ULP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def rand(shape, seed, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(TD[dtype])


def np64(t):
    return t.detach().double().cpu().numpy()


class Cache:
    """A KVCache with values of its own, in fp64 beside it."""

    def __init__(self, pages, kv, page, d, dtype, layout="head", seed=0, empty=False):
        self.dtype = dtype
        shape = (pages, kv, page, d) if layout == "head" else (pages, page, kv, d)

        def make(s):
            t = torch.empty(shape, dtype=TD[dtype], device="cuda")
            t = t if layout == "head" else t.transpose(1, 2)
            if empty:
                t.copy_(torch.full((1,), float("nan")).to(TD[dtype]).cuda())
            else:
                t.copy_(rand((pages, kv, page, d), s, "f16", 100.0 if dtype == "e4m3" else 1.0)
                        .float().clamp(-448, 448).to(TD[dtype]).cuda())
            return t

        self.k, self.v = make(seed), make(seed + 1)
        self.ks = self.vs = None
        if dtype == "e4m3":
            g = torch.Generator().manual_seed(seed + 2)
            self.ks, self.vs = ((0.01 * (0.2 + torch.rand((pages, kv, page), generator=g))).cuda()
                                for _ in range(2))
            if empty:
                self.ks.fill_(float("nan"))
                self.vs.fill_(float("nan"))
        self.c = wq.KVCache(self.k, self.v, self.ks, self.vs)

    def values(self):
        out = []
        for t, s in ((self.k, self.ks), (self.v, self.vs)):
            x = np64(t.float())
            out.append(x if s is None else x * np64(s)[..., None])
        return out


def table_of(lens, page, seed, extra=0):
    """(table, pages in the cache): shuffled pages, none shared."""
    counts = [max(0, -(-n // page)) for n in lens]
    g = np.random.default_rng(seed)
    total = sum(counts) + 2
    order = g.permutation(total)
    table = g.integers(-5, total + 5, (len(lens), max(max(counts), 1) + extra))   # unused: anything
    at = 0
    for i, n in enumerate(counts):
        table[i, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(table.astype(np.int32)).cuda(), total


def check(y, lse, q, kv, rows, scale, window, sinks, r, dtype, table):
    """rows: (row of q, sequence, position, tokens)."""
    d = q.shape[-1]
    k, v = kv
    qn, yn = np64(q), np64(y)
    ln = None if lse is None else np64(lse)
    seen = {}
    worst = 0.0
    for row, seq, pos, n in rows:
        if seq not in seen:
            seen[seq] = (oracle.tokens(k, table[seq], n), oracle.tokens(v, table[seq], n))
        ks, vs = seen[seq]
        ref, rl, w, mag = oracle.attend(qn[row], ks, vs, pos, scale, window, sinks)
        nv = (w > 0).sum(1).max() if n else 0
        group = ref.shape[0] // k.shape[1]
        for h in range(ref.shape[0]):
            dz = (d + 12) * 2.0 ** -24 * (mag[h].max() if n else 0.0)
            rel = 2 * dz + r + 2.0 ** -20 + (nv + 64) * 2.0 ** -22
            av = np.abs(vs[:, h // group])
            err = rel * (w[h] @ av) if n else np.zeros(d)
            if r == 2.0 ** -11 and n:
                err = err + 2.0 ** -25 * av[w[h] > 0].sum(0) * w[h].max() if w[h].any() else err
            tol = err + ULP[dtype] * (np.abs(ref[h]) + err) + TINY[dtype]
            off = np.abs(yn[row, h] - ref[h])
            assert np.all(off <= tol), (row, h, float((off / tol).max()))
            worst = max(worst, float((off / tol).max()))
            if ln is not None:
                if np.isinf(rl[h]):
                    assert ln[row, h] == rl[h]
                else:
                    lt = dz + (nv + 64) * 2.0 ** -23 + 2.0 ** -21 * abs(rl[h]) + 2.0 ** -22
                    assert abs(ln[row, h] - rl[h]) <= lt, (row, h, ln[row, h], rl[h])
    return worst


DECODE_R = 2.0 ** -16


def prompt_r(dtype, cdtype):
    return DECODE_R if (dtype, cdtype) == ("f16", "e4m3") else ULP[dtype]


def workspace(n):
    return torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") if n else None


def run_decode(q, c, table, lens, window=0, sinks=0, scale=None, lse=True, ws=None):
    m, heads, _ = q.shape
    y = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    ls = torch.full((m, heads), float("nan"), device="cuda") if lse else None
    ws = workspace(wq.wq_attention_decode_workspace(m, heads, c.c)) if ws is None else ws
    wq.wq_attention_decode(q, c.c, table, lens, y, ws, scale=scale, window=window, sinks=sinks,
                           lse=ls)
    torch.cuda.synchronize()
    return y, ls


def run_prompt(q, starts, c, table, lens, window=0, sinks=0, scale=None, lse=True):
    m, heads, _ = q.shape
    y = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    ls = torch.full((m, heads), float("nan"), device="cuda") if lse else None
    ws = workspace(wq.wq_attention_prompt_workspace(m, heads, len(lens), c.c))
    wq.wq_attention_prompt(q, starts, c.c, table, lens, y, ws, scale=scale, window=window,
                           sinks=sinks, lse=ls)
    torch.cuda.synchronize()
    return y, ls


def i32(a):
    return torch.tensor(list(a), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ append
APPEND = [
    # m, heads, kv, d, rot, interleaved, page, layout
    (1, 32, 8, 128, 128, False, 64, "head"), (1, 4, 4, 64, 64, True, 16, "token"),
    (3, 7, 1, 128, 96, False, 1, "head"), (5, 64, 8, 64, 32, False, 32, "head"),
    (33, 5, 5, 128, 16, True, 16, "token"), (70, 28, 4, 64, 48, True, 128, "head"),
    (130, 3, 3, 128, 0, False, 8, "token"), (9, 40, 40, 128, 112, True, 16, "head"),
    # more heads per thread
    (512, 5, 1, 64, 64, False, 64, "head"), (600, 30, 9, 128, 64, True, 16, "token"),
    (700, 1, 16, 64, 32, False, 16, "head"),
]


def inputs(m, heads, kv, d, rot, dtype, seed):
    qkv = rand((m, heads + 2 * kv, d), seed, dtype).cuda()
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    pos = torch.randint(0, 50, (m,), generator=torch.Generator().manual_seed(seed)).int().cuda()
    ang = torch.rand((50, rot // 2), generator=torch.Generator().manual_seed(seed + 1)) * 7
    table = torch.cat((ang.cos(), ang.sin()), 1).cuda()
    return q, k, v, pos, table


def rotated(x, pos, table, inter):
    """(fp64 rotation, what bounds its fp32 form)."""
    xn, tn, p = np64(x), np64(table), pos.cpu().numpy()
    return oracle.rotate(xn, p, tn, inter), (
        3 * 2.0 ** -24 * oracle.rotate(np.abs(xn), p, np.concatenate(
            (np.abs(tn[:, :tn.shape[1] // 2]), 0 * tn[:, tn.shape[1] // 2:]), 1), inter)
        + 3 * 2.0 ** -24 * np.abs(oracle.rotate(np.abs(xn), p, np.concatenate(
            (0 * tn[:, :tn.shape[1] // 2], np.abs(tn[:, tn.shape[1] // 2:])), 1), inter)))


@pytest.mark.parametrize("dtype,cdtype", [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"),
                                          ("bf16", "e4m3")])
@pytest.mark.parametrize("shape", APPEND)
def test_append(shape, dtype, cdtype):
    m, heads, kv, d, rot, inter, page, layout = shape
    say(f"append {shape} {dtype} {cdtype}")
    q, k, v, pos, table = inputs(m, heads, kv, d, rot, dtype, 11)
    pages = m // page + 3
    c = Cache(pages, kv, page, d, cdtype, layout, seed=20)
    before = [t.clone() for t in (c.k, c.v)] + [c.ks, c.vs]
    before[2:] = [t.clone() if t is not None else None for t in before[2:]]
    slots = np.random.default_rng(3).permutation(pages * page)[:m].astype(np.int32)
    if m > 2:
        slots[1], slots[m - 1] = -7, pages * page                       # rows that are not stored
        pos[0], pos[2] = -4, 1000                                        # past the table
    q_out = torch.full((m, heads, d), float("nan"), dtype=q.dtype, device="cuda")
    args = dict(positions=pos, cos_sin=table, interleaved=inter) if rot else {}
    wq.wq_append_kv(q, k, v, c.c, i32(slots), q_out=q_out, **args)
    torch.cuda.synchronize()
    if rot:
        (qr, qe), (kr, ke) = rotated(q, pos, table, inter), rotated(k, pos, table, inter)
    else:
        qr, kr = np64(q), np64(k)
        qe, ke = 0 * qr, 0 * kr
    u = ULP[dtype]
    assert np.all(np.abs(np64(q_out) - qr) <= qe + u * (np.abs(qr) + qe) + TINY[dtype])
    if rot < d:
        assert torch.equal(q_out[..., rot:], q[..., rot:])
    rows, pg, at = oracle.slots_of(slots, pages, page)
    pg, at = torch.from_numpy(pg).cuda(), torch.from_numpy(at).cuda()
    raw = (lambda t: t.view(torch.uint8)) if cdtype == "e4m3" else (lambda t: t.view(torch.int16))
    gk, gv = raw(c.k)[pg, :, at], raw(c.v)[pg, :, at]
    if cdtype == "e4m3":
        sk, sv = np64(c.ks[pg, :, at]), c.vs[pg, :, at].cpu().numpy()
        vf = v.float().cpu().numpy()[rows].reshape(-1, d)
        pad = np.zeros((vf.shape[0], 128), np.float32)
        pad[:, :d] = vf
        codes, scales = fp8.quantize_rows(pad)
        assert np.array_equal(gv.cpu().numpy().reshape(-1, d), codes[:, :d])
        assert np.array_equal(sv.reshape(-1), scales[0])
        kr, ke = kr[rows], ke[rows]
        big = np.abs(kr).max(-1)
        assert np.all(np.abs(sk - big / 448) <= ke.max(-1) / 448 + 2.0 ** -22 * sk)
        val = fp8.decode(gk.cpu().numpy()) * sk[..., None]
        assert np.all(np.abs(val - kr) <= 2.0 ** -4 * np.abs(kr) + 2 * ke + 2.0 ** -20 * np.abs(kr)
                      + 2.0 ** -10 * sk[..., None])
    else:
        assert torch.equal(gv, raw(v)[torch.from_numpy(rows).cuda()])
        got = np64(c.k[pg, :, at])
        kr, ke = kr[rows], ke[rows]
        assert np.all(np.abs(got - kr) <= ke + u * (np.abs(kr) + ke) + TINY[dtype])
    # every other place is as it was
    raw(before[0])[pg, :, at], raw(before[1])[pg, :, at] = gk, gv
    assert torch.equal(raw(c.k), raw(before[0])) and torch.equal(raw(c.v), raw(before[1]))
    if cdtype == "e4m3":
        for s, b in ((c.ks, before[2]), (c.vs, before[3])):
            b[pg, :, at] = s[pg, :, at]
            assert torch.equal(s, b)


@pytest.mark.parametrize("inter", [False, True])
def test_append_in_place_and_without_queries(inter):
    m, heads, kv, d = 37, 6, 2, 128
    q, k, v, pos, table = inputs(m, heads, kv, d, 128, "bf16", 31)
    slots = i32(range(m))
    a, b = Cache(5, kv, 16, d, "bf16"), Cache(5, kv, 16, d, "bf16")
    out = torch.empty((m, heads, d), dtype=q.dtype, device="cuda")
    wq.wq_append_kv(q, k, v, a.c, slots, pos, table, out, inter)
    wq.wq_append_kv(None, k, v, b.c, slots, pos, table, None, inter)
    torch.cuda.synchronize()
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    wq.wq_append_kv(q, k, v, a.c, slots, pos, table, q, inter)
    torch.cuda.synchronize()
    assert torch.equal(q, out) and torch.equal(a.k, b.k)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_append_not_finite(bad):
    """They stay in their head; zeros have scale 1 and values near the smallest keep theirs."""
    q, k, v, pos, table = inputs(6, 2, 2, 128, 128, "bf16", 41)
    c, ref = Cache(2, 2, 8, 128, "e4m3"), Cache(2, 2, 8, 128, "e4m3")
    slots = i32(range(6))
    out, out2 = (torch.empty((6, 2, 128), dtype=q.dtype, device="cuda") for _ in range(2))
    wq.wq_append_kv(q, k, v, ref.c, slots, pos, table, out)
    v[1, 0, 5] = bad
    k[2, 1, 70] = bad
    q[3, 0, 9] = bad
    v[4, 1] = 0
    wq.wq_append_kv(q, k, v, c.c, slots, pos, table, out2)
    torch.cuda.synchronize()
    kd, vd = c.values()
    assert not np.isfinite(vd[0, 0, 1, 5]) and not np.isfinite(kd[0, 1, 2, 70])
    assert not torch.isfinite(out2[3, 0, 9]).item() and not torch.isfinite(out2[3, 0, 73]).item()
    assert c.vs[0, 1, 4].item() == 1.0 and not vd[0, 1, 4].any()
    out[3, 0] = out2[3, 0]
    assert torch.equal(out.view(torch.int16), out2.view(torch.int16))
    for t, r, (h, at) in ((c.k, ref.k, (1, 2)), (c.v, ref.v, (0, 1))):
        t, r = t.view(torch.uint8).clone(), r.view(torch.uint8).clone()
        r[0, h, at] = t[0, h, at]
        if t.data_ptr() and (h, at) == (0, 1):
            r[0, 1, 4] = t[0, 1, 4]
        assert torch.equal(t, r)


# ------------------------------------------------------------------ decode
LENS = {
    "one": [1], "short": [2, 31, 32, 33], "mixed": [0, 1, 17, 64, 100, 129, 255, 256, 257, 3],
    "long": [5000, 1, 1300], "same": [77] * 5, "none": [0, -3],
}
DECODE = [
    # heads, kv, d, page, layout, lens, window, sinks
    (32, 8, 128, 64, "head", "one", 0, 0), (8, 8, 128, 16, "token", "mixed", 0, 0),
    (4, 1, 64, 32, "head", "mixed", 0, 0), (28, 4, 128, 16, "head", "mixed", 0, 0),
    (64, 8, 64, 128, "token", "short", 0, 0), (40, 2, 128, 8, "head", "short", 0, 0),
    (71, 1, 64, 1, "head", "mixed", 0, 0), (8, 2, 128, 16, "head", "long", 0, 0),
    (16, 1, 128, 32, "token", "long", 0, 0), (8, 4, 64, 64, "head", "long", 200, 4),
    (5, 5, 128, 2, "head", "mixed", 1, 0), (6, 2, 128, 16, "token", "mixed", 33, 3),
    (33, 3, 64, 4, "head", "mixed", 100, 50), (8, 2, 128, 16, "head", "long", 2000, 4999),
    (2, 2, 64, 16, "head", "none", 0, 0), (12, 4, 128, 256, "head", "same", 7, 1),
]


@pytest.mark.parametrize("dtype,cdtype", [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"),
                                          ("bf16", "e4m3")])
@pytest.mark.parametrize("case", DECODE)
def test_decode(case, dtype, cdtype):
    heads, kv, d, page, layout, lens, window, sinks = case
    lens = LENS[lens]
    say(f"decode {case} {dtype} {cdtype}")
    table, pages = table_of(lens, page, 5, extra=3)
    c = Cache(pages, kv, page, d, cdtype, layout, seed=50)
    q = rand((len(lens), heads, d), 60, dtype, 2.0).cuda()
    y, lse = run_decode(q, c, table, i32(lens), window, sinks)
    rows = [(i, i, n - 1, max(n, 0)) for i, n in enumerate(lens)]
    w = check(y, lse, q, c.values(), rows, d ** -0.5, window, sinks, DECODE_R, dtype,
              table.cpu().numpy())
    say(f"  {w:.3f} of the tolerance")


@pytest.mark.parametrize("scale", [1.0, 30.0, 1e-3])
def test_decode_scales(scale):
    """Flat and sharp weights; z spread over thousands (scale 30)."""
    lens = [700, 40, 1]
    table, pages = table_of(lens, 16, 6)
    c = Cache(pages, 2, 16, 128, "bf16", seed=51)
    q = rand((3, 8, 128), 61, "bf16", 2.0).cuda()
    y, lse = run_decode(q, c, table, i32(lens), scale=scale)
    check(y, lse, q, c.values(), [(i, i, n - 1, n) for i, n in enumerate(lens)], scale, 0, 0,
          DECODE_R, "bf16", table.cpu().numpy())


def far_cache(cdtype):
    """k and v of more than 2^32 bytes each, of which two pages are used."""
    big = {"bf16": (1 << 31) + (1 << 27), "e4m3": (1 << 32) + (1 << 28)}[cdtype]
    page, kv, d = 64, 2, 128
    pages = big // (page * kv * d)
    t = [torch.zeros((pages, kv, page, d), dtype=torch.uint8 if cdtype == "e4m3" else TD[cdtype],
                     device="cuda") for _ in range(2)]
    s = [torch.ones((pages, kv, page), device="cuda") for _ in range(2)] if cdtype == "e4m3" else []
    return pages, t, s


@pytest.mark.parametrize("cdtype", ["bf16", "e4m3"])
def test_far_pages(cdtype):
    """Offsets past 32 bits, for the append, the decode and the prompt call."""
    pages, t, s = far_cache(cdtype)
    c = wq.KVCache(*t, *s)
    near = Cache(2, 2, 64, 128, cdtype)
    nc = near.c
    m, d = 100, 128
    q, k, v, pos, table = inputs(m, 4, 2, d, 128, "bf16", 71)
    far = torch.tensor([[pages - 1, pages // 2 + 3]], dtype=torch.int32, device="cuda")
    low = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    j = torch.arange(m, device="cuda")
    out = torch.empty((m, 4, d), dtype=q.dtype, device="cuda")
    for cc, tab in ((c, far), (nc, low)):
        wq.wq_append_kv(q, k, v, cc, (tab[0, j // 64] * 64 + j % 64).int(), pos, table, out)
    res = []
    for cc, tab in ((c, far), (nc, low)):
        y, yp = torch.empty((1, 4, d), dtype=q.dtype, device="cuda"), torch.empty_like(out)
        wq.wq_attention_decode(out[:1], cc, tab, i32([m]), y,
                               workspace(wq.wq_attention_decode_workspace(1, 4, cc)))
        wq.wq_attention_prompt(out, i32([0, m]), cc, tab, i32([m]), yp,
                               workspace(wq.wq_attention_prompt_workspace(m, 4, 1, cc)))
        res.append((y, yp))
    torch.cuda.synchronize()
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
    assert torch.equal(c.k[far[0].long()].view(torch.uint8)[0],
                       nc.k[low[0].long()].view(torch.uint8)[0])


# ------------------------------------------------------------------ prompt
PROMPT = [
    # heads, kv, d, page, layout, rows of each sequence, tokens before them, window, sinks
    (4, 4, 128, 16, "head", [1], [0], 0, 0), (8, 2, 128, 64, "head", [70], [0], 0, 0),
    (4, 2, 64, 32, "token", [33, 1, 0, 65], [0, 10, 9, 100], 0, 0),
    (7, 1, 128, 16, "head", [5, 40], [300, 0], 0, 0), (16, 2, 64, 16, "head", [130], [7], 0, 0),
    (5, 5, 128, 8, "token", [64, 63, 2], [64, 1, 500], 0, 0),
    (6, 2, 128, 16, "head", [150, 3], [0, 400], 50, 0),
    (4, 4, 64, 32, "head", [200], [33], 20, 5), (8, 1, 128, 1, "head", [20, 11], [90, 0], 1, 1),
    (2, 1, 64, 128, "token", [300], [0], 64, 64), (8, 8, 128, 16, "head", [260, 129], [0, 1], 0, 0),
    (32, 2, 64, 64, "head", [17], [2000], 0, 0), (64, 8, 128, 16, "head", [3] * 9, [50] * 9, 0, 0),
    (12, 4, 128, 16, "head", [4, 9], [1500, 700], 300, 4),
    (3, 3, 64, 16, "head", [0, 0, 5], [3, 0, 0], 0, 0),
    # many parts of many rows
    (32, 8, 128, 64, "head", [100], [1500], 0, 0),
    # enough sequences and kv heads for workgroups of 256 rows
    (8, 4, 128, 16, "head", [200, 1, 140] + [2, 1, 3] * 43, [0, 300, 77] + [1, 40, 0] * 43, 0, 0),
    (12, 4, 64, 32, "token", [190] + [1, 0, 4] * 50, [100] + [30, 5, 0] * 50, 61, 5),
    (4, 4, 128, 64, "head", [520, 257] + [1] * 130, [0, 64] + [3] * 130, 0, 0),
    (4, 4, 64, 16, "token", [600] + [2] * 129, [30] + [9] * 129, 200, 70),
    # the same for up to 64 sequences: the longest come first
    (64, 64, 64, 16, "head", [40, 1, 0, 300, 77, 130, 5, 64, 3],
     [0, 200, 5, 10, 0, 30, 400, 0, 90], 0, 0),
    (128, 64, 64, 32, "head", [70, 2, 70, 33, 1, 0, 90, 12, 4], [5, 100, 5, 0, 30, 2, 5, 5, 5],
     20, 2),
    (56, 8, 128, 16, "head", [9, 1, 30] * 16, [0, 33, 4] * 16, 0, 0),
]


def prompt_case(case, dtype, cdtype, lead=0, tail=0):
    heads, kv, d, page, layout, new, ctx, window, sinks = case
    lens = [a + b for a, b in zip(new, ctx)]
    starts = [lead]
    for n in new:
        starts.append(starts[-1] + n)
    table, pages = table_of(lens, page, 8, extra=2)
    c = Cache(pages, kv, page, d, cdtype, layout, seed=80)
    q = rand((max(1, starts[-1] + tail), heads, d), 90, dtype, 2.0).cuda()
    rows = [(starts[s] + i, s, ctx[s] + i, lens[s]) for s, n in enumerate(new) for i in range(n)]
    return q, starts, c, table, lens, rows


@pytest.mark.parametrize("dtype,cdtype", [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"),
                                          ("bf16", "e4m3")])
@pytest.mark.parametrize("case", PROMPT)
def test_prompt(case, dtype, cdtype):
    window, sinks, d = case[7], case[8], case[2]
    say(f"prompt {case} {dtype} {cdtype}")
    q, starts, c, table, lens, rows = prompt_case(case, dtype, cdtype)
    y, lse = run_prompt(q, i32(starts), c, table, i32(lens), window, sinks)
    w = check(y, lse, q, c.values(), rows, d ** -0.5, window, sinks, prompt_r(dtype, cdtype), dtype,
              table.cpu().numpy())
    say(f"  {w:.3f} of the tolerance")


def test_prompt_leaves_other_rows():
    """Rows before the first and behind the last sequence, and rows that see nothing."""
    case = (4, 2, 128, 16, "head", [30, 5], [0, 40], 0, 0)
    q, starts, c, table, lens, rows = prompt_case(case, "bf16", "bf16", lead=3, tail=6)
    q[:3], q[38:] = float("nan"), float("nan")
    y, lse = run_prompt(q, i32(starts), c, table, i32(lens))
    assert torch.isnan(y[:3]).all() and torch.isnan(y[38:]).all()
    assert torch.isnan(lse[:3]).all() and torch.isnan(lse[38:]).all()
    check(y, lse, q, c.values(), rows, 128 ** -0.5, 0, 0, ULP["bf16"], "bf16", table.cpu().numpy())
    # more rows than tokens: the first ones are before the sequence
    y, lse = run_prompt(q, i32(starts), c, table, i32([12, 45]))
    assert not y[3:21].any() and torch.all(lse[3:21] == -float("inf"))
    rows = [(3 + i, 0, i - 18, 12) for i in range(30)] + [(33 + i, 1, 40 + i, 45) for i in range(5)]
    check(y, lse, q, c.values(), rows, 128 ** -0.5, 0, 0, ULP["bf16"], "bf16", table.cpu().numpy())
    y, lse = run_prompt(q, i32(starts), c, table, i32([0, -5]))
    assert not y[3:38].any() and torch.all(lse[3:38] == -float("inf"))


def test_rows_before_their_sequences():
    """More rows than tokens in several sequences, with many workgroups."""
    case = (64, 64, 64, 16, "head", [150, 3, 140, 40, 9, 300, 1], [0] * 7, 0, 0)
    q, starts, c, table, _, _ = prompt_case(case, "bf16", "bf16")
    lens = [20, 0, 140, 1, -2, 33, 1]
    y, lse = run_prompt(q, i32(starts), c, table, i32(lens))
    rows = [(starts[s] + i, s, lens[s] - n + i if lens[s] > 0 else -1, max(lens[s], 0))
            for s, n in enumerate(case[5]) for i in range(n)]
    check(y, lse, q, c.values(), rows, 0.125, 0, 0, ULP["bf16"], "bf16", table.cpu().numpy())


def test_tables_and_lens_past_their_ends():
    """Pages outside the cache are the nearest inside, lens stop at the table's end."""
    c = Cache(4, 2, 16, 128, "bf16", seed=100)
    q = rand((3, 4, 128), 101, "bf16", 2.0).cuda()
    table = torch.tensor([[1, 99, -7], [2, 0, 3], [0, 0, 0]], dtype=torch.int32, device="cuda")
    y, lse = run_decode(q, c, table, i32([45, 1 << 30, 48]))
    rows = [(0, 0, 44, 45), (1, 1, 47, 48), (2, 2, 47, 48)]
    tn = table.cpu().numpy()
    check(y, lse, q, c.values(), rows, 128 ** -0.5, 0, 0, DECODE_R, "bf16", tn)
    y, lse = run_prompt(q, i32([0, 1, 2, 3]), c, table, i32([45, 1 << 30, 48]))
    check(y, lse, q, c.values(), rows, 128 ** -0.5, 0, 0, ULP["bf16"], "bf16", tn)


@pytest.mark.parametrize("dtype,cdtype", [("bf16", "bf16"), ("f16", "e4m3")])
def test_places_that_no_row_sees_may_hold_anything(dtype, cdtype):
    lens, page, kv, d = [37, 5, 130], 16, 2, 128
    table, pages = table_of(lens, page, 9)
    full = Cache(pages, kv, page, d, cdtype, seed=110)
    c = Cache(pages, kv, page, d, cdtype, empty=True)
    tn = table.cpu().numpy()
    window, sinks = 40, 3
    for i, n in enumerate(lens):
        for j in range(n):
            # the windowed calls below see the last 40 and the first 3 tokens
            if j < sinks or j >= n - window - 9:
                p, a = int(tn[i, j // page]), j % page
                c.k[p, :, a], c.v[p, :, a] = full.k[p, :, a], full.v[p, :, a]
                if cdtype == "e4m3":
                    c.ks[p, :, a], c.vs[p, :, a] = full.ks[p, :, a], full.vs[p, :, a]
    q = rand((3, 4, d), 111, dtype, 2.0).cuda()
    rows = [(i, i, n - 1, n) for i, n in enumerate(lens)]
    a, b = run_decode(q, c, table, i32(lens), window, sinks), run_decode(q, full, table, i32(lens),
                                                                        window, sinks)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check(*a, q, full.values(), rows, d ** -0.5, window, sinks, DECODE_R, dtype, tn)
    q = rand((10 + 5 + 7, 4, d), 112, dtype, 2.0).cuda()
    starts = i32([0, 10, 15, 22])
    a = run_prompt(q, starts, c, table, i32(lens), window, sinks)
    b = run_prompt(q, starts, full, table, i32(lens), window, sinks)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.isfinite(a[0]).all()


@pytest.mark.parametrize("many", [0, 260])
@pytest.mark.parametrize("what", ["k", "v", "vs"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_not_finite_tokens_reach_the_rows_that_see_them(bad, what, many):
    """A token that is not finite among many rows of a prompt, and in a decoded batch;
    with `many` sequences of one token behind, the workgroups have 256 rows."""
    cdtype = "e4m3" if what == "vs" else "bf16"
    n, at, kv, heads, d = 150, 90, 2, 4, 128
    table, pages = table_of([n, 20] + [1] * many, 16, 10)
    tn = table.cpu().numpy()
    c = Cache(pages, kv, 16, d, cdtype, seed=120)
    q = rand((n + 20 + many, heads, d), 121, "bf16", 2.0).cuda()
    starts = i32([0, n] + list(range(n + 20, n + 21 + many)))
    lens = i32([n, 20] + [1] * many)
    for window, sinks in ((0, 0), (25, 2)):
        before, lb = run_prompt(q, starts, c, table, lens, window, sinks)
        t = getattr(c, what)
        place = (int(tn[0, at // 16]), 1, at % 16) + (() if what == "vs" else (7,))
        keep = t[place].clone()
        t[place] = bad
        y, lse = run_prompt(q, starts, c, table, lens, window, sinks)
        sees = torch.zeros(n + 20 + many, dtype=torch.bool, device="cuda")
        sees[at:(at + window if window else n)] = True
        other = ~sees[:, None].expand(-1, heads).clone()
        other[:, :2] = True                                          # the other kv head's
        assert torch.equal(y[other], before[other]) and torch.equal(lse[other], lb[other])
        if what == "k":
            finite = torch.isfinite(y[sees, 2:]).all(-1)
            # an infinite key gives z = +inf (NaN) or -inf (left out)
            assert not finite.any() if bad != bad else (~finite).any()
        else:
            assert not torch.isfinite(y[sees, 2:, 7]).any()
        if what == "v":
            mine = [i for i in range(d) if i != 7]
            assert torch.equal(y[sees][:, 2:, mine], before[sees][:, 2:, mine])
        yd, _ = run_decode(q[n - 1:n + 1], c, table[:2], lens[:2], window, sinks)
        assert torch.isfinite(yd[1]).all() and torch.isfinite(yd[0, :2]).all()
        assert torch.isfinite(yd[0, 2:]).all().item() == (window > 0) or what == "k"
        t[place] = keep


def test_infinite_scores():
    """z = -inf leaves a token out, z = +inf makes its row NaN."""
    c = Cache(2, 1, 16, 64, "bf16", seed=130)
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    q = torch.ones((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    q[0, 1] = -1
    c.k[0, 0, 3, 0] = -float("inf")
    for run in (lambda: run_decode(q, c, table, i32([20])),
                lambda: run_prompt(q, i32([0, 1]), c, table, i32([20]))):
        y, lse = run()
        k, v = c.values()
        ks, vs = oracle.tokens(k, [0, 1], 20), oracle.tokens(v, [0, 1], 20)
        keep = [j for j in range(20) if j != 3]
        ref, rl, _, _ = oracle.attend(np64(q)[0, :1], ks[keep], vs[keep], 18, 0.125)
        assert np.abs(np64(y)[0, 0] - ref[0]).max() < 2.0 ** -7 and abs(lse[0, 0].item() - rl[0]) < 1e-4
        assert torch.isnan(y[0, 1]).all()
    c.k[:] = -float("inf")
    q.fill_(1.0)
    for run in (lambda: run_decode(q, c, table, i32([20])),
                lambda: run_prompt(q, i32([0, 1]), c, table, i32([20]))):
        y, lse = run()
        assert not y.any() and torch.all(lse == -float("inf"))


# ------------------------------------------------------- together, graphs, streams
def test_decode_is_a_prompt_of_one_row():
    lens = [300, 1, 64]
    table, pages = table_of(lens, 32, 12)
    c = Cache(pages, 4, 32, 128, "f16", seed=140)
    q = rand((3, 8, 128), 141, "f16", 2.0).cuda()
    a, la = run_decode(q, c, table, i32(lens))
    b, lb = run_prompt(q, i32(range(4)), c, table, i32(lens))
    assert np.abs(np64(a) - np64(b)).max() <= 2.0 ** -9 * np.abs(np64(a)).max()
    assert np.abs(np64(la) - np64(lb)).max() <= 1e-4


def test_graph_with_growing_sequences():
    """A captured step: append, then decode; lens and slots change between replays."""
    b, heads, kv, d, page, steps = 3, 8, 2, 128, 16, 4
    table = i32(range(b * 5)).view(b, 5)
    q, k, v, pos, cs = inputs(b, heads, kv, d, 128, "bf16", 150)
    start = [30, 15, 60]

    def make():
        return Cache(b * 5, kv, page, d, "e4m3", seed=151)

    def slots_at(step):
        return [(int(table[i, (n + step) // page]) * page + (n + step) % page)
                for i, n in enumerate(start)]

    out, y = (torch.empty((b, heads, d), dtype=q.dtype, device="cuda") for _ in range(2))
    lens, slots = i32(start), i32(slots_at(0))

    def call(c, ws):
        wq.wq_append_kv(q, k, v, c.c, slots, pos, cs, out)
        wq.wq_attention_decode(out, c.c, table, lens, y, ws)

    eager, c = [], make()
    ws = workspace(wq.wq_attention_decode_workspace(b, heads, c.c))
    for step in range(steps):
        lens.copy_(i32([n + step + 1 for n in start]))
        slots.copy_(i32(slots_at(step)))
        call(c, ws)
        torch.cuda.synchronize()
        eager.append(y.clone())
    assert not torch.equal(eager[0], eager[1])
    c = make()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    slots.fill_(-1)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        call(c, ws)
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            call(c, ws)
    for step in range(steps):
        lens.copy_(i32([n + step + 1 for n in start]))
        slots.copy_(i32(slots_at(step)))
        y.fill_(0)
        ws.fill_(step) if ws is not None else None      # nothing in it is kept between calls
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager[step]), step


def test_graph_of_a_prompt():
    case = (8, 2, 128, 16, "head", [40, 3, 100], [0, 200, 17], 0, 0)
    q, starts, c, table, lens, _ = prompt_case(case, "bf16", "bf16")
    st, ln = i32(starts), i32(lens)
    ws = workspace(wq.wq_attention_prompt_workspace(q.shape[0], 8, 3, c.c))
    y = torch.empty_like(q)
    refs = []
    for lv in (lens, [n - 2 for n in lens]):
        ln.copy_(i32(lv))
        wq.wq_attention_prompt(q, st, c.c, table, ln, y, ws)
        torch.cuda.synchronize()
        refs.append(y.clone())
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            wq.wq_attention_prompt(q, st, c.c, table, ln, y, ws)
    for i in (0, 1, 0, 1):
        ln.copy_(i32(lens if i == 0 else [n - 2 for n in lens]))
        y.fill_(0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, refs[i])


def test_two_streams():
    """Calls on two streams at once, each with its own buffers, against one stream."""
    sets = []
    for i in range(2):
        lens = [900 + 300 * i, 70, 2500]
        table, pages = table_of(lens, 16, 13 + i)
        c = Cache(pages, 2, 16, 128, "bf16", seed=160 + i)
        q = rand((3, 8, 128), 161 + i, "bf16", 2.0).cuda()
        qp = rand((60, 8, 128), 163 + i, "bf16", 2.0).cuda()
        sets.append((q, qp, c, table, i32(lens), i32([0, 20, 21, 60]),
                     workspace(wq.wq_attention_decode_workspace(3, 8, c.c)),
                     workspace(wq.wq_attention_prompt_workspace(60, 8, 3, c.c)),
                     torch.empty_like(q), torch.empty_like(qp)))

    def issue(t, s):
        q, qp, c, table, lens, starts, w0, w1, y, yp = t
        for _ in range(3):
            wq.wq_attention_decode(q, c.c, table, lens, y, w0, stream=s)
            wq.wq_attention_prompt(qp, starts, c.c, table, lens, yp, w1, stream=s)

    torch.cuda.synchronize()
    for t in sets:
        issue(t, torch.cuda.current_stream())
    torch.cuda.synchronize()
    ref = [(t[-2].clone(), t[-1].clone()) for t in sets]
    for t in sets:
        t[-2].fill_(float("nan"))
        t[-1].fill_(float("nan"))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(2):
        for t, s in zip(sets, streams):
            issue(t, s)
    torch.cuda.synchronize()
    for t, r in zip(sets, ref):
        assert torch.equal(t[-2], r[0]) and torch.equal(t[-1], r[1])
