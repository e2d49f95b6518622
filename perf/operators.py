"""The FP8 and mixture-of-experts operators of libwq as cases that can be timed.

Five operators of one transformer block, in the order a block runs them:

  norm    residual addition and root-mean-square norm, with 16-bit and / or
          FP8 outputs (``wq_add_rmsnorm``)
  rows    FP8 quantization of activation rows, plain or of silu(x) * up
          (``wq_quantize_fp8_rows``)
  linear  the FP8 x FP8 product with a scale per 128 activations of a row and
          per 128 x 128 weights (``wq_linear_fp8``)
  moe     router, top-k, gate/up, SiLU product, down and combination of a
          mixture-of-experts layer for a few tokens, INT4 or FP8 experts
          (``wq_moe``)

``own = False`` computes them with elementary torch operations in fp32;
``own = True`` calls the library.  ``exact`` is the definition in fp64.
"""

import math

import torch

own = False

F8 = torch.float8_e4m3fn
F8_MAX = 448.0
B = 128                      # elements that share an FP8 scale
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decoded token of a 4096-wide model before its FP8 projections
        {"name": "norm m1 k4096", "op": "norm", "m": 1, "k": 4096, "dtype": "bf16",
         "residual": True, "y16": False, "fp8": True},
        # a ragged prompt batch where both a 16-bit consumer (router) and an
        # FP8 one (projections) read the norm
        {"name": "norm m509 k5008", "op": "norm", "m": 509, "k": 5008, "dtype": "f16",
         "residual": True, "y16": True, "fp8": True},
        # a long prompt of the 8192-wide model
        {"name": "norm m8192 k8192", "op": "norm", "m": 8192, "k": 8192, "dtype": "bf16",
         "residual": True, "y16": False, "fp8": True},
        # the gated product of a decode batch on its way to an FP8 down projection
        {"name": "rows silu m16 k11008", "op": "rows", "m": 16, "k": 11008, "dtype": "f16",
         "gated": True},
        # the same for a prompt
        {"name": "rows silu m2048 k14336", "op": "rows", "m": 2048, "k": 14336,
         "dtype": "bf16", "gated": True},
        # one decoded token, an attention projection
        {"name": "linear m1 4096x4096", "op": "linear", "m": 1, "n": 4096, "k": 4096,
         "ydt": "bf16"},
        # a decode batch through the down projection
        {"name": "linear m16 4096x11008", "op": "linear", "m": 16, "n": 4096, "k": 11008,
         "ydt": "f16"},
        # a short prompt, sizes that end inside tiles and scale blocks
        {"name": "linear m333 5000x4112", "op": "linear", "m": 333, "n": 5000, "k": 4112,
         "ydt": "f32"},
        # a long prompt through a gate or up projection
        {"name": "linear m4096 14336x4096", "op": "linear", "m": 4096, "n": 14336, "k": 4096,
         "ydt": "bf16"},
        # one token through 8 of 64 small experts
        {"name": "moe int4 t1 e64", "op": "moe", "t": 1, "experts": 64, "top_k": 8, "h": 2048,
         "i": 1024, "fmt": "int4", "group": 128, "dtype": "bf16"},
        # a decode batch that touches most of the small experts
        {"name": "moe fp8 t24 e64", "op": "moe", "t": 24, "experts": 64, "top_k": 6, "h": 2048,
         "i": 1024, "fmt": "fp8", "group": 128, "dtype": "bf16"},
        # the largest decode batch, 2 of 8 large experts for each token
        {"name": "moe int4 t64 e8", "op": "moe", "t": 64, "experts": 8, "top_k": 2, "h": 4096,
         "i": 14336, "fmt": "int4", "group": 128, "dtype": "f16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "rows", "linear", "linear", "moe", "moe"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "norm":
        m, k = _log(rng, 1, 8192), 8 * _log(rng, 32, 1024)
        y16, fp8 = rng.choice([(False, True), (True, True), (True, False)])
        return {"op": op, "m": m, "k": k, "dtype": dtype, "residual": rng.random() < 0.75,
                "y16": y16, "fp8": fp8}
    if op == "rows":
        return {"op": op, "m": _log(rng, 1, 2048), "k": 16 * _log(rng, 16, 896), "dtype": dtype,
                "gated": rng.random() < 0.7}
    if op == "linear":
        m, n, k = _log(rng, 1, 4096), _log(rng, 128, 14336), 16 * _log(rng, 16, 256)
        return {"op": op, "m": m, "n": n, "k": k, "ydt": rng.choice(["f16", "bf16", "f32"])}
    fmt = rng.choice(["int4", "int4", "fp8"])
    group = rng.choice([128, 128, 64, 32]) if fmt == "int4" else 128
    if rng.random() < 0.5:
        e, top_k = rng.choice([16, 60, 64, 128]), rng.choice([4, 6, 8])
        h, i = 128 * rng.randint(8, 32), 128 * rng.randint(4, 12)
    else:
        e, top_k = 8, rng.choice([1, 2])
        h, i = 4096, 128 * rng.randint(32, 112)
    while e * h * i > 8 * 4096 * 14336 or (fmt == "fp8" and e * h * i > 4 * 4096 * 14336):
        i -= 128
    return {"op": op, "t": _log(rng, 1, 64), "experts": e, "top_k": top_k, "h": h, "i": i,
            "fmt": fmt, "group": group, "dtype": dtype}


# ------------------------------------------------------------------ inputs
def _randn(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _activations(g, m, k, dtype):
    """N(0, 1) rows with a few channels of larger magnitude, as hidden states have."""
    x = _randn(g, m, k)
    at = torch.randint(0, k, (4,), device="cuda", generator=g)
    x[:, at] = x[:, at] * 20.0
    return x.to(DT[dtype])


def _int4(g, n, k, group):
    """INT4 codes, fp16 scales and packed 4-bit zero points of an [n][k] weight
    whose values are near N(0, 0.016)."""
    codes = torch.empty((n, k // 8), dtype=torch.int32, device="cuda")
    step = max(1, (1 << 25) // k)
    for r in range(0, n, step):
        c = (_randn(g, min(step, n - r), k // 8, 8) * 2.7 + 7.5).round_().clamp_(0, 15)
        c = c.to(torch.int32)
        c <<= torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
        codes[r:r + step] = c.sum(-1).to(torch.int32)
    ng = k // group
    u = torch.rand((n, ng), device="cuda", generator=g)
    z = torch.randint(6, 10, (n, 2 * ((ng + 1) // 2)), device="cuda", generator=g)
    if ng % 2:
        z[:, -1] = 0
    z = (z[:, 0::2] | (z[:, 1::2] << 4)).to(torch.uint8)
    return {"codes": codes, "scales": (0.006 * (0.8 + 0.4 * u)).half(), "zeros": z}


def _fp8(g, n, k):
    """E4M3 codes and fp32 scales per 128 x 128 block of an [n][k] weight near N(0, 0.02)."""
    codes = torch.empty((n, k), dtype=F8, device="cuda")
    step = max(1, (1 << 25) // k)
    for r in range(0, n, step):
        c = _randn(g, min(step, n - r), k) * (F8_MAX / 4.5)
        codes[r:r + step] = c.clamp_(-F8_MAX, F8_MAX).to(F8)
    u = torch.rand((-(-n // B), -(-k // B)), device="cuda", generator=g)
    return {"codes": codes, "scales": 0.02 * 4.5 / F8_MAX * (0.8 + 0.4 * u)}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op in ("norm", "rows"):
        m, k, dt = case["m"], case["k"], DT[case["dtype"]]
        s["x"] = _activations(g, m, k, case["dtype"])
        if op == "norm":
            s["gain"] = (1.0 + 0.1 * _randn(g, k)).to(dt)
            s["eps"] = 1e-5
            s["res"] = _activations(g, m, k, case["dtype"]) if case["residual"] else None
            s["res_out"] = torch.empty_like(s["x"]) if case["residual"] else None
            s["y"] = torch.empty_like(s["x"]) if case["y16"] else None
        else:
            s["up"] = _randn(g, m, k).to(dt) if case["gated"] else None
        fp8 = case.get("fp8", True)
        s["q"] = torch.empty((m, k), dtype=F8, device="cuda") if fp8 else None
        s["scales"] = torch.empty((-(-k // B), m), device="cuda") if fp8 else None
    elif op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        x = _activations(g, m, k, "bf16").float()
        v = torch.nn.functional.pad(x, (0, -k % B)).view(m, -1, B)
        a = v.abs().amax(-1) / F8_MAX
        s["xq"] = (v / a[..., None]).view(m, -1)[:, :k].to(F8).contiguous()
        s["xs"] = a.t().contiguous()
        w = _fp8(g, n, k)
        s["codes"], s["wscales"] = w["codes"], w["scales"]
        s["y"] = torch.empty((m, n), dtype=DT[case["ydt"]], device="cuda")
        # scratch, as a program that runs many layers keeps it once
        s["ws"] = torch.empty((64 << 20,), dtype=torch.uint8, device="cuda")
    else:
        t, e, h, i = case["t"], case["experts"], case["h"], case["i"]
        dt = DT[case["dtype"]]
        s["x"] = _randn(g, t, h).to(dt)
        s["router"] = (0.03 * _randn(g, e, h)).to(dt)
        pack = (lambda n, k: _int4(g, n, k, case["group"])) if case["fmt"] == "int4" else (
            lambda n, k: _fp8(g, n, k))
        s["gate"], s["up"], s["down"] = pack(e * i, h), pack(e * i, h), pack(e * h, i)
        s["y"] = torch.empty((t, h), dtype=dt, device="cuda")
        s["ids"] = torch.empty((t, case["top_k"]), dtype=torch.int32, device="cuda")
        s["probs"] = torch.empty((t, case["top_k"]), device="cuda")
        s["ws"] = torch.empty((64 << 20,), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------- plain forms
def _plain_rows_fp8(v):
    """fp32 [m][k] -> E4M3 rows and their scales [ceil(k / 128)][m]."""
    m, k = v.shape
    v = torch.nn.functional.pad(v, (0, -k % B)).view(m, -1, B)
    a = v.abs().amax(-1) / F8_MAX
    a = torch.where(a == 0, torch.ones_like(a), a)
    q = (v / a[..., None]).view(m, -1)[:, :k].to(F8)
    return q.contiguous(), a.t().contiguous()


def _plain_norm(s):
    v = s["x"].float()
    out = {}
    if s["res"] is not None:
        v = v + s["res"].float()
        out["residual"] = v.to(s["x"].dtype)
    v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + s["eps"]) * s["gain"].float()
    if s["y16"]:
        out["y"] = v.to(s["x"].dtype)
    if s["fp8"]:
        out["q"], out["scales"] = _plain_rows_fp8(v)
    return out


def _plain_rows(s):
    v = s["x"].float()
    if s["up"] is not None:
        v = v / (1.0 + torch.exp(-v)) * s["up"].float()
    q, scales = _plain_rows_fp8(v)
    return {"q": q, "scales": scales}


def _plain_fp8_weight(codes, scales):
    n, k = codes.shape
    e = scales.repeat_interleave(B, 0)[:n].repeat_interleave(B, 1)[:, :k]
    return codes.float() * e


def _plain_linear(s):
    m, k = s["xq"].shape
    x = s["xq"].float() * s["xs"].t().repeat_interleave(B, 1)[:, :k]
    w = _plain_fp8_weight(s["codes"], s["wscales"])
    return {"y": torch.matmul(x, w.t()).to(s["y"].dtype)}


def _plain_int4_weight(w, group):
    n = w["codes"].shape[0]
    shift = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    q = ((w["codes"][..., None] >> shift) & 15).float().view(n, -1, group)
    ng = q.shape[1]
    z = torch.stack((w["zeros"] & 15, w["zeros"] >> 4), -1).view(n, -1)[:, :ng].float()
    return ((q - z[..., None]) * w["scales"].float()[..., None]).view(n, -1)


def _plain_moe(s):
    t, e, h, i, top = s["t"], s["experts"], s["h"], s["i"], s["top_k"]
    x = s["x"].float()
    p = torch.softmax(torch.matmul(x, s["router"].float().t()), -1)
    p, ids = torch.sort(p, dim=-1, descending=True, stable=True)
    p, ids = p[:, :top], ids[:, :top]
    p = p / p.sum(-1, keepdim=True)
    if s["fmt"] == "int4":
        gate, up, down = (_plain_int4_weight(s[n], s["group"]) for n in ("gate", "up", "down"))
    else:
        gate, up, down = (_plain_fp8_weight(s[n]["codes"], s[n]["scales"])
                          for n in ("gate", "up", "down"))
    a = torch.matmul(x, gate.t())
    a = a / (1.0 + torch.exp(-a)) * torch.matmul(x, up.t())
    share = torch.zeros((t, e), device="cuda").scatter_(1, ids, p)
    a = (a.view(t, e, i) * share[..., None]).transpose(0, 1).contiguous()     # [e][t][i]
    y = torch.bmm(a, down.view(e, h, i).transpose(1, 2).contiguous()).sum(0)
    return {"y": y.to(s["y"].dtype), "ids": ids.int(), "probs": p}


# ------------------------------------------------------------ library calls
def _weight(wq, w, n, k, group):
    if group:
        return wq.QuantizedWeight(wq.FMT_INT4_ASYM, n, k, group, w["codes"], w["scales"],
                                  w["zeros"])
    return wq.QuantizedWeight(wq.FMT_FP8_BLOCK, n, k, B, w["codes"], w["scales"])


def _own(s):
    import bit_quantized_linear_int4_amd as wq
    op = s["op"]
    if op == "norm":
        wq.wq_add_rmsnorm(s["x"], s["gain"], s["eps"], residual=s["res"],
                          residual_out=s["res_out"], y=s["y"], q=s["q"], scales=s["scales"])
        out = {"residual": s["res_out"], "y": s["y"], "q": s["q"], "scales": s["scales"]}
        return {n: v for n, v in out.items() if v is not None}
    if op == "rows":
        wq.wq_quantize_fp8_rows(s["x"], s["q"], s["scales"], up=s["up"])
        return {"q": s["q"], "scales": s["scales"]}
    if op == "linear":
        w = wq.QuantizedWeight(wq.FMT_FP8_BLOCK, s["n"], s["k"], B, s["codes"], s["wscales"])
        wq.wq_linear_fp8(s["xq"], s["xs"], w, s["y"], s["ws"])
        return {"y": s["y"]}
    e, h, i = s["experts"], s["h"], s["i"]
    group = s["group"] if s["fmt"] == "int4" else 0
    wq.wq_moe(s["x"], s["router"], s["top_k"], _weight(wq, s["gate"], e * i, h, group),
              _weight(wq, s["up"], e * i, h, group), _weight(wq, s["down"], e * h, i, group),
              s["y"], s["ws"], renormalize=True, ids=s["ids"], probs=s["probs"])
    return {"y": s["y"], "ids": s["ids"], "probs": s["probs"]}


PLAIN = {"norm": _plain_norm, "rows": _plain_rows, "linear": _plain_linear, "moe": _plain_moe}


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# -------------------------------------------------------------------- work
def work(case):
    """Bytes: each input once, each output once.  Flops: two per multiply-add."""
    op = case["op"]
    if op in ("norm", "rows"):
        m, k = case["m"], case["k"]
        fp8 = m * k + 4 * m * -(-k // B)
        if op == "rows":
            return {"bytes": (4 if case["gated"] else 2) * m * k + fp8,
                    "flops": (6 if case["gated"] else 2) * m * k}
        n16 = 1 + 2 * case["residual"] + case["y16"]
        return {"bytes": 2 * n16 * m * k + 2 * k + (fp8 if case["fp8"] else 0),
                "flops": 6 * m * k}
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // B)
        out = 4 if case["ydt"] == "f32" else 2
        return {"bytes": m * k + 4 * m * kb + n * k + 4 * kb * -(-n // B) + out * m * n,
                "flops": 2 * m * n * k}
    t, e, top, h, i = (case[n] for n in ("t", "experts", "top_k", "h", "i"))
    # experts that t tokens reach when each takes top of e at random
    hit = e * (1.0 - (1.0 - top / e) ** t)
    per = 1.0 / B / B * 4 + 1 if case["fmt"] == "fp8" else 0.5 + 2.5 / case["group"]
    return {"bytes": hit * 3 * h * i * per + 2 * e * h + 4 * t * h + 8 * t * top,
            "flops": 2 * t * (e * h + top * 3 * h * i)}


# ------------------------------------------------------- definition in fp64
def _e4m3(v):
    """fp64 -> the nearest E4M3 value, ties to even, saturating."""
    _, ex = torch.frexp(v)                      # |v| = f * 2^ex, f in [1/2, 1)
    step = torch.exp2((ex - 4).clamp(min=-9).double())
    return (torch.round(v / step) * step).clamp(-F8_MAX, F8_MAX)


def _exact_fp8(v):
    m, k = v.shape
    kb = -(-k // B)
    scales = torch.empty((kb, m), dtype=torch.float64, device=v.device)
    q = torch.empty_like(v)
    for b in range(kb):
        part = v[:, b * B:(b + 1) * B]
        a = part.abs().max(1).values / F8_MAX
        scales[b] = torch.where(a > 0, a, 1.0)
        q[:, b * B:(b + 1) * B] = _e4m3(part / scales[b][:, None])
    return {"q": q, "scales": scales}


def _exact_weight(s, name, rows, group):
    """Rows [r0, r1) of a packed weight in fp64."""
    w, (r0, r1) = s[name], rows
    codes = w["codes"][r0:r1]
    if s["fmt"] == "fp8":
        r = torch.arange(r0, r1, device="cuda") // B
        c = torch.arange(codes.shape[1], device="cuda") // B
        return codes.double() * w["scales"].double()[r][:, c]
    n, words = codes.shape
    out = torch.empty((n, words * 8), dtype=torch.float64, device="cuda")
    wide = codes.long() & 0xFFFFFFFF
    for j in range(8):
        out[:, j::8] = torch.bitwise_and(wide >> (4 * j), 15).double()
    for gi in range(words * 8 // group):
        byte = w["zeros"][r0:r1, gi // 2].long()
        z = (byte >> (4 * (gi % 2))) % 16
        cols = slice(gi * group, (gi + 1) * group)
        out[:, cols] = (out[:, cols] - z[:, None]) * w["scales"][r0:r1, gi].double()[:, None]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        v = s["x"].double()
        out = {}
        if case["residual"]:
            v = v + s["res"].double()
            out["residual"] = v
        rms = torch.sqrt(v.square().sum(1) / case["k"] + s["eps"])
        v = v / rms[:, None] * s["gain"].double()
        if case["y16"]:
            out["y"] = v
        return {**out, **(_exact_fp8(v) if case["fp8"] else {})}
    if op == "rows":
        v = s["x"].double()
        if case["gated"]:
            v = v * torch.sigmoid(v) * s["up"].double()
        return _exact_fp8(v)
    if op == "linear":
        y = torch.zeros((case["m"], case["n"]), dtype=torch.float64, device="cuda")
        for b in range(s["xs"].shape[0]):
            cols = slice(b * B, (b + 1) * B)
            part = torch.matmul(s["xq"][:, cols].double(), s["codes"][:, cols].double().t())
            sw = s["wscales"][:, b].double().repeat_interleave(B)[:case["n"]]
            y += part * s["xs"][b].double()[:, None] * sw
        return {"y": y}
    t, e, h, i, top = (case[n] for n in ("t", "experts", "h", "i", "top_k"))
    x = s["x"].double()
    logits = torch.matmul(x, s["router"].double().t())
    ids = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :top]
    chosen = torch.gather(logits, 1, ids)
    chosen = torch.exp(chosen - chosen[:, :1])
    probs = chosen / chosen.sum(1, keepdim=True)
    y = torch.zeros((t, h), dtype=torch.float64, device="cuda")
    for ex in torch.unique(ids).tolist():
        tok, pick = torch.nonzero(ids == ex, as_tuple=True)
        a = torch.matmul(x[tok], _exact_weight(s, "gate", (ex * i, ex * i + i), case["group"]).t())
        u = torch.matmul(x[tok], _exact_weight(s, "up", (ex * i, ex * i + i), case["group"]).t())
        a = a * torch.sigmoid(a) * u * probs[tok, pick][:, None]
        d = _exact_weight(s, "down", (ex * h, ex * h + h), case["group"])
        y.index_add_(0, tok, torch.matmul(a, d.t()))
    return {"y": y, "ids": ids.int(), "probs": probs}
