"""examples/attention_block.py on the GPU: each stage against the fp64 oracle on the
values the stage before it left, with the tolerances of the operators' own tests, for
prompts, for chunks behind them and for single tokens, and replays of a decoding step's
graph against eager calls, bit for bit.  A whole layer: the attention half and the MLP
half of mlp_block.py, one after the other on one residual stream."""

import os
import sys

import numpy as np
import pytest
import torch

import bit_quantized_linear_int4_amd as wq
from gpu_util import say
from test_gpu_attention import DECODE_R, check, np64, prompt_r, rotated
from test_gpu_fp8 import TINY, ULP, check_codes, check_linear, rand
from test_gpu_mlp_block import norm_of

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

pytestmark = pytest.mark.gpu

TD = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


class Setup:
    def __init__(self, batch, heads, kv, d, hidden, dtype, cdtype, max_len=160, page=16, window=0,
                 sinks=0):
        import attention_block as ab
        self.ab, self.dtype, self.cdtype = ab, dtype, cdtype
        self.hidden, self.window, self.sinks = hidden, window, sinks
        torch.manual_seed(5)
        self.seqs = ab.Sequences(batch, max_len, page)
        self.cache = wq.alloc_kv_cache(self.seqs.count, kv, page, d, TD[cdtype])
        self.table = ab.rotary_table(max_len, d)
        self.gain = rand((hidden,), 1, dtype).cuda()
        self.weights = (rand(((heads + 2 * kv) * d, hidden), 2, dtype, 0.06).cuda(),
                        rand((hidden, heads * d), 3, dtype, 0.06).cuda())
        self.heads = heads

    def block(self, rows):
        return self.ab.AttentionBlock(self.gain, *self.weights, self.heads, self.cache, self.table,
                                      rows, self.window, self.sinks)

    def values(self):
        out = []
        for t, s in ((self.cache.k, self.cache.k_scales), (self.cache.v, self.cache.v_scales)):
            x = np64(t.float())
            out.append(x if s is None else x * np64(s)[..., None])
        return out

    def check(self, b, x, r, before, pos, slots, rows, tolerance, y):
        """The stages of a call that has just run."""
        h, kv = b.heads, b.kv
        hs, v, tol = norm_of(x, before, self.gain, b.eps, self.dtype)
        assert np.all(np.abs(np64(r) - hs) <= (ULP[self.dtype] + 2.0 ** -23) * np.abs(hs)
                      + TINY[self.dtype])
        check_codes(b.q8, b.s, v, tol)
        check_linear(b.qkv.view(len(x), -1), b.q8, b.s, b.w_qkv, self.dtype)
        qr, qe = rotated(b.qkv[:, :h], pos, self.table, False)
        kr, ke = rotated(b.qkv[:, h:h + kv], pos, self.table, False)
        u = ULP[self.dtype]
        assert np.all(np.abs(np64(b.q) - qr) <= qe + u * (np.abs(qr) + qe) + TINY[self.dtype])
        size = self.cache.shape[2]
        pg, at = slots.long() // size, slots.long() % size
        k8, v8 = self.values()
        k8, v8 = k8[pg.cpu(), :, at.cpu()], v8[pg.cpu(), :, at.cpu()]
        vr = np64(b.qkv[:, h + kv:])
        step = 2.0 ** -4 if self.cdtype == "e4m3" else u
        for got, ref, err in ((k8, kr, ke), (v8, vr, 0 * vr)):
            small = 2.0 ** -10 * np.abs(ref).max(-1, keepdims=True) / 448
            assert np.all(np.abs(got - ref) <= step * (1 + 2.0 ** -10) * (np.abs(ref) + err) + 2 * err
                          + small * (1 + 2.0 ** -10) + TINY[self.dtype])
        check(b.a, None, b.q, self.values(), rows, b.d ** -0.5, self.window, self.sinks, tolerance,
              self.dtype, self.seqs.pages.cpu().numpy())
        check_codes(b.a8, b.s2, np64(b.a).reshape(len(x), -1), 2.0 ** -22)
        check_linear(y, b.a8, b.s2, b.w_o, self.dtype)


@pytest.mark.parametrize("dtype,cdtype", [("bf16", "e4m3"), ("f16", "f16"), ("f16", "e4m3")])
@pytest.mark.parametrize("heads,kv,d,window,sinks", [(8, 2, 64, 0, 0), (4, 4, 128, 30, 2)])
def test_prompts_chunks_and_tokens(heads, kv, d, window, sinks, dtype, cdtype):
    say(f"attention block {heads} {kv} {d} {window} {dtype} {cdtype}")
    s = Setup(3, heads, kv, d, 256, dtype, cdtype, window=window, sinks=sinks)
    # prompts; then a chunk for two of the sequences; then two tokens for each
    for new in ([50, 1, 97], [20, 0, 3]):
        n = torch.tensor(new).cuda()
        ctx = s.seqs.lens.tolist()
        pos, slots, starts = s.seqs.add(n)
        m = int(n.sum())
        x, r = rand((m, 256), 11, dtype).cuda(), rand((m, 256), 12, dtype).cuda()
        before, b = r.clone(), s.block(m)
        y = b.prompt(x, r, pos, slots, starts, s.seqs.pages, s.seqs.lens)
        torch.cuda.synchronize()
        rows, at = [], 0
        for i, k in enumerate(new):
            rows += [(at + j, i, ctx[i] + j, ctx[i] + k) for j in range(k)]
            at += k
        s.check(b, x, r, before, pos, slots, rows, prompt_r(dtype, cdtype), y)
    b = s.block(3)
    for _ in range(2):
        pos, slots, _ = s.seqs.add(torch.ones(3, dtype=torch.int64, device="cuda"))
        x, r = rand((3, 256), 13, dtype).cuda(), rand((3, 256), 14, dtype).cuda()
        before = r.clone()
        y = b.decode(x, r, pos, slots, s.seqs.pages, s.seqs.lens)
        torch.cuda.synchronize()
        lens = s.seqs.lens.tolist()
        s.check(b, x, r, before, pos, slots, [(i, i, n - 1, n) for i, n in enumerate(lens)],
                DECODE_R, y)


def test_layer_replays():
    """Attention half, then MLP half, on one residual stream: a captured decoding step
    against eager steps on a second cache."""
    import mlp_block
    b, heads, kv, d, hidden, steps = 3, 4, 2, 64, 256, 3
    gate, up = (rand((384, hidden), 30 + i, "bf16", 0.06).cuda() for i in range(2))
    down = rand((hidden, 384), 32, "bf16", 0.06).cuda()
    xs = [rand((b, hidden), 40 + i, "bf16").cuda() for i in range(steps)]

    def make():
        s = Setup(b, heads, kv, d, hidden, "bf16", "e4m3")
        m = mlp_block.DenseMLP(s.gain, gate, up, down, b)
        n = torch.tensor([33, 5, 70]).cuda()
        pos, slots, starts = s.seqs.add(n)
        x = rand((108, hidden), 50, "bf16").cuda()
        s.block(108).prompt(x, torch.zeros_like(x), pos, slots, starts, s.seqs.pages,
                               s.seqs.lens)
        return s, s.block(b), m

    s, att, mlp = make()
    want = []
    for x in xs:
        r = torch.zeros_like(x)
        pos, slots, _ = s.seqs.add(torch.ones(b, dtype=torch.int64, device="cuda"))
        y = mlp(att.decode(x, r, pos, slots, s.seqs.pages, s.seqs.lens), r)
        torch.cuda.synchronize()
        want.append((y.clone(), r.clone()))
    assert not torch.equal(want[0][0], want[1][0])

    s, att, mlp = make()
    x, r = torch.zeros((b, hidden), dtype=torch.bfloat16, device="cuda"), torch.zeros(
        (b, hidden), dtype=torch.bfloat16, device="cuda")
    pos, slots = (torch.full((b,), -1, dtype=torch.int32, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        mlp(att.decode(x, r, pos, slots, s.seqs.pages, s.seqs.lens), r)
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            mlp(att.decode(x, r, pos, slots, s.seqs.pages, s.seqs.lens), r)
    for token, (y, after) in zip(xs, want):
        p1, s1, _ = s.seqs.add(torch.ones(b, dtype=torch.int64, device="cuda"))
        pos.copy_(p1)
        slots.copy_(s1)
        x.copy_(token)
        r.zero_()
        (x @ x.t().contiguous()).sum()                   # other work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(mlp.y, y) and torch.equal(r, after)
