"""The MLP half of a transformer block on quantized weights.

  dense:    residual += x; q = FP8(RMSNorm(residual)); y = down(FP8(silu(gate q) * up q))
            with E4M3 weights, one scale per 128 x 128 block
  experts:  residual += x; v = RMSNorm(residual); y = mixture of experts of v
            with INT4 weights, groups of 128

Both take the output x of the attention half and the residual stream, update
the stream in place and return y, which the next block adds.  Every buffer is
allocated once, so a call only launches kernels and can be captured in a graph.

    python examples/mlp_block.py --tokens 16 --hidden 4096 --inner 11008
    python examples/mlp_block.py --experts 64 --top-k 8 --hidden 2048 --inner 1024
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_linear_int4_amd as wq  # noqa: E402


def pack_fp8(w):
    q = wq.alloc_fp8(*w.shape, device=w.device)
    wq.wq_quantize_fp8_block(w, q.codes, q.scales)
    return q


def pack_int4(w, group=128):
    q = wq.alloc_int4(*w.shape, group, device=w.device)
    wq.wq_quantize_groupwise(w, 4, group, 0, q.codes, q.scales, q.zeros)
    return q


class DenseMLP:
    """gate, up [inner][hidden] and down [hidden][inner] in 16 bits, for `tokens`
    rows a call."""

    def __init__(self, gain, gate, up, down, tokens, eps=1e-6):
        inner, hidden = gate.shape
        dt, dev = gate.dtype, gate.device
        self.gain, self.eps = gain, eps
        self.gate, self.up, self.down = pack_fp8(gate), pack_fp8(up), pack_fp8(down)
        self.q, self.s = wq.alloc_fp8_rows(tokens, hidden, dev)
        self.q2, self.s2 = wq.alloc_fp8_rows(tokens, inner, dev)
        self.g = torch.empty((tokens, inner), dtype=dt, device=dev)
        self.u = torch.empty_like(self.g)
        self.y = torch.empty((tokens, hidden), dtype=dt, device=dev)
        need = max(wq.wq_linear_fp8_workspace(tokens, w) for w in (self.gate, self.down))
        self.ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None

    def __call__(self, x, residual):
        wq.wq_add_rmsnorm(x, self.gain, self.eps, residual=residual, residual_out=residual,
                          q=self.q, scales=self.s)
        wq.wq_linear_fp8(self.q, self.s, self.gate, self.g, self.ws)
        wq.wq_linear_fp8(self.q, self.s, self.up, self.u, self.ws)
        wq.wq_quantize_fp8_rows(self.g, self.q2, self.s2, up=self.u)
        wq.wq_linear_fp8(self.q2, self.s2, self.down, self.y, self.ws)
        return self.y


class ExpertsMLP:
    """router [experts][hidden], gate and up [experts][inner][hidden], down
    [experts][hidden][inner] in 16 bits, for `tokens` <= 64 rows a call."""

    def __init__(self, gain, router, gate, up, down, top_k, tokens, eps=1e-6):
        e, inner, hidden = gate.shape
        dt, dev = gate.dtype, gate.device
        self.gain, self.eps, self.router, self.top_k = gain, eps, router, top_k
        self.gate, self.up, self.down = (pack_int4(w.reshape(-1, w.shape[-1]))
                                         for w in (gate, up, down))
        self.v = torch.empty((tokens, hidden), dtype=dt, device=dev)
        self.y = torch.empty_like(self.v)
        self.ws = torch.empty(wq.wq_moe_workspace(tokens, top_k, self.gate, e),
                              dtype=torch.uint8, device=dev)

    def __call__(self, x, residual):
        wq.wq_add_rmsnorm(x, self.gain, self.eps, residual=residual, residual_out=residual,
                          y=self.v)
        wq.wq_moe(self.v, self.router, self.top_k, self.gate, self.up, self.down, self.y, self.ws)
        return self.y


def capture(block, x, residual):
    """A graph of one call on these tensors; the residual stream is put back."""
    keep, stream = residual.clone(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        block(x, residual)
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            block(x, residual)
    residual.copy_(keep)
    return graph


def plain(x, residual, gain, eps, mlp):
    h = x.double() + residual.double()
    return mlp(h * torch.rsqrt(h.square().mean(-1, keepdim=True) + eps) * gain.double())


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=16)
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--inner", type=int, default=11008)
    p.add_argument("--experts", type=int, default=0)
    p.add_argument("--top-k", type=int, default=2)
    p.add_argument("--steps", type=int, default=50)
    a = p.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)

    def rand(*shape, scale=1.0):
        return (torch.randn(shape, device="cuda", generator=g) * scale).bfloat16()

    x, r, gain = rand(a.tokens, a.hidden), rand(a.tokens, a.hidden), rand(a.hidden, scale=0.1) + 1
    lead = (a.experts,) if a.experts else ()
    gate, up = (rand(*lead, a.inner, a.hidden, scale=0.02) for _ in range(2))
    down = rand(*lead, a.hidden, a.inner, scale=0.02)
    silu = torch.nn.functional.silu
    if a.experts:
        router = rand(a.experts, a.hidden, scale=0.05)
        block = ExpertsMLP(gain, router, gate, up, down, a.top_k, a.tokens)

        def mlp(v):
            v16 = v.bfloat16().double()
            probs, ids = (v16 @ router.double().t()).softmax(-1).topk(a.top_k)
            probs = probs / probs.sum(-1, keepdim=True)
            rows = []
            for t in range(a.tokens):
                rows.append(sum(
                    pr * (down[e].double() @ (silu(gate[e].double() @ v[t]) * (up[e].double() @ v[t])))
                    for pr, e in zip(probs[t], ids[t].tolist())))
            return torch.stack(rows)
    else:
        block = DenseMLP(gain, gate, up, down, a.tokens)

        def mlp(v):
            gv, uv = v @ gate.double().t(), v @ up.double().t()
            return (silu(gv) * uv) @ down.double().t()

    ref = plain(x, r, gain, block.eps, mlp)
    graph = capture(block, x, r)
    graph.replay()
    torch.cuda.synchronize()
    err = float((block.y.double() - ref).norm() / ref.norm())
    e0, e1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    r.zero_()
    e0.record()
    for _ in range(a.steps):
        graph.replay()
    e1.record()
    torch.cuda.synchronize()
    kind = f"{a.experts} experts, top {a.top_k}, INT4" if a.experts else "dense, FP8"
    print(f"{kind}: {a.tokens} tokens, {a.hidden} x {a.inner}: "
          f"{e0.elapsed_time(e1) / a.steps * 1e3:.1f} us a call, "
          f"{err:.3f} from the unquantized product")


if __name__ == "__main__":
    main()
