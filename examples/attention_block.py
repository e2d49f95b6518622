"""The attention half of a transformer block on quantized weights, with a paged cache.

  residual += x; q, k, v = FP8(RMSNorm(residual)) W_qkv; rotation; k, v into the cache
  (16 bits, or E4M3 with a scale per token and head); attention of the new rows over the
  cache; y = FP8(attention) W_o

takes the output x of the block before and the residual stream, updates the stream in
place and returns y, which the MLP half adds.  The same object takes prompts (any
number of rows per sequence, behind tokens that are in the cache already) and single
tokens.  Every buffer is allocated once, so a call only launches kernels: a decoding
step is captured in a graph and replayed while its lens, slots and positions grow.

    python examples/attention_block.py --batch 8 --prompt 500 --new 64
    python examples/attention_block.py --cache bf16 --window 256 --sinks 4
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_linear_int4_amd as wq  # noqa: E402
from mlp_block import pack_fp8  # noqa: E402


def rotary_table(max_pos, rot, theta=10000.0, device="cuda"):
    """cos and sin of position * theta^(-2 i / rot): angles in fp64, rounded once."""
    freq = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat((angle.cos(), angle.sin()), 1).float()


class Sequences:
    """The pages of a batch of sequences in a cache, and what the calls read of them."""

    def __init__(self, batch, max_len, page_size, device="cuda"):
        self.page_size, width = page_size, -(-max_len // page_size)
        # pages in a mixed order, as a server that gives them out over time has them
        order = torch.randperm(batch * width, device=device)
        self.pages = order.view(batch, width).int()
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.count = batch * width

    def add(self, new):
        """(positions, slots, starts) of `new` more tokens of each sequence; lens grows."""
        starts = torch.nn.functional.pad(torch.cumsum(new, 0), (1, 0)).int()
        seq = torch.repeat_interleave(torch.arange(len(new), device=new.device), new)
        pos = torch.arange(len(seq), device=new.device) - starts[seq] + self.lens[seq]
        slots = (self.pages[seq, pos // self.page_size] * self.page_size
                 + pos % self.page_size)
        self.lens += new.int()
        return pos.int(), slots.int(), starts


def _first_rows(codes, scales, rows):
    """(codes, scales) of `rows` rows in the buffers of alloc_fp8_rows for as many or more:
    scales stand [block][row] without gaps."""
    blocks = scales.shape[0]
    return codes[:rows], scales.view(-1)[:blocks * rows].view(blocks, rows)


class AttentionBlock:
    """w_qkv [(heads + 2 kv_heads) * head_dim][hidden], w_o [hidden][heads * head_dim] in
    16 bits; at most `tokens` rows a call, which use the first rows of every buffer."""

    def __init__(self, gain, w_qkv, w_o, heads, cache, table, tokens, window=0, sinks=0,
                 eps=1e-6):
        _, self.kv, _, d = cache.shape
        dt, dev = w_qkv.dtype, w_qkv.device
        hidden = w_o.shape[0]
        self.gain, self.eps, self.heads, self.d = gain, eps, heads, d
        self.cache, self.table, self.window, self.sinks = cache, table, window, sinks
        self.tokens = tokens
        self.w_qkv, self.w_o = pack_fp8(w_qkv), pack_fp8(w_o)
        self.q8, self.s = wq.alloc_fp8_rows(tokens, hidden, dev)
        self.qkv = torch.empty((tokens, heads + 2 * self.kv, d), dtype=dt, device=dev)
        self.q = torch.empty((tokens, heads, d), dtype=dt, device=dev)
        self.a = torch.empty_like(self.q)
        self.a8, self.s2 = wq.alloc_fp8_rows(tokens, heads * d, dev)
        self.y = torch.empty((tokens, hidden), dtype=dt, device=dev)
        # a linear of few rows, which splits k, may need more than one of many
        need = max(max(wq.wq_linear_fp8_workspace(rows, self.w_qkv),
                       wq.wq_linear_fp8_workspace(rows, self.w_o),
                       wq.wq_attention_decode_workspace(rows, heads, cache))
                   for rows in range(1, tokens + 1))
        need = max(need, wq.wq_attention_prompt_workspace(tokens, heads, 1, cache))
        self.ws = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)

    def _project(self, x, residual, positions, slots):
        rows, h, kv = len(x), self.heads, self.kv
        if rows > self.tokens:
            raise ValueError(f"{rows} rows in a block for {self.tokens}")
        q8, s = _first_rows(self.q8, self.s, rows)
        qkv, q = self.qkv[:rows], self.q[:rows]
        wq.wq_add_rmsnorm(x, self.gain, self.eps, residual=residual, residual_out=residual,
                          q=q8, scales=s)
        wq.wq_linear_fp8(q8, s, self.w_qkv, qkv.view(rows, -1), self.ws)
        wq.wq_append_kv(qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:], self.cache, slots,
                        positions=positions, cos_sin=self.table, q_out=q)
        return q, self.a[:rows]

    def _output(self, a):
        y = self.y[:len(a)]
        a8, s2 = _first_rows(self.a8, self.s2, len(a))
        wq.wq_quantize_fp8_rows(a.view(len(a), -1), a8, s2)
        wq.wq_linear_fp8(a8, s2, self.w_o, y, self.ws)
        return y

    def prompt(self, x, residual, positions, slots, starts, pages, lens):
        q, a = self._project(x, residual, positions, slots)
        wq.wq_attention_prompt(q, starts, self.cache, pages, lens, a, self.ws,
                               window=self.window, sinks=self.sinks)
        return self._output(a)

    def decode(self, x, residual, positions, slots, pages, lens):
        q, a = self._project(x, residual, positions, slots)
        wq.wq_attention_decode(q, self.cache, pages, lens, a, self.ws, window=self.window,
                               sinks=self.sinks)
        return self._output(a)


def plain(xs, gain, w_qkv, w_o, heads, kv, d, table, eps, window, sinks):
    """y of the last token of one sequence from its residual stream xs [n][hidden], fp64."""
    n, group = len(xs), heads // kv
    v = xs * torch.rsqrt(xs.square().mean(-1, keepdim=True) + eps) * gain.double()
    qkv = (v @ w_qkv.double().t()).view(n, heads + 2 * kv, d)
    t, half = table[:n].double(), d // 2
    c, s = t[:, None, :half], t[:, None, half:]
    r = qkv[:, :heads + kv]
    r = torch.cat((r[..., :half] * c - r[..., half:] * s, r[..., half:] * c + r[..., :half] * s), -1)
    q, k, val = r[-1, :heads], r[:, heads:], qkv[:, heads + kv:]
    j = torch.arange(n, device=xs.device)
    seen = (n - 1 - j < window) | (j < sinks) if window else j >= 0
    out = []
    for h in range(heads):
        z = (k[:, h // group] @ q[h]) * d ** -0.5
        z[~seen] = -float("inf")
        out.append(z.softmax(0) @ val[:, h // group])
    return w_o.double() @ torch.cat(out)


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--batch", type=int, default=8)
    p.add_argument("--prompt", type=int, default=500)
    p.add_argument("--new", type=int, default=32)
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--heads", type=int, default=32)
    p.add_argument("--kv-heads", type=int, default=8)
    p.add_argument("--head-dim", type=int, default=128)
    p.add_argument("--page-size", type=int, default=64)
    p.add_argument("--cache", choices=("bf16", "e4m3"), default="e4m3")
    p.add_argument("--window", type=int, default=0)
    p.add_argument("--sinks", type=int, default=0)
    a = p.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)

    def rand(*shape, scale=1.0):
        return (torch.randn(shape, device="cuda", generator=g) * scale).bfloat16()

    b, kv, d, hidden = a.batch, a.kv_heads, a.head_dim, a.hidden
    total = a.prompt + a.new
    gain = rand(hidden, scale=0.1) + 1
    w_qkv = rand((a.heads + 2 * kv) * d, hidden, scale=0.03)
    w_o = rand(hidden, a.heads * d, scale=0.02)
    table = rotary_table(total, d)
    seqs = Sequences(b, total, a.page_size)
    dt = torch.bfloat16 if a.cache == "bf16" else torch.float8_e4m3fn
    cache = wq.alloc_kv_cache(seqs.count, kv, a.page_size, d, dt)
    weights = (gain, w_qkv, w_o, a.heads, cache, table)
    block = AttentionBlock(*weights, b * a.prompt, a.window, a.sinks)
    step = AttentionBlock(*weights, b, a.window, a.sinks)

    # prompts of all sequences in one call
    x, r = rand(b * a.prompt, hidden), torch.zeros((b * a.prompt, hidden), dtype=torch.bfloat16,
                                                   device="cuda")
    where = seqs.add(torch.full((b,), a.prompt, device="cuda"))
    stream = x.view(b, a.prompt, hidden)
    e0, e1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    block.prompt(x, r.clone(), *where, seqs.pages, seqs.lens)
    e0.record()
    block.prompt(x, r, *where, seqs.pages, seqs.lens)
    e1.record()
    torch.cuda.synchronize()
    print(f"prompt: {b} x {a.prompt} tokens, {e0.elapsed_time(e1) * 1e3:.0f} us")

    # single tokens: one graph, whose inputs are refilled between its replays
    x1 = torch.zeros((b, hidden), dtype=torch.bfloat16, device="cuda")
    r1 = torch.zeros_like(x1)
    pos, slots = (torch.zeros(b, dtype=torch.int32, device="cuda") for _ in range(2))
    slots.fill_(-1)                                      # the first run stores nothing
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step.decode(x1, r1, pos, slots, seqs.pages, seqs.lens)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            step.decode(x1, r1, pos, slots, seqs.pages, seqs.lens)
    times, new = [], []
    for _ in range(a.new):
        token = rand(b, hidden)
        new.append(token)
        x1.copy_(token)
        r1.zero_()
        p1, s1, _ = seqs.add(torch.ones(b, dtype=torch.int64, device="cuda"))
        pos.copy_(p1)
        slots.copy_(s1)
        e0.record()
        graph.replay()
        e1.record()
        torch.cuda.synchronize()
        times.append(e0.elapsed_time(e1) * 1e3)
    full = torch.cat((stream, torch.stack(new, 1)), 1)[0].double()
    ref = plain(full, gain, w_qkv, w_o, a.heads, kv, d, table, step.eps, a.window, a.sinks)
    err = float((step.y[0].double() - ref).norm() / ref.norm())
    print(f"decode: {b} sequences of {a.prompt} to {total} tokens, {a.cache} cache: "
          f"{sorted(times)[len(times) // 2]:.1f} us a step, {err:.3f} from the unquantized block")


if __name__ == "__main__":
    main()
