"""Prompt calls whose tokens are split into parts: rows outside the sequences stay as they
were, windows and rows that see nothing of some parts agree with the fp64 oracle, and a
captured call whose lens change between its replays, from many parts to one and back, gives
the bits of calls with a workspace of their own."""

import numpy as np
import pytest
import torch

import bit_quantized_linear_int4_amd as wq
from gpu_util import say
from test_gpu_attention import Cache, check, i32, prompt_r, rand, table_of, workspace

pytestmark = pytest.mark.gpu

NAN = float("nan")


def call(q, starts, c, table, lens, ws, window=0, sinks=0):
    y = torch.full(q.shape, NAN, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], NAN, device="cuda")
    wq.wq_attention_prompt(q, starts, c.c, table, lens, y, ws, window=window, sinks=sinks, lse=lse)
    torch.cuda.synchronize()
    return y, lse


def fresh(q, c, table):
    return workspace(wq.wq_attention_prompt_workspace(q.shape[0], q.shape[1], len(table), c.c))


# rows and lens of the sequences, heads, kv heads, head size, window, sinks
CASES = [
    ([3, 0, 7, 2], [900, 500, 7, -3], 4, 2, 128, 0, 0),
    ([90, 4, 30], [1000, 2, 600], 8, 2, 128, 0, 0),
    ([64, 9], [1500, 800], 2, 1, 128, 513, 0),
    ([64, 9], [1500, 800], 3, 3, 64, 300, 70),
    ([128, 40], [1281, 513], 12, 4, 64, 0, 0),
]


@pytest.mark.parametrize("dtype,cdtype", [("bf16", "bf16"), ("f16", "f16"), ("f16", "e4m3")])
@pytest.mark.parametrize("case", CASES)
def test_rows_of_a_split_prompt(case, dtype, cdtype):
    new, lens, heads, kv, d, window, sinks = case
    say(f"split prompt {case} {dtype} {cdtype}")
    lead, tail = 2, 3
    table, pages = table_of(lens, 16, 400, extra=50)
    c = Cache(pages, kv, 16, d, cdtype, seed=400)
    starts = np.cumsum([lead] + new)
    q = rand((int(starts[-1]) + tail, heads, d), 403, dtype, 2.0).cuda()
    q[:lead], q[starts[-1]:] = NAN, NAN
    ws = fresh(q, c, table)
    y, lse = call(q, i32(starts), c, table, i32(lens), ws, window, sinks)
    assert (ws != 0xA5).any()
    for t in (y, lse):
        assert torch.isnan(t[:lead]).all() and torch.isnan(t[starts[-1]:]).all()
    rows = [(int(starts[s]) + i, s, lens[s] - n + i if lens[s] > 0 else -1, max(lens[s], 0))
            for s, n in enumerate(new) for i in range(n) if n < 20 or i % 9 in (0, 8)]
    check(y, lse, q, c.values(), rows, d ** -0.5, window, sinks, prompt_r(dtype, cdtype), dtype,
          table.cpu().numpy())


@pytest.mark.parametrize("window", [0, 200])
@pytest.mark.parametrize("heads,kv", [(4, 2), (16, 4)])
def test_a_captured_split_prompt(heads, kv, window):
    say(f"captured split prompt {heads} {kv} {window}")
    new, steps = [30, 8], [[1400, 900], [30, 900], [1400, 8], [200, 129], [0, 300], [1400, 900]]
    table, pages = table_of(steps[0], 16, 410)
    c = Cache(pages, kv, 16, 128, "bf16", seed=410)
    q, starts = rand((38, heads, 128), 413, "bf16", 2.0).cuda(), i32([0, 30, 38])
    want = [call(q, starts, c, table, i32(s), fresh(q, c, table), window, 3) for s in steps]
    ws, lens = fresh(q, c, table), i32(steps[0])
    y, lse = torch.empty_like(q), torch.empty((38, heads), device="cuda")

    def run():
        wq.wq_attention_prompt(q, starts, c.c, table, lens, y, ws, window=window, sinks=3, lse=lse)

    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        run()
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            run()
    assert (ws != 0xA5).any()
    for at, (wy, wl) in zip(steps, want):
        lens.copy_(i32(at))
        y.fill_(NAN)
        lse.fill_(NAN)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, wy) and torch.equal(lse, wl), at
