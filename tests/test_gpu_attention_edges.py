"""Calls at the ends of what wq.h allows, against the fp64 oracle with the tolerances of
test_gpu_attention: many sequences (more than a wave scans, more items than workgroups),
the most heads, groups larger than a workgroup's rows, pages that sequences share, caches
whose keys and values are one tensor, byte caches, graphs that share a workspace, and
prompts whose parts follow lens below what the page table could hold."""

import numpy as np
import pytest
import torch

import bit_quantized_linear_int4_amd as wq
from gpu_util import say
from test_gpu_attention import (DECODE_R, Cache, check, i32, prompt_r, rand, run_decode,
                                run_prompt, table_of, workspace)

pytestmark = pytest.mark.gpu


def rows_of(lens):
    return [(i, i, n - 1, max(n, 0)) for i, n in enumerate(lens)]


@pytest.mark.parametrize("m,heads,kv,d,page,cdtype,window,sinks", [
    (65, 4, 2, 64, 16, "bf16", 0, 0), (300, 4, 4, 128, 16, "e4m3", 0, 0),
    (700, 6, 2, 64, 32, "e4m3", 90, 4), (1500, 2, 1, 128, 64, "bf16", 0, 0),
    (129, 28, 4, 64, 32, "e4m3", 100, 4), (513, 1, 1, 64, 1, "bf16", 0, 0),
])
def test_decode_of_many_sequences(m, heads, kv, d, page, cdtype, window, sinks):
    say(f"many {m} {heads} {kv} {d} {page} {cdtype} {window}")
    g = np.random.default_rng(m)
    lens = [int(n) for n in g.integers(0, 300, m)]
    lens[3], lens[m // 2], lens[m - 1], lens[m - 2] = 1400, 0, 900, -4
    table, pages = table_of(lens, page, 5, extra=1)
    c = Cache(pages, kv, page, d, cdtype, seed=70)
    q = rand((m, heads, d), 71, "bf16", 2.0).cuda()
    y, lse = run_decode(q, c, table, i32(lens), window, sinks)
    some = sorted(set(list(range(8)) + list(range(60, 68)) + [m // 2, m - 2, m - 1]
                      + [int(i) for i in g.integers(0, m, 60)]))
    some = [i for i in some if i < m]
    check(y, lse, q, c.values(), [rows_of(lens)[i] for i in some], d ** -0.5, window, sinks,
          DECODE_R, "bf16", table.cpu().numpy())
    assert not torch.isnan(y).any() and not torch.isnan(lse).any()
    # each sequence by itself: the same sums, in other parts
    i = 3
    alone, _ = run_decode(q[i:i + 1], c, table[i:i + 1], i32([lens[i]]), window, sinks)
    check(alone, None, q[i:i + 1], c.values(), [(0, 0, lens[i] - 1, lens[i])], d ** -0.5, window,
          sinks, DECODE_R, "bf16", table[i:i + 1].cpu().numpy())


@pytest.mark.parametrize("heads,kv,d,cdtype", [(8, 4, 128, "bf16"), (66, 4, 64, "e4m3"),
                                               (8, 1, 128, "bf16"), (20, 20, 64, "bf16")])
def test_one_long_sequence_among_many(heads, kv, d, cdtype):
    """Its items have many parts, those of the others one or two."""
    say(f"one long {heads} {kv} {d} {cdtype}")
    heads = heads // kv * kv
    lens = [5, 200, 9000, 0, 130] + [int(n) for n in np.random.default_rng(2).integers(1, 60, 60)]
    table, pages = table_of(lens, 16, 14)
    c = Cache(pages, kv, 16, d, cdtype, seed=91)
    q = rand((len(lens), heads, d), 92, "bf16", 2.0).cuda()
    y, lse = run_decode(q, c, table, i32(lens))
    check(y, lse, q, c.values(), rows_of(lens)[:8], d ** -0.5, 0, 0, DECODE_R, "bf16",
          table.cpu().numpy())
    assert not torch.isnan(y).any()


@pytest.mark.parametrize("heads,kv,d", [(1024, 1, 64), (1024, 1024, 64), (1000, 8, 128),
                                        (272, 1, 128)])
def test_many_heads(heads, kv, d):
    say(f"heads {heads} {kv} {d}")
    lens, page = [70, 3], 16
    table, pages = table_of(lens, page, 9)
    c = Cache(pages, kv, page, d, "bf16", seed=72)
    q = rand((2, heads, d), 73, "bf16", 2.0).cuda()
    y, lse = run_decode(q, c, table, i32(lens))
    check(y, lse, q, c.values(), rows_of(lens), d ** -0.5, 0, 0, DECODE_R, "bf16",
          table.cpu().numpy())
    q = rand((5, heads, d), 74, "bf16", 2.0).cuda()
    y, lse = run_prompt(q, i32([0, 3, 5]), c, table, i32(lens), 40, 1)
    rows = [(0, 0, 67, 70), (1, 0, 68, 70), (2, 0, 69, 70), (3, 1, 1, 3), (4, 1, 2, 3)]
    check(y, lse, q, c.values(), rows, d ** -0.5, 40, 1, prompt_r("bf16", "bf16"), "bf16",
          table.cpu().numpy())


@pytest.mark.parametrize("cdtype", ["bf16", "e4m3"])
def test_shared_and_repeated_pages(cdtype):
    """A common prefix: its pages stand in several tables, one of them twice in one."""
    say(f"shared {cdtype}")
    c = Cache(7, 2, 16, 64, cdtype, seed=75)
    table = torch.tensor([[3, 1, 4, 0], [3, 1, 5, 5], [3, 1, 4, 2]], dtype=torch.int32).cuda()
    lens = [50, 64, 61]
    q = rand((3, 8, 64), 76, "bf16", 2.0).cuda()
    y, lse = run_decode(q, c, table, i32(lens))
    check(y, lse, q, c.values(), rows_of(lens), 0.125, 0, 0, DECODE_R, "bf16", table.cpu().numpy())
    q = rand((30, 8, 64), 77, "bf16", 2.0).cuda()
    y, lse = run_prompt(q, i32([0, 10, 20, 30]), c, table, i32(lens))
    rows = [(10 * s + i, s, n - 10 + i, n) for s, n in enumerate(lens) for i in range(10)]
    check(y, lse, q, c.values(), rows, 0.125, 0, 0, prompt_r("bf16", cdtype), "bf16",
          table.cpu().numpy())


@pytest.mark.parametrize("layout", ["pages", "heads"])
def test_keys_and_values_of_one_tensor(layout):
    """[pages][2][...] or [...][2 d]: strides between, no two places overlap."""
    say(f"one tensor {layout}")
    pages, kv, page, d = 6, 2, 16, 64
    if layout == "pages":
        both = rand((pages, 2, kv, page, d), 78, "f16").cuda()
        k, v = both[:, 0], both[:, 1]
    else:
        both = rand((pages, page, kv, 2 * d), 79, "f16").cuda().transpose(1, 2)
        k, v = both[..., :d], both[..., d:]
    cache = wq.KVCache(k, v)
    rows = rand((20, 8, d), 80, "f16").cuda()
    slots = i32(list(range(16, 32)) + list(range(80, 84)))
    want = [t.clone() for t in (k, v)]
    wq.wq_append_kv(rows[:, :4], rows[:, 4:6], rows[:, 6:], cache, slots,
                    q_out=torch.empty((20, 4, d), dtype=torch.float16, device="cuda"))
    torch.cuda.synchronize()
    for w, r in ((want[0], rows[:, 4:6]), (want[1], rows[:, 6:])):
        for i, s in enumerate(slots.tolist()):
            w[s // page, :, s % page] = r[i]
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    table = torch.tensor([[1, 5]], dtype=torch.int32).cuda()
    y = torch.empty((1, 4, d), dtype=torch.float16, device="cuda")
    ws = workspace(wq.wq_attention_decode_workspace(1, 4, cache))
    wq.wq_attention_decode(rows[:1, :4], cache, table, i32([20]), y, ws)
    torch.cuda.synchronize()
    check(y, None, rows[:1, :4], [t.double().cpu().numpy() for t in (k, v)], [(0, 0, 19, 20)],
          0.125, 0, 0, DECODE_R, "f16", table.cpu().numpy())


def test_byte_cache_is_the_e4m3_cache():
    say("bytes")
    lens = [100, 30]
    table, pages = table_of(lens, 16, 11)
    c = Cache(pages, 2, 16, 64, "e4m3", seed=81)
    b = wq.KVCache(c.k.view(torch.uint8), c.v.view(torch.uint8), c.ks, c.vs)
    q = rand((2, 4, 64), 82, "f16", 2.0).cuda()
    y, _ = run_decode(q, c, table, i32(lens))
    y2 = torch.empty_like(y)
    wq.wq_attention_decode(q, b, table, i32(lens), y2,
                           workspace(wq.wq_attention_decode_workspace(2, 4, b)))
    torch.cuda.synchronize()
    assert torch.equal(y, y2)


def test_graphs_that_share_a_workspace():
    """A prompt's and a decoding step's graph, replayed in turn, with eager calls between:
    all on one workspace, as the layers of a model would."""
    say("shared workspace")
    lens = [900, 40, 333]
    table, pages = table_of(lens, 16, 12)
    c = Cache(pages, 2, 16, 128, "bf16", seed=83)
    n = i32(lens)
    qd, qp = rand((3, 8, 128), 84, "bf16", 2.0).cuda(), rand((20, 8, 128), 85, "bf16", 2.0).cuda()
    starts = i32([0, 7, 8, 20])
    yd, yp = torch.zeros_like(qd), torch.zeros_like(qp)
    ws = workspace(max(wq.wq_attention_decode_workspace(3, 8, c.c),
                       wq.wq_attention_prompt_workspace(20, 8, 3, c.c)))

    def decode():
        wq.wq_attention_decode(qd, c.c, table, n, yd, ws)

    def prompt():
        wq.wq_attention_prompt(qp, starts, c.c, table, n, yp, ws)

    decode()
    prompt()
    torch.cuda.synchronize()
    want = yd.clone(), yp.clone()
    side, graphs = torch.cuda.Stream(), []
    for fn in (decode, prompt):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            fn()
            side.synchronize()
            with torch.cuda.graph(g, stream=side):
                fn()
        graphs.append(g)
    for i in range(4):
        yd.zero_()
        yp.zero_()
        ws.fill_(0x5A)
        torch.cuda.synchronize()
        for g in graphs if i % 2 else graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(yd, want[0]) and torch.equal(yp, want[1])
        prompt()
        decode()
        torch.cuda.synchronize()
        assert torch.equal(yd, want[0]) and torch.equal(yp, want[1])


@pytest.mark.parametrize("dtype,cdtype", [("bf16", "bf16"), ("f16", "e4m3")])
@pytest.mark.parametrize("d,heads,kv", [(128, 8, 2), (64, 6, 6)])
def test_prompt_under_a_long_table(d, heads, kv, dtype, cdtype):
    """The table has room for many times the tokens: parts are planned for that room, and
    most of them find none.  Lens of some sequences fill a few, one a single tile."""
    say(f"long table {d} {heads} {dtype} {cdtype}")
    new, ctx = [5, 1, 0, 9], [700, 20, 30, 0]
    lens = [a + b for a, b in zip(new, ctx)]
    table, pages = table_of(lens, 16, 13, extra=4000)
    c = Cache(pages, kv, 16, d, cdtype, seed=86)
    starts = [0, 5, 6, 6, 15]
    q = rand((15, heads, d), 87, dtype, 2.0).cuda()
    y, lse = run_prompt(q, i32(starts), c, table, i32(lens))
    rows = [(starts[s] + i, s, ctx[s] + i, lens[s]) for s, n in enumerate(new) for i in range(n)]
    check(y, lse, q, c.values(), rows, d ** -0.5, 0, 0, prompt_r(dtype, cdtype), dtype,
          table.cpu().numpy())
    again, _ = run_prompt(q, i32(starts), c, table, i32(lens))
    assert torch.equal(y, again)


def test_one_page_of_many_tokens():
    """The largest page, partly filled; a table of one entry."""
    say("page 65536")
    c = Cache(2, 1, 65536, 64, "bf16", seed=88)
    table = torch.tensor([[1]], dtype=torch.int32).cuda()
    q = rand((1, 2, 64), 89, "bf16", 2.0).cuda()
    y, lse = run_decode(q, c, table, i32([3000]), 700, 9)
    check(y, lse, q, c.values(), [(0, 0, 2999, 3000)], 0.125, 700, 9, DECODE_R, "bf16",
          table.cpu().numpy())
    q = rand((40, 2, 64), 90, "bf16", 2.0).cuda()
    y, lse = run_prompt(q, i32([0, 40]), c, table, i32([65536]), 700, 9)
    check(y, lse, q, c.values(), [(i, 0, 65496 + i, 65536) for i in (0, 17, 39)], 0.125, 700, 9,
          prompt_r("bf16", "bf16"), "bf16", table.cpu().numpy())
