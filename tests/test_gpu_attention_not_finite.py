"""Queries, keys, values and scales that are not finite in calls whose tokens are split into
parts and joined.  They reach every row that sees them, also where nothing else of a part
is visible to the row, and no other row.  Expected are the places alone, from what a row
sees, and the bits of the same call without them everywhere else; the leaving out of
z = -inf is compared with the fp64 oracle, with the tolerances of test_gpu_attention."""

import numpy as np
import pytest
import torch

import bit_quantized_linear_int4_amd as wq
from gpu_util import say
from test_gpu_attention import (DECODE_R, Cache, check, i32, prompt_r, rand, run_decode,
                                table_of)

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def bits(t):
    return t.view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def prompt(q, starts, c, table, lens, window=0, sinks=0):
    """(y, lse, whether parts went through the workspace)."""
    m, heads, _ = q.shape
    y = torch.zeros(q.shape, dtype=q.dtype, device="cuda")
    lse = torch.zeros((m, heads), device="cuda")
    n = wq.wq_attention_prompt_workspace(m, heads, len(lens), c.c)
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    wq.wq_attention_prompt(q, starts, c.c, table, lens, y, ws, window=window, sinks=sinks, lse=lse)
    torch.cuda.synchronize()
    return y, lse, bool((ws != 0xA5).any())


def places(table, seq, tokens, page):
    """(pages, places in them) of tokens of a sequence."""
    tokens = np.asarray(tokens)
    at = table.cpu().numpy()[seq, tokens // page]
    return torch.from_numpy(at).long().cuda(), torch.from_numpy(tokens % page).cuda()


def poison(c, what, table, seq, tokens, page, head, bad):
    t = getattr(c, what)
    pg, at = places(table, seq, tokens, page)
    if what in ("ks", "vs"):
        t[pg, head, at] = bad
    else:
        one = torch.full((1,), bad, device="cuda").to(t.dtype)
        if t.dtype == torch.float8_e4m3fn:
            t, one = t.view(torch.uint8), one.view(torch.uint8)
        t[pg, head, at, 5] = one


def reached(got, clean, hit, values_only=False):
    """NaN in y and lse of the rows and heads `hit` (with values_only in y alone, and there
    where a component that is not finite enters), the bits of `clean` everywhere else."""
    (y, lse), (y0, lse0) = got, clean
    assert torch.isfinite(y0).all() and torch.isfinite(lse0).all()
    keep = ~hit
    assert torch.equal(bits(y)[keep], bits(y0)[keep])
    if values_only:
        assert torch.equal(bits(lse), bits(lse0))
        assert not torch.isfinite(y[hit][:, 5]).any()
        return
    assert torch.equal(bits(lse)[keep], bits(lse0)[keep])
    assert torch.isnan(y[hit]).all() and torch.isnan(lse[hit]).all()


# (rows of two sequences, their lens, heads, kv, d): few rows, whose parts eight groups of
# threads join, and more of them, one group a row
SPLIT = [
    ([3, 2], [1000, 700], 4, 2, 128), ([1, 4], [3000, 600], 6, 2, 64),
    ([100, 60], [1000, 900], 8, 2, 128), ([150, 30], [1200, 800], 12, 2, 64),
]


def case_of(shape, dtype, cdtype, seed):
    new, lens, heads, kv, d = shape
    table, pages = table_of(lens, 16, seed, extra=3)
    c = Cache(pages, kv, 16, d, cdtype, seed=seed)
    q = rand((sum(new), heads, d), seed + 3, dtype, 2.0).cuda()
    return q, i32(np.cumsum([0] + new)), c, table, i32(lens)


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("dtype,cdtype", [("bf16", "bf16"), ("f16", "f16"), ("f16", "e4m3")])
@pytest.mark.parametrize("i", range(len(SPLIT)))
def test_a_query_of_a_split_prompt(i, dtype, cdtype, bad):
    say(f"split prompt, query {SPLIT[i]} {dtype} {cdtype} {bad}")
    args = case_of(SPLIT[i], dtype, cdtype, 200)
    q = args[0]
    y0, l0, split = prompt(*args)
    assert split
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    hit[1, 2] = hit[q.shape[0] - 1, 0] = True
    q[hit, 7] = bad
    y, lse, _ = prompt(*args)
    reached((y, lse), (y0, l0), hit)


@pytest.mark.parametrize("what,cdtype", [("k", "bf16"), ("v", "bf16"), ("k", "e4m3"),
                                         ("ks", "e4m3"), ("vs", "e4m3")])
@pytest.mark.parametrize("i", range(len(SPLIT)))
def test_tokens_that_fill_parts_of_a_prompt(i, what, cdtype):
    """Tokens 128 to 511, whole parts among them, of one kv head of one sequence."""
    new, _, heads, kv, _ = SPLIT[i]
    say(f"split prompt, tokens {SPLIT[i]} {what} {cdtype}")
    args = case_of(SPLIT[i], "bf16", cdtype, 210)
    q, _, c, table, _ = args
    y0, l0, split = prompt(*args)
    assert split
    poison(c, what, table, 0, range(128, 512), 16, 1, NAN)
    y, lse, _ = prompt(*args)
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    hit[:new[0], heads // kv:] = True
    reached((y, lse), (y0, l0), hit, what in ("v", "vs"))


@pytest.mark.parametrize("what,cdtype", [("k", "bf16"), ("k", "f16"), ("ks", "e4m3")])
@pytest.mark.parametrize("heads", [2, 4])
def test_the_only_token_of_a_part(heads, what, cdtype):
    """128 rows at 448 to 575, every head with keys of its own: 448 starts the last of five
    parts, and is all that its own row sees of it."""
    say(f"split prompt, one token {heads} {what} {cdtype}")
    dtype = "f16" if cdtype == "f16" else "bf16"
    table, pages = table_of([576], 16, 220)
    c = Cache(pages, heads, 16, 128, cdtype, seed=220)
    q = rand((128, heads, 128), 223, dtype, 2.0).cuda()
    args = (q, i32([0, 128]), c, table, i32([576]))
    y0, l0, split = prompt(*args)
    assert split
    poison(c, what, table, 0, [448], 16, 1, NAN)
    y, lse, _ = prompt(*args)
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    hit[:, 1] = True
    reached((y, lse), (y0, l0), hit)


def test_the_only_token_of_a_part_in_a_window():
    """64 rows at 1000 to 1063 with a window of 513: of the first part, 488 to 551, the last
    row sees 551 alone; 487 is seen by none."""
    say("split prompt, one token in a window")
    table, pages = table_of([1064], 16, 230)
    c = Cache(pages, 1, 16, 128, "bf16", seed=230)
    q = rand((64, 2, 128), 233, "bf16", 2.0).cuda()
    args = (q, i32([0, 64]), c, table, i32([1064]), 513)
    y0, l0, split = prompt(*args)
    assert split
    poison(c, "k", table, 0, [487], 16, 0, NAN)
    y, lse, _ = prompt(*args)
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    reached((y, lse), (y0, l0), hit)
    poison(c, "k", table, 0, [551], 16, 0, NAN)
    y, lse, _ = prompt(*args)
    reached((y, lse), (y0, l0), ~hit)


@pytest.mark.parametrize("what", ["q", "k", "v"])
def test_wide_and_narrow_tables(what):
    """What is not finite comes out the same whether the table has room for parts or not."""
    say(f"wide and narrow tables {what}")
    n, m = 200, 5
    table, pages = table_of([n], 16, 240, extra=500)
    c = Cache(pages, 2, 16, 128, "bf16", seed=240)
    q = rand((m, 4, 128), 243, "bf16", 2.0).cuda()
    if what == "q":
        q[2, 1, 9], q[4, 3, 0] = NAN, INF
    else:
        poison(c, what, table, 0, range(128, n), 16, 1, NAN)
    outs = []
    for width in (table.shape[1], -(-n // 16)):
        y, lse, split = prompt(q, i32([0, m]), c, table[:, :width], i32([n]))
        assert split == (width == table.shape[1])
        outs.append((torch.isnan(y), torch.isnan(lse)))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert outs[0][0].any() and not outs[0][0].all()


@pytest.mark.parametrize("every", [False, True])
@pytest.mark.parametrize("i", range(len(SPLIT)))
def test_infinite_scores_of_a_split_prompt(i, every):
    """z = -inf leaves out the tokens of whole parts; of all tokens: y = 0, lse = -inf."""
    say(f"split prompt, z = -inf {SPLIT[i]} {every}")
    new, lens, heads, kv, d = SPLIT[i]
    args = case_of(SPLIT[i], "bf16", "bf16", 250)
    q, _, c, table, _ = args
    q[:, :, 5] = 1.0
    clean = c.values()
    out = list(range(lens[0] if every else 512))
    poison(c, "k", table, 0, out, 16, 0, -INF)
    y, lse, split = prompt(*args)
    assert split and torch.isfinite(y).all()
    group = heads // kv
    if every:
        assert not y[:new[0], :group].any() and torch.all(lse[:new[0], :group] == -INF)
        return
    # the tokens from 512 on are a sequence of their own with the same results
    rows = [(r, 0, lens[0] - 512 - new[0] + r, lens[0] - 512) for r in range(0, new[0], 7)]
    check(y[:, :group], lse[:, :group], q[:, :group], [x[:, :1] for x in clean], rows, d ** -0.5,
          0, 0, prompt_r("bf16", "bf16"), "bf16", table.cpu().numpy()[:, 32:])


@pytest.mark.parametrize("what,cdtype", [("q", "bf16"), ("k", "bf16"), ("v", "f16"), ("k", "e4m3"),
                                         ("ks", "e4m3"), ("vs", "e4m3")])
@pytest.mark.parametrize("tokens", [range(128, 900), [1024]])
def test_a_split_decode(tokens, what, cdtype):
    """Tokens that fill units, and the last token, alone in its unit of 128."""
    say(f"split decode {what} {cdtype} {len(tokens)}")
    dtype = "f16" if cdtype == "f16" else "bf16"
    lens = [1025, 3, 900]
    table, pages = table_of(lens, 16, 260)
    c = Cache(pages, 2, 16, 128, cdtype, seed=260)
    q = rand((3, 8, 128), 263, dtype, 2.0).cuda()
    before = run_decode(q, c, table, i32(lens))
    hit = torch.zeros((3, 8), dtype=torch.bool, device="cuda")
    if what == "q":
        hit[0, 5] = hit[2, 0] = True
        q[hit, 7] = NAN
    else:
        hit[0, 4:] = True
        poison(c, what, table, 0, tokens, 16, 1, NAN)
    reached(run_decode(q, c, table, i32(lens)), before, hit, what in ("v", "vs"))


def test_a_key_that_is_nan_in_a_decoded_batch():
    """Unsplit: one NaN key makes NaN of its kv head's rows where it is visible."""
    say("decode, one key")
    lens = [150, 20]
    table, pages = table_of(lens, 16, 270)
    c = Cache(pages, 2, 16, 128, "bf16", seed=270)
    q = rand((2, 4, 128), 273, "bf16", 2.0).cuda()
    for window, seen in ((0, True), (25, False), (60, False), (61, True)):
        before = run_decode(q, c, table, i32(lens), window)
        t, (pg, at) = c.k, places(table, 0, [89], 16)
        keep = t[pg, 1, at, 5].clone()
        t[pg, 1, at, 5] = NAN
        hit = torch.zeros((2, 4), dtype=torch.bool, device="cuda")
        hit[0, 2:] = seen
        reached(run_decode(q, c, table, i32(lens), window), before, hit)
        t[pg, 1, at, 5] = keep
