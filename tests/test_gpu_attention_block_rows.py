"""One attention block of examples/attention_block.py for calls of different numbers of
rows, up to those it was made for: a prompt, a chunk and single tokens give the bits of
blocks that were made for just these rows, also behind a larger call's leftovers."""

import pytest
import torch

from gpu_util import say
from test_gpu_attention_block import Setup
from test_gpu_fp8 import rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hidden", [256, 1024])
@pytest.mark.parametrize("dtype,cdtype", [("bf16", "e4m3"), ("f16", "f16")])
def test_fewer_rows_than_the_block_was_made_for(dtype, cdtype, hidden):
    say(f"attention block, fewer rows {dtype} {cdtype} {hidden}")
    one, exact = (Setup(3, 8, 2, 64, hidden, dtype, cdtype) for _ in range(2))
    block = one.block(300)
    for step, new in enumerate([[90, 1, 140], [20, 0, 3], [1, 1, 1], [0, 1, 0]]):
        say(f"rows {new}")
        outs = []
        for s in (one, exact):
            n = torch.tensor(new, device="cuda")
            pos, slots, starts = s.seqs.add(n)
            m = len(pos)
            x, r = (rand((m, hidden), 20 + 2 * step + i, dtype).cuda() for i in range(2))
            b = block if s is one else s.block(m)
            if step == 2:
                y = b.decode(x, r, pos, slots, s.seqs.pages, s.seqs.lens)
            else:
                y = b.prompt(x, r, pos, slots, starts, s.seqs.pages, s.seqs.lens)
            torch.cuda.synchronize()
            assert y.shape == (m, hidden) and torch.isfinite(y).all()
            outs.append((y.clone(), r))
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_more_rows_than_the_block_was_made_for():
    s = Setup(1, 2, 2, 64, 256, "bf16", "bf16")
    b = s.block(4)
    pos, slots, starts = s.seqs.add(torch.tensor([5], device="cuda"))
    x, r = (rand((5, 256), 30 + i, "bf16").cuda() for i in range(2))
    for call in (lambda: b.prompt(x, r, pos, slots, starts, s.seqs.pages, s.seqs.lens),
                 lambda: b.decode(x, r, pos, slots, s.seqs.pages, s.seqs.lens)):
        with pytest.raises(ValueError, match="5 rows"):
            call()
