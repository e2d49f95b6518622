"""Small weights next to a large one.  One token of each row has z = 0 and a value of 0;
the others have z = -e ln 2, so their weights are 2^-e of the largest, and y is theirs
alone.  The calls keep a weight to r of itself (decode 2^-16, prompt half a step of the
products' type), in f16 products no finer than 2^-32 of the row's largest weight: these are
held 2^7 larger and round to multiples of 2^-24 at worst.  So y is off by at most
  sum_j |v_j| (w_j (r + dz) + 2^-32) / sum w,
with dz the tolerance of z itself: (d + 12) 2^-24 of what is summed to it, twice, and 2^-20
and (n + 64) 2^-22 of the sums as in test_gpu_attention; then half a step of its type."""

import numpy as np
import pytest
import torch

from gpu_util import say
from oracle import attention as oracle
from test_gpu_attention import (DECODE_R, TINY, ULP, Cache, i32, np64, prompt_r, rand, run_decode,
                                run_prompt, table_of)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,cdtype", [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3")])
@pytest.mark.parametrize("e", [10, 18, 24, 28, 33])
@pytest.mark.parametrize("n", [100, 2000])
def test_small_weights(n, e, dtype, cdtype):
    say(f"small weights {n} {e} {dtype} {cdtype}")
    d, heads, first = 64, 2, n // 3
    table, pages = table_of([n], 16, 300, extra=200)
    c = Cache(pages, 1, 16, d, cdtype, seed=300)
    # q has one component, keys hold -e/8 there or 0: z = q k scale, a multiple of ln 2
    # up to the rounding of the scale
    q = torch.zeros((1, heads, d), dtype=rand((1,), 1, dtype).dtype, device="cuda")
    q[:, 0, 3], q[:, 1, 3] = 8.0, 4.0
    c.k[:] = torch.zeros((), device="cuda").to(c.k.dtype)
    c.k[:, :, :, 3] = torch.full((), -e / 8, device="cuda").to(c.k.dtype)
    if c.ks is not None:
        c.ks.fill_(1.0)
        c.vs.fill_(1.0)
    pg, at = int(table[0, first // 16]), first % 16
    zero = torch.zeros((), device="cuda").to(c.k.dtype)
    c.k[pg, 0, at, 3] = zero
    c.v[pg, 0, at] = zero
    scale = float(np.float32(np.log(2.0)))
    k, v = c.values()
    ks, vs = oracle.tokens(k, table.cpu().numpy()[0], n), oracle.tokens(v, table.cpu().numpy()[0], n)
    ref, _, w, mag = oracle.attend(np64(q)[0], ks, vs, n - 1, scale)
    for name, run, r in (("decode", run_decode(q, c, table, i32([n]), scale=scale), DECODE_R),
                         ("prompt", run_prompt(q, i32([0, 1]), c, table, i32([n]), scale=scale),
                          prompt_r(dtype, cdtype))):
        y = np64(run[0])[0]
        for h in range(heads):
            dz = (d + 12) * 2.0 ** -24 * mag[h].max()
            rel = 2 * dz + r + 2.0 ** -20 + (n + 64) * 2.0 ** -22
            least = 2.0 ** -32 * w[h].max() if (dtype, cdtype) == ("f16", "f16") else 0.0
            err = (w[h] * rel + least) @ np.abs(vs[:, 0])
            tol = err + ULP[dtype] * (np.abs(ref[h]) + err) + TINY[dtype]
            off = np.abs(y[h] - ref[h])
            assert np.all(off <= tol), (name, h, float((off / tol).max()))
