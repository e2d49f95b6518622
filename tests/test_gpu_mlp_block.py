"""examples/mlp_block.py on the GPU: each stage against the fp64 oracle on the
values the stage before it left, with the tolerances of the operators' own
tests, and replays of its graph against the eager call, bit for bit."""

import os
import sys

import numpy as np
import pytest
import torch

from gpu_util import say
from oracle import fp8
from test_gpu_fp8 import ULP, TINY, check_codes, check_linear, rand
from test_gpu_moe import check as check_experts, Experts

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

pytestmark = pytest.mark.gpu


def norm_of(x, r, gain, eps, dtype):
    """fp64 residual sum and norm, and the norm's relative tolerance."""
    h, v = fp8.add_rmsnorm(x.double().cpu().numpy(), gain.double().cpu().numpy(), eps,
                           r.double().cpu().numpy())
    return h, v, (x.shape[1] / 256 + 40) * 2.0 ** -24


def replays(mlp_block, block, x, r):
    before = r.clone()
    y = block(x, r).clone()
    after = r.clone()
    torch.cuda.synchronize()
    r.copy_(before)
    graph = mlp_block.capture(block, x, r)
    assert torch.equal(r, before)
    for i in range(3):
        block.y.fill_(i)
        r.copy_(before)
        (x @ x.t().contiguous()).sum()               # other work between the replays
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(block.y, y) and torch.equal(r, after)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,h,i", [(1, 256, 384), (5, 512, 400), (70, 272, 640)])
def test_dense(m, h, i, dtype):
    import mlp_block
    say(f"dense mlp m={m} h={h} i={i} {dtype}")
    x, r = rand((m, h), 70, dtype).cuda(), rand((m, h), 71, dtype).cuda()
    gain = rand((h,), 72, dtype).cuda()
    gate, up = rand((i, h), 73, dtype, 0.06).cuda(), rand((i, h), 74, dtype, 0.06).cuda()
    block = mlp_block.DenseMLP(gain, gate, up, rand((h, i), 75, dtype, 0.06).cuda(), m)
    hs, v, tol = norm_of(x, r, gain, block.eps, dtype)
    y = block(x, r)
    torch.cuda.synchronize()
    assert np.all(np.abs(r.double().cpu().numpy() - hs)
                  <= (ULP[dtype] + 2.0 ** -23) * np.abs(hs) + TINY[dtype])
    check_codes(block.q, block.s, v, tol)
    check_linear(block.g, block.q, block.s, block.gate, dtype)
    check_linear(block.u, block.q, block.s, block.up, dtype)
    check_codes(block.q2, block.s2, fp8.silu_product(block.g.double().cpu().numpy(),
                                                     block.u.double().cpu().numpy()), 2.0 ** -19)
    check_linear(y, block.q2, block.s2, block.down, dtype)
    replays(mlp_block, block, x, r)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("t,e,top_k", [(1, 4, 2), (9, 8, 3)])
def test_experts(t, e, top_k, dtype):
    import mlp_block
    say(f"experts mlp t={t} e={e} top_k={top_k} {dtype}")
    h, i = 256, 384
    x, r = rand((t, h), 80, dtype).cuda(), rand((t, h), 81, dtype).cuda()
    gain = rand((h,), 82, dtype).cuda()
    # an integer router with powers of two: logits far enough apart to rank alike
    router = (2.0 * torch.eye(e, h)).to(x.dtype).cuda()
    ex = Experts(e, h, i, "int4", 128, 83)
    w16 = [rand((e * n, k), 83 + j, "f16", 0.05).to(x.dtype).reshape(e, n, k).cuda()
           for j, (n, k) in enumerate(((i, h), (i, h), (h, i)))]
    block = mlp_block.ExpertsMLP(gain, router, *w16, top_k, t)
    block.gate, block.up, block.down = ex.w          # the oracle's values are of these
    hs, v, tol = norm_of(x, r, gain, block.eps, dtype)
    y = block(x, r)
    torch.cuda.synchronize()
    got = block.v.double().cpu().numpy()
    assert np.all(np.abs(got - v) <= (ULP[dtype] * (1 + 2.0 ** -10) + tol) * np.abs(v)
                  + TINY[dtype])
    logits = block.v.double() @ router.double().t()
    from oracle import moe
    ids, probs = moe.route(logits.cpu().numpy(), top_k, True)
    # one product per logit is not zero: exact
    check_experts(block.v, ex, logits.cpu().numpy(), top_k, dtype, (y, ids, probs), True, dtype)
    replays(mlp_block, block, x, r)
