"""Calls of lp_moe.h held to what their arithmetic can make of the result, and the
ways through them that sizes choose (GPU)."""
import numpy as np
import pytest
import torch

from test_gpu_moe import same_runs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,E,H", [(1500, 8, 400, 4112), (1024, 8, 256, 4224), (700, 8, 1024, 6160)])
@pytest.mark.parametrize("weighted", [False, True])
def test_gather_quant_of_short_runs_past_the_caches(lp, T, k, E, H, weighted):
    """More than 64 MB of rows, 32 an expert at the most on average; some experts with more, some pairs of nobody's."""
    g = torch.Generator(device="cuda").manual_seed(T)
    assert 2 * T * k * H > 64 << 20 and T * k <= 32 * E
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    e = torch.randint(-1, E, (T, k), generator=g, device="cuda").int()
    e[:, 0] = torch.where(torch.rand(T, generator=g, device="cuda") < 0.2, E // 2, e[:, 0])
    off, rows, order = lp.lp_moe_sort(e, E)
    w = torch.rand(T, k, generator=g, device="cuda") if weighted else None
    plain, n = lp.lp_moe_combine_bwd(x, None, rows, w, need_dw=False)[0], int(off[-1])
    out = lp.lp_moe_gather_quant(x, order, off, k, weights=w)
    for q in out:
        q.codes.fill_(99)
    same_runs(lp, lp.lp_moe_gather_quant(x, order, off, k, weights=w, out=out), lp.lp_r128_quant_dual(plain, off), off, H)
    assert all((q.codes[0, n:] == 99).all() for q in out)
