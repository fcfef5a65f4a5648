"""Tensors of another shape than a call of lp_moe.h reads or writes are refused by
the binding: the C calls take bare pointers and would go through them at the pitch
of the right shape (CPU only, stand-ins for device tensors; no kernel is
launched)."""
import pytest
import torch

import fp8_gemm_backward_amd as lp
from test_moe_binding import F, I, made, refused, t  # noqa: F401


def test_results_of_gather_and_combine_have_their_width(made):  # noqa: F811
    rows, w = t(7, 2, dtype=I), t(7, 2, dtype=F)
    lp.lp_moe_gather(t(7, 32), rows, out=t(14, 32))
    lp.lp_moe_combine(t(14, 32), rows, w, out=t(7, 32))
    made.clear()
    refused(made, lambda: lp.lp_moe_gather(t(7, 32), rows, out=t(14, 48)), lambda: lp.lp_moe_combine(t(14, 32), rows, w, out=t(7, 48)))


def test_the_rows_of_combines_gradient_have_its_width(made):  # noqa: F811
    rows, w = t(7, 2, dtype=I), t(7, 2, dtype=F)
    lp.lp_moe_combine_bwd(t(7, 32), t(14, 32), rows, w, grad_y=t(14, 32))
    lp.lp_moe_combine_bwd(t(7, 32), t(15, 32), rows, w, grad_y=t(14 * 32))          # (more rows than are read; flat memory)
    made.clear()
    refused(made, lambda: lp.lp_moe_combine_bwd(t(7, 32), t(14, 48), rows, w), lambda: lp.lp_moe_combine_bwd(t(7, 32), t(7, 64), rows, w),
            lambda: lp.lp_moe_combine_bwd(t(7, 32), t(14, 32), rows, w, grad_y=t(14, 48)),
            lambda: lp.lp_moe_combine_bwd(t(7, 32), t(14, 32), rows, w, grad_y=t(28, 16)))
