"""The binding's own checks of the calls of lp_moe.h, with stand-ins for device
tensors and for the C functions (CPU only; no kernel is launched)."""
import pytest
import torch

import fp8_gemm_backward_amd as lp
from test_train_binding import DeviceTensor

BF, F, I, U = torch.bfloat16, torch.float32, torch.int32, torch.uint8
NAMES = ["lp_moe_gate", "lp_moe_gate_bwd", "lp_moe_sort_workspace", "lp_moe_sort", "lp_moe_gather", "lp_moe_gather_quant",
         "lp_moe_combine", "lp_moe_combine_bwd", "lp_linear_fwd_w4", "lp_grouped_fwd_w4"]


@pytest.fixture
def made(monkeypatch):
    """The C calls made, as (name, arguments); none is carried out."""
    calls = []
    for name in NAMES:
        monkeypatch.setattr(lp.lib, name, lambda *a, _n=name: calls.append((_n, a)) or 0)
    monkeypatch.setattr(lp, "_stream", lambda s: 0)
    return calls


class Tensor(DeviceTensor):
    def new_empty(self, shape, dtype=None):
        return Tensor(shape, dtype or self.dtype)

    def split_with_sizes(self, sizes):
        return [Tensor((n,), self.dtype) for n in sizes]

    def view(self, shape):
        return Tensor(shape, self.dtype)


def t(*shape, dtype=BF, ptr=0x10000):
    return Tensor(shape, dtype, ptr)


def refused(made, *calls):
    for call in calls:
        with pytest.raises((ValueError, lp.LpError)):
            call()
    assert not made


def test_gate(made):
    w, e = lp.lp_moe_gate(t(5, 12), 3, renorm=False)
    assert (w.shape, w.dtype, e.shape, e.dtype) == ((5, 3), F, (5, 3), I)
    assert made.pop()[1][1:6] == (1, 5, 12, 3, 0)
    lp.lp_moe_gate(t(5, 12, dtype=F), 3)
    assert made.pop()[1][1:6] == (0, 5, 12, 3, 1)
    g = lp.lp_moe_gate_bwd(t(5, 3, dtype=F), t(5, 12), w, e)
    assert (g.shape, g.dtype) == ((5, 12), BF)
    made.clear()
    refused(made, lambda: lp.lp_moe_gate(t(5, 12, dtype=torch.float16), 3), lambda: lp.lp_moe_gate(t(5, 12), 3, weights=t(5, 3), chosen=e),
            lambda: lp.lp_moe_gate(t(5, 12), 3, weights=t(4, 3, dtype=F), chosen=e),
            lambda: lp.lp_moe_gate(t(5, 12), 3, weights=w, chosen=t(5, 3, dtype=torch.int64)),
            lambda: lp.lp_moe_gate(t(60), 3),
            lambda: lp.lp_moe_gate_bwd(t(5, 3), t(5, 12), w, e), lambda: lp.lp_moe_gate_bwd(t(5, 2, dtype=F), t(5, 12), w, e),
            lambda: lp.lp_moe_gate_bwd(w, t(5, 12), w, e, grad_logits=t(5, 12, dtype=F)),
            lambda: lp.lp_moe_gate_bwd(w, t(5, 12), w, t(5, 4, dtype=I)), lambda: lp.lp_moe_gate_bwd(w, t(5, 12), w, t(15, dtype=I)))


def test_sort(made):
    off, rows, order = lp.lp_moe_sort(t(7, 2, dtype=I), 4)
    assert [v.shape for v in (off, rows, order)] == [(4,), (7, 2), (14,)] and all(v.dtype == I for v in (off, rows, order))
    made.clear()
    refused(made, lambda: lp.lp_moe_sort(t(7, 2, dtype=torch.int64), 4), lambda: lp.lp_moe_sort(t(7, 2, dtype=F), 4))


def test_rows(made):
    rows, w = t(7, 2, dtype=I), t(7, 2, dtype=F)
    assert lp.lp_moe_gather(t(7, 32), rows).shape == (14, 32) and made.pop()[1][1:4] == (7, 2, 32)
    assert lp.lp_moe_combine(t(14, 32), rows, w).shape == (7, 32)
    gy, gw = lp.lp_moe_combine_bwd(t(7, 32), t(14, 32), rows, w)
    assert gy.shape == (14, 32) and (gw.shape, gw.dtype) == ((7, 2), F)
    assert lp.lp_moe_combine_bwd(t(7, 32), None, rows, w, need_dw=False)[1] is None
    assert lp.lp_moe_combine_bwd(t(7, 32), t(14, 32), rows, need_dy=False)[0] is None
    made.clear()
    refused(made, lambda: lp.lp_moe_gather(t(6, 32), rows), lambda: lp.lp_moe_gather(t(7, 32, dtype=F), rows),
            lambda: lp.lp_moe_gather(t(7, 32), t(14, dtype=I)), lambda: lp.lp_moe_gather(t(7, 32), t(7, 2, dtype=torch.int64)),
            lambda: lp.lp_moe_gather(t(7, 32), rows, out=t(13, 32)), lambda: lp.lp_moe_gather(t(7, 32), rows, out=t(14, 16)),
            lambda: lp.lp_moe_combine(t(13, 32), rows, w), lambda: lp.lp_moe_combine(t(14, 32), rows, t(7, 2)),
            lambda: lp.lp_moe_combine(t(14, 32), rows, t(7, dtype=F)), lambda: lp.lp_moe_combine(t(14, 32), rows, w, out=t(7, 16)),
            lambda: lp.lp_moe_combine_bwd(t(6, 32), t(14, 32), rows, w), lambda: lp.lp_moe_combine_bwd(t(7, 32), None, rows, w),
            lambda: lp.lp_moe_combine_bwd(t(7, 32), t(13, 32), rows, w), lambda: lp.lp_moe_combine_bwd(t(7, 32), t(14, 32, dtype=F), rows, w),
            lambda: lp.lp_moe_combine_bwd(t(7, 32), t(14, 32), rows, w, grad_y=t(13, 32)),
            lambda: lp.lp_moe_combine_bwd(t(7, 32), t(14, 32), rows, w, grad_weights=t(7, 2)))


def test_gather_quant(made):
    order, off, w = t(14, dtype=I), t(3, dtype=I), t(14, dtype=F)
    cols, toks = out = lp.lp_moe_gather_quant(t(7, 144), order, off, 2, weights=w)
    assert cols.codes.shape == toks.codes.shape == (1, 14, 144) and (cols.axis, toks.axis, toks.run_groups) == (-1, -2, 3)
    assert cols.scales.shape == (1, 2, 14) and toks.scales.shape == (1, 14 // 128 + 3, 144)
    assert lp.lp_moe_gather_quant(t(7, 144), order, off, 2, out=out) is out
    made.clear()
    short = lp.QTensor("fp8_r128", toks.codes, t(1, 2, 144, dtype=F), None, (1, 14, 144), -2, 3)
    refused(made, lambda: lp.lp_moe_gather_quant(t(7, 144), t(13, dtype=I), off, 2), lambda: lp.lp_moe_gather_quant(t(7, 144, dtype=F), order, off, 2),
            lambda: lp.lp_moe_gather_quant(t(7, 144), order, t(0, dtype=I), 2), lambda: lp.lp_moe_gather_quant(t(7, 144), order, off, 2, weights=t(13, dtype=F)),
            lambda: lp.lp_moe_gather_quant(t(7, 144), order, off, 2, out=(toks, cols)),
            lambda: lp.lp_moe_gather_quant(t(7, 144), order, off, 2, out=(cols, short)),
            lambda: lp.lp_moe_gather_quant(t(7, 144), order, off, 2, out=(cols, cols)))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_w4(made, fmt):
    def weight(batch, N, K, short=0):
        return lp.QTensor(fmt, t(batch, N, K // 2, dtype=U), t(batch, N, K // (32 if fmt == "mxfp4" else 16) - short, dtype=U),
                          t(1, dtype=F) if fmt == "nvfp4" else None, (batch, N, K))
    assert lp.lp_linear_fwd_w4(t(3, 64), weight(1, 48, 64)).shape == (3, 48)
    assert lp.lp_grouped_fwd_w4(t(3, 64), weight(5, 48, 64), t(5, dtype=I)).shape == (3, 48)
    made.clear()
    refused(made, lambda: lp.lp_linear_fwd_w4(t(3, 32), weight(1, 48, 64)), lambda: lp.lp_linear_fwd_w4(t(3, 64, dtype=F), weight(1, 48, 64)),
            lambda: lp.lp_linear_fwd_w4(t(3, 64), weight(1, 48, 64), y=t(2, 48)), lambda: lp.lp_linear_fwd_w4(t(192), weight(1, 48, 64)),
            lambda: lp.lp_linear_fwd_w4(t(3, 64), weight(1, 48, 64), y=t(3, 48, dtype=torch.float16)),
            lambda: lp.lp_grouped_fwd_w4(t(3, 64), weight(5, 48, 64), t(5, dtype=torch.int64)),
            lambda: lp.lp_linear_fwd_w4(t(3, 64), weight(1, 48, 64, short=1)))
