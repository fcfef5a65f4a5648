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


def test_results_of_the_4_bit_forward_have_its_width(made):  # noqa: F811
    def weight(batch):
        return lp.QTensor("mxfp4", t(batch, 48, 32, dtype=torch.uint8), t(batch, 48, 2, dtype=torch.uint8), None, (batch, 48, 64))
    lp.lp_linear_fwd_w4(t(3, 64), weight(1), y=t(5, 48))
    lp.lp_grouped_fwd_w4(t(3, 64), weight(2), t(2, dtype=I), y=t(3 * 48))
    made.clear()
    refused(made, lambda: lp.lp_linear_fwd_w4(t(3, 64), weight(1), y=t(3, 64)), lambda: lp.lp_linear_fwd_w4(t(3, 64), weight(1), y=t(48, 3)),
            lambda: lp.lp_grouped_fwd_w4(t(3, 64), weight(2), t(2, dtype=I), y=t(3, 64)))


def test_numbers_by_pair_and_gradients_of_logits_have_their_width(made):  # noqa: F811
    """A slot more a token than the call has: refused; the same numbers in another shape: taken."""
    rows, w, e, wide = t(7, 2, dtype=I), t(7, 2, dtype=F), t(7, 2, dtype=I), t(7, 3, dtype=F)
    order, off = t(14, dtype=I), t(3, dtype=I)
    for same in (w, t(14, dtype=F), t(14, 1, dtype=F), t(1, 7, 2, dtype=F), t(9, 2, dtype=F)):
        lp.lp_moe_combine(t(14, 32), rows, same)
        lp.lp_moe_combine_bwd(t(7, 32), t(14, 32), rows, same)
        lp.lp_moe_gather_quant(t(7, 144), order, off, 2, weights=same)
        lp.lp_moe_gate_bwd(same, t(7, 12), same, e)
        lp.lp_moe_gate(t(7, 12), 2, weights=same, chosen=e)
    lp.lp_moe_gate_bwd(w, t(7, 12), w, e, grad_logits=t(8, 12))
    made.clear()
    refused(made, lambda: lp.lp_moe_combine(t(14, 32), rows, wide), lambda: lp.lp_moe_combine_bwd(t(7, 32), t(14, 32), rows, wide),
            lambda: lp.lp_moe_combine_bwd(t(7, 32), t(14, 32), rows, w, grad_weights=wide),
            lambda: lp.lp_moe_gather_quant(t(7, 144), order, off, 2, weights=wide),
            lambda: lp.lp_moe_gate(t(7, 12), 2, weights=wide, chosen=e), lambda: lp.lp_moe_gate(t(7, 12), 2, weights=w, chosen=t(7, 3, dtype=I)),
            lambda: lp.lp_moe_gate_bwd(wide, t(7, 12), w, e), lambda: lp.lp_moe_gate_bwd(w, t(7, 12), wide, e),
            lambda: lp.lp_moe_gate_bwd(w, t(7, 12), w, e, grad_logits=t(7, 16)))


def test_the_two_fp8_copies_are_told_apart_by_place(made):  # noqa: F811
    """One tensor given for both would be written twice: its scales are large enough for both where rows are short."""
    order, off = t(2000, dtype=I), t(3, dtype=I)
    cols, toks = lp.lp_moe_gather_quant(t(1000, 16), order, off, 2)
    assert cols.scales.nbytes >= toks.scales.nbytes
    made.clear()
    refused(made, lambda: lp.lp_moe_gather_quant(t(1000, 16), order, off, 2, out=(cols, cols)),
            lambda: lp.lp_moe_gather_quant(t(1000, 16), order, off, 2, out=(toks, toks)),
            lambda: lp.lp_moe_gather_quant(t(1000, 16), order, off, 2, out=(toks, cols)))


def test_combines_gradient_of_nothing_needs_no_rows(made):  # noqa: F811
    """No token, or rows of no column: the C call reads no y, and none has to be given."""
    for T, H in ((0, 32), (7, 0)):
        gy, gw = lp.lp_moe_combine_bwd(t(T, H), None, t(T, 2, dtype=I))
        assert gy.shape == (2 * T, H) and gw.shape == (T, 2) and made.pop()[1][1] is None


def test_the_sorts_workspace_is_what_the_library_asks_for(made, monkeypatch):  # noqa: F811
    """Up to any number of pairs: the binding has no limit of its own."""
    asked = []

    def workspace(pairs, groups, nbytes):
        asked.append((pairs, groups))
        nbytes._obj.value = 0 if pairs <= 100 else 16 * pairs
        return 0
    monkeypatch.setattr(lp.lib, "lp_moe_sort_workspace", workspace)
    lp._sort_workspace.cache_clear()
    try:
        for pairs in (0, 8, 100, 101, 65536, 65537):
            lp.lp_moe_sort(t(pairs, dtype=I), 4)
            name, args = made.pop()
            assert name == "lp_moe_sort" and args[1:3] == (pairs, 4)
            assert (args[6] is None, args[7]) == ((True, 0) if pairs <= 100 else (False, 16 * pairs))
        assert asked == [(n, 4) for n in (0, 8, 100, 101, 65536, 65537)]
    finally:
        lp._sort_workspace.cache_clear()


def test_the_sorts_workspace_is_refused_as_the_sort_is():
    for pairs, groups in ((8, 0), (8, 1025), (1 << 30, 4)):
        with pytest.raises(lp.LpError) as e:
            lp._sort_workspace(pairs, groups)
        assert "lp_moe_sort" in str(e.value)


def test_the_fp8_copies_have_their_width(made):  # noqa: F811
    """Codes and scales whose rows are longer: refused; as many in another shape, or more rows: taken."""
    order, off, x = t(2000, dtype=I), t(3, dtype=I), t(1000, 144)

    def copies(codes=(1, 2000, 144), cols=(1, 2, 2000), rows=(1, 18, 144), codes_rows=(1, 2000, 144)):
        return (lp.QTensor("fp8_r128", t(*codes, dtype=torch.uint8), t(*cols, dtype=F), None, (1, 2000, 144), -1),
                lp.QTensor("fp8_r128", t(*codes_rows, dtype=torch.uint8), t(*rows, dtype=F), None, (1, 2000, 144), -2))
    for kw in ({}, dict(codes=(2000 * 144,)), dict(cols=(1, 4000)), dict(rows=(1, 19, 144)), dict(cols=(3, 2000))):
        lp.lp_moe_gather_quant(x, order, off, 2, out=copies(**kw))
    made.clear()
    refused(made, *(lambda kw=kw: lp.lp_moe_gather_quant(x, order, off, 2, out=copies(**kw))
                    for kw in (dict(codes=(1, 2000, 160)), dict(codes_rows=(1, 2000, 160)), dict(cols=(1, 2, 2048)), dict(rows=(1, 18, 160)))))


def test_tensors_of_another_gpu_than_the_current_one_are_refused(made, monkeypatch):  # noqa: F811
    """Without a stream a call runs on the current GPU, which cannot reach the other one's memory.  (A given stream says
    where it runs.)"""
    monkeypatch.setattr(lp, "_several_gpus", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

    def on(at, x):
        x.device = torch.device("cuda", at)
        return x
    q = lp.QTensor("mxfp4", t(2, 48, 32, dtype=torch.uint8), t(2, 48, 2, dtype=torch.uint8), None, (2, 48, 64))
    one = lp.QTensor("mxfp4", t(1, 48, 32, dtype=torch.uint8), t(1, 48, 2, dtype=torch.uint8), None, (1, 48, 64))
    rows, w, e, order, off = t(7, 2, dtype=I), t(7, 2, dtype=F), t(7, 2, dtype=I), t(14, dtype=I), t(2, dtype=I)
    calls = [lambda at, s: lp.lp_moe_gate(on(at, t(7, 12)), 2, stream=s), lambda at, s: lp.lp_moe_gate_bwd(w, on(at, t(7, 12)), w, e, stream=s),
             lambda at, s: lp.lp_moe_sort(on(at, t(7, 2, dtype=I)), 4, stream=s), lambda at, s: lp.lp_moe_gather(on(at, t(7, 32)), rows, stream=s),
             lambda at, s: lp.lp_moe_gather_quant(on(at, t(7, 144)), order, off, 2, stream=s),
             lambda at, s: lp.lp_moe_combine(on(at, t(14, 32)), rows, w, stream=s),
             lambda at, s: lp.lp_moe_combine_bwd(on(at, t(7, 32)), t(14, 32), rows, w, stream=s),
             lambda at, s: lp.lp_linear_fwd_w4(on(at, t(3, 64)), one, stream=s), lambda at, s: lp.lp_grouped_fwd_w4(on(at, t(3, 64)), q, off, stream=s)]
    for call in calls:
        call(0, None), call(1, 0x500)
    made.clear()
    refused(made, *(lambda c=c: c(1, None) for c in calls))
