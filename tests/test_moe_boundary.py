"""lp_moe.h on the host: exports, documented refusals before anything touches the
GPU, and the oracle of these calls against its definitions (CPU only; no kernel
is launched)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import fp8_gemm_backward_amd as lp
from fp8_gemm_backward_amd import _QTensorC
from oracle import moe as O

OK, NULL, SHAPE, FORMAT, ALIGN = 0, 1, 2, 3, 4
FAKE = 0x10000          # 16-byte aligned stand-in pointer; never dereferenced here
F32, BF16 = 0, 1


def test_library_exports_every_function_of_the_header():
    text = open(os.path.join(os.path.dirname(lp.HEADER_PATH), "lp_moe.h")).read()
    names = re.findall(r"^lp_status\s+(lp_\w+)\s*\(", text, re.M)
    assert len(names) == 10
    for n in names:
        assert hasattr(lp.lib, n) and (n == "lp_moe_sort_workspace" or hasattr(lp, n)), n


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=2), FORMAT), (dict(dtype=-1), FORMAT), (dict(T=-1), SHAPE), (dict(T=1 << 30), SHAPE), (dict(T=1 << 29), SHAPE),
    (dict(T=1 << 25, E=1024), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(k=0), SHAPE), (dict(k=9), SHAPE),
    (dict(E=100, k=65), SHAPE), (dict(logits=None), NULL), (dict(weights=None), NULL), (dict(chosen=None), NULL),
    (dict(logits=FAKE + 2), ALIGN), (dict(weights=FAKE + 2), ALIGN), (dict(chosen=FAKE + 1), ALIGN),
    (dict(T=0, logits=None, weights=None, chosen=None), OK),
])
def test_gate_rejects(kw, expect):
    a = {**dict(logits=FAKE, dtype=F32, T=4, E=8, k=2, renorm=1, weights=FAKE, chosen=FAKE), **kw}
    assert lp.lib.lp_moe_gate(*a.values(), None) == expect
    grad = None if a["T"] == 0 else FAKE
    args = [grad, a["logits"], a["dtype"], a["T"], a["E"], a["k"], 1, a["weights"], a["chosen"], grad]
    assert lp.lib.lp_moe_gate_bwd(*args, None) == expect
    if expect == OK:
        return
    for at in (0, 9):
        good = [FAKE, FAKE, F32, 4, 8, 2, 1, FAKE, FAKE, FAKE, None]
        good[at] = None
        assert lp.lib.lp_moe_gate_bwd(*good) == NULL
        good[at] = FAKE + 2
        assert lp.lib.lp_moe_gate_bwd(*good) == ALIGN


def need(pairs, groups):
    n = ctypes.c_size_t(7)
    return lp.lib.lp_moe_sort_workspace(pairs, groups, ctypes.byref(n)), n.value


def test_sort_workspace():
    assert lp.lib.lp_moe_sort_workspace(8, 2, None) == NULL
    for pairs, groups in ((-1, 4), (1 << 30, 4), (8, 0), (8, 1025)):
        assert need(pairs, groups) == (SHAPE, 0)
    assert need(0, 4) == (OK, 0) and need(96, 64) == (OK, 0)
    assert need(1 << 16, 256) == (OK, 0)                 # (one launch, which needs none)
    big = [need(n, 256)[1] for n in ((1 << 16) + 1, 1 << 20, (1 << 30) - 1)]
    assert 0 < big[0] < big[1] < big[2]


@pytest.mark.parametrize("kw,expect", [
    (dict(pairs=-1), SHAPE), (dict(pairs=1 << 30), SHAPE), (dict(groups=0), SHAPE), (dict(groups=1025), SHAPE),
    (dict(experts=None), NULL), (dict(offsets=None), NULL), (dict(rows=None), NULL), (dict(order=None), NULL),
    (dict(offsets=None, pairs=0), NULL), (dict(experts=FAKE + 2), ALIGN), (dict(offsets=FAKE + 2), ALIGN),
    (dict(rows=FAKE + 2), ALIGN), (dict(order=FAKE + 1), ALIGN), (dict(ws=None, size=0), NULL), (dict(ws=FAKE + 8), ALIGN),
    (dict(size=-1), SHAPE),
])
def test_sort_rejects(kw, expect):
    a = {**dict(experts=FAKE, pairs=1 << 20, groups=64, offsets=FAKE, rows=FAKE, order=FAKE, ws=FAKE, size=0), **kw}
    a["size"] += need(1 << 20, 64)[1]
    assert lp.lib.lp_moe_sort(*a.values(), None) == expect


BAD_ROWS = [(dict(T=-1), SHAPE), (dict(k=0), SHAPE), (dict(k=65), SHAPE), (dict(T=1 << 30), SHAPE), (dict(T=1 << 29), SHAPE),
            (dict(cols=-8), SHAPE), (dict(cols=12), SHAPE), (dict(cols=1 << 22), SHAPE), (dict(T=1 << 20, k=8, cols=2048), SHAPE)]


def rows_call(name, T=4, k=2, cols=16, **kw):
    p = {**dict(x=FAKE, y=FAKE, rows=FAKE, out=FAKE, w=FAKE, gw=FAKE, order=FAKE, off=FAKE, G=3, c=(FAKE,) * 4), **kw}
    args = {"gather": (p["x"], T, k, cols, p["rows"], p["out"]),
            "combine": (p["y"], T, k, cols, p["rows"], p["w"], p["out"]),
            "combine_bwd": (p["x"], p["y"], T, k, cols, p["rows"], p["w"], p["out"], p["gw"]),
            "gather_quant": (p["x"], T, k, cols, p["order"], p["w"], p["off"], p["G"], *p["c"])}[name]
    return getattr(lp.lib, "lp_moe_" + name)(*args, None)


@pytest.mark.parametrize("name", ["gather", "combine", "combine_bwd", "gather_quant"])
def test_rows_reject_sizes(name):
    for kw, expect in BAD_ROWS:
        assert rows_call(name, **kw) == expect, kw


@pytest.mark.parametrize("name,kw,expect", [
    ("gather", dict(x=None), NULL), ("gather", dict(rows=None), NULL), ("gather", dict(out=None), NULL),
    ("gather", dict(x=FAKE + 8), ALIGN), ("gather", dict(rows=FAKE + 2), ALIGN), ("gather", dict(out=FAKE + 8), ALIGN),
    ("gather", dict(T=0, x=None, rows=None, out=None), OK), ("gather", dict(cols=0, x=None, out=None), OK),
    ("combine", dict(y=None), NULL), ("combine", dict(rows=None), NULL), ("combine", dict(out=None), NULL),
    ("combine", dict(y=FAKE + 4), ALIGN), ("combine", dict(w=FAKE + 2), ALIGN), ("combine", dict(out=FAKE + 2), ALIGN),
    ("combine", dict(T=0, y=None, rows=None, out=None, w=None), OK),
    ("combine_bwd", dict(x=None), NULL), ("combine_bwd", dict(y=None), NULL), ("combine_bwd", dict(rows=None), NULL),
    ("combine_bwd", dict(x=FAKE + 8), ALIGN), ("combine_bwd", dict(y=FAKE + 8), ALIGN), ("combine_bwd", dict(out=FAKE + 8), ALIGN),
    ("combine_bwd", dict(gw=FAKE + 2), ALIGN), ("combine_bwd", dict(w=FAKE + 2), ALIGN),
    ("combine_bwd", dict(out=None, gw=None), OK), ("combine_bwd", dict(T=0, x=None, y=None, rows=None), OK),
    ("gather_quant", dict(x=None), NULL), ("gather_quant", dict(order=None), NULL), ("gather_quant", dict(off=None), NULL),
    ("gather_quant", dict(c=(FAKE, None, FAKE, FAKE)), NULL), ("gather_quant", dict(c=(FAKE, FAKE, FAKE + 4, FAKE)), ALIGN),
    ("gather_quant", dict(w=FAKE + 2), ALIGN), ("gather_quant", dict(off=FAKE + 2), ALIGN), ("gather_quant", dict(order=FAKE + 1), ALIGN),
    ("gather_quant", dict(G=0), SHAPE), ("gather_quant", dict(G=1025), SHAPE), ("gather_quant", dict(cols=24), SHAPE),
    ("gather_quant", dict(T=(1 << 30) - 1, k=1, cols=16, G=1), SHAPE), ("gather_quant", dict(T=0, x=None, order=None), OK),
])
def test_rows_reject(name, kw, expect):
    assert rows_call(name, **kw) == expect


def q(fmt, rows=32, cols=64, batch=1, axis=-1, codes=FAKE, scales=FAKE, ts=FAKE):
    return _QTensorC(lp.FMT[fmt], axis, batch, rows, cols, codes, scales, ts)


@pytest.mark.parametrize("w,kw,expect", [
    (q("bf16"), {}, FORMAT), (q("fp8_b128"), {}, FORMAT), (q("mxfp8"), {}, FORMAT), (q("fp8_r128"), {}, FORMAT),
    (q("mxfp4", axis=-2), {}, FORMAT), (q("nvfp4", axis=-2), {}, FORMAT), (q("mxfp4", rows=24), {}, SHAPE),
    (q("mxfp4", cols=48), {}, SHAPE), (q("nvfp4", cols=48), {}, SHAPE), (q("nvfp4", rows=8), {}, SHAPE),
    (q("mxfp4", cols=1 << 22), {}, SHAPE), (q("mxfp4", rows=1 << 22), {}, SHAPE), (q("mxfp4", batch=2), {}, SHAPE),
    (q("mxfp4"), dict(M=-1), SHAPE), (q("mxfp4"), dict(M=1 << 30), SHAPE), (q("mxfp4", rows=1 << 20), dict(M=1 << 26), SHAPE),
    (q("mxfp4", codes=None), {}, NULL), (q("mxfp4", scales=None), {}, NULL), (q("nvfp4", ts=None), {}, NULL),
    (q("mxfp4"), dict(x=None), NULL), (q("mxfp4"), dict(y=None), NULL), (q("mxfp4", codes=FAKE + 8), {}, ALIGN),
    (q("mxfp4"), dict(x=FAKE + 8), ALIGN), (q("mxfp4"), dict(y=FAKE + 8), ALIGN), (q("nvfp4", ts=FAKE + 2), {}, ALIGN),
    (q("nvfp4", cols=0, ts=None), {}, NULL),                          # read whatever the contraction's length
    (q("mxfp4"), dict(M=0, x=None, y=None), OK), (q("mxfp4", rows=0, codes=None, scales=None), dict(y=None), OK),
])
def test_w4_rejects(w, kw, expect):
    a = {**dict(x=FAKE, M=4, y=FAKE), **kw}
    assert lp.lib.lp_linear_fwd_w4(a["x"], a["M"], ctypes.byref(w), a["y"], None) == expect
    groups = 1 if w.batch == 1 else 3
    assert lp.lib.lp_grouped_fwd_w4(a["x"], a["M"], ctypes.byref(w), FAKE, groups, a["y"], None) == expect


def test_grouped_w4_rejects():
    grp = lp.lib.lp_grouped_fwd_w4
    assert lp.lib.lp_linear_fwd_w4(FAKE, 4, None, FAKE, None) == NULL
    w = q("mxfp4", batch=2)
    for groups, off, expect in ((0, FAKE, SHAPE), (1025, FAKE, SHAPE), (3, FAKE, SHAPE), (2, None, NULL), (2, FAKE + 2, ALIGN)):
        assert grp(FAKE, 4, ctypes.byref(w), off, groups, FAKE, None) == expect


def test_binding_rejects_host_tensors_and_mismatches():
    f, i, b = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 16, dtype=torch.bfloat16)
    w = lp.QTensor("mxfp4", torch.zeros(32, 8, dtype=torch.uint8), torch.zeros(32, 1, dtype=torch.uint8))
    for call in (lambda: lp.lp_moe_gate(f, 2), lambda: lp.lp_moe_gate(f.half(), 2),
                 lambda: lp.lp_moe_gate_bwd(f[:, :2], f, f[:, :2], i), lambda: lp.lp_moe_sort(i, 4), lambda: lp.lp_moe_gather(b, i),
                 lambda: lp.lp_moe_gather(b, i[0]), lambda: lp.lp_moe_combine(b, i), lambda: lp.lp_moe_combine_bwd(b, b, i),
                 lambda: lp.lp_moe_gather_quant(b, i, i[0], 2), lambda: lp.lp_linear_fwd_w4(b, w),
                 lambda: lp.lp_linear_fwd_w4(torch.zeros(4, 32, dtype=torch.bfloat16), w)):
        with pytest.raises(ValueError):
            call()


# ---------------------------------------------------------------- the oracle itself

@pytest.mark.parametrize("renorm", [False, True])
def test_oracle_gate_gradient_against_differences(renorm):
    rng = np.random.default_rng(0)
    l, g, h = rng.standard_normal((3, 7)), rng.standard_normal((3, 2)), 1e-5
    w, e = O.gate(l, 2, renorm)
    assert np.array_equal(e, np.argsort(-l, 1, kind="stable")[:, :2])
    assert np.allclose(w.sum(1), 1) == renorm
    grad = O.gate_bwd(g, l, e, renorm)
    for i in range(7):
        d = np.zeros_like(l)
        d[:, i] = h
        diff = (O.gate(l + d, 2, renorm)[0] - O.gate(l - d, 2, renorm)[0]) / (2 * h)
        assert np.abs((diff * g).sum(1) - grad[:, i]).max() < 1e-8


def test_oracle_gate_ties_masks_and_nan():
    inf, nan = np.inf, np.nan
    l = np.array([[1.0, 2.0, 2.0, 0.0], [-inf, 3.0, -inf, -inf], [-inf] * 4, [0.0, nan, inf, 1.0]])
    w, e = O.gate(l, 3, True)
    assert e.tolist() == [[1, 2, 0], [1, -1, -1], [-1, -1, -1], [1, 2, 3]]
    assert w[1].tolist() == [1, 0, 0] and not w[2].any() and np.isnan(w[3]).all()


def test_oracle_sort_and_rows():
    rng = np.random.default_rng(1)
    e = rng.integers(-1, 6, (50, 3)).astype(np.int32)
    off, rows, order = O.sort(e, 5)
    flat = e.reshape(-1)
    live = np.flatnonzero((flat >= 0) & (flat < 5))
    assert order.tolist() == sorted(live, key=lambda p: (flat[p], p)) and off[-1] == live.size
    assert all(rows.reshape(-1)[p] == r for r, p in enumerate(order)) and (rows.reshape(-1)[flat == 5] == -1).all()
    # gather and the unweighted combine are adjoint; combine's gradients are those of its formula
    x, y, w = rng.standard_normal((50, 4)), rng.standard_normal((150, 4)), rng.standard_normal((50, 3))
    assert abs((O.gather(x, rows) * y).sum() - (x * O.combine(y, rows)[0]).sum()) < 1e-10
    dots = O.combine_dots(x, y, rows)[0]
    assert abs((O.combine(y, rows, w)[0] * x).sum() - (dots * w).sum()) < 1e-10
