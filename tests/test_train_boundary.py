"""lp_train.h on the host: exports, documented refusals before anything touches
the GPU, and the oracle of these calls against brute force (CPU only; no
kernel is launched)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import fp8_gemm_backward_amd as lp
from fp8_gemm_backward_amd import _AdamWTensorC, _QTensorC
from oracle import train as O
from oracle.formats import E4M3_TABLE

OK, NULL, SHAPE, FORMAT, ALIGN = 0, 1, 2, 3, 4
FAKE = 0x10000          # 16-byte aligned stand-in pointer; never dereferenced here
R, B = "fp8_r128", "fp8_b128"


def q(fmt, rows, cols, batch=1, axis=-1, codes=FAKE, scales=FAKE):
    return _QTensorC(lp.FMT[fmt], axis, batch, rows, cols, codes, scales, None)


def test_library_exports_every_function_of_the_header():
    text = open(os.path.join(os.path.dirname(lp.HEADER_PATH), "lp_train.h")).read()
    names = re.findall(r"^lp_status\s+(lp_\w+)\s*\(", text, re.M)
    assert len(names) == 7
    for n in names:
        assert hasattr(lp.lib, n) and hasattr(lp, "AdamWPlan" if n == "lp_adamw_plan" else n), n


@pytest.mark.parametrize("args,expect", [
    ((None, 1, 4, 64, -1, None, 0, FAKE, FAKE), NULL),
    ((FAKE, 1, 4, 64, -1, None, 0, None, FAKE), NULL),
    ((FAKE, 1, 4, 64, -1, None, 0, FAKE, None), NULL),
    ((FAKE, 1, 4, 40, -1, None, 0, FAKE, FAKE), SHAPE),           # cols % 16
    ((FAKE, 1, -4, 64, -1, None, 0, FAKE, FAKE), SHAPE),
    ((FAKE, 1, 1 << 31, 64, -1, None, 0, FAKE, FAKE), SHAPE),
    ((FAKE, 1 << 20, 1 << 10, 16, -1, None, 0, FAKE, FAKE), SHAPE),   # 2^34 elements
    ((FAKE, 1 << 24, 1, 16, -2, None, 0, FAKE, FAKE), SHAPE),     # too many tiles
    ((FAKE, 1 << 23, 1, 16, -2, None, 0, FAKE, FAKE), SHAPE),
    ((FAKE, 1, 4, 64, 0, None, 0, FAKE, FAKE), FORMAT),
    ((FAKE, 1, 4, 64, -1, FAKE, 2, FAKE, FAKE), FORMAT),          # offsets are for token runs
    ((FAKE, 2, 4, 64, -2, FAKE, 2, FAKE, FAKE), FORMAT),          # one batch entry only
    ((FAKE, 1, 4, 64, -2, FAKE, 0, FAKE, FAKE), SHAPE),
    ((FAKE, 1, 4, 64, -2, FAKE, 1025, FAKE, FAKE), SHAPE),
    ((FAKE, 1, 4, 64, -2, FAKE + 2, 2, FAKE, FAKE), ALIGN),
    ((FAKE + 8, 1, 4, 64, -1, None, 0, FAKE, FAKE), ALIGN),
    ((FAKE, 1, 4, 64, -1, None, 0, FAKE, FAKE + 4), ALIGN),
    ((None, 1, 0, 64, -1, None, 0, None, None), OK),              # empty
])
def test_r128_quant_rejects(args, expect):
    assert lp.lib.lp_r128_quant(*args, None) == expect


def test_dual_and_block_quantizers_reject():
    dual, block = lp.lib.lp_r128_quant_dual, lp.lib.lp_b128_quant
    for k in range(4):
        out = [FAKE] * 4
        out[k] = None
        assert dual(FAKE, 1, 4, 64, None, 0, *out, None) == NULL
        out[k] = FAKE + 4
        assert dual(FAKE, 1, 4, 64, None, 0, *out, None) == ALIGN
    assert dual(FAKE, 1, 4, 72, None, 0, FAKE, FAKE, FAKE, FAKE, None) == SHAPE
    assert dual(FAKE, 2, 4, 64, FAKE, 3, FAKE, FAKE, FAKE, FAKE, None) == FORMAT
    assert block(None, 1, 4, 64, FAKE, FAKE, None) == NULL
    assert block(FAKE, 1, 4, 8, FAKE, FAKE, None) == SHAPE
    assert block(FAKE, 1, 4, 64, FAKE + 1, FAKE, None) == ALIGN


def lin(g, x, w, dx=FAKE, dw=FAKE):
    r = [ctypes.byref(t) if t is not None else None for t in (g, x, w)]
    return lp.lib.lp_linear_bwd(*r, dx, dw, None)


@pytest.mark.parametrize("g,x,w,dx,dw,expect", [
    (q(R, 8, 32), q(R, 8, 64, axis=-2), q(B, 32, 64), FAKE, FAKE, FORMAT),     # one copy serves one product
    (q(R, 8, 32, axis=-2), None, q(B, 32, 64), FAKE, None, FORMAT),            # scales along the other axis
    (q(R, 8, 32), q(R, 8, 64, axis=-2), None, None, FAKE, FORMAT),
    (q(R, 8, 32), None, q("bf16", 32, 64), FAKE, None, FORMAT),
    (q(R, 8, 32), None, q(R, 32, 64), FAKE, None, FORMAT),
    (q(R, 8, 32, axis=-2), q(R, 8, 64), None, None, FAKE, FORMAT),
    (q(R, 8, 32, axis=-2), q("bf16", 8, 64), None, None, FAKE, FORMAT),
    (q("bf16", 8, 32), q(R, 8, 64, axis=-2), None, None, FAKE, FORMAT),
    (q("bf16", 8, 32), None, q(R, 32, 64), FAKE, None, FORMAT),
    (q(R, 8, 32), None, q(B, 48, 64), FAKE, None, SHAPE),
    (q(R, 8, 40), None, q(B, 40, 64), FAKE, None, SHAPE),
    (q(R, 8, 32, axis=-2), q(R, 9, 64, axis=-2), None, None, FAKE, SHAPE),
    (q(R, 8, 32, scales=None), None, q(B, 32, 64), FAKE, None, NULL),
    (q(R, 8, 32, scales=FAKE + 4), None, q(B, 32, 64), FAKE, None, ALIGN),
    (q(R, 8, 32), None, q(B, 32, 64), FAKE + 2, None, ALIGN),
    (q(R, 0, 32, codes=None, scales=None), None, q(B, 32, 64), FAKE, None, OK),   # no token: nothing to do
])
def test_linear_bwd_rejects(g, x, w, dx, dw, expect):
    assert lin(g, x, w, dx, dw) == expect


def test_split_workspace():
    """Asked for only where few tiles meet a long contraction."""
    def need(g, x, w, dx, dw):
        n = ctypes.c_size_t(7)
        args = [None if t is None else ctypes.byref(t) for t in (g, x, w)]
        assert lp.lib.lp_linear_bwd_workspace(*args, dx, dw, ctypes.byref(n)) == OK
        return n.value
    for M, N, K, expect in ((16, 8192, 64, True), (16, 1024, 64, False), (4096, 8192, 4096, False)):
        assert (need(q(R, M, N), None, q(B, N, K), FAKE, None) > 4096) == expect, "grad_X"
        assert (need(q(R, N, M, axis=-2), q(R, N, K, axis=-2), None, None, FAKE) > 4096) == expect, "grad_W"
    assert need(q(R, 8, 1024), None, q(B, 1024, 64), FAKE, None) == 0


@pytest.mark.parametrize("x,w,expect", [
    (q(R, 8, 64, axis=-2), q(B, 32, 64), FORMAT),
    (q(R, 8, 64), q("bf16", 32, 64), FORMAT),
    (q("mxfp8", 8, 64), q(B, 32, 64), FORMAT),
    (q(R, 8, 64), q(B, 40, 64), SHAPE),
    (q(R, 8, 64), q(B, 32, 80), SHAPE),
    (q(R, 8, 64), q(B, 32, 64, batch=2), SHAPE),
    (q(R, 0, 64, codes=None, scales=None), q(B, 32, 64), OK),
])
def test_linear_fwd_rejects(x, w, expect):
    assert lp.lib.lp_linear_fwd(ctypes.byref(x), ctypes.byref(w), FAKE, None) == expect


def test_forwards_that_quantize_reject():
    lin_, grp = lp.lib.lp_linear_fwd_dyn, lp.lib.lp_grouped_fwd_dyn

    def w(**kw):
        return ctypes.byref(q(**{"fmt": B, "rows": 32, "cols": 64, **kw}))
    assert lin_(FAKE, 8, None, FAKE, FAKE, FAKE, None) == NULL
    for at in (0, 3, 4, 5):
        a = [FAKE, 8, w(), FAKE, FAKE, FAKE, None]
        a[at] = None
        assert lin_(*a) == NULL
        a[at] = FAKE + 2
        assert lin_(*a) == ALIGN
    assert lin_(FAKE, 4, w(), None, None, None, None) == NULL      # few rows need no scratch, but an output
    assert lin_(FAKE, 4, w(cols=16400), None, None, FAKE, None) == NULL
    assert lin_(FAKE, 8, w(fmt="bf16"), FAKE, FAKE, FAKE, None) == FORMAT
    assert lin_(FAKE, -1, w(), FAKE, FAKE, FAKE, None) == SHAPE
    assert lin_(FAKE, 8, w(rows=40), FAKE, FAKE, FAKE, None) == SHAPE
    assert lin_(FAKE, 8, w(batch=2), FAKE, FAKE, FAKE, None) == SHAPE
    assert lin_(None, 0, w(), None, None, None, None) == OK
    assert grp(FAKE, 8, w(batch=2), FAKE, 0, FAKE, FAKE, FAKE, None) == SHAPE
    assert grp(FAKE, 8, w(batch=2), FAKE, 1025, FAKE, FAKE, FAKE, None) == SHAPE
    assert grp(FAKE, 8, w(batch=2), FAKE, 3, FAKE, FAKE, FAKE, None) == SHAPE
    assert grp(FAKE, 8, w(batch=2), None, 2, FAKE, FAKE, FAKE, None) == NULL
    assert grp(FAKE, 8, w(batch=2), FAKE + 2, 2, FAKE, FAKE, FAKE, None) == ALIGN


def tensor(n=8, param=FAKE, grad=FAKE, m=FAKE, v=FAKE, ms=None, vs=None, copy=None, ls=1.0, wd=0.0):
    return _AdamWTensorC(param, grad, m, v, ms, vs, copy, n, ls, wd)


def plan(tensors=None, count=None, pd=0, gd=0, sd=0, table=None, size=0):
    tensors = [tensor()] if tensors is None else tensors
    c = (_AdamWTensorC * max(len(tensors), 1))(*tensors)
    need, chunks = ctypes.c_size_t(size), ctypes.c_int64(-1)
    st = lp.lib.lp_adamw_plan(c, len(tensors) if count is None else count, pd, gd, sd, table, ctypes.byref(need),
                              ctypes.byref(chunks))
    return st, need.value, chunks.value


@pytest.mark.parametrize("kw,expect", [
    (dict(count=-1), SHAPE), (dict(pd=2), FORMAT), (dict(gd=-1), FORMAT), (dict(sd=2), FORMAT),
    (dict(tensors=[tensor(n=-1)]), SHAPE), (dict(tensors=[tensor(n=1 << 34)]), SHAPE),
    (dict(tensors=[tensor(n=(1 << 34) - 1)] * 4), SHAPE),          # too many chunks together
    (dict(tensors=[tensor(wd=-1.0)]), SHAPE), (dict(tensors=[tensor(ls=float("inf"))]), SHAPE),
    (dict(tensors=[tensor(wd=float("nan"))]), SHAPE),
    (dict(tensors=[tensor(param=None)]), NULL), (dict(tensors=[tensor(grad=None)]), NULL),
    (dict(tensors=[tensor(m=None)]), NULL), (dict(tensors=[tensor(v=None)]), NULL),
    (dict(sd=1), NULL), (dict(sd=1, tensors=[tensor(ms=FAKE)]), NULL),
    (dict(tensors=[tensor(param=FAKE + 2)]), ALIGN), (dict(gd=1, tensors=[tensor(grad=FAKE + 1)]), ALIGN),
    (dict(tensors=[tensor(m=FAKE + 1)]), ALIGN), (dict(sd=1, tensors=[tensor(ms=FAKE, vs=FAKE + 2)]), ALIGN),
    (dict(pd=1, tensors=[tensor(copy=FAKE)]), FORMAT),
    (dict(tensors=[tensor(n=0), tensor(m=None)]), NULL),           # every tensor is checked
    (dict(table=FAKE + 4), ALIGN), (dict(table=FAKE, size=8), SHAPE),
    (dict(tensors=[tensor(n=0, param=None, grad=None, m=None, v=None)]), OK), (dict(tensors=[]), OK),
])
def test_adamw_plan_rejects(kw, expect):
    assert plan(**kw)[0] == expect


def test_adamw_plan_chunks_and_size():
    st, need, chunks = plan([tensor(n=n) for n in (1, 4096, 4097, 0, 10000)])
    assert (st, chunks) == (OK, 1 + 1 + 2 + 0 + 3) and need >= 5 * 64 + 7 * 4
    buf = ctypes.create_string_buffer(need + 8)
    assert plan([tensor(n=n) for n in (1, 4096, 4097, 0, 10000)], table=(ctypes.addressof(buf) + 7) // 8 * 8, size=need)[0] == OK
    c = (_AdamWTensorC * 1)(tensor())
    assert lp.lib.lp_adamw_plan(c, 1, 0, 0, 0, None, None, ctypes.byref(ctypes.c_int64())) == NULL


@pytest.mark.parametrize("kw,expect", [
    (dict(count=-1), SHAPE), (dict(chunks=-1), SHAPE), (dict(chunks=1 << 24), SHAPE), (dict(step=0), SHAPE),
    (dict(b1=1.0), SHAPE), (dict(b2=-0.1), SHAPE), (dict(b1=float("nan")), SHAPE), (dict(lr=-1.0), SHAPE),
    (dict(lr=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE), (dict(pd=2), FORMAT), (dict(gd=-1), FORMAT),
    (dict(sd=2), FORMAT), (dict(table=None), NULL), (dict(table=FAKE + 4), ALIGN), (dict(gs=FAKE + 2), ALIGN),
    (dict(table=None, chunks=0), OK),
])
def test_adamw_rejects(kw, expect):
    a = {**dict(table=FAKE, count=1, chunks=1, pd=0, gd=0, sd=0, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, step=1, gs=None), **kw}
    assert lp.lib.lp_adamw(*a.values(), None) == expect


def test_binding_rejects_host_tensors_and_mismatches():
    h = torch.zeros(8, 64, dtype=torch.bfloat16)
    for call in (lambda: lp.lp_r128_quant(h), lambda: lp.lp_r128_quant_dual(h), lambda: lp.lp_b128_quant(h),
                 lambda: lp.lp_linear_fwd_dyn(h, lp.QTensor(B, torch.zeros(32, 64, dtype=torch.uint8), torch.ones(1, 1)))):
        with pytest.raises(ValueError):
            call()
    f = torch.zeros(8)
    for bad in (dict(grads=[]), dict(exp_avg_scales=[f]), dict(weight_decay=[0.1, 0.2]), dict()):
        with pytest.raises(ValueError):
            lp.AdamWPlan(**{**dict(params=[f], grads=[f], exp_avgs=[f], exp_avg_sqs=[f]), **bad})
    with pytest.raises(ValueError):
        lp.AdamWPlan([f.half()], [f], [f], [f])


# ---------------------------------------------------------------- the oracle itself

def test_oracle_quantization_is_the_nearest_code():
    rng = np.random.default_rng(0)
    v = rng.standard_normal(128) * np.exp(rng.standard_normal(128) * 4)
    codes, s = O.quant_set(v)
    assert s == np.float32(np.abs(v).max() / 448)
    t = (v / np.float64(s)).astype(np.float32).astype(np.float64)
    finite = E4M3_TABLE[np.isfinite(E4M3_TABLE)]
    assert np.array_equal(np.abs(E4M3_TABLE[codes] - t), np.abs(finite[None] - t[:, None]).min(1))
    assert O.quant_set(np.zeros(5))[1] == np.float32(2.0 ** -64 / 448) and not O.quant_set(np.zeros(5))[0].any()
    codes, s = O.quant_set(np.array([1.0, -np.inf, -2.0]))
    assert np.isnan(s) and codes.tolist() == [0x7F, 0xFF, 0xFF]


def test_oracle_runs_of_groups_are_disjoint_and_in_range():
    rng = np.random.default_rng(1)
    for _ in range(200):
        sizes = rng.integers(0, 400, rng.integers(1, 9))
        rows = int(sizes.sum() + rng.integers(0, 50))
        got = O.spans(rows, np.cumsum(sizes))
        runs = [r for r, _, _ in got]
        assert len(set(runs)) == len(runs) and all(0 <= r < rows // 128 + len(sizes) for r in runs)
        assert sum(b - a for _, a, b in got) == sizes.sum() and all(0 < b - a <= 128 for _, a, b in got)


def test_oracle_adamw_against_a_scalar_loop():
    p, m, v = 0.5, 0.0, 0.0
    P, M, V = (np.array([x]) for x in (p, m, v))
    for t in range(1, 6):
        g = 0.3 * t - 1
        P, M, V = O.adamw(P, np.array([g]), M, V, 0.01, 0.9, 0.99, 1e-8, t, 0.1)
        m, v = 0.9 * m + 0.1 * g, 0.99 * v + 0.01 * g * g
        p = p * (1 - 0.01 * 0.1) - 0.01 * (m / (1 - 0.9 ** t)) / ((v / (1 - 0.99 ** t)) ** 0.5 + 1e-8)
        assert abs(P[0] - p) < 1e-15
