"""The calls around a mixture of experts' grouped products (lp_moe.h) against the
fp64 oracle (GPU): indices and copies bit for bit, sums within bounds derived
from the arithmetic."""
import numpy as np
import pytest
import torch

import workloads as W
from gpu_util import assert_bits_equal, bf16_dev, bits_host, dev
from oracle import moe as O
from oracle.formats import bf16_bits_to_f64, f32_to_bf16_bits

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24                 # half a step of fp32
U16 = 2.0 ** -8                  # half a step of bf16
TINY = 2.0 ** -126


def bits(rng, shape, sigma=1.0):
    return W.bf16_bits((rng.standard_normal(shape) * sigma).astype(np.float32))


# ---------------------------------------------------------------- gate

def logits_of(rng, T, E, dtype, kind):
    """(device tensor, its values in fp64)."""
    v = (rng.standard_normal((T, E)) * 2).astype(np.float32)
    if kind == "ties":
        v = np.round(v)
    elif kind == "masked":
        v[rng.random((T, E)) < 0.8] = -np.inf
        v[0] = -np.inf
        v[T - 1, :] = -np.inf
        v[T - 1, E - 1] = 3e38 if dtype == torch.float32 else 2.0 ** 127      # (the largest left alone)
    elif kind == "wide":
        v *= 30
    elif kind == "lowest":                               # a mask of the type's lowest value: chosen last, but chosen
        v[rng.random((T, E)) < 0.7] = torch.finfo(dtype).min
    if dtype == torch.bfloat16:
        b = W.bf16_bits(v)
        return bf16_dev(b), bf16_bits_to_f64(b)
    return dev(v), v.astype(np.float64)


def gate_rtol(values, E):
    """Relative error of one weight: the exponential's argument is rounded by half a step of its size (-104 and below give
    0), the exponential by at most 2 ulp, sums of E such terms by log-depth rounding within a wave, then a division."""
    return U32 * (104 + 4 + (E / 64 + 8) * 2 + 2)


GATES = [(1, 1, 1), (1, 64, 8), (3, 2, 2), (65, 40, 6), (130, 64, 64), (33, 65, 5), (17, 100, 10), (9, 256, 8), (9, 300, 1),
         (5, 512, 33), (4, 1000, 16), (3, 1024, 64)]


@pytest.mark.parametrize("T,E,k", GATES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["normal", "ties", "masked", "wide", "lowest"])
def test_gate(lp, T, E, k, dtype, kind):
    rng = np.random.default_rng(T * 10007 + E * 31 + k)
    l, lv = logits_of(rng, T, E, dtype, kind)
    g = rng.standard_normal((T, k)).astype(np.float32)
    for renorm in (False, True):
        w, e = lp.lp_moe_gate(l, k, renorm=renorm)
        gl = lp.lp_moe_gate_bwd(dev(g), l, w, e, renorm=renorm)
        rw, re_ = O.gate(lv, k, renorm)
        assert_bits_equal(e.cpu().numpy(), re_, "chosen")
        wv, rtol = w.cpu().numpy().astype(np.float64), gate_rtol(lv, E)
        assert (np.abs(wv - rw) <= rtol * rw + TINY).all(), np.abs(wv / np.maximum(rw, 1e-300) - 1).max()
        # dl_i = sum over slots of w (g [own] - q_i g): twice the weights' error, k products and sums, one rounding
        ref = O.gate_bwd(g.astype(np.float64), lv, re_, renorm)
        size = np.zeros((T, E))
        q = np.zeros((T, E))
        for t in range(T):
            for j in range(k):
                if re_[t, j] >= 0:
                    size[t, re_[t, j]] += rw[t, j] * abs(g[t, j])
                    q[t, re_[t, j]] = rw[t, j]
            if not renorm and (re_[t] >= 0).any():
                q[t] = np.exp(lv[t] - lv[t].max())
                q[t] /= q[t].sum()
        size += q * (rw * np.abs(g)).sum(1, keepdims=True)
        tol = (2 * rtol + (k + 8) * U32) * size + (U16 if dtype == torch.bfloat16 else U32) * np.abs(ref)
        # (below the normal range of the type a rounding is half the smallest step)
        tol += 2.0 ** -134 if dtype == torch.bfloat16 else 2.0 ** -149
        got = gl.float().cpu().numpy().astype(np.float64)
        assert gl.dtype == dtype and (np.abs(got - ref) <= tol + k * TINY).all()


@pytest.mark.parametrize("T,E,k", [(7, 203, 8), (6, 203, 12), (5, 144, 9), (9, 136, 8), (4, 1001, 5), (3, 1001, 20), (66, 12, 12), (5, 520, 8), (2, 509, 64)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["normal", "ties", "masked"])
def test_gate_of_odd_rows(lp, T, E, k, dtype, kind):
    test_gate(lp, T, E, k, dtype, kind)


@pytest.mark.parametrize("E,k", [(64, 8), (256, 8), (256, 10), (512, 8), (1024, 9)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gate_of_logits_beside_a_16_byte_border(lp, E, k, dtype):
    """What an aligned copy gives: the same experts, weights and gradients up to the order of the softmax's sum."""
    rng = np.random.default_rng(E + k)
    off = 4 // torch.empty(0, dtype=dtype).element_size()
    l = dev(rng.standard_normal(33 * E + off).astype(np.float32)).to(dtype)[off:].view(33, E)
    g, out = dev(rng.standard_normal((33, k)).astype(np.float32)), torch.empty(33 * E + off, dtype=dtype, device="cuda")[off:].view(33, E)
    assert l.data_ptr() % 16 == 4 and out.data_ptr() % 16 == 4
    for renorm in (False, True):
        (w, e), (cw, ce) = lp.lp_moe_gate(l, k, renorm=renorm), lp.lp_moe_gate(l.clone(), k, renorm=renorm)
        rtol = 2 * gate_rtol(None, E)
        assert torch.equal(e, ce) and ((w - cw).abs() <= rtol * cw).all()
        a, b = lp.lp_moe_gate_bwd(g, l, cw, ce, renorm=renorm, grad_logits=out), lp.lp_moe_gate_bwd(g, l.clone(), cw, ce, renorm=renorm)
        # (each p of the softmax times the inner product, and a rounding to bf16)
        size = (cw * g.abs()).sum(1, keepdim=True)
        assert ((a - b).float().abs() <= 2 * rtol * size + 2 * (U16 if dtype == torch.bfloat16 else U32) * b.float().abs()).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_gate_of_a_row_that_is_not_finite(lp, dtype, bad):
    """NaN weights in that row, whose NaN or infinity is chosen first; the other rows as without it."""
    rng = np.random.default_rng(5)
    l = dev(rng.standard_normal((6, 70)).astype(np.float32)).to(dtype)
    clean = [lp.lp_moe_gate(l, 4, renorm=r) for r in (False, True)]
    l[2, 66] = bad
    l[4] = float("nan")
    for renorm, (cw, ce) in zip((False, True), clean):
        w, e = lp.lp_moe_gate(l, 4, renorm=renorm)
        assert e[2, 0] == 66 and torch.isnan(w[2]).all() and torch.isnan(w[4]).all()
        assert e[4].tolist() == [0, 1, 2, 3]
        keep = [0, 1, 3, 5]
        assert torch.equal(w[keep], cw[keep]) and torch.equal(e[keep], ce[keep])
        gl = lp.lp_moe_gate_bwd(torch.ones(6, 4, device="cuda"), l, w, e, renorm=renorm)
        assert torch.isfinite(gl[keep].float()).all() and torch.isnan(gl[2, 66].float())


def test_gate_bwd_ignores_experts_out_of_range(lp):
    """Slots of nobody's have no gradient, whatever their weight and incoming gradient hold."""
    l = torch.randn(5, 32, device="cuda")
    w, e = lp.lp_moe_gate(l, 4, renorm=False)
    g = torch.randn(5, 4, device="cuda")
    part = lp.lp_moe_gate_bwd(torch.where(torch.arange(4, device="cuda") < 3, g, 0.0), l, w, e, renorm=False)
    for bad in (-1, 32, 1 << 30, -(1 << 31)):
        e2, w2, g2 = e.clone(), w.clone(), g.clone()
        e2[:, 3], w2[:, 3], g2[:, 3] = bad, float("nan"), float("nan")
        assert torch.equal(lp.lp_moe_gate_bwd(g2, l, w2, e2, renorm=False), part)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", [(6, 40, 5), (9, 256, 8), (3, 700, 20), (2, 5, 3)])
def test_gate_bwd_of_an_expert_chosen_twice(lp, T, E, k, renorm):
    """Slots of one expert add up: w_j (g_j - sum w g) each, or p_i times their g and once the inner product."""
    rng = np.random.default_rng(T)
    lv, g = rng.standard_normal((T, E)).astype(np.float32), rng.standard_normal((T, k)).astype(np.float32)
    e, w = rng.integers(0, min(E, 4), (T, k)).astype(np.int32), rng.random((T, k)).astype(np.float32)
    e[0, 0], w[0, 0] = -1, np.nan
    got = lp.lp_moe_gate_bwd(dev(g), dev(lv), dev(w), dev(e), renorm=renorm).cpu().numpy().astype(np.float64)
    w64, g64 = np.where(e >= 0, w, 0).astype(np.float64), g.astype(np.float64)
    inner = (w64 * g64).sum(1)
    p = np.exp(lv.astype(np.float64) - lv.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    want = np.zeros((T, E)) if renorm else -p * inner[:, None]
    size = np.zeros((T, E)) if renorm else p * (w64 * np.abs(g64)).sum(1)[:, None]
    for t in range(T):
        for j in range(k):
            if e[t, j] >= 0:
                # (without renorm the slots' weights are the softmax's; here any, and each counts as it is)
                want[t, e[t, j]] += w64[t, j] * (g64[t, j] - inner[t] if renorm else g64[t, j])
                size[t, e[t, j]] += w64[t, j] * (abs(g64[t, j]) + (w64[t] * np.abs(g64[t])).sum())
    assert (np.abs(got - want) <= (2 * gate_rtol(lv, E) + (k + 8) * U32) * size + U32 * np.abs(want) + 1e-37).all()


@pytest.mark.parametrize("renorm", [False, True])
def test_gate_gradient_against_differences(lp, renorm):
    """Central differences of fp32 weights with a step of 2^-7: truncation (third derivatives at most 2 of a probability)
    below 2 h^2 / 6, rounding 2 rtol / (2 h)."""
    torch.manual_seed(3)
    T, E, k, h = 7, 12, 3, 2.0 ** -7
    l = torch.randn(T, E, device="cuda")
    w, e = lp.lp_moe_gate(l, k, renorm=renorm)
    g = torch.randn(T, k, device="cuda")
    grad = lp.lp_moe_gate_bwd(g, l, w, e, renorm=renorm)
    tol = (2 * h * h / 6 + gate_rtol(None, E) / h) * g.abs().sum(1)
    for i in range(E):
        d = []
        for s in (h, -h):
            moved = l.clone()
            moved[:, i] += s
            mw, me = lp.lp_moe_gate(moved, E, renorm=False)
            full = torch.zeros(T, E, device="cuda").scatter_(1, me.long(), mw)
            part = full.gather(1, e.long())                          # the same experts' weights
            d.append((part / part.sum(1, keepdim=True) if renorm else part).double())
        diff = (((d[0] - d[1]) / (2 * h)) * g).sum(1)
        assert ((diff - grad[:, i]).abs() <= tol).all()


# ---------------------------------------------------------------- sort

def check_sort(lp, experts, groups):
    off, rows, order = lp.lp_moe_sort(dev(experts), groups)
    ro, rr, rp = O.sort(experts, groups)
    assert_bits_equal(off.cpu().numpy(), ro, "offsets")
    assert_bits_equal(rows.cpu().numpy(), rr, "rows")
    assert_bits_equal(order.cpu().numpy()[:rp.size], rp, "order")


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (12, 8, 64), (63, 1, 2), (64, 1, 3), (65, 3, 7), (511, 8, 1),
                                   (512, 8, 5), (513, 8, 129), (4099, 1, 1024), (5000, 7, 40), (40000, 6, 256),
                                   (70000, 8, 1000)])
def test_sort(lp, T, k, E):
    rng = np.random.default_rng(T + k + E)
    even = rng.integers(0, E, (T, k)).astype(np.int32)
    check_sort(lp, even, E)
    few = np.where(rng.random((T, k)) < 0.9, E // 2, even).astype(np.int32)        # nearly all one expert's
    few[rng.random((T, k)) < 0.3] = -1
    few.reshape(-1)[0] = E                                                         # out of range on every side
    few.reshape(-1)[-1] = np.iinfo(np.int32).max
    few.reshape(-1)[T * k // 2] = np.iinfo(np.int32).min
    check_sort(lp, few, E)


@pytest.mark.parametrize("n", [1, 63, 1023, 1024, 1025, 2047, 2048, 2049, 3071, 65535, 65536, 65537])
@pytest.mark.parametrize("E", [1, 3, 256, 257, 1024])
def test_sort_at_the_borders_of_its_workgroups(lp, n, E):
    """Evenly spread and all but one of one expert; some of nobody's."""
    rng = np.random.default_rng(n + E)
    for kind in range(2):
        e = rng.integers(-1, E + 1, n).astype(np.int32) if kind == 0 else np.full(n, E - 1, np.int32)
        if kind:
            e[n // 2] = 0
        off, rows, order = lp.lp_moe_sort(dev(e), E)
        live = np.flatnonzero((e >= 0) & (e < E))
        want = live[np.argsort(e[live], kind="stable")]
        assert_bits_equal(off.cpu().numpy(), np.cumsum(np.bincount(e[live], minlength=E)).astype(np.int32), "offsets")
        assert_bits_equal(order.cpu().numpy()[:live.size], want.astype(np.int32), "order")
        at = np.full(n, -1, np.int32)
        at[want] = np.arange(live.size)
        assert_bits_equal(rows.cpu().numpy(), at, "rows")


@pytest.mark.parametrize("n", [0, 1, 4096, 4097, 10000])
def test_sort_of_nobodys_pairs(lp, n):
    experts = torch.full((n, 1), -1, dtype=torch.int32, device="cuda")
    off, rows, _ = lp.lp_moe_sort(experts, 9)
    assert off.tolist() == [0] * 9 and (rows == -1).all() and rows.shape == experts.shape


def test_sort_leaves_the_tail_of_order(lp):
    """Entries past the last offset are left as they were."""
    e = np.array([[2, -1, 0], [7, 0, 3]], np.int32)
    order = torch.full((6,), 77, dtype=torch.int32, device="cuda")
    off, rows = torch.empty(4, dtype=torch.int32, device="cuda"), torch.empty(2, 3, dtype=torch.int32, device="cuda")
    t = dev(e)
    assert lp.lib.lp_moe_sort(t.data_ptr(), 6, 4, off.data_ptr(), rows.data_ptr(), order.data_ptr(), None, 0,
                              lp._stream(None)) == 0
    assert off.tolist() == [2, 2, 3, 4] and rows.tolist() == [[2, -1, 0], [-1, 1, 3]]
    assert order.tolist() == [2, 4, 0, 5, 77, 77]


# ---------------------------------------------------------------- rows there and back

ROWS = [(1, 1, 1, 8, 0.0), (1, 8, 64, 7168, 0.0), (12, 8, 64, 2048, 0.0), (3, 2, 4, 16, 0.5), (65, 6, 40, 1040, 0.2),
        (130, 9, 16, 264, 0.1), (40, 17, 20, 48, 0.3), (5, 64, 70, 24, 0.0), (700, 2, 8, 512, 1.0), (33, 3, 5, 4096, 0.9)]


def routing(rng, T, k, E, drop):
    e = np.stack([rng.permutation(max(E, k))[:k] for _ in range(T)]).astype(np.int32)
    e[rng.random((T, k)) < drop] = -1
    return e, max(E, k)


@pytest.mark.parametrize("T,k,E,H,drop", ROWS)
def test_rows_there_and_back(lp, T, k, E, H, drop):
    rng = np.random.default_rng(T * 13 + k + H)
    experts, E = routing(rng, T, k, E, drop)
    ro, rr, rp = O.sort(experts, E)
    rows = dev(rr)
    xb, yb, gb = bits(rng, (T, H)), bits(rng, (T * k, H)), bits(rng, (T, H), 0.01)
    yb[rp.size:] = 0x7FC0                                # NaN in rows that no pair has: never read
    w = rng.standard_normal((T, k)).astype(np.float32)
    w[experts < 0] = np.nan                              # nor the weight of a pair without a row
    live = np.arange(T * k) < rp.size

    out = torch.full((T * k, H), 7.0, dtype=torch.bfloat16, device="cuda")
    lp.lp_moe_gather(bf16_dev(xb), rows, out=out)
    want = np.where(live[:, None], O.gather(xb, rr), W.bf16_bits(np.float32([7.0]))[0])
    assert_bits_equal(bits_host(out), want, "gather")

    y, x64, y64, g64 = bf16_dev(yb), bf16_bits_to_f64(xb), bf16_bits_to_f64(yb), bf16_bits_to_f64(gb)
    for weights in (w, None):
        got = lp.lp_moe_combine(y, rows, None if weights is None else dev(weights))
        ref, size = O.combine(y64, rr, weights)
        err = np.abs(got.float().cpu().numpy() - ref)
        assert (err <= U16 * np.abs(ref) + k * U32 * (1 + U16) * size + 2.0 ** -134).all(), (weights is None, err.max())
        assert not got[torch.from_numpy((rr < 0).all(1)).cuda()].any()

        gy = torch.full((T * k, H), 7.0, dtype=torch.bfloat16, device="cuda")
        _, gw = lp.lp_moe_combine_bwd(bf16_dev(gb), y, rows, None if weights is None else dev(weights), grad_y=gy)
        rows_of_grad = O.gather(np.float32(g64), rr)
        if weights is not None:
            by_row = np.zeros((T * k, 1), np.float32)
            by_row[:rp.size, 0] = weights.reshape(-1)[rp]
            rows_of_grad = rows_of_grad * by_row                     # one fp32 rounding, as the kernel's
        want = np.where(live[:, None], f32_to_bf16_bits(rows_of_grad), W.bf16_bits(np.float32([7.0]))[0])
        assert_bits_equal(bits_host(gy), want, "grad_y")
        ref, size = O.combine_dots(g64, y64, rr)
        assert (np.abs(gw.cpu().numpy() - ref) <= (H / 256 + 8 + 16) * U32 * size).all()

    only, none = lp.lp_moe_combine_bwd(bf16_dev(gb), None, rows, dev(w), need_dw=False)
    assert none is None and torch.equal(only[:rp.size].view(torch.int16), lp.lp_moe_combine_bwd(
        bf16_dev(gb), y, rows, dev(w))[0][:rp.size].view(torch.int16))
    none, dots = lp.lp_moe_combine_bwd(bf16_dev(gb), y, rows, dev(w), need_dy=False)
    assert none is None and torch.equal(dots, gw)


@pytest.mark.parametrize("T,k,E,H,drop", [(1027, 3, 8, 264, 0.1), (1030, 9, 16, 136, 0.1), (1024, 1, 3, 1024, 0.0), (2049, 2, 5, 1032, 0.2),
                                          (8195, 2, 8, 256, 0.1), (8193, 5, 7, 24, 0.2), (8191, 1, 2, 256, 0.0)])
def test_rows_of_many_tokens(lp, T, k, E, H, drop):
    test_rows_there_and_back(lp, T, k, E, H, drop)


@pytest.mark.parametrize("bad", [-1, -7, 24, 1 << 20, (1 << 31) - 1, -(1 << 31)])
def test_rows_out_of_range_are_no_rows(lp, bad):
    rng = np.random.default_rng(9)
    T, k, H = 12, 2, 40
    rows = rng.permutation(T * k).astype(np.int32).reshape(T, k)
    without, withbad = rows.copy(), rows.copy()
    hit = rng.random((T, k)) < 0.4
    without[hit], withbad[hit] = -1, bad
    x, y, g = (bf16_dev(bits(rng, (n, H))) for n in (T, T * k, T))
    w = torch.randn(T, k, device="cuda")
    a, b = dev(without), dev(withbad)
    zero = lambda: torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    assert torch.equal(lp.lp_moe_gather(x, a, out=zero()), lp.lp_moe_gather(x, b, out=zero()))
    assert torch.equal(lp.lp_moe_combine(y, a, w), lp.lp_moe_combine(y, b, w))
    for p, q in zip(lp.lp_moe_combine_bwd(g, y, a, w, grad_y=zero()), lp.lp_moe_combine_bwd(g, y, b, w, grad_y=zero())):
        assert torch.equal(p, q)


def test_empty_rows(lp):
    """No token; rows of no column."""
    rows0 = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    e = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    assert lp.lp_moe_gather(e, rows0).shape == (0, 16) and lp.lp_moe_combine(e, rows0).shape == (0, 16)
    assert lp.lp_moe_combine_bwd(e, e, rows0)[1].shape == (0, 3)
    assert lp.lp_moe_gate(torch.empty(0, 4, device="cuda"), 2)[0].shape == (0, 2)
    rows = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    n = torch.empty(6, 0, dtype=torch.bfloat16, device="cuda")
    assert lp.lp_moe_combine(n, rows).shape == (2, 0)
    assert lp.lp_moe_combine_bwd(n[:2], n, rows)[1].tolist() == [[0.0] * 3] * 2


# ---------------------------------------------------------------- rows straight into FP8

def same_runs(lp, got, want, off, H):
    """Everything that lp_r128_quant_dual writes, in both copies."""
    n = int(off[-1])
    assert torch.equal(got[0].codes[0, :n], want[0].codes[0, :n])
    assert torch.equal(got[0].scales[0, :, :n].view(torch.int32), want[0].scales[0, :, :n].view(torch.int32))
    assert torch.equal(got[1].codes[0, :n], want[1].codes[0, :n])
    start = 0
    for g, end in enumerate(off.tolist()):
        at = slice(start // 128 + g, start // 128 + g + -(-(end - start) // 128))
        assert torch.equal(got[1].scales[0, at].view(torch.int32), want[1].scales[0, at].view(torch.int32)), g
        start = end


@pytest.mark.parametrize("T,k,E,H,drop", [(1, 1, 1, 16, 0.0), (12, 8, 64, 2048, 0.0), (300, 3, 4, 144, 0.2), (65, 6, 40, 1040, 0.3),
                                          (1000, 2, 3, 272, 0.0), (50, 4, 8, 128, 1.0)])
@pytest.mark.parametrize("weighted", [False, True])
def test_gather_quant_is_gather_then_quant(lp, T, k, E, H, drop, weighted):
    rng = np.random.default_rng(T + H)
    experts, E = routing(rng, T, k, E, drop)
    off, rows, order = lp.lp_moe_sort(dev(experts), E)
    xb = bits(rng, (T, H))
    xb[T // 2, ::3] = 0
    if H > 16:
        xb[T // 3, 5], xb[0, 7] = 0x7F80, 0xFFC1                     # an infinity and a NaN
    x, w = bf16_dev(xb), dev(rng.random((T, k)).astype(np.float32)) if weighted else None
    plain = lp.lp_moe_combine_bwd(x, None, rows, w, need_dw=False)[0]
    same_runs(lp, lp.lp_moe_gather_quant(x, order, off, k, weights=w), lp.lp_r128_quant_dual(plain, off), off, H)


@pytest.mark.parametrize("T,E,H", [(200, 64, 2192), (511, 64, 2048), (300, 300, 400), (16, 1000, 144)])
@pytest.mark.parametrize("weighted", [False, True])
def test_gather_quant_of_many_short_runs(lp, T, E, H, weighted):
    """Most experts with a row or none, one with every token's first slot: runs of 1 to 128 rows beside one another."""
    rng = np.random.default_rng(T + E)
    experts = rng.integers(0, E, (T, 2)).astype(np.int32)
    experts[:, 0] = E // 3
    experts[rng.random((T, 2)) < 0.1] = -1
    off, rows, order = lp.lp_moe_sort(dev(experts), E)
    xb = bits(rng, (T, H))
    xb[T // 3, 5], xb[0, 7], xb[T - 1, H - 1] = 0x7F80, 0xFFC1, 0x7FC0
    x, w = bf16_dev(xb), dev(rng.random((T, 2)).astype(np.float32)) if weighted else None
    plain = lp.lp_moe_combine_bwd(x, None, rows, w, need_dw=False)[0]
    out = (lp.QTensor("fp8_r128", torch.full((1, 2 * T, H), 99, dtype=torch.uint8, device="cuda"),
                      torch.full((1, -(-H // 128), 2 * T), 5.0, device="cuda"), None, (1, 2 * T, H), -1),
           lp.QTensor("fp8_r128", torch.full((1, 2 * T, H), 99, dtype=torch.uint8, device="cuda"),
                      torch.full((1, 2 * T // 128 + E, H), 5.0, device="cuda"), None, (1, 2 * T, H), -2))
    got, n = lp.lp_moe_gather_quant(x, order, off, 2, weights=w, out=out), int(off[-1])
    same_runs(lp, got, lp.lp_r128_quant_dual(plain, off), off, H)
    assert (got[0].codes[0, n:] == 99).all() and (got[1].codes[0, n:] == 99).all() and (got[0].scales[0, :, n:] == 5).all()


def test_gather_quant_leaves_what_no_expert_has(lp):
    T, k, H, E = 100, 3, 160, 4
    rng = np.random.default_rng(2)
    experts, _ = routing(rng, T, k, E, 0.5)
    off, rows, order = lp.lp_moe_sort(dev(experts), E)
    n = int(off[-1])
    out = (lp.QTensor("fp8_r128", torch.full((1, T * k, H), 99, dtype=torch.uint8, device="cuda"),
                      torch.full((1, 2, T * k), 5.0, device="cuda"), None, (1, T * k, H), -1),
           lp.QTensor("fp8_r128", torch.full((1, T * k, H), 99, dtype=torch.uint8, device="cuda"),
                      torch.full((1, T * k // 128 + E, H), 5.0, device="cuda"), None, (1, T * k, H), -2))
    got = lp.lp_moe_gather_quant(bf16_dev(bits(rng, (T, H))), order, off, k, out=out)
    assert got[1].run_groups == E
    for q in got:
        assert (q.codes[0, n:] == 99).all()
    assert (got[0].scales[0, :, n:] == 5).all()
    used, start = set(), 0
    for g, end in enumerate(off.tolist()):
        used |= {start // 128 + g + i for i in range(-(-(end - start) // 128))}
        start = end
    for run in range(T * k // 128 + E):
        assert (got[1].scales[0, run] == 5).all() == (run not in used)


def test_gather_quant_of_pairs_out_of_range(lp):
    """A row whose pair is none has zeros: code 0 under its own scale."""
    T, k, H = 40, 2, 128
    rng = np.random.default_rng(3)
    off = torch.tensor([30, 80], dtype=torch.int32, device="cuda")
    order = rng.permutation(T * k).astype(np.int32)
    bad = order.copy()
    bad[[0, 31, 79]] = -1, T * k, (1 << 31) - 1
    x = bf16_dev(bits(rng, (T, H)))
    rows = np.empty(T * k, np.int32)
    rows[order] = np.arange(T * k)
    plain = lp.lp_moe_gather(x, dev(rows.reshape(T, k)))
    plain[[0, 31, 79]] = 0
    same_runs(lp, lp.lp_moe_gather_quant(x, dev(bad), off, k), lp.lp_r128_quant_dual(plain, off), off, H)


@pytest.mark.parametrize("H", [128, 144])
def test_gather_quant_of_pairs_out_of_range_beside_a_nan_weight(lp, H):
    """Pair 0's NaN reaches its own row's runs only, neither a row of no pair nor one past the group's end."""
    T, k = 40, 2
    rng = np.random.default_rng(4)
    off = torch.tensor([30, 75], dtype=torch.int32, device="cuda")
    order = rng.permutation(T * k).astype(np.int32)
    bad = order.copy()
    bad[[1, 33, 74]] = -1, T * k, -(1 << 31)
    x, w = bf16_dev(bits(rng, (T, H))), rng.random((T, k)).astype(np.float32)
    for value in (0.5, np.nan, np.inf):
        w[0, 0] = value
        rows = np.empty(T * k, np.int32)
        rows[order] = np.arange(T * k)
        plain = lp.lp_moe_combine_bwd(x, None, dev(rows.reshape(T, k)), dev(w), need_dw=False)[0]
        plain[[1, 33, 74]] = 0
        same_runs(lp, lp.lp_moe_gather_quant(x, dev(bad), off, k, weights=dev(w)), lp.lp_r128_quant_dual(plain, off), off, H)


@pytest.mark.parametrize("H", [144, 4096])
@pytest.mark.parametrize("ends", [[5, 2, 9], [-3, 4, 1 << 30], [0, 0, 0], [1 << 30, 0, -1], [30, 20, 80]])
def test_gather_quant_of_bad_offsets(lp, ends, H):
    """Ends that fall, below zero or past the rows: taken as the largest so far, within the rows, as the quantizer takes
    them (64 groups and more of them empty, so that both ways of sharing out the tiles are met)."""
    T, k = 40, 2
    rng = np.random.default_rng(6)
    ends = ends + [ends[-1]] * 61
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    clean = torch.from_numpy(np.maximum.accumulate(np.clip(ends, 0, T * k))).int()
    order = rng.permutation(T * k).astype(np.int32)
    rows = np.empty(T * k, np.int32)
    rows[order] = np.arange(T * k)
    x = bf16_dev(bits(rng, (T, H)))
    plain = lp.lp_moe_gather(x, dev(rows.reshape(T, k)))
    got = lp.lp_moe_gather_quant(x, dev(order), off, k)
    same_runs(lp, got, lp.lp_r128_quant_dual(plain, clean.cuda()), clean, H)
