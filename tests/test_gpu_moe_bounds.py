"""Calls of lp_moe.h held to what their arithmetic can make of the result, and the
ways through them that sizes choose (GPU)."""
import numpy as np
import pytest
import torch

from oracle import moe as O
from test_gpu_moe import same_runs
from test_gpu_moe_layer import Weights, f64
from test_gpu_train_streams import busy, segment_stream  # noqa: F401

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


# ---------------------------------------------------------------- gate

U32, U16 = 2.0 ** -24, 2.0 ** -8                         # half a step of fp32 and bf16
GATES = [(40, 12, 12), (33, 16, 5), (50, 64, 64), (21, 100, 33), (17, 203, 64), (30, 256, 64), (20, 256, 8), (9, 300, 64), (9, 1001, 64), (8, 1024, 64)]


def far_logits(T, E, k, dtype, seed):
    """fp32 [T, E] from a peak down to 70 below it, most of the k largest far below; differences of two are exact in fp32
    (multiples of 2^-10, of 1/4 in bf16's range)."""
    rng = np.random.default_rng(seed)
    unit = 4 if dtype == torch.bfloat16 else 1024
    v = -40 * unit + rng.integers(0, 8 * unit, (T, E))
    v[:, rng.permutation(E)[:k]] = rng.integers(-40 * unit, 30 * unit, (T, k))
    v[np.arange(T), rng.integers(0, E, T)] = 30 * unit
    return (v / unit).astype(np.float32)


def adds(E):
    """Roundings on the way of a term into the sum over a row: those of a lane, then those over the lanes."""
    return (max(1, -(-E // 16)) - 1 + 4) if E <= 256 else -(-E // 64) - 1 + 6


def weights_bound(l, k, E, renorm):
    """Relative error of a weight e^d / sum, in fp32.

    The exponential: the instruction's 2^t is within a step (2 U32); t = d log2 e is split into a rounded part and its
    residual, whose own rounding is 2^-24 of half a step of t < 128 and whose square term is below 2^-36: nothing; one
    rounding puts the residual in.  3 U32, and below 0.01 of them for the rest.
    The sum: of the chosen, the same exponentials, at most 4 a lane, then 6 times over the lanes.  Of all, exponentials
    without the residual: half a step of t times ln 2, |d| U32, and |d| 2^-26 0.9 for what log2 e has beyond fp32; in the
    sum the mean of |d| by weight counts.  The quotient is correctly rounded."""
    if renorm:
        return (3.01 + 3.01 + 9 + 1) * U32
    d = np.abs(l - l.max(1, keepdims=True))
    p = np.exp(-d)
    mean = (p * d).sum(1, keepdims=True) / p.sum(1, keepdims=True)
    return (3.01 + 2 + 1.23 * mean + adds(E) + 1) * U32


def exact_weights(l, e, renorm):
    """fp64 [T, k] of the chosen e, and the softmax [T, E]."""
    p = np.exp(l.astype(np.float64) - l.max(1, keepdims=True))
    top = np.take_along_axis(p, e, 1)
    return top / (top if renorm else p).sum(1, keepdims=True), p / p.sum(1, keepdims=True)


@pytest.mark.parametrize("T,E,k", GATES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [False, True])
def test_gate_far_below_the_peak(lp, T, E, k, dtype, renorm):
    lv = far_logits(T, E, k, dtype, E + k)
    l = torch.from_numpy(lv).cuda().to(dtype)
    assert np.array_equal(l.float().cpu().numpy(), lv)
    w, e = lp.lp_moe_gate(l, k, renorm=renorm)
    eh = e.cpu().numpy().astype(np.int64)
    assert np.array_equal(eh, np.argsort(-lv, 1, kind="stable")[:, :k])
    want, p = exact_weights(lv, eh, renorm)
    wh = w.cpu().numpy().astype(np.float64)
    assert (np.abs(wh - want) <= weights_bound(lv, k, E, renorm) * want).all(), (np.abs(wh / want - 1) / U32).max()

    # The gradient, from the weights as they are: sum w g in fp32 (a product's rounding, at most 3 sums a lane and 6 over
    # the lanes: 10 U32), then w (g - that) by two roundings; or p times it, p = e^d / sum by its own exponentials (those
    # of bf16 logits without the residual), a quotient and a product, and w g added to it.
    g = np.random.default_rng(k).standard_normal((T, k)).astype(np.float32)
    got = lp.lp_moe_gate_bwd(torch.from_numpy(g).cuda(), l, w, e, renorm=renorm).float().cpu().numpy().astype(np.float64)
    g = g.astype(np.float64)
    inner, size = (wh * g).sum(1, keepdims=True), (wh * np.abs(g)).sum(1, keepdims=True)
    ref, tol = np.zeros((T, E)), np.zeros((T, E))
    if renorm:
        np.put_along_axis(ref, eh, wh * (g - inner), 1)
        np.put_along_axis(tol, eh, wh * (10 * size + 2.01 * (np.abs(g) + size)) * U32, 1)
    else:
        own = np.zeros((T, E))
        np.put_along_axis(own, eh, wh * g, 1)
        d = np.abs(lv.astype(np.float64) - lv.max(1, keepdims=True))
        one = 3.01 if dtype == torch.float32 else 2 + 1.23 * d
        mean = (p * one).sum(1, keepdims=True) if dtype == torch.bfloat16 else 3.01
        ref = own - p * inner
        tol = (p * size * (one + mean + adds(E) + 10 + 2) + np.abs(own) + np.abs(ref)) * U32 * 1.01
    tol += np.abs(ref) * (U16 if dtype == torch.bfloat16 else 0)
    assert (np.abs(got - ref) <= tol).all(), (np.abs(got - ref) / np.maximum(tol, 1e-300)).max()


# ---------------------------------------------------------------- 4-bit forward

# (M, N, K, groups; 0: dense) that go to the 256 x 256 tiles.
LARGE_TILES = [(1348, 8832, 96, 0), (3100, 6000, 32, 2)]


def rows_and_weight(lp, fmt, M, N, K, G, seed):
    """x, a weight over `G` groups (0: one, dense) and its bf16 values in fp64."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    run, n = 32 if fmt == "mxfp4" else 16, max(G, 1)
    codes = torch.randint(0, 256, (n, N, K // 2), generator=g, dtype=torch.uint8, device="cuda")
    scales = torch.randint(*((118, 126) if fmt == "mxfp4" else (0x20, 0x40)), (n, N, K // run), generator=g, dtype=torch.uint8, device="cuda")
    w = lp.QTensor(fmt, codes, scales, torch.tensor([0.03], device="cuda") if fmt == "nvfp4" else None, shape=(n, N, K))
    return torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_(generator=g), w


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K,G", LARGE_TILES)
@pytest.mark.parametrize("raw", [False, True])
def test_large_tiles_on_another_stream(lp, busy, fmt, M, N, K, G, raw):  # noqa: F811
    """The bits of the current stream, whose late writes to freed memory miss the result; the result is that stream's."""
    x, w = rows_and_weight(lp, fmt, M, N, K, G, M)
    off = torch.tensor([M // 3, M - 7], dtype=torch.int32, device="cuda")

    def call(stream):
        return lp.lp_grouped_fwd_w4(x, w, off, stream=stream) if G else lp.lp_linear_fwd_w4(x, w, stream=stream)
    n = M - 7 if G else M
    want = call(None)[:n].clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    mine = [torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    busy()
    for t in mine:
        t.fill_(7)
    del mine, t
    got = call(s.cuda_stream if raw else s)
    s.synchronize()
    assert segment_stream(got.data_ptr()) == s.cuda_stream
    torch.cuda.synchronize()
    assert torch.equal(got[:n], want)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K,G", LARGE_TILES)
def test_captured_large_tiles(lp, fmt, M, N, K, G):
    x, w = rows_and_weight(lp, fmt, M, N, K, G, M)
    off = torch.tensor([M // 3, M - 7], dtype=torch.int32, device="cuda")
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")

    def call(y):
        return lp.lp_grouped_fwd_w4(x, w, off, y=y) if G else lp.lp_linear_fwd_w4(x, w, y=y)
    call(torch.empty_like(y))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(y)
    for k in range(3):
        x.copy_(torch.roll(x, 1, 0))
        off.copy_(torch.tensor([M // (2 + k), M - 7], dtype=torch.int32))
        graph.replay()
        want = call(torch.full_like(y, 7.0))
        torch.cuda.synchronize()
        assert torch.equal(y, want), k


def close(y, x, w):
    """y against x w^T in fp64, w the bf16 values that the kernel multiplies: exact products, K sums in fp32 in any order (a
    step each, should the matrix core cut off rather than round) and one rounding to bf16."""
    want, size = x.double() @ w.double().T, x.double().abs() @ w.double().abs().T
    off = (y.double() - want).abs()
    assert (off <= U16 * want.abs() + x.shape[1] * 2 * U32 * size).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_w4_weights_past_2_to_32_bytes(lp, fmt):
    """Every group's rows, those of the last groups past 2^32 bytes of codes."""
    G, N, K, M = 40, 16400, 14336, 57
    x, q = rows_and_weight(lp, fmt, M, N, K, G, 5)
    off = torch.zeros(G, dtype=torch.int32, device="cuda")
    off[1:20], off[20:G - 1], off[G - 1] = 3, 20, M
    y = lp.lp_grouped_fwd_w4(x, q, off)
    for e, r in ((1, slice(0, 3)), (20, slice(3, 20)), (G - 1, slice(20, M))):
        one = lp.QTensor(fmt, q.codes[e:e + 1], q.scales[e:e + 1], q.tensor_scale, shape=(1, N, K))
        close(y[r], x[r], lp.lp_dequant(one)[0])
    torch.cuda.empty_cache()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K,G", LARGE_TILES)
def test_large_tiles_against_the_decoded_weight(lp, fmt, M, N, K, G):
    x, w = rows_and_weight(lp, fmt, M, N, K, G, N)
    if not G:
        close(lp.lp_linear_fwd_w4(x, w), x, lp.lp_dequant(w)[0])
        return
    off = torch.tensor([M // 3, M], dtype=torch.int32, device="cuda")
    y, dec = lp.lp_grouped_fwd_w4(x, w, off), lp.lp_dequant(w)
    close(y[:M // 3], x[:M // 3], dec[0])
    close(y[M // 3:], x[M // 3:], dec[1])


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("T,E,k,width,hidden", [(1, 8, 2, 256, 512), (9, 16, 4, 288, 160), (200, 8, 3, 256, 544)])
def test_served_layer_within_its_roundings(lp, fmt, T, E, k, width, hidden):
    """fp64 with the bf16 values that both formats' weights stand for.  h, y and the result are rounded to bf16, half a step
    each, times |W| for h; the sums in fp32 are off by a step for each of their terms at the most.  The gate's weights: 17
    half steps (weights_bound), and 12 more in the exponential and in the sum for rounded differences of logits within 12 of
    one another."""
    gen = torch.Generator(device="cuda").manual_seed(300 + T)
    layer = Weights(lp, fmt, E, k, width, hidden, gen)
    x = torch.randn(T, width, generator=gen, device="cuda").bfloat16()
    out = f64(layer.forward(x))
    logits = f64(x.float() @ layer.router.T)
    assert np.ptp(logits, axis=1).max() < 12
    w, chosen = O.gate(logits, k, True)
    xv, (W1, W2) = f64(x), layer.values
    for t in range(T):
        want, bound = np.zeros(width), np.zeros(width)
        for j, e in enumerate(chosen[t]):
            h = W1[e] @ xv[t]
            bh = width * 2 * U32 * np.abs(W1[e]) @ np.abs(xv[t])
            bh += U16 * (np.abs(h) + bh)
            y = W2[e] @ np.maximum(h, 0)
            b = np.abs(W2[e]) @ bh + hidden * 2 * U32 * np.abs(W2[e]) @ (np.abs(h) + bh)
            b += U16 * (np.abs(y) + b)
            want += w[t, j] * y
            bound += w[t, j] * b + (41 + 2 * k) * U32 * np.abs(w[t, j] * y)
        bound += U16 * (np.abs(want) + bound)
        assert (np.abs(out[t] - want) <= bound).all(), (t, (np.abs(out[t] - want) / bound).max())
