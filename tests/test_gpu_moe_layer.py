"""The calls of lp_moe.h run together as a mixture-of-experts layer does: trained in
block-scaled FP8, served from 4-bit weights, captured into graphs, on other streams
(GPU)."""
import os
import sys

import numpy as np
import pytest
import torch

from oracle import moe as O
from oracle import train as OT
from oracle.formats import bf16_bits_to_f64, dequant
from test_gpu_train_streams import busy, segment_stream  # noqa: F401

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

U16, U32, U8 = 2.0 ** -8, 2.0 ** -24, 2.0 ** -4      # half a step of bf16, fp32, E4M3


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def masked(T, E, gen):
    """Some tokens barred from most experts, one from all: fewer than topk pairs."""
    mask = torch.zeros(T, E, device="cuda")
    mask[torch.rand(T, E, generator=gen, device="cuda") < 0.3] = -torch.inf
    mask[T // 2] = -torch.inf
    mask[0, 1:] = -torch.inf
    return mask


def norm(a, axis=None):
    return np.linalg.norm(a, axis=axis)


def spectral(a):
    return np.linalg.norm(a, 2) if a.size else 0.0


class Reference:
    """The layer in fp64 with the weights that the FP8 codes stand for, the experts that were chosen, the ReLU's side as the
    GPU took it and, for the gate's gradient (a difference of near products, beside which e8 below is large), its rows y;
    and for every result a bound of what E4M3 and bf16 roundings can make of it, in the Euclidean norm:

      a run of v, scale s = amax / 448: each code is off by at most half a step, 2^-4 of the value, or below the normal
      codes 2^-10 s <= 2^-18 amax; so the row by at most (2^-4 + sqrt(128 n) 2^-18) of its norm, n its runs: e8 below
      (along the tokens the same by column);  W v: at most |W| (its largest singular value) times that, plus half a step
      of bf16 of the result;  fp32 sums stay below 2^-20 of the products' magnitudes, for which e8 is rounded up.
    """

    def __init__(self, layer, s, x, grad):
        self.E, self.k = layer.experts, layer.topk
        T, K = x.shape
        self.x, self.g = f64(x), f64(grad)
        self.R = f64(layer.router.copy)
        W1, W2 = (np.stack([OT.values_blocks(c, v) for c, v in zip(m.weight.codes.cpu().numpy(), m.weight.scales.cpu().numpy())])
                  for m in (layer.up, layer.down))
        e8 = U8 + np.sqrt(max(W1.shape[1], K)) * 2.0 ** -18 + 2.0 ** -10
        u16 = U16 + 2.0 ** -12
        logits = f64(s["logits"])
        w, chosen = O.gate(logits, self.k, True)
        assert np.array_equal(chosen, s["chosen"].cpu().numpy())
        offsets, rows, order = O.sort(chosen, self.E)
        for name, v in (("offsets", offsets), ("rows", rows)):
            assert np.array_equal(s[name].cpu().numpy(), v), name
        n = order.size
        assert np.array_equal(s["order"].cpu().numpy()[:n], order)
        ends = [0, *offsets]
        h_gpu, a_gpu, y_gpu = (f64(s[v])[:n] for v in ("h", "a", "y"))
        side = h_gpu > 0
        tok, wr = order // self.k, w.reshape(-1)[order]
        xs, gy = self.x[tok], wr[:, None] * self.g[tok]
        h, y, ga, gx = np.zeros_like(h_gpu), np.zeros_like(y_gpu), np.zeros_like(h_gpu), np.zeros_like(xs)
        self.gW1, self.gW2 = np.zeros_like(W1), np.zeros_like(W2)
        self.bW1, self.bW2 = np.zeros(self.E), np.zeros(self.E)
        by, bgx = np.zeros(n), np.zeros(n)
        for e in range(self.E):
            r = slice(ends[e], ends[e + 1])
            s1, s2 = spectral(W1[e]), spectral(W2[e])
            h[r] = xs[r] @ W1[e].T
            a = side[r] * h[r]
            y[r] = a @ W2[e].T
            bh = s1 * e8 * norm(xs[r], 1) + u16 * norm(h_gpu[r], 1)
            by[r] = s2 * (bh + e8 * norm(a_gpu[r], 1)) + u16 * norm(y_gpu[r], 1)
            # gy is rounded to bf16 before its codes, and w by the gate's own error, below 2^-16
            bgy = (e8 + u16) * norm(gy[r], 1)
            ga[r] = gy[r] @ W2[e]
            bga = s2 * bgy + u16 * (norm(ga[r], 1) + s2 * bgy)
            gh = side[r] * ga[r]
            gx[r] = gh @ W1[e]
            bgh = bga + e8 * (norm(gh, 1) + bga)
            bgx[r] = s1 * bgh + u16 * (norm(gx[r], 1) + s1 * bgh)
            self.gW1[e], self.gW2[e] = gh.T @ xs[r], gy[r].T @ a
            # |A'^T B' - A^T B| <= |A' - A| |B'| + |A| |B' - B|, in the Frobenius and the spectral norm
            for out, bound, A, dA, B, dB in ((self.gW2, self.bW2, gy[r], norm(bgy), a, norm(bh) + e8 * norm(a_gpu[r])),
                                             (self.gW1, self.bW1, gh, norm(bga) + e8 * (norm(gh) + norm(bga)), xs[r],
                                              e8 * norm(xs[r]))):
                bound[e] = dA * (spectral(B) + dB) + spectral(A) * dB
                bound[e] += u16 * (norm(out[e]) + bound[e])
        self.out, self.bout = np.zeros((T, y.shape[1])), np.zeros(T)
        self.gx, self.bgx = np.zeros_like(self.x), np.zeros(T)
        gw, bgw = np.zeros((T, self.k)), np.zeros((T, self.k))
        for t in range(T):
            for j, r in enumerate(rows[t]):
                if r >= 0:
                    self.out[t] += w[t, j] * y[r]
                    self.bout[t] += w[t, j] * by[r]
                    self.gx[t] += gx[r]
                    self.bgx[t] += bgx[r]
                    gw[t, j], bgw[t, j] = self.g[t] @ y_gpu[r], 2.0 ** -16 * norm(self.g[t]) * norm(y_gpu[r])
        self.bout += u16 * (norm(self.out, 1) + self.bout)
        self.bgx += u16 * (norm(self.gx, 1) + self.bgx)
        gl = O.gate_bwd(gw, logits, chosen, True)
        # |dl_i| <= w_i (|dg_i| + sum w |dg|)
        bgl = np.zeros_like(gl)
        for t in range(T):
            mean = (w[t] * bgw[t]).sum()
            for j, e in enumerate(chosen[t]):
                if e >= 0:
                    bgl[t, e] = w[t, j] * (bgw[t, j] + mean) + 2.0 ** -14 * np.abs(gw[t]).max()
        self.gx += gl @ self.R
        self.bgx += norm(bgl, 1) * spectral(self.R) + 2.0 ** -18 * norm(gl, 1) * spectral(self.R)
        self.gR = gl.T @ self.x
        self.bR = (1 + u16) * norm(bgl) * spectral(self.x) + u16 * norm(self.gR) + 2.0 ** -15 * norm(gl) * norm(self.x)


@pytest.mark.parametrize("T,E,k,width,hidden,barred", [(300, 4, 2, 256, 384, False), (257, 8, 3, 128, 272, True), (5, 6, 2, 144, 128, False),
                                                       (40, 3, 3, 256, 128, True)])
def test_layer_against_its_formula(lp, T, E, k, width, hidden, barred):
    """Output and every gradient of a whole layer.  Its own output as the incoming gradient (of |out|^2 / 2), so that the
    weights' gradients are sums of one sign."""
    import route_experts as X
    gen = torch.Generator(device="cuda").manual_seed(T)
    layer = X.RoutedExperts(E, k, width, hidden, gen)
    x = torch.randn(T, width, generator=gen, device="cuda").bfloat16()
    out, s = layer.forward(x, masked(T, E, gen) if barred else None)
    grad_x = layer.backward(out, s)
    ref = Reference(layer, s, x, out)
    d = norm(f64(out) - ref.out, 1)
    assert (d <= ref.bout).all(), (d / np.maximum(ref.bout, 1e-300)).max()
    d = norm(f64(grad_x) - ref.gx, 1)
    assert (d <= ref.bgx).all(), (d / np.maximum(ref.bgx, 1e-300)).max()
    for name, got, want, bound in (("up", layer.up.grad, ref.gW1, ref.bW1), ("down", layer.down.grad, ref.gW2, ref.bW2)):
        d = norm((f64(got) - want).reshape(E, -1), 1)
        assert (d <= bound).all(), (name, d / np.maximum(bound, 1e-300))
    assert norm(f64(layer.router.grad) - ref.gR) <= ref.bR
    if barred:                                           # the token that no expert has
        assert not out[T // 2].any() and not grad_x[T // 2].any()


def test_example_runs(lp):
    import route_experts as X
    layer, x, losses = X.train(steps=4)
    assert len(losses) == 5 and np.isfinite(losses).all()
    for m in layer.layers():
        assert torch.isfinite(m.grad.float()).all() and m.grad.any()
    served = X.Served(layer).forward(x[:7])
    assert served.shape == (7, 256) and torch.isfinite(served.float()).all()


# ---------------------------------------------------------------- served

class Weights:
    """A served layer of given 4-bit weights; forward as the example's."""

    def __init__(self, lp, fmt, E, k, width, hidden, gen):
        import route_experts as X
        self.experts, self.topk = E, k
        self.router = torch.randn(E, width, generator=gen, device="cuda") * width ** -0.5

        def weight(N, K):
            codes = torch.randint(0, 256, (E, N, K // 2), generator=gen, dtype=torch.uint8, device="cuda")
            if fmt == "mxfp4":
                scales = torch.randint(118, 122, (E, N, K // 32), generator=gen, dtype=torch.uint8, device="cuda")
                return lp.QTensor(fmt, codes, scales, shape=(E, N, K))
            scales = torch.randint(0x20, 0x38, (E, N, K // 16), generator=gen, dtype=torch.uint8, device="cuda")
            return lp.QTensor(fmt, codes, scales, torch.tensor([0.03], device="cuda"), shape=(E, N, K))
        self.up, self.down = weight(hidden, width), weight(width, hidden)
        self.values = [bf16_bits_to_f64(dequant(fmt, q.codes.cpu().numpy(), q.scales.cpu().numpy(),
                                                None if q.tensor_scale is None else 0.03, -1)) for q in (self.up, self.down)]
        self.forward = lambda x, mask=None: X.Served.forward(self, x, mask)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("T,E,k,width,hidden,barred", [(1, 8, 2, 256, 512, False), (1, 4, 4, 128, 96, True), (9, 16, 4, 288, 160, True),
                                                       (33, 4, 2, 512, 1024, False), (200, 8, 3, 256, 544, True)])
def test_served_layer_against_its_formula(lp, fmt, T, E, k, width, hidden, barred):
    """fp64 with the values of the 4-bit weights.  Rounded to bf16 are nvfp4's values (by a step of 2^-8 at the most, in the
    oracle's dequant, not in the products), h, y and the result: half a step each, times |W| for h."""
    gen = torch.Generator(device="cuda").manual_seed(100 + T)
    layer = Weights(lp, fmt, E, k, width, hidden, gen)
    x = torch.randn(T, width, generator=gen, device="cuda").bfloat16()
    mask = None
    if barred and T > 1:
        mask = masked(T, E, gen)
    elif barred:
        mask = torch.zeros(T, E, device="cuda")
        mask[:, 1:3] = -torch.inf
    out = f64(layer.forward(x, mask))
    logits = x.float() @ layer.router.T
    w, chosen = O.gate(f64(logits if mask is None else logits + mask), k, True)
    W1, W2 = layer.values
    xv, uw = f64(x), (U16 if fmt == "nvfp4" else 0.0) + 2.0 ** -14
    for t in range(T):
        want, bound = np.zeros(width), np.zeros(width)
        for j, e in enumerate(chosen[t]):
            if e < 0:
                continue
            h = W1[e] @ xv[t]
            bh = uw * np.abs(W1[e]) @ np.abs(xv[t])
            bh += U16 * (np.abs(h) + bh)
            y = W2[e] @ np.maximum(h, 0)
            b = np.abs(W2[e]) @ bh + uw * np.abs(W2[e]) @ (np.abs(h) + bh)
            b += U16 * (np.abs(y) + b)
            want += w[t, j] * y
            bound += w[t, j] * b + 2.0 ** -16 * np.abs(y)
        bound += U16 * (np.abs(want) + bound)
        assert (np.abs(out[t] - want) <= bound + 1e-30).all(), (t, (np.abs(out[t] - want) / (bound + 1e-30)).max())


# ---------------------------------------------------------------- captured

def test_captured_layer(lp):
    """Replays on new inputs give the eager step's bits, with eager steps between."""
    import route_experts as X
    gen = torch.Generator(device="cuda").manual_seed(3)
    layer = X.RoutedExperts(8, 2, 256, 128, gen)
    layer.router.forward = lambda x: logits              # (library products stay out of the graph)
    layer.router.backward = lambda x, g: g
    x, logits = torch.empty(150, 256, dtype=torch.bfloat16, device="cuda"), torch.empty(150, 8, device="cuda")
    x_in = [torch.randn(150, 256, generator=gen, device="cuda").bfloat16() for _ in range(4)]
    l_in = [torch.randn(150, 8, generator=gen, device="cuda") for _ in range(4)]
    lp_w4 = [lp.lp_mx_quant(m.copy, -1, "mxfp4") for m in (layer.up, layer.down)]

    def step():
        out, s = layer.forward(x)
        y = lp.lp_grouped_fwd_w4(lp.lp_moe_gather(x, s["rows"]), lp_w4[0], s["offsets"])
        y = lp.lp_moe_combine(lp.lp_grouped_fwd_w4(y, lp_w4[1], s["offsets"]), s["rows"], s["weights"])
        _, gw = lp.lp_moe_combine_bwd(out, s["y"], s["rows"], s["weights"], need_dy=False)
        q, _ = lp.lp_moe_gather_quant(out, s["order"], s["offsets"], 2, weights=s["weights"])
        gy, _ = lp.lp_moe_combine_bwd(out, None, s["rows"], s["weights"], need_dw=False)
        gl = lp.lp_moe_gate_bwd(gw, logits, s["weights"], s["chosen"])
        return [out, y, gw, q.codes, q.scales, gy, gl, s["chosen"], s["rows"]]
    want = []
    for a, b in zip(x_in, l_in):
        x.copy_(a), logits.copy_(b)
        want.append([t.clone() for t in step()])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for k in (0, 1, 2, 3, 1):
        x.copy_(x_in[k]), logits.copy_(l_in[k])
        graph.replay()
        held = [t.clone() for t in got]
        eager = step()
        torch.cuda.synchronize()
        for i, (a, b, c) in enumerate(zip(held, eager, want[k])):
            assert torch.equal(a, c) and torch.equal(b, c), (k, i)


def test_captured_sorts_have_workspaces_of_their_own(lp):
    """Two graphs of sorts beyond one launch's pairs, replayed at once on two streams."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    inputs = [[torch.randint(-1, 40, (n, 3), generator=gen, device="cuda").int() for _ in range(3)] for n in (30001, 50000)]
    at = [torch.empty_like(v[0]) for v in inputs]
    graphs, outs = [], []
    for a, v in zip(at, inputs):
        a.copy_(v[0])
        lp.lp_moe_sort(a, 40)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(lp.lp_moe_sort(a, 40))
    streams = [torch.cuda.Stream() for _ in graphs]
    for k in (0, 1, 2, 0):
        for a, v in zip(at, inputs):
            a.copy_(v[k])
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for v, (off, rows, order) in zip(inputs, outs):
            eoff, erows, eorder = lp.lp_moe_sort(v[k], 40)
            n = int(eoff[-1])
            flat = v[k].reshape(-1)
            live = (flat >= 0).nonzero()[:, 0]
            assert torch.equal(eorder[:n].long(), live[flat[live].sort(stable=True).indices])
            assert torch.equal(off, eoff) and torch.equal(rows, erows) and torch.equal(order[:n], eorder[:n])


@pytest.mark.parametrize("n", [7, 2000, 5000, 65536, 70000])
def test_captured_sort_over_the_most_experts(lp, n):
    """1024 experts: the counters take more LDS than 64 KB."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    e_in = [torch.randint(-1, 1024, (n, 1), generator=gen, device="cuda").int() for _ in range(3)]
    e = e_in[0].clone()
    lp.lp_moe_sort(e, 1024)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        off, rows, order = lp.lp_moe_sort(e, 1024)
    for v in e_in + e_in[:1]:
        e.copy_(v)
        graph.replay()
        want = lp.lp_moe_sort(v, 1024)
        torch.cuda.synchronize()
        live = int(want[0][-1])
        assert torch.equal(off, want[0]) and torch.equal(rows, want[1]) and torch.equal(order[:live], want[2][:live])


# ---------------------------------------------------------------- other streams

NAMES = ["lp_moe_gate", "lp_moe_gate_bwd", "lp_moe_sort", "lp_moe_gather", "lp_moe_gather_quant", "lp_moe_combine",
         "lp_moe_combine_bwd", "lp_linear_fwd_w4", "lp_grouped_fwd_w4"]


def calls_of(lp):
    """name -> call(stream), every call with everything left to it to allocate, and the inputs."""
    gen = torch.Generator(device="cuda").manual_seed(6)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")
    x, grad, y, logits, g = randn(50, 144).bfloat16(), randn(50, 144).bfloat16(), randn(100, 144).bfloat16(), randn(50, 6), randn(50, 2)
    w, e = lp.lp_moe_gate(logits, 2)
    off, rows, order = lp.lp_moe_sort(e, 6)
    many = torch.randint(0, 6, (40000, 2), generator=gen, device="cuda").int()       # (a workspace)
    wq = lp.lp_mx_quant(randn(6, 96, 288).bfloat16(), -1, "mxfp4")
    w1 = lp.QTensor("mxfp4", wq.codes[:1].contiguous(), wq.scales[:1].contiguous(), shape=(1, 96, 288))
    xr = randn(100, 288).bfloat16()
    keep = dict(locals())
    calls = {
        "gate": lambda s: lp.lp_moe_gate(logits, 2, stream=s),
        "gate_bwd": lambda s: [lp.lp_moe_gate_bwd(g, logits, w, e, stream=s)],
        "sort": lambda s: lp.lp_moe_sort(e, 6, stream=s),
        "sort many": lambda s: lp.lp_moe_sort(many, 6, stream=s),
        "gather": lambda s: [lp.lp_moe_gather(x, rows, stream=s)],
        "gather_quant": lambda s: [t for q in lp.lp_moe_gather_quant(x, order, off, 2, stream=s) for t in (q.codes, q.scales)],
        "combine": lambda s: [lp.lp_moe_combine(y, rows, w, stream=s)],
        "combine_bwd": lambda s: lp.lp_moe_combine_bwd(grad, y, rows, w, stream=s),
        "linear_w4": lambda s: [lp.lp_linear_fwd_w4(xr[:3], w1, stream=s)],
        "linear_w4 tile": lambda s: [lp.lp_linear_fwd_w4(xr, w1, stream=s)],
        "grouped_w4": lambda s: [lp.lp_grouped_fwd_w4(xr, wq, off, stream=s)],
    }
    return calls, keep


@pytest.mark.parametrize("raw", [False, True])
def test_what_a_call_allocates_is_memory_of_its_stream(lp, monkeypatch, raw):
    """Results and hidden scratch: no address that a C call is given, but the inputs', is the current stream's memory."""
    calls, keep = calls_of(lp)
    inputs = set()
    for v in keep.values():
        for t in [v.codes, v.scales] if isinstance(v, lp.QTensor) else [v]:
            if isinstance(t, torch.Tensor):
                inputs.add(t.data_ptr())
    seen = []
    for name in NAMES:
        def wrapped(*args, _f=getattr(lp.lib, name)):
            seen.extend(a for a in args if isinstance(a, int) and a not in inputs)
            return _f(*args)
        monkeypatch.setattr(lp.lib, name, wrapped)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for name, call in calls.items():
        seen.clear()
        out = call(s.cuda_stream if raw else s)
        assert {segment_stream(p) for p in seen if segment_stream(p) is not None} == {s.cuda_stream}, name
        assert {segment_stream(t.data_ptr()) for t in out} == {s.cuda_stream}, name
    torch.cuda.synchronize()


def written(name, out):
    """What of a call's results it writes."""
    if name.startswith("gather_quant"):                  # (whole runs only where an expert has rows)
        return out[:3]
    return out


def test_results_on_another_stream(lp, busy):  # noqa: F811
    """The same bits as on the current one, whose late writes to freed memory hit none of them."""
    calls, keep = calls_of(lp)
    want = {name: [t.clone() for t in written(name, call(None))] for name, call in calls.items()}
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for name, call in calls.items():
        mine = [torch.empty(t.nbytes, dtype=torch.uint8, device="cuda") for t in want[name] for _ in range(2)]
        busy()
        for t in mine:
            t.fill_(0x55)
        del mine, t
        got = written(name, call(s))
        s.synchronize()
        torch.cuda.synchronize()
        for a, b in zip(want[name], got):
            assert torch.equal(a, b), name
