"""Calls on a stream other than the current one (GPU): what they allocate, and
what has to stay until that stream is done with it."""
import numpy as np
import pytest
import torch

from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def busy():
    """busy(): keeps the current stream at work for some 50 ms."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda._sleep(1000)
    cycles = 1 << 20
    start.record()
    torch.cuda._sleep(cycles)
    end.record()
    torch.cuda.synchronize()
    n = int(cycles * 50 / max(start.elapsed_time(end), 1e-3))
    return lambda: torch.cuda._sleep(n)


def test_raw_default_stream_is_the_default_stream(lp):
    s = torch.cuda.Stream()
    assert lp._torch_stream(0) == torch.cuda.default_stream()
    assert lp._torch_stream(s) is s and lp._torch_stream(s.cuda_stream).cuda_stream == s.cuda_stream


@pytest.mark.parametrize("raw", [True, False])
def test_adamw_table_of_another_stream_outlives_a_step_on_the_default_one(lp, busy, raw):
    """The plan is made on a side stream, the step waits on the default stream while set_grads replaces the table and the
    side stream writes over whatever memory it is given next."""
    n = 5000
    p0, g1, g2 = np.random.default_rng(17).standard_normal((3, n), dtype=np.float32)

    def run(side):
        p, m, v = dev(p0), torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
        a, b = dev(g1), dev(g2)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            plan = lp.AdamWPlan([p], [a], [m], [v])
        torch.cuda.synchronize()
        busy()
        lp.lp_adamw(plan, lr=0.1, step=1, stream=0 if raw else None)
        with torch.cuda.stream(side):
            plan.set_grads([b])
            junk = [torch.full((64,), -1, dtype=torch.int64, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        del junk
        return torch.stack([p, m, v])
    want = run(torch.cuda.default_stream())
    assert torch.equal(run(torch.cuda.Stream()), want)


def test_a_captured_adamw_step_outlives_set_grads(lp):
    """Replays after set_grads, with memory given out in between, step with the gradients of the capture."""
    n = 5000
    p0, g1, g2 = np.random.default_rng(18).standard_normal((3, n), dtype=np.float32)

    def fresh(g):
        t = [dev(p0), torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")]
        return t, lp.AdamWPlan(t[:1], [dev(g)], t[1:2], t[2:])
    want_t, want_plan = fresh(g1)
    t, plan = fresh(g1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lp.lp_adamw(plan, lr=0.1, step=1)
    for _ in range(3):
        plan.set_grads([dev(g2)])
        junk = [torch.full((k,), -1, dtype=torch.int64, device="cuda") for k in (16, 64, 2500) for _ in range(4)]
        graph.replay()
        torch.cuda.synchronize()
        del junk
        lp.lp_adamw(want_plan, lr=0.1, step=1)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(t, want_t))
    lp.lp_adamw(plan, lr=0.1, step=2)                    # an eager step takes the new gradients
    want_plan.set_grads([dev(g2)])
    lp.lp_adamw(want_plan, lr=0.1, step=2)
    assert all(torch.equal(a, b) for a, b in zip(t, want_t))


# ---------------------------------------------------------------- what a call allocates

def products(lp):
    """name -> (call(stream), input tensors): every call of the binding that allocates, with everything left to it."""
    torch.manual_seed(5)
    M, N, K, G = 40, 272, 400, 3

    def randn(*shape):
        return torch.randn(shape, device="cuda").bfloat16()
    x, g, w = randn(M, K), randn(M, N), randn(G, N, K)
    off = dev(np.array([10, 10, 40], np.int32))
    wq, w1 = lp.lp_b128_quant(w), lp.lp_b128_quant(w[0])
    (gc, gr), (gc1, gr1) = lp.lp_r128_quant_dual(g, off), lp.lp_r128_quant_dual(g)
    (xc, xr), xr1 = lp.lp_r128_quant_dual(x, off), lp.lp_r128_quant(x, -2)
    long_g, long_x = (lp.lp_r128_quant(randn(12000, 16), -2) for _ in range(2))     # split: a workspace
    sq = randn(96, 128)
    hist, scale = torch.ones(4, device="cuda"), torch.ones(1, device="cuda")
    rings = [hist.clone() for _ in range(4)]             # (the call writes its own)
    mx, t8 = lp.lp_mx_quant(sq, -1), lp.lp_tensor_quant(sq, "fp8t_e4m3", scale)
    b16 = lp.QTensor("bf16", g, shape=(1, M, N))
    wm = randn(2, 64, 64)
    gm, offm = lp.lp_mx_quant(randn(64, 64), -1), dev(np.array([30, 64], np.int32))
    keep = dict(locals())
    calls = {
        "dequant": lambda s: [lp.lp_dequant(gr1, stream=s)],
        "mx_quant": lambda s: parts(lp.lp_mx_quant(sq, -2, stream=s)),
        "mx_quant_dual": lambda s: parts(*lp.lp_mx_quant_dual(sq, stream=s)),
        "tensor_amax": lambda s: [lp.lp_tensor_amax(sq, stream=s)],
        "tensor_quant": lambda s: [lp.lp_tensor_quant(sq, "fp8t_e5m2", scale, stream=s).codes],
        "tensor_quant_delayed": lambda s: [lp.lp_tensor_quant_delayed(sq, "fp8t_e4m3", rings.pop(), 0, stream=s).codes],
        "scale_from_history": lambda s: [lp.lp_scale_from_history(hist, "fp8t_e4m3", stream=s)],
        "r128_quant": lambda s: parts(lp.lp_r128_quant(x, -1, stream=s)),
        "r128_quant rows": lambda s: parts(lp.lp_r128_quant(x, -2, stream=s)),
        "r128_quant_dual": lambda s: parts(*lp.lp_r128_quant_dual(x, stream=s)),
        "b128_quant": lambda s: parts(lp.lp_b128_quant(w, stream=s)),
        "linear_fwd": lambda s: [lp.lp_linear_fwd(xc, w1, stream=s)],
        "grouped_fwd": lambda s: [lp.lp_grouped_fwd(xc, wq, off, stream=s)],
        "linear_fwd_dyn": lambda s: [lp.lp_linear_fwd_dyn(x, w1, stream=s)],
        "linear_fwd_dyn fused": lambda s: [lp.lp_linear_fwd_dyn(x[:3], w1, stream=s)],
        "grouped_fwd_dyn": lambda s: [lp.lp_grouped_fwd_dyn(x, wq, off, stream=s)],
        "linear_bwd dX": lambda s: [lp.lp_linear_bwd(gc1, None, w1, need_dw=False, stream=s)[0]],
        "linear_bwd dW": lambda s: [lp.lp_linear_bwd(gr1, xr1, None, need_dx=False, stream=s)[1]],
        "linear_bwd dW split": lambda s: [lp.lp_linear_bwd(long_g, long_x, None, need_dx=False, stream=s)[1]],
        "linear_bwd bf16": lambda s: [lp.lp_linear_bwd(b16, None, w1, need_dw=False, stream=s)[0]],
        "linear_bwd_noalloc": lambda s: [lp.lp_linear_bwd_noalloc(b16, None, w1, need_dw=False, stream=s)[0]],
        "grouped_bwd dX": lambda s: [lp.lp_grouped_bwd(gc, None, wq, off, need_dw=False, stream=s)[0]],
        "grouped_bwd dW": lambda s: [lp.lp_grouped_bwd(gr, xr, None, off, need_dx=False, stream=s)[1]],
        "grouped_dx_deferred": lambda s: [lp.lp_grouped_dx_deferred(gm, wm, offm, fuse_rows=0, stream=s)],
    }
    return calls, keep


def parts(*tensors):
    return [t for q in tensors for t in (q.codes, q.scales)]


def segment_stream(ptr):
    """The stream whose memory an address lies in (None: no device memory of torch's)."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= ptr < seg["address"] + seg["total_size"]:
            return seg["stream"]
    return None


@pytest.mark.parametrize("raw", [False, True])
def test_what_a_call_allocates_is_memory_of_its_stream(lp, monkeypatch, raw):
    """Results and hidden scratch: no address that a C call is given, but the inputs', is the current stream's memory."""
    calls, keep = products(lp)
    inputs = set()
    for v in [*keep.values(), *keep["rings"]]:
        for t in parts(v) + [v.tensor_scale] if isinstance(v, lp.QTensor) else [v]:
            if isinstance(t, torch.Tensor):
                inputs.add(t.data_ptr())
    seen = []
    for name in [n for n in lp.header_functions() if n != "lp_status_string"] + [
            "lp_r128_quant", "lp_r128_quant_dual", "lp_b128_quant", "lp_linear_fwd_dyn", "lp_grouped_fwd_dyn"]:
        def wrapped(*args, _f=getattr(lp.lib, name)):
            seen.extend(a for a in args if isinstance(a, int) and a not in inputs)
            return _f(*args)
        monkeypatch.setattr(lp.lib, name, wrapped)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for name, call in calls.items():
        seen.clear()
        out = call(s.cuda_stream if raw else s)
        streams = {segment_stream(p) for p in seen if segment_stream(p) is not None}
        assert streams == {s.cuda_stream}, name
        assert {segment_stream(t.data_ptr()) for t in out} == {s.cuda_stream}, name
    torch.cuda.synchronize()


def test_results_are_not_overwritten_by_work_of_the_current_stream(lp, busy):
    """The current stream has a late write to memory that was then freed: no result of a call on another stream lies
    there.  And the other way round: a result freed while the current stream still has to read it is not given away."""
    calls, keep = products(lp)
    want = {name: [t.clone() for t in call(None)] for name, call in calls.items()}
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for name, call in calls.items():
        sizes = [t.nbytes for t in want[name]]
        mine = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
        busy()
        for t in mine:
            t.fill_(0x55)
        del mine, t
        got = call(s)
        s.synchronize()
        torch.cuda.synchronize()
        for a, b in zip(want[name], got):
            assert torch.equal(a, b), name
        busy()
        late = [t.clone() for t in got]                  # on the current stream, behind the wait
        sizes = [(t.shape, t.dtype) for t in got]
        del got, b
        with torch.cuda.stream(s):
            junk = [torch.zeros(shape, dtype=dtype, device="cuda") for shape, dtype in sizes]
        torch.cuda.synchronize()
        for a, b in zip(want[name], late):
            assert torch.equal(a, b), name
        del junk
