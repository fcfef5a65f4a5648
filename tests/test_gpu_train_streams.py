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
