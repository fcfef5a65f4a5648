"""What the bounds of test_gpu_moe_bounds.py tell apart (CPU only)."""
import numpy as np
import pytest
import torch

import test_gpu_moe_bounds as B

LOG2E, LOW = np.float32(float.fromhex("0x1.715476p+0")), np.float32(float.fromhex("0x1.4ae0bep-26"))


def power(d, residual):
    """e^d of fp32 d by a rounded t = d log2 e, with or without what the rounding left; rounded to fp32."""
    t = (d * LOG2E).astype(np.float32)
    left = d.astype(np.float64) * (float(LOG2E) + float(LOW)) - t
    return (np.exp2(t.astype(np.float64)) * (1 + left * np.log(2) * residual)).astype(np.float32).astype(np.float64)


@pytest.mark.parametrize("T,E,k", B.GATES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [False, True])
def test_a_gate_without_the_exponentials_residual_is_seen(T, E, k, dtype, renorm):
    l = B.far_logits(T, E, k, dtype, E + k)
    e = np.argsort(-l, 1, kind="stable")[:, :k]
    d = np.take_along_axis(l, e, 1) - l.max(1, keepdims=True)
    want, p = B.exact_weights(l, e, renorm)
    total = np.exp(l.astype(np.float64) - l.max(1, keepdims=True))
    total = (np.take_along_axis(total, e, 1) if renorm else total).sum(1, keepdims=True)
    bound = B.weights_bound(l, k, E, renorm)
    off = [np.abs(power(d, r) / total / want - 1) / bound for r in (1, 0)]
    assert off[0].max() < 0.2 and off[1].max() > 1.2, (off[0].max(), off[1].max())
