"""The ends of the ranges that the block-scaled FP8 training calls admit, and
the rules between their kernels there (GPU)."""
import numpy as np
import pytest
import torch

from gpu_util import assert_bits_equal, bits_host
from oracle import train as O

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [2 ** 31 - 128, 2 ** 31 - 112, 2 ** 31 - 16])
def test_quantizer_along_the_longest_rows(lp, cols):
    """One row of almost 2^31 columns: every run's scale is written, the last (partial) runs' right."""
    src = torch.zeros(1, cols, dtype=torch.bfloat16, device="cuda")
    src[0, :300] = torch.randn(300, device="cuda")
    src[0, -300:] = torch.randn(300, device="cuda")
    runs = -(-cols // 128)
    codes = torch.full((1, cols), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((runs,), -1.0, device="cuda")
    assert lp.lib.lp_r128_quant(src.data_ptr(), 1, 1, cols, -1, None, 0, codes.data_ptr(), scales.data_ptr(), lp._stream(None)) == 0
    assert (scales > 0).all()
    for at in (slice(0, 512), slice(cols // 128 * 128 - 512, cols)):
        want_c, want_s = O.quant_cols(bits_host(src[:, at]))
        assert_bits_equal(codes[:, at].cpu().numpy(), want_c, "codes")
        got = scales[at.start // 128:at.start // 128 + len(want_s)].cpu().numpy()
        assert_bits_equal(got.view(np.uint32), want_s[:, 0].view(np.uint32), "scales")
