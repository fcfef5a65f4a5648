"""The ends of the ranges that the block-scaled FP8 training calls admit, and
the rules between their kernels there (GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from gpu_util import assert_bits_equal, bf16_dev, bits_host, dev
from oracle import train as O
from oracle.formats import E4M3_TABLE
from test_gpu_train import assert_product, bits, decoded, decoded_rows, weight

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


# rows x contraction: the most that is quantized inside the product (512 runs in all, with more than 64 KiB of LDS), and
# the least that is not
@pytest.mark.parametrize("M,K,fused", [(4, 16384, True), (3, 21760, True), (2, 32768, True), (1, 65536, True), (1, 65424, True),
                                       (4, 16400, False), (3, 21776, False), (1, 65552, False), (5, 16384, False)])
def test_forward_of_few_rows_over_the_longest_contractions(lp, M, K, fused):
    rng = np.random.default_rng(M + K)
    for N in (16, 144):
        w, wv = weight(lp, rng, 1, N, K)
        x = bf16_dev(bits(rng, (M, K)))
        xq = lp.lp_r128_quant(x, -1)
        assert_product(lp.lp_linear_fwd_dyn(x, w), decoded(xq), wv[0].T, f"y from bf16, {N} columns")
        assert_product(lp.lp_linear_fwd(xq, w), decoded(xq), wv[0].T, f"y, {N} columns")
        y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        wc = w.c()
        st = lp.lib.lp_linear_fwd_dyn(x.data_ptr(), M, ctypes.byref(wc), None, None, y.data_ptr(), lp._stream(None))
        assert st == (0 if fused else 1)                 # without scratch: LP_ERR_NULL unless it needs none
        if fused:
            assert_product(y, decoded(xq), wv[0].T, "y without scratch")


# either side of 64 groups (one wave's scan) and of 256 (the most that are ranked by size); grad_W on every tile size
@pytest.mark.parametrize("G,N,K", [(64, 272, 400), (65, 272, 400), (100, 272, 400), (200, 128, 128), (70, 16, 16), (256, 16, 32),
                                   (257, 16, 32)])
def test_grouped_products_of_many_groups(lp, G, N, K):
    rng = np.random.default_rng(G)
    sizes = [int(v) for v in rng.choice([0, 0, 1, 5, 128, 129, 300], G)]
    sizes[3], sizes[-1] = 0, 0
    M, ends = sum(sizes) + 7, np.cumsum(sizes).astype(np.int32)
    w, wv = weight(lp, rng, G, N, K)
    x, g, off = bf16_dev(bits(rng, (M, K))), bf16_dev(bits(rng, (M, N), 1e-3)), dev(ends)
    xq, (gc, gr), (_, xr) = lp.lp_r128_quant(x, -1), lp.lp_r128_quant_dual(g, off), lp.lp_r128_quant_dual(x, off)
    dw = torch.full((G, N, K), 3.0, dtype=torch.bfloat16, device="cuda")
    lp.lp_grouped_bwd(gr, xr, None, off, need_dx=False, grad_w=dw)
    dx, _ = lp.lp_grouped_bwd(gc, None, w, off, need_dw=False)
    y = lp.lp_grouped_fwd(xq, w, off)
    xv, gv, xrv, grv = decoded(xq), decoded(gc), decoded_rows(xr, ends), decoded_rows(gr, ends)
    for k, (a, b) in enumerate(O.groups(M, ends)):
        if a == b:
            assert not dw[k].any(), k
            continue
        assert_product(dw[k], grv[a:b].T, xrv[a:b], f"dW of group {k}")
        assert_product(dx[a:b], gv[a:b], wv[k], f"dX of group {k}")
        assert_product(y[a:b], xv[a:b], wv[k].T, f"y of group {k}")


@pytest.mark.parametrize("M,N,K", [(0, 272, 400), (5, 272, 0), (40, 272, 0), (300, 272, 0), (5, 0, 400), (300, 0, 400)])
def test_sizes_of_zero(lp, M, N, K):
    """No token: grad_W is zero; no input or output feature: y or grad_X is zero."""
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    x, g, w = torch.randn(M, K, **bf16), torch.randn(M, N, **bf16), lp.lp_b128_quant(torch.randn(N, K, **bf16))
    (xc, xr), (gc, gr) = lp.lp_r128_quant_dual(x), lp.lp_r128_quant_dual(g)
    outs = [torch.full(s, 3.0, **bf16) for s in ((M, N), (M, N), (M, K), (N, K))]
    lp.lp_linear_fwd(xc, w, y=outs[0])
    lp.lp_linear_fwd_dyn(x, w, y=outs[1])
    lp.lp_linear_bwd(gc, None, w, need_dw=False, grad_x=outs[2])
    lp.lp_linear_bwd(gr, xr, None, need_dx=False, grad_w=outs[3])
    torch.cuda.synchronize()
    for t in outs:
        assert not t.any()


@pytest.mark.parametrize("M", [3, 40])
@pytest.mark.parametrize("small", [1, 9, 24, 57, 65])
def test_bits_dropped_inside_an_instruction_stay_within_the_bound(lp, M, small):
    """Two products of 448 x 448 that cancel, among equal small ones: the matrix core aligns all of them to the large
    ones, and what it drops is less than 2^-10 of the magnitudes' sum."""
    N, K = 16, 128
    for big, other in ((0, 1), (0, 64), (5, 100)):
        x, w = np.full((M, K), small, np.uint8), np.full((N, K), 57, np.uint8)
        x[:, big], x[:, other], w[:, big], w[:, other] = 0x7E, 0xFE, 0x7E, 0x7E
        ones = torch.ones(1, 1, 1, device="cuda")
        y = lp.lp_linear_fwd(lp.QTensor("fp8_r128", dev(x), ones.expand(1, 1, M).contiguous()), lp.QTensor("fp8_b128", dev(w), ones))
        a, b = E4M3_TABLE[x], E4M3_TABLE[w].T
        bound = 2.0 ** -8 * np.abs(a @ b) + 2.0 ** -10 * (np.abs(a) @ np.abs(b))
        assert (np.abs(y.float().cpu().numpy() - a @ b) <= bound).all(), (big, other)
