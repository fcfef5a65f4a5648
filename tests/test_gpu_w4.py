"""Forwards of a bf16 x by a 4-bit weight (lp_linear_fwd_w4, lp_grouped_fwd_w4)
against fp64 over the decoded weight (GPU)."""
import numpy as np
import pytest
import torch

import workloads as W
from gpu_util import bf16_dev, dev, quantize
from oracle import formats as F
from oracle.formats import bf16_bits_to_f64

pytestmark = pytest.mark.gpu


def weight(lp, fmt, G, N, K, seed):
    """(tensor, its decoded values [G, N, K] in fp64): random codes, scales over a wide range."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (G, N, K // 2), dtype=np.uint8)
    ts = None
    if fmt == "mxfp4":
        scales = rng.integers(115, 130, (G, N, K // 32), dtype=np.uint8)
    else:
        scales = rng.integers(0, 0x7F, (G, N, K // 16), dtype=np.uint8)      # subnormal scales and 448 among them
        ts = np.float32(0.0123)
    dec = bf16_bits_to_f64(F.dequant(fmt, codes, scales, None if ts is None else float(ts)))
    q = lp.QTensor(fmt, dev(codes), dev(scales), None if ts is None else torch.tensor([ts], device="cuda"), shape=(G, N, K))
    return q, dec.reshape(G, N, K)


def rows_of(M, K, seed):
    b = W.bf16_bits(np.random.default_rng(seed).standard_normal((M, K)).astype(np.float32))
    return bf16_dev(b), bf16_bits_to_f64(b)


def check(got, x, w, what):
    """One rounding to bf16, and fp32 sums of K exact products in any order: at most K roundings (a step each, should the
    matrix core cut off rather than round) of partial sums no larger than the products' magnitudes together."""
    ref, size = x @ w.T, np.abs(x) @ np.abs(w).T
    err = np.abs(got.float().cpu().numpy() - ref)
    assert (err <= 2.0 ** -8 * np.abs(ref) + x.shape[1] * 2.0 ** -23 * size + 1e-30).all(), (what, (err / size).max())


SHAPES = [(1, 16, 32), (1, 4096, 4096), (2, 48, 96), (3, 1040, 288), (4, 256, 7168), (5, 8192, 2048), (15, 272, 544),
          (16, 4096, 1024), (17, 4112, 256), (24, 8192, 2048), (31, 144, 4128), (33, 2048, 512), (48, 528, 1056), (64, 16, 8192),
          (65, 272, 544), (100, 512, 160), (257, 528, 288), (600, 272, 96)]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(lp, fmt, M, N, K):
    w, dec = weight(lp, fmt, 1, N, K, M + N + K)
    x, xv = rows_of(M, K, M * N + K)
    guard = torch.full((M + 3, N), 7.0, dtype=torch.bfloat16, device="cuda")
    y = lp.lp_linear_fwd_w4(x, w, y=guard[:M])
    check(y, xv, dec[0], (fmt, M, N, K))
    assert (guard[M:] == 7).all()
    assert torch.equal(y, lp.lp_linear_fwd_w4(x, w))                 # the same bits again


# Sizes that take each of the workgroup shapes in turn, then the large tiles.
DENSE = [(16, 16, 32), (101, 608, 160), (175, 768, 160), (853, 80, 32), (1394, 144, 320), (2207, 112, 416), (2634, 288, 32),
         (2329, 288, 480), (3214, 528, 448), (306, 8832, 32), (289, 6464, 32), (388, 9472, 288), (517, 7216, 32), (1106, 7200, 32)]
GROUPED = [(3, 16, 32, 2), (34, 128, 160, 33), (282, 496, 160, 2), (109, 592, 32, 2), (2269, 96, 320, 9), (2222, 128, 416, 5),
           (4076, 80, 64, 33), (3927, 80, 288, 70), (2960, 528, 480, 5), (456, 3904, 32, 9), (3396, 304, 32, 70), (836, 4640, 288, 2),
           (1390, 1616, 32, 33), (3223, 2336, 32, 5)]


# Those of the shapes that take middling sizes, and the large tiles.
MIDDLING = [(2713, 288, 416), (212, 3488, 1024), (97, 9280, 2464), (393, 9392, 416), (2181, 288, 32), (1266, 6992, 32), (1348, 8832, 96),
            (489, 9344, 32), (197, 8320, 672), (294, 8368, 416)]
MIDDLING_GROUPED = [(2099, 336, 416, 2), (205, 1632, 1056, 9), (98, 9312, 2464, 2), (398, 9360, 416, 2), (2059, 336, 32, 2), (971, 8848, 32, 2),
                    (49, 1616, 1056, 9), (157, 9520, 32, 5), (3100, 6000, 32, 2), (175, 9232, 32, 5), (1178, 288, 672, 70), (71, 3792, 32, 33)]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K", MIDDLING)
def test_middling_shapes(lp, fmt, M, N, K):
    test_linear(lp, fmt, M, N, K)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K,G", MIDDLING_GROUPED)
def test_middling_shapes_grouped(lp, fmt, M, N, K, G):
    test_grouped(lp, fmt, M, N, K, G, "uneven")


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,G", [(1, 70), (2, 33), (17, 40), (33, 9)])
def test_fewer_rows_than_groups(lp, fmt, M, G):
    """One row a group, the last groups' too, and all rows in the last one: as many row tiles as there can be."""
    w, dec = weight(lp, fmt, G, 144, 96, M + G)
    x, xv = rows_of(M, 96, M)
    sizes = np.zeros((2, G), np.int64)
    sizes[0, G - min(M, G):] = 1
    sizes[0, G - 1] += M - sizes[0].sum()
    sizes[1, G - 1] = M
    for n in sizes:
        ends = np.cumsum(n)
        y = lp.lp_grouped_fwd_w4(x, w, dev(ends.astype(np.int32)))
        for g in np.flatnonzero(n):
            rows = slice(ends[g] - n[g], ends[g])
            check(y[rows], xv[rows], dec[g], (fmt, M, G, g))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K", DENSE)
def test_every_shape_of_a_workgroup(lp, fmt, M, N, K):
    test_linear(lp, fmt, M, N, K)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K,G", GROUPED)
def test_every_shape_of_a_workgroup_grouped(lp, fmt, M, N, K, G):
    test_grouped(lp, fmt, M, N, K, G, "uneven")


def spread(rng, M, G, kind):
    if kind == "empty":
        return np.zeros(G, np.int64)
    if kind == "one":
        s = np.zeros(G, np.int64)
        s[G // 2] = M
        return s
    p = rng.dirichlet(np.full(G, 0.3))
    return rng.multinomial(M, p)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K,G", [(1, 16, 32, 1), (7, 272, 96, 3), (16, 2048, 1024, 8), (96, 528, 544, 64), (40, 144, 288, 100),
                                     (300, 272, 160, 7), (513, 64, 64, 65), (1000, 144, 96, 130)])
@pytest.mark.parametrize("kind", ["uneven", "one", "empty"])
def test_grouped(lp, fmt, M, N, K, G, kind):
    rng = np.random.default_rng(M + N + G)
    w, dec = weight(lp, fmt, G, N, K, M * 3 + N)
    x, xv = rows_of(M, K, M + K)
    used = M if M < 7 else M - 5                                     # rows past the last offset
    ends = np.cumsum(spread(rng, used, G, kind)).astype(np.int32)
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    lp.lp_grouped_fwd_w4(x, w, dev(ends), y=y)
    start = 0
    for g, e in enumerate(ends):
        if e > start:
            check(y[start:e], xv[start:e], dec[g], (fmt, g))
        start = e
    assert (y[start:] == 7).all()


@pytest.mark.parametrize("M", [3, 20, 90])
@pytest.mark.parametrize("ends", [[5, 2, 9], [-3, 4, 1 << 30], [0, 0, 0], [1 << 30, 0, -1]])
def test_bad_offsets_stay_in_bounds(lp, M, ends):
    """Clamped as everywhere: end_g = clamp(offsets[g], end_{g-1}, M)."""
    w, dec = weight(lp, "mxfp4", 3, 48, 64, 1)
    x, xv = rows_of(M, 64, 2)
    y = torch.full((M, 48), 7.0, dtype=torch.bfloat16, device="cuda")
    lp.lp_grouped_fwd_w4(x, w, dev(np.array(ends, np.int32)), y=y)
    start = 0
    for g, e in enumerate(ends):
        e = min(max(e, start), M)
        if e > start:
            check(y[start:e], xv[start:e], dec[g], g)
        start = e
    assert (y[start:] == 7).all()


@pytest.mark.parametrize("M", [1, 20, 70])
@pytest.mark.parametrize("fmt,nan", [("mxfp4", 0xFF), ("nvfp4", 0x7F), ("nvfp4", 0xFF)])
def test_a_nan_scale_reaches_its_column_only(lp, fmt, nan, M):
    N, K = 64, 352
    w, _ = weight(lp, fmt, 1, N, K, 4)
    x, _ = rows_of(M, K, 5)
    clean = lp.lp_linear_fwd_w4(x, w)
    w.scales[0, 37, -1] = nan
    y = lp.lp_linear_fwd_w4(x, w)
    assert torch.isnan(y[:, 37]).all()
    keep = [n for n in range(N) if n != 37]
    assert torch.equal(y[:, keep], clean[:, keep])


@pytest.mark.parametrize("M", [2, 19, 70])
def test_a_nan_or_infinite_x_reaches_its_row_only(lp, M):
    w, _ = weight(lp, "mxfp4", 1, 48, 96, 6)
    w.codes[0, :, 47] |= 0x66                                        # (no zero weight there: inf * 0 would be NaN)
    x, _ = rows_of(M, 96, 7)
    clean = lp.lp_linear_fwd_w4(x, w)
    x[1, 95] = float("inf")
    y = lp.lp_linear_fwd_w4(x, w)
    keep = [m for m in range(M) if m != 1]
    assert torch.isinf(y[1].float()).all() and torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_the_ends_of_the_scales(lp, fmt):
    """The smallest and the largest scales a format has, exact in bf16 (mxfp4: 2^-127 to 2^120)."""
    N, K = 16, 64
    codes = np.tile(np.arange(16, dtype=np.uint8), (1, N, K // 16))
    codes = codes[..., 0::2] | (codes[..., 1::2] << 4)
    bytes_ = [0, 1, 2, 127, 240, 247] if fmt == "mxfp4" else [0, 1, 7, 8, 0x38, 0x7E]
    for s in bytes_:
        scales = np.full((1, N, K // (32 if fmt == "mxfp4" else 16)), s, np.uint8)
        ts = None if fmt == "mxfp4" else 1.0
        dec = bf16_bits_to_f64(F.dequant(fmt, codes, scales, ts)).reshape(N, K)
        q = lp.QTensor(fmt, dev(codes), dev(scales), None if ts is None else torch.ones(1, device="cuda"), shape=(1, N, K))
        x = torch.zeros(2, K, dtype=torch.bfloat16, device="cuda")
        x[0, 5], x[1, 38] = 1.0, 2.0
        y = lp.lp_linear_fwd_w4(x, q).float().cpu().numpy()
        assert np.array_equal(y[0], dec[:, 5]) and np.array_equal(y[1], 2 * dec[:, 38]), s


@pytest.mark.parametrize("M", [1, 33, 300])
def test_no_contraction_gives_zeros(lp, M):
    for fmt in ("mxfp4", "nvfp4"):
        e = torch.empty(1, 32, 0, dtype=torch.uint8, device="cuda")
        q = lp.QTensor(fmt, e, e, torch.ones(1, device="cuda"), shape=(1, 32, 0))
        y = lp.lp_linear_fwd_w4(torch.empty(M, 0, dtype=torch.bfloat16, device="cuda"), q)
        assert y.shape == (M, 32) and not y.any()


def test_no_row(lp):
    w, _ = weight(lp, "mxfp4", 2, 32, 64, 8)
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert lp.lp_grouped_fwd_w4(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), w, off).shape == (0, 32)


def test_quantized_weights_of_the_library(lp):
    """A weight that lp_mx_quant made, and the same decoded by lp_dequant."""
    rng = np.random.default_rng(11)
    wb = bf16_dev(W.bf16_bits((rng.standard_normal((1, 80, 256)) * 0.02).astype(np.float32)))
    q = lp.lp_mx_quant(wb, -1, "mxfp4")
    x, xv = rows_of(6, 256, 12)
    check(lp.lp_linear_fwd_w4(x, q), xv, lp.lp_dequant(q)[0].float().cpu().numpy().astype(np.float64), "mx_quant")
