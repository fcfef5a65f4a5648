"""Oracle of block-scaled FP8 training: E4M3 with fp32 scales per 128
elements, its products, and the AdamW step, in numpy fp64.

Quantization of a set of values with largest magnitude a:
s = RNE_fp32(max(a, 2^-64) / 448), code = E4M3(RNE_fp32(v / s)), saturating; a
set with a NaN or an infinity gets s = NaN and codes 0x7F with each element's
sign.  Sets are runs of 128 along an axis (cut at the tensor's edge; along the
rows, restarting at each group's first row) or 128 x 128 blocks.
"""
from __future__ import annotations

import numpy as np

from .formats import E4M3_TABLE, bf16_bits_to_f64, round_f32, round_to_grid

RUN = 128
FLOOR = 2.0 ** -64


def quant_set(v: np.ndarray):
    """(codes like v, scale) of one set of fp64 values."""
    v = np.asarray(v, dtype=np.float64)
    if not np.isfinite(v).all():
        return (0x7F | (np.signbit(v).astype(np.uint8) << 7)).astype(np.uint8), np.float32(np.nan)
    s = np.float32(round_f32(max(np.abs(v).max(initial=0.0), FLOOR) / 448.0))
    return round_to_grid(round_f32(v / np.float64(s)).astype(np.float64), "e4m3"), s


def spans(rows: int, ends=None) -> list:
    """[(run index, first row, end row)] of the runs along the rows; ends: clamped cumulative group ends."""
    out, start = [], 0
    for g, e in enumerate([rows] if ends is None else ends):
        e = min(max(int(e), start), rows)
        first = 0 if ends is None else start // RUN + g
        for i, r in enumerate(range(start, e, RUN)):
            out.append((first + i, r, min(r + RUN, e)))
        start = e
    return out


def quant_cols(bits: np.ndarray):
    """bf16 bits [R, C] -> codes [R, C], scales [ceil(C / 128), R]."""
    v = bf16_bits_to_f64(bits)
    R, C = v.shape
    codes, scales = np.zeros((R, C), np.uint8), np.zeros((-(-C // RUN), R), np.float32)
    for r in range(R):
        for b in range(scales.shape[0]):
            codes[r, b * RUN:(b + 1) * RUN], scales[b, r] = quant_set(v[r, b * RUN:(b + 1) * RUN])
    return codes, scales


def quant_rows(bits: np.ndarray, ends=None):
    """bf16 bits [R, C] -> codes [R, C], scales {run index: [C]}; rows of no group keep code 0."""
    v = bf16_bits_to_f64(bits)
    codes, scales = np.zeros(v.shape, np.uint8), {}
    for run, a, b in spans(v.shape[0], ends):
        scales[run] = np.zeros(v.shape[1], np.float32)
        for c in range(v.shape[1]):
            codes[a:b, c], scales[run][c] = quant_set(v[a:b, c])
    return codes, scales


def quant_blocks(bits: np.ndarray):
    """bf16 bits [R, C] -> codes [R, C], scales [ceil(R / 128), ceil(C / 128)]."""
    v = bf16_bits_to_f64(bits)
    R, C = v.shape
    codes, scales = np.zeros((R, C), np.uint8), np.zeros((-(-R // RUN), -(-C // RUN)), np.float32)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = np.s_[i * RUN:(i + 1) * RUN, j * RUN:(j + 1) * RUN]
            codes[at], scales[i, j] = quant_set(v[at])
    return codes, scales


def values_cols(codes, scales):
    """fp64 values of a tensor scaled along its columns (scales [runs, R])."""
    return E4M3_TABLE[codes] * np.repeat(scales.astype(np.float64).T, RUN, 1)[:, :codes.shape[1]]


def values_rows(codes, scales, ends=None):
    out = np.zeros(codes.shape)
    for run, a, b in spans(codes.shape[0], ends):
        out[a:b] = E4M3_TABLE[codes[a:b]] * scales[run].astype(np.float64)
    return out


def values_blocks(codes, scales):
    R, C = codes.shape
    return E4M3_TABLE[codes] * np.repeat(np.repeat(scales.astype(np.float64), RUN, 0), RUN, 1)[:R, :C]


def groups(rows: int, ends) -> list:
    out, start = [], 0
    for e in ends:
        e = min(max(int(e), start), rows)
        out.append((start, e))
        start = e
    return out


def adamw(p, g, m, v, lr, beta1, beta2, eps, step, weight_decay):
    """One step in fp64: (p, m, v)."""
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    p = (1 - lr * weight_decay) * p - lr * (m / (1 - beta1 ** step)) / (np.sqrt(v / (1 - beta2 ** step)) + eps)
    return p, m, v


def quant_state(x: np.ndarray, keep: bool = False):
    """1-D values -> (codes, scales) in runs of 128; keep: a positive value is at least code 1."""
    codes, scales = np.zeros(x.size, np.uint8), np.zeros(-(-x.size // RUN), np.float32)
    for b in range(scales.size):
        at = slice(b * RUN, (b + 1) * RUN)
        codes[at], scales[b] = quant_set(x[at])
    if keep:
        codes = np.where((x > 0) & (codes == 0), 1, codes).astype(np.uint8)
    return codes, scales


def state_values(codes, scales):
    return E4M3_TABLE[codes] * np.repeat(scales.astype(np.float64), RUN)[:codes.size]


