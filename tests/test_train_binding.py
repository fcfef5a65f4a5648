"""The binding's own checks of the block-scaled FP8 training calls, with
stand-ins for device tensors and for the C functions (CPU only; no kernel is
launched)."""
import ctypes

import pytest
import torch

import fp8_gemm_backward_amd as lp

FAKE = 0x10000


class DeviceTensor:
    """What the binding looks at of a contiguous device tensor; its memory is never touched."""
    is_cuda = True

    def __init__(self, shape, dtype=torch.uint8, ptr=FAKE):
        self.shape, self.dtype, self.device, self.ptr = tuple(shape), dtype, torch.device("meta"), ptr

    def numel(self):
        return torch.Size(self.shape).numel()

    def dim(self):
        return len(self.shape)

    def element_size(self):
        return self.dtype.itemsize

    @property
    def nbytes(self):
        return self.numel() * self.dtype.itemsize

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.ptr if self.numel() else 0

    def new_empty(self, shape, dtype=None):
        return DeviceTensor(shape, dtype or self.dtype)


@pytest.fixture
def calls(monkeypatch):
    """The C calls made, as (name, arguments); none is carried out."""
    made = []
    for name in ("lp_r128_quant", "lp_r128_quant_dual", "lp_linear_bwd", "lp_grouped_bwd", "lp_dequant", "lp_adamw"):
        monkeypatch.setattr(lp.lib, name, lambda *a, _n=name: made.append((_n, a)) or 0)
    monkeypatch.setattr(lp, "_stream", lambda s: 0)
    return made


def runs_tensor(rows, cols, runs, axis=-2, **kw):
    """An "fp8_r128" tensor whose scales hold `runs` runs."""
    shape = (1, runs, cols) if axis == -2 else (1, -(-cols // 128), rows)
    return lp.QTensor("fp8_r128", DeviceTensor((1, rows, cols)), DeviceTensor(shape, torch.float32), axis=axis, **kw)


def offsets(groups):
    return DeviceTensor((groups,), torch.int32)


@pytest.mark.parametrize("rows,groups,runs,ok", [
    (4096, 64, 32, False),            # quantized without offsets
    (4096, 64, 95, False), (4096, 64, 96, True), (4096, 64, 97, True),
    (100, 3, 1, False), (100, 3, 2, False), (100, 3, 3, True),
    (130, 1, 1, False), (130, 1, 2, True), (128, 1, 1, True),     # one group: the layout without offsets
])
@pytest.mark.parametrize("short", ["grad_out", "x"])
def test_grouped_grad_w_needs_scales_of_every_run(calls, rows, groups, runs, ok, short):
    """Group g's runs begin at its first row / 128 + g, so the kernel reads up to rows / 128 + groups of them."""
    enough = rows // 128 + groups
    g = runs_tensor(rows, 256, runs if short == "grad_out" else enough)
    x = runs_tensor(rows, 144, runs if short == "x" else enough)

    def call():
        return lp.lp_grouped_bwd(g, x, None, offsets(groups), need_dx=False)
    if ok:
        call()
        assert [n for n, _ in calls] == ["lp_grouped_bwd"]
    else:
        with pytest.raises(ValueError, match="scales"):
            call()
        assert not calls
