"""The binding's own checks of the block-scaled FP8 training calls, with
stand-ins for device tensors and for the C functions (CPU only; no kernel is
launched)."""
import gc
import weakref

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


# ---------------------------------------------------------------- which groups a token-run tensor was made for

def test_quantizers_note_the_groups(calls):
    src = DeviceTensor((300, 256), torch.bfloat16)
    assert lp.lp_r128_quant(src, -2).run_groups == 0 and lp.lp_r128_quant(src, -2, offsets(5)).run_groups == 5
    assert lp.lp_r128_quant(src, -1).run_groups is None
    for off, n in ((None, 0), (offsets(7), 7)):
        cols, rows = lp.lp_r128_quant_dual(src, off)
        assert cols.run_groups is None and rows.run_groups == n


@pytest.mark.parametrize("made_for,ok", [(None, True), (0, True), (1, True), (2, False), (5, False)])
def test_calls_without_offsets_refuse_runs_of_groups(calls, made_for, ok):
    """The dense calls find a row's run at row / 128; runs that restart at a group's first row are elsewhere."""
    def q():
        return runs_tensor(300, 256, 3 + 5, run_groups=made_for)
    out = DeviceTensor((300, 256), torch.bfloat16)
    for call in (lambda: lp.lp_dequant(q(), out), lambda: lp.lp_linear_bwd(q(), runs_tensor(300, 256, 3), None, need_dx=False),
                 lambda: lp.lp_linear_bwd(runs_tensor(300, 256, 3), q(), None, need_dx=False)):
        calls.clear()
        if ok:
            call()
            assert len(calls) == 1
        else:
            with pytest.raises(ValueError, match="groups"):
                call()
            assert not calls


@pytest.mark.parametrize("made_for,groups,ok", [(None, 4, True), (4, 4, True), (3, 4, False), (5, 4, False), (0, 4, False),
                                                (1, 4, False), (0, 1, True), (1, 1, True), (None, 1, True), (2, 1, False)])
def test_grouped_grad_w_refuses_runs_of_other_groups(calls, made_for, groups, ok):
    for k in range(2):
        ops = [runs_tensor(300, 256, 9), runs_tensor(300, 256, 9)]
        ops[k].run_groups = made_for
        calls.clear()
        if ok:
            lp.lp_grouped_bwd(*ops, None, offsets(groups), need_dx=False)
            assert len(calls) == 1
        else:
            with pytest.raises(ValueError, match="groups"):
                lp.lp_grouped_bwd(*ops, None, offsets(groups), need_dx=False)
            assert not calls


@pytest.mark.parametrize("ptr", [0, FAKE])
def test_quantizers_refuse_offsets_of_no_group(monkeypatch, ptr):
    """An empty offsets tensor has a null address, with which the C call would quantize without groups: into scales of
    rows // 128 runs, one too few."""
    made = []
    for name in ("lp_r128_quant", "lp_r128_quant_dual"):
        monkeypatch.setattr(lp.lib, name, lambda *a: made.append(a) or 0)
    monkeypatch.setattr(lp, "_stream", lambda s: 0)
    none = offsets(0)
    monkeypatch.setattr(none, "data_ptr", lambda: ptr, raising=False)
    src = DeviceTensor((300, 256), torch.bfloat16)
    for call in (lambda: lp.lp_r128_quant(src, -2, none), lambda: lp.lp_r128_quant_dual(src, none)):
        with pytest.raises(lp.LpError) as e:
            call()
        assert e.value.status == 2
    assert not made


# ---------------------------------------------------------------- AdamW

def adamw_lists(*params):
    return [list(params)] + [[DeviceTensor(p.shape, torch.float32) for p in params] for _ in range(3)]


def test_adamw_table_goes_where_the_parameters_are(calls):
    """An empty parameter may be anywhere (it is not touched); the table may not."""
    p = DeviceTensor((300,), torch.float32)
    for params in ([p], [torch.zeros(0), p], [p, torch.zeros(0)]):
        assert lp.AdamWPlan(*adamw_lists(*params))._table.device == p.device
    assert lp.AdamWPlan(*adamw_lists(torch.zeros(0)))._table is None


@pytest.mark.parametrize("captured", [True, False])
def test_adamw_keeps_what_a_captured_step_reads(calls, monkeypatch, captured):
    """A graph that holds a step reads that step's table, and through it the gradients, at every replay: set_grads must
    not free them."""
    capturing = captured
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    lists = adamw_lists(DeviceTensor((300,), torch.float32))
    first = weakref.ref(lists[1][0])
    plan = lp.AdamWPlan(*lists)
    lists[1] = None
    table = weakref.ref(plan._table)
    lp.lp_adamw(plan, lr=0.1)
    capturing = False
    for _ in range(3):
        plan.set_grads([DeviceTensor((300,), torch.float32)])
        lp.lp_adamw(plan, lr=0.1)
    gc.collect()
    assert (table() is not None) == (first() is not None) == captured


@pytest.mark.parametrize("private", [True, False])
def test_current_stream_without_torch_s_private_lookup(monkeypatch, private):
    """The handle comes from a private call of torch's where there is one, from the public stream object otherwise."""
    class Stream:
        cuda_stream = 77
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream)
    monkeypatch.setattr(lp, "_raw_stream", (lambda device: 1000 + device) if private else None)
    assert lp._stream(None) == (1003 if private else 77)
    assert lp._stream(Stream) == 77 and lp._stream(5) == 5
