"""Host-side checks whose every call ends at a refusal, and the rule that keeps made-up device addresses off a GPU."""
import ctypes
import types

import pytest
import torch

import conftest
from bit_quantized_base_nf4_b200 import _capi
from bit_quantized_base_nf4_b200 import build as libbuild

P = ctypes.c_void_p
ARG, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return _capi.load()


def _err(lib):
    return lib.qlora_last_error().decode()


def _tensor(at=0, **kw):
    t = dict(param=0x10000 + at, grad=0x20000 + at, exp_avg=0x30000 + at, exp_avg_sq=0x40000 + at, numel=1000, lr_scale=1.0,
             weight_decay=0.0, flags=0)
    t.update(kw)
    return _capi.AdamWTensorC(**t)


class _Item:
    """As much of a collected test as the collection hook looks at."""

    def __init__(self, file, name, *marks):
        self.path, self.originalname, self.name = types.SimpleNamespace(name=file), name, name
        self.keywords, self.added = set(marks), []

    def add_marker(self, m):
        self.added.append(m.name)


@pytest.mark.parametrize("has_gpu", [True, False])
def test_made_up_addresses_stay_off_a_gpu(monkeypatch, has_gpu):
    monkeypatch.setattr(torch.cuda, "is_available", lambda: has_gpu)
    fakes = [_Item("test_capi_cpu.py", "test_format_flags_are_validated"),
             _Item("test_training_capi_cpu.py", "test_neighbouring_buffers_and_shared_gradients_are_not_refused")]
    other, gpu = _Item("test_capi_cpu.py", "test_validation_rejects_before_launch"), _Item("test_gpu_parity.py", "test_x", "gpu")
    conftest.pytest_collection_modifyitems(None, fakes + [other, gpu])
    assert [i.added for i in fakes] == ([["skip"]] * 2 if has_gpu else [[]] * 2)
    assert other.added == [] and gpu.added == ([] if has_gpu else ["skip"])


def test_neighbours_and_shared_gradients_pass_the_overlap_check(lib):
    # the buffer's size is looked at after the overlaps: one byte short, the list itself was fine
    arr = (_capi.AdamWTensorC * 3)(_tensor(), _tensor(0x100000, param=0x10000 + 4000), _tensor(0x200000, grad=0x20000))
    plan, need = _capi.AdamWPlanC(), lib.qlora_adamw_plan_bytes(arr, 3)
    assert need > 0
    assert lib.qlora_adamw_plan_init(arr, 3, P(0x1000000), need - 1, ctypes.byref(plan), None) == WORKSPACE, _err(lib)
    assert plan.magic == 0


def test_no_second_level_scales_without_double_quantization(lib):
    # the output's alignment is looked at after the weight: a NULL scales2 passed
    w = _capi.Nf4WeightC(256, 512, 0x1000, 0x2000, None)
    w.format = 2
    assert lib.qlora_dequant(ctypes.byref(w), P(0x20008), 0, None) == ALIGN and "out must" in _err(lib)
    w.format = 0
    assert lib.qlora_dequant(ctypes.byref(w), P(0x20008), 0, None) == ARG


def _huge(at):
    """A tensor of 2^40 elements whose buffers lie far apart."""
    return _tensor(numel=1 << 40, **{k: at + (i << 50) for i, k in enumerate(("param", "grad", "exp_avg", "exp_avg_sq"), 1)})


@pytest.mark.parametrize("tensors", [
    [_huge(0), _huge(1 << 60)],                   # more elements than a plan takes
])
def test_plan_bytes_are_zero_for_a_list_that_plan_init_refuses(lib, tensors):
    arr, plan = (_capi.AdamWTensorC * len(tensors))(*tensors), _capi.AdamWPlanC()
    assert lib.qlora_adamw_plan_init(arr, len(tensors), P(0x1000000), 1 << 62, ctypes.byref(plan), None) in (ARG, SHAPE)
    assert lib.qlora_adamw_plan_bytes(arr, len(tensors)) == 0


def test_a_list_whose_elements_pass_64_bits_is_refused(lib):
    # 2^23 tensors of 2^40 elements: the sum of the elements would wrap
    n = 1 << 23
    one = bytes(_tensor(numel=1 << 40, grad=0x20000, flags=8))               # gradients alone, which may share memory
    arr = (_capi.AdamWTensorC * n).from_buffer(bytearray(one * n))
    assert lib.qlora_adamw_plan_bytes(arr, n) == 0 and "too many elements" in _err(lib)


@pytest.mark.parametrize("tensors", [[_tensor(), _tensor()], [_tensor(exp_avg_sq=0x30000)]])
def test_overlaps_are_found_by_plan_init_alone(lib, tensors):
    # as the header says: the bytes are those of the list, whatever its buffers do to one another
    arr, plan = (_capi.AdamWTensorC * len(tensors))(*tensors), _capi.AdamWPlanC()
    need = lib.qlora_adamw_plan_bytes(arr, len(tensors))
    assert need > 0
    assert lib.qlora_adamw_plan_init(arr, len(tensors), P(0x1000000), need, ctypes.byref(plan), None) == ARG and "overlaps" in _err(lib)
