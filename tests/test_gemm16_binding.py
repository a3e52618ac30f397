"""Types, devices and streams of the 16-bit calls' arguments, without a GPU: stand-ins for tensors, and sizes that the
library refuses, so that a call that goes through returns a status and launches nothing."""

import pytest
import torch

import dense_fp32_gemm_sm_gb300 as fg
from test_mxfp4_binding import INVALID, Tensor, gpu, only_gpu  # noqa: F401

H, F, I = torch.bfloat16, torch.float32, torch.int32  # noqa: E741

# Every call with M = -1, its tensors by name and type (None: any).
CALLS = {
    "gemm16": (lambda t: fg.gemm16(fg.BF16, fg.F32, 0, 0, -1, 8, 8, 1.0, t["A"], 8, t["B"], 8, t["b"], 0, t["Z"], 8, 0.0, t["R"], 8,
                                   t["Y"], 8, t["w"], 64, check=False), dict(A=H, B=H, b=F, Z=H, R=F, Y=F, w=None)),
    "gemm16_grad": (lambda t: fg.gemm16_grad(fg.BF16, fg.BF16, 0, 0, -1, 8, 8, 1.0, t["A"], 8, t["B"], 8, 0, t["Z"], 8, t["Y"], 8, t["s"],
                                             t["w"], 64, check=False), dict(A=H, B=H, Z=H, Y=H, s=F, w=None)),
    "grouped": (lambda t: fg.gemm16_grouped(fg.BF16, fg.F32, 0, 2, -1, 8, 8, t["o"], 1.0, t["A"], 8, t["B"], 8, 64, t["b"], 0, t["Z"], 8,
                                            0.0, t["R"], 8, t["Y"], 8, t["w"], 64, check=False),
                dict(o=I, A=H, B=H, b=F, Z=H, R=F, Y=F, w=None)),
    "grouped_grad": (lambda t: fg.gemm16_grouped_grad(fg.BF16, fg.BF16, 0, 2, -1, 8, 8, t["o"], 1.0, t["A"], 8, t["B"], 8, 64, 0, t["Z"], 8,
                                                      t["Y"], 8, t["s"], t["w"], 64, check=False),
                     dict(o=I, A=H, B=H, Z=H, Y=H, s=F, w=None)),
    "weight_grad": (lambda t: fg.gemm16_weight_grad(fg.BF16, fg.F32, 2, -1, 8, 8, t["o"], 1.0, t["A"], 8, t["G"], 8, 0.0, t["C"], 8, 64,
                                                    t["w"], 64, check=False), dict(o=I, A=H, G=H, C=F, w=None)),
    "act16_grad": (lambda t: fg.act16_grad(fg.BF16, 2, -1, 8, t["o"], 0, t["G"], 8, t["Z"], 8, t["D"], 8, t["s"], t["w"], 64, check=False),
                   dict(o=I, G=H, Z=H, D=H, s=F, w=None)),
}
ALL = [(n, k) for n, (_, types) in CALLS.items() for k in types]


def tensors(types, index=0):
    return {k: Tensor(index, t or torch.uint8) for k, t in types.items()}


@pytest.mark.parametrize("name", CALLS)
def test_tensors_on_the_current_device(gpu, name):  # noqa: F811
    call, types = CALLS[name]
    for index in (0, 1):
        gpu.current = index
        assert call(tensors(types, index)) == INVALID
    assert gpu.asked == [0, 1]


@pytest.mark.parametrize("name", CALLS)
def test_tensors_on_another_device_are_refused(gpu, name):  # noqa: F811
    call, types = CALLS[name]
    for current, index in ((0, 1), (1, 0)):
        gpu.current = current
        with pytest.raises(ValueError):
            call(tensors(types, index))


@pytest.mark.parametrize("name,odd", ALL)
def test_tensors_on_several_devices_are_refused(gpu, name, odd):  # noqa: F811
    call, types = CALLS[name]
    with pytest.raises(ValueError):
        call(tensors(types) | {odd: Tensor(1, types[odd] or torch.uint8)})


@pytest.mark.parametrize("name,odd", ALL)
def test_another_element_type_is_a_type_error(only_gpu, name, odd):  # noqa: F811
    call, types = CALLS[name]
    if types[odd] is None:
        assert call(tensors(types) | {odd: Tensor(0, torch.float64)}) == INVALID
        return
    for dtype in (torch.float16, torch.int64, torch.float64):
        with pytest.raises(TypeError):
            call(tensors(types) | {odd: Tensor(0, dtype)})


@pytest.mark.parametrize("name,odd", ALL)
def test_what_is_no_cuda_tensor_is_a_type_error(only_gpu, name, odd):  # noqa: F811
    call, types = CALLS[name]
    for bad in (torch.zeros(4, dtype=types[odd] or torch.uint8), object(), "x", 1.5):
        with pytest.raises(TypeError):
            call(tensors(types) | {odd: bad})


@pytest.mark.parametrize("name,odd", ALL)
def test_one_tensor_among_addresses_gives_its_stream(gpu, name, odd):  # noqa: F811
    call, types = CALLS[name]
    gpu.current = 1
    assert call({k: Tensor(1, t or torch.uint8) if k == odd else 0x10000 for k, t in types.items()}) == INVALID
    assert gpu.asked == [1]


def test_numbers_out_of_range():
    with pytest.raises(OverflowError):
        fg.gemm16_grad(fg.BF16, fg.BF16, 0, 0, 1 << 40, 8, 8, 1.0, 16, 8, 16, 8, 0, 16, 8, 16, 8, check=False)
    with pytest.raises(OverflowError):
        fg.gemm16_weight_grad(fg.BF16, fg.F32, 2, 4, 8, 8, 16, 1.0, 16, 8, 16, 8, 0.0, 16, 8, 1 << 70, check=False)
