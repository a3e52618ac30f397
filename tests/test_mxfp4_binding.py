"""The devices and streams of the MXFP4 calls' arguments, without a GPU: stand-ins for tensors, and
sizes that the library refuses, so that a call that goes through returns a status and launches
nothing."""

import pytest
import torch

import dense_fp32_gemm_sm_gb300 as fg
from dense_fp32_gemm_sm_gb300 import _binding

INVALID = fg.ERR_INVALID_VALUE


class Tensor:
    """What a CUDA tensor shows of itself."""

    is_cuda = True

    def __init__(self, index=0, dtype=torch.float32):
        self.index, self.dtype, self.device = index, dtype, "cuda:%d" % index

    def data_ptr(self):
        return 0x10000

    def get_device(self):
        return self.index


@pytest.fixture
def gpu(monkeypatch):
    """Two devices: the current one, and those whose current stream was asked for."""
    state = type("State", (), dict(current=0, asked=[]))()
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)

    def stream(index):
        state.asked.append(index)
        return 0x5000 + index

    torch_c = pytest.importorskip("torch._C")
    monkeypatch.setattr(torch_c, "_cuda_getCurrentRawStream", stream, raising=False)
    monkeypatch.setattr(torch_c, "_cuda_getDevice", lambda: state.current, raising=False)
    monkeypatch.setattr(_binding, "_calls", None)  # (bound anew to these, and again after the test)
    yield state
    monkeypatch.undo()
    _binding._calls = None


@pytest.fixture
def only_gpu(gpu, monkeypatch):
    """The same with one device, of which nobody asks whether it is current."""
    def asked():
        raise AssertionError("asked for the current device")
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 1)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", asked, raising=False)
    return gpu


def u8(index=0):
    return Tensor(index, torch.uint8)


# Every call with M = -1, its tensors by name.
CALLS = {
    "quantize": (lambda t: fg.mxfp4_quantize(fg.F32, -1, 40, t["X"], 40, t["r"], 32, t["rs"], t["c"], 16, t["cs"], check=False),
                 dict(X=Tensor, r=u8, rs=u8, c=u8, cs=u8)),
    "quantize_grad": (lambda t: fg.mxfp4_quantize_grad(fg.F32, -1, 40, t["X"], 40, t["Y"], 40, t["r"], 32, t["rs"], t["c"], 16, t["cs"],
                                                       t["b"], t["w"], 160, check=False),
                      dict(X=Tensor, Y=Tensor, r=u8, rs=u8, c=u8, cs=u8, b=Tensor, w=u8)),
    "dequantize": (lambda t: fg.mxfp4_dequantize(fg.F32, -1, 40, t["r"], 32, t["rs"], t["X"], 40, check=False),
                   dict(r=u8, rs=u8, X=Tensor)),
    "gemm": (lambda t: fg.mxfp4_gemm(fg.F32, -1, 5, 40, 1.0, t["r"], 32, t["rs"], t["c"], 32, t["cs"], 0.0, t["X"], 5, t["b"], check=False),
             dict(r=u8, rs=u8, c=u8, cs=u8, X=Tensor, b=Tensor)),
    "linear": (lambda t: fg.mxfp4_linear(fg.F32, -1, 5, 40, t["X"], 40, t["c"], 32, t["cs"], t["b"], False, t["Y"], 5, t["w"], 64,
                                         check=False),
               dict(X=Tensor, c=u8, cs=u8, b=Tensor, Y=Tensor, w=u8)),
}


@pytest.mark.parametrize("name", CALLS)
def test_tensors_on_the_current_device(gpu, name):
    call, makers = CALLS[name]
    for index in (0, 1):
        gpu.current = index
        assert call({k: make(index) for k, make in makers.items()}) == INVALID
    assert gpu.asked == [0, 1]


@pytest.mark.parametrize("name", CALLS)
def test_tensors_on_the_only_device(only_gpu, name):
    call, makers = CALLS[name]
    assert call({k: make() for k, make in makers.items()}) == INVALID
    assert only_gpu.asked == [0]


@pytest.mark.parametrize("name", CALLS)
def test_tensors_on_another_device_are_refused(gpu, name):
    # the library launches on the current device, whatever device an address belongs to
    call, makers = CALLS[name]
    for current, index in ((0, 1), (1, 0)):
        gpu.current = current
        with pytest.raises(ValueError):
            call({k: make(index) for k, make in makers.items()})


@pytest.mark.parametrize("name,odd", [(n, k) for n, (_, makers) in CALLS.items() for k in makers])
def test_tensors_on_several_devices_are_refused(gpu, name, odd):
    call, makers = CALLS[name]
    for current in (0, 1):
        gpu.current = current
        with pytest.raises(ValueError):
            call({k: make(1 if k == odd else 0) for k, make in makers.items()})


def test_addresses_are_taken_as_they_are(gpu):
    for name, (call, makers) in CALLS.items():
        assert call({k: 0x10000 for k in makers}) == INVALID
    assert not gpu.asked


@pytest.mark.parametrize("devices", ["gpu", "only_gpu"])
def test_what_is_no_cuda_tensor_is_a_type_error(devices, request):
    request.getfixturevalue(devices)
    call, makers = CALLS["quantize"]
    for bad in (torch.zeros(4, 40), torch.zeros(4, 40, device="meta"), object(), "x", 1.5):
        for k in ("X", "rs"):
            with pytest.raises(TypeError):
                call({n: bad if n == k else make() for n, make in makers.items()})
    with pytest.raises(TypeError):
        call({n: make() for n, make in makers.items()} | dict(X=Tensor(0, torch.float16)))


@pytest.mark.parametrize("name,odd", [(n, k) for n, (_, makers) in CALLS.items() for k in makers])
def test_one_tensor_among_addresses_gives_its_stream(gpu, name, odd):
    # whichever argument it is: work that made it is on that stream
    call, makers = CALLS[name]
    gpu.current = 1
    assert call({k: make(1) if k == odd else 0x10000 for k, make in makers.items()}) == INVALID
    assert gpu.asked == [1]
