"""What the MXFP4 layer refuses and passes on, without a GPU: its calls are replaced by ones that
only look at their arguments, so that no bad argument ever reaches a kernel."""

import pytest
import torch

from dense_fp32_gemm_sm_gb300 import mxfp4_layer
from dense_fp32_gemm_sm_gb300.mxfp4_layer import Mxfp4Layer

K, N = 64, 32


class Calls(list):
    """(name, arguments) of the calls made, in order."""

    def named(self, name):
        return [args for n, args in self if n == name]


@pytest.fixture
def calls(monkeypatch):
    made = Calls()
    for name in ("quantize", "quantize_grad", "gemm", "linear"):
        monkeypatch.setattr(mxfp4_layer.fg, "mxfp4_" + name, lambda *a, name=name: made.append((name, a)))
    return made


def overlapping(rows, cols):
    """Matrices of rows x cols whose rows share elements: a row repeated, and a sliding window."""
    row = torch.randn(cols)
    return [row.expand(rows, cols), row[None].expand(rows, cols), torch.randn(rows + cols).as_strided((rows, cols), (1, 1)),
            torch.randn(rows * cols).as_strided((rows, cols), (cols - 1, 1))]


@pytest.mark.parametrize("which", range(4))
def test_rows_that_overlap_are_refused(calls, which):
    layer = Mxfp4Layer(torch.randn(K, N))
    x, g, y = overlapping(5, K)[which], overlapping(5, N)[which], torch.ones(5, N)
    layer.forward(torch.randn(5, K))
    del calls[:]
    for call in (lambda: layer.forward(x), lambda: layer.decode(x), lambda: layer.backward(g, y),
                 lambda: layer.backward(y, g)):
        with pytest.raises(ValueError):
            call()
    assert not calls


def test_leading_dimensions(calls):
    layer = Mxfp4Layer(torch.randn(K, N))
    for x, ld in ((torch.randn(3, K), K), (torch.randn(3, K + 5)[:, :K], K + 5), (torch.randn(6, K)[::2], 2 * K),
                  (torch.randn(K).expand(1, K), K)):
        del calls[:]
        layer.decode(x)
        (args,) = calls.named("linear")
        assert args[4] is x and args[5] == ld


@pytest.mark.parametrize("rows", [0, 1, 4, 6])
def test_backward_wants_as_many_outputs_as_gradients(calls, rows):
    layer = Mxfp4Layer(torch.randn(K, N))
    layer.forward(torch.randn(5, K))
    del calls[:]
    with pytest.raises(ValueError):
        layer.backward(torch.randn(5, N), torch.ones(rows, N))
    assert not calls


@pytest.mark.parametrize("bias", [torch.zeros(N - 1), torch.zeros(N + 1), torch.zeros(2 * N)[::2], torch.zeros(2, N), torch.zeros(N, 2)[:, :1],
                                  torch.zeros(1).expand(N), torch.zeros(N).double(), torch.zeros(N).half(),
                                  torch.zeros(N, device="meta"), [0.0] * N])
def test_bias_is_n_consecutive_floats(calls, bias):
    with pytest.raises(ValueError):
        Mxfp4Layer(torch.randn(K, N), bias)
    assert not calls


def test_a_good_bias_goes_to_the_calls(calls):
    for b in (None, torch.zeros(N), torch.zeros(3, N)[1], torch.zeros(1, N), torch.zeros(N, 1)):
        layer = Mxfp4Layer(torch.randn(K, N).bfloat16(), b)
        del calls[:]
        layer.decode(torch.randn(2, K).bfloat16())
        assert calls.named("linear")[0][9] is b


def test_backward_without_its_forward_is_refused(calls):
    layer = Mxfp4Layer(torch.randn(K, N))
    del calls[:]
    with pytest.raises(ValueError):
        layer.backward(torch.randn(5, N), torch.ones(5, N))
    y = layer.forward(torch.randn(5, K))
    del calls[:]
    with pytest.raises(ValueError):
        layer.backward(torch.randn(4, N), y[:4])
    assert not calls
    layer.backward(torch.randn(5, N), y)
    assert [name for name, _ in calls] == ["quantize_grad", "gemm", "gemm"]


def held(layer):
    """Bytes of the tensors that the layer keeps, besides what it was given."""
    seen, stack, total = set(), [layer], 0
    while stack:
        o = stack.pop()
        if id(o) in seen or o is layer.weight or o is layer.bias:
            continue
        seen.add(id(o))
        if isinstance(o, torch.Tensor):
            total += o.numel() * o.element_size()
        elif isinstance(o, dict):
            stack.extend(o.values())
        elif isinstance(o, (list, tuple)):
            stack.extend(o)
        elif type(o).__module__ == mxfp4_layer.__name__:
            stack.extend(getattr(o, n, None) for n in (*vars(o), *getattr(type(o), "__slots__", ())))
    return total


def test_many_sizes_do_not_fill_the_memory(calls):
    layer = Mxfp4Layer(torch.randn(K, N))
    weights = held(layer)
    most = 0
    layer.backward(torch.randn(200, N), layer.forward(torch.randn(200, K)))  # the largest size
    one = held(layer) - weights
    for M in range(1, 201):
        layer.backward(torch.randn(M, N), layer.forward(torch.randn(M, K)))
        most = max(most, held(layer) - weights)
    assert 0 < one and most <= 4 * one


def test_a_few_sizes_may_be_under_way_at_once(calls):
    layer = Mxfp4Layer(torch.randn(K, N))
    sizes = (5, 17, 130, 40)
    outs = [layer.forward(torch.randn(M, K)) for M in sizes]
    for y in outs:
        del calls[:]
        layer.backward(torch.randn(len(y), N), y)
        assert calls.named("gemm")[1][3] == len(y)


def test_an_output_whose_tokens_were_replaced_is_refused(calls):
    layer = Mxfp4Layer(torch.randn(K, N))
    first = layer.forward(torch.randn(5, K))
    second = layer.forward(torch.randn(5, K))
    del calls[:]
    with pytest.raises(ValueError):
        layer.backward(torch.randn(5, N), first)
    assert not calls
    layer.backward(torch.randn(5, N), second)
    layer.backward(torch.randn(5, N), second.detach())
    assert len(calls) == 6


def test_forwards_kept_by_the_caller(calls):
    # several forwards of one size before their backwards, each with tokens of its own
    layer = Mxfp4Layer(torch.randn(K, N))
    outs, saved = [], []
    for M in (5, 5, 9, 5):
        outs.append(layer.forward(torch.randn(M, K)))
        saved.append(layer.saved)
    addresses = []
    for y, s in zip(outs, saved):
        del calls[:]
        layer.backward(torch.randn(len(y), N), y.clone(), s)  # (a copy of the output will do then)
        addresses.append(calls.named("gemm")[1][5].data_ptr())
    assert len(set(addresses)) == 4
    del calls[:]
    layer.forward(torch.randn(5, K))
    assert calls.named("quantize")[0][8].data_ptr() not in addresses
    for wrong in (saved[2], object()):
        with pytest.raises(ValueError):
            layer.backward(torch.randn(5, N), outs[0], wrong)
    other = Mxfp4Layer(torch.randn(K, N))
    with pytest.raises(ValueError):  # another layer's tokens
        other.backward(torch.randn(5, N), outs[0], saved[0])


def test_without_relu_no_output_is_needed(calls):
    layer = Mxfp4Layer(torch.randn(K, N), relu=False)
    first = layer.forward(torch.randn(5, K))
    layer.backward(torch.randn(5, N), None)
    layer.forward(torch.randn(5, K))
    with pytest.raises(ValueError):
        layer.backward(torch.randn(5, N), first)


def test_no_tokens_leave_nothing(calls):
    layer = Mxfp4Layer(torch.randn(K, N))
    layer.forward(torch.randn(5, K))
    y = layer.forward(torch.empty(0, K))
    assert layer.saved is None
    dx, dw, db = layer.backward(torch.empty(0, N), y, layer.saved)
    assert dx.shape == (0, K) and not dw.any() and not db.any()
