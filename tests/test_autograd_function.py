"""DualWeightGlu under torch's own machinery -- forward-mode differentiation,
tracing, function transforms -- without a GPU: the library's calls are replaced by
ones that write their output where torch does not see it, as the library does."""
import ctypes

import numpy as np
import pytest
import torch
import torch.autograd.forward_ad as fwd

import memory_bound_glu_gb300 as mb
from memory_bound_glu_gb300 import binding

ROWS = [1, 64, 65, 130]   # around the change from glu_gemv to glu_gemm
K, N = 5, 3


def _array(t):
    """t's memory as numpy sees it (row-major, fp32)."""
    return np.ctypeslib.as_array((ctypes.c_float * t.numel()).from_address(t.data_ptr())).reshape(tuple(t.shape))


def _glu(h, gate_w, up_w):
    g, u = (_array(h).astype(np.float64) @ _array(w).astype(np.float64).T for w in (gate_w, up_w))
    return (g / (1 + np.exp(-g)) * u).astype(np.float32)


@pytest.fixture
def calls(monkeypatch):
    """The forward calls that were made: (name, whether g and u are kept)."""
    made = []

    def forward(name):
        def call(h, gate_w, up_w, out=None, mode="fused", gu=None, stream=None):
            made.append((name, gu is not None))
            out = torch.empty((h.shape[0], gate_w.shape[0]))
            _array(out)[:] = _glu(h, gate_w, up_w)
            return out
        return call

    class Quick:   # the extension module: its node is invisible to the tracer
        @staticmethod
        def wide_glu(h, gate_w, up_w, mode):
            made.append(("wide_glu", True))
            out = torch.empty((h.shape[0], gate_w.shape[0]))
            _array(out)[:] = _glu(h, gate_w, up_w)
            return out.requires_grad_(True)

    monkeypatch.setattr(binding, "glu_gemv", forward("glu_gemv"))
    monkeypatch.setattr(binding, "glu_gemm", forward("glu_gemm"))
    monkeypatch.setattr(binding, "_quick_module", Quick)
    return made


def operands(M, seed=0, grad=False):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(*s, generator=g).requires_grad_(grad) for s in ((M, K), (N, K), (N, K))]


def right(out, ops):
    want = _glu(*(t.detach() for t in ops))
    return np.array_equal(_array(out.detach()), want)


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("grad", [False, True])
def test_values_and_what_is_kept(calls, M, grad):
    ops = operands(M, grad=grad)
    out = mb.DualWeightGlu.apply(*ops)
    assert right(out, ops) and out.requires_grad == grad
    wide = ("wide_glu", True) if grad else ("glu_gemm", False)
    assert calls == [wide if M > mb.MAX_M else ("glu_gemv", False)]
    del calls[:]
    with torch.no_grad():
        out = mb.DualWeightGlu.apply(*ops, mode="hf")
    assert right(out, ops) and not out.requires_grad
    assert calls == [("glu_gemm" if M > mb.MAX_M else "glu_gemv", False)]   # nothing is kept for a backward


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("which", [0, 1, 2])
def test_forward_mode_is_refused(calls, M, which):
    """There is no forward-mode derivative: a dual operand is an error, not a zero tangent."""
    ops = operands(M)
    with fwd.dual_level():
        ops[which] = fwd.make_dual(ops[which], torch.ones_like(ops[which]))
        with pytest.raises((NotImplementedError, RuntimeError), match="jvp"):
            mb.DualWeightGlu.apply(*ops)


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("mode", ["fused", "hf"])
def test_a_trace_computes_again(calls, M, grad, mode):
    """A traced call computes on the inputs that it is given, with and without gradients."""
    traced = torch.jit.trace(lambda *a: mb.DualWeightGlu.apply(*a, mode), tuple(operands(M, grad=grad)), check_trace=False)
    for seed, again in ((1, False), (2, grad)):
        ops = operands(M, seed=seed, grad=again)
        before = len(calls)
        out = traced(*ops)
        assert len(calls) > before, "the trace does not call the operator"
        assert right(out, ops) and out.requires_grad == again


@pytest.mark.parametrize("M", ROWS)
def test_function_transforms_are_refused(calls, M):
    h, gate_w, up_w = operands(M)
    with pytest.raises(RuntimeError):
        torch.func.grad(lambda x: mb.DualWeightGlu.apply(x, gate_w, up_w).sum())(h)
    with pytest.raises(RuntimeError):
        torch.func.vmap(lambda x: mb.DualWeightGlu.apply(x, gate_w, up_w))(torch.stack([h, h]))


@pytest.mark.parametrize("M", [4, 100])
@pytest.mark.parametrize("grad", [False, True])
def test_inside_a_compiled_function(calls, M, grad):
    torch._dynamo.reset()
    f = torch.compile(lambda *a: mb.DualWeightGlu.apply(*a) * 2, backend="eager")
    for seed in (0, 1):
        ops = operands(M, seed=seed, grad=grad)
        out = f(*ops)
        assert right(out / 2, ops) and out.requires_grad == grad
        with torch.no_grad():
            assert right(f(*ops) / 2, ops)
    torch._dynamo.reset()
