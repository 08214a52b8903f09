"""DualWeightGlu as torch drives it: gradients of any layout, forward mode, traces
and compiled functions, on both sides of the change from glu_gemv to glu_gemm."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import memory_bound_glu_gb300 as mb
from test_glu_gemm_gpu import BF, DEV, backward_reference, operands, rand
import dense_ref as R

pytestmark = pytest.mark.gpu
ROWS = [33, 100]


def leaves_of(ops):
    return [t.clone().requires_grad_(True) for t in ops]


@pytest.mark.parametrize("M", [1, *ROWS])
@pytest.mark.parametrize("N", [1, 2, 40])
@pytest.mark.parametrize("layout", ["rows", "columns", "strided", "broadcast", "row of any stride"])
def test_gradients_of_any_layout(M, N, layout):
    """What arrives at the node is the caller's tensor: a transposed one, one column of
    a wider matrix, a single value for all."""
    K = 48
    ops = operands(M, N, K, seed=M + N)
    if layout == "columns":
        d = rand(N, M, seed=7).t()
    elif layout == "strided":
        d = rand(M, 2 * N, seed=7)[:, ::2]
    elif layout == "row of any stride":
        d = rand(M, N, seed=7).as_strided((M, N), (1, 1)) if M == 1 else rand(M, N, seed=7)
    elif layout == "broadcast":
        d = rand(1, 1, seed=7).expand(M, N)
    else:
        d = rand(M, N, seed=7)
    leaves = leaves_of(ops)
    got = torch.autograd.grad(mb.DualWeightGlu.apply(*leaves), leaves, d)
    for name, x, (ref, err) in zip(("grad_h", "grad_gate", "grad_up"), got, backward_reference(*ops, d)):
        R.assert_bf16(x, ref, err, name)
    assert mb.read_device_error() == 0


@pytest.mark.parametrize("M", ROWS)
def test_a_column_through_a_transposed_product(M):
    ops = operands(M, 1, 48, seed=M)
    w = rand(1, M, seed=8)
    leaves = leaves_of(ops)
    (mb.DualWeightGlu.apply(*leaves).t() * w).sum().backward()
    for t, (ref, err) in zip(leaves, backward_reference(*ops, w.t())):
        R.assert_bf16(t.grad, ref, err)


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("grad", [False, True])
def test_forward_mode_is_refused(M, grad):
    h, gw, uw = operands(M, 24, 16, seed=M)
    gw.requires_grad_(grad)
    with fwd.dual_level():
        with pytest.raises((NotImplementedError, RuntimeError), match="jvp"):
            mb.DualWeightGlu.apply(fwd.make_dual(h, torch.ones_like(h)), gw, uw)


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("grad", [False, True])
def test_trace_and_compile(M, grad):
    def f(h, gw, uw):
        return mb.DualWeightGlu.apply(h, gw, uw) * 2

    first, then = operands(M, 24, 16, seed=1), operands(M, 24, 16, seed=2)
    d = rand(M, 24, seed=3)
    runs = [torch.jit.trace(f, tuple(leaves_of(first) if grad else first), check_trace=False)]
    torch._dynamo.reset()
    runs.append(torch.compile(f, backend="eager"))
    for run in runs:
        for ops in (first, then):
            assert torch.equal(run(*ops), f(*ops))
            leaves, plain = leaves_of(ops), leaves_of(ops)
            out, want = run(*leaves), f(*plain)
            assert torch.equal(out, want)
            assert all(torch.equal(a, b) for a, b in zip(torch.autograd.grad(out, leaves, d), torch.autograd.grad(want, plain, d)))
    torch._dynamo.reset()
