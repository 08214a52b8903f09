"""DualWeightGlu as torch drives it: gradients of any layout, forward mode, traces
and compiled functions, on both sides of the change from glu_gemv to glu_gemm."""
import pytest
import torch
import torch.autograd.forward_ad as fwd
import torch.utils.checkpoint

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


@pytest.mark.parametrize("M", ROWS)
def test_saved_tensors_elsewhere_and_computed_again(M):
    """Saved tensors on the host, and a forward that is run again in the backward."""
    ops, d = operands(M, 40, 48, seed=M), rand(M, 40, seed=9)
    leaves = leaves_of(ops)
    want = torch.autograd.grad(mb.DualWeightGlu.apply(*leaves), leaves, d)
    with torch.autograd.graph.save_on_cpu():
        out = mb.DualWeightGlu.apply(*leaves)
    runs = [torch.autograd.grad(out, leaves, d)]
    for reentrant in (False, True):
        out = torch.utils.checkpoint.checkpoint(mb.DualWeightGlu.apply, *leaves, use_reentrant=reentrant)
        for t in leaves:
            t.grad = None
        out.backward(d)   # a reentrant checkpoint takes no other call
        runs.append([t.grad for t in leaves])
    for got in runs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("which", [0, 1, 2])
def test_an_operand_changed_before_the_backward_is_an_error(M, which):
    leaves = leaves_of(operands(M, 40, 48, seed=M))
    out = mb.DualWeightGlu.apply(*leaves)
    with torch.no_grad():
        leaves[which].add_(1)
    with pytest.raises(RuntimeError, match="inplace"):
        out.sum().backward()


@pytest.mark.parametrize("M", ROWS)
def test_used_twice_and_kept(M):
    """Gradients of two uses of the same weights add up; a kept graph gives the same again
    and a freed one is an error."""
    ops, d = operands(M, 40, 48, seed=M), rand(M, 40, seed=9)
    leaves = leaves_of(ops)
    h = leaves[0]
    out = mb.DualWeightGlu.apply(h, leaves[1], leaves[1]) + mb.DualWeightGlu.apply(h, leaves[1], leaves[2])
    one = torch.autograd.grad(out, leaves, d, retain_graph=True)
    two = torch.autograd.grad(out, leaves, d)
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    first = backward_reference(ops[0], ops[1], ops[1], d)
    second = backward_reference(*ops, d)
    for got, terms in zip(one, ([first[0], second[0]], [first[1], first[2], second[1]], [second[2]])):
        # each term rounds to bf16, and so may each partial sum of them
        ref, err = sum(t[0] for t in terms), sum(t[1] + R.EPS_BF16 * (t[0].abs() + t[1]) for t in terms)
        for _ in terms[1:]:
            err = err + R.EPS_BF16 * (sum(t[0].abs() for t in terms) + err)
        assert ((got.double() - ref).abs() <= err + 1e-37).all()
    with pytest.raises(RuntimeError, match="second time"):
        torch.autograd.grad(out, leaves, d)
