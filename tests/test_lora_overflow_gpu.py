"""glu_lora and linear_lora where p = scale (x A^T) leaves bf16's range or fp32's: p is carried
as two bf16 terms on the tensor cores, and neither may turn a large number or an infinity
into NaN.  In blocks of rows with one adapter, with several, and in small batches."""
import pytest
import torch

import dense_ref as R
import memory_bound_glu_gb300 as mb
import rows_ref as Q

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
LARGEST = 3.3895313892515355e38   # of bf16


def rand(*shape, seed=0, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(BF)


def operands(M, r, sides, how, N=264, K=136, L=4):
    """B is small and nowhere 0, so that a large p leaves finite outputs."""
    g = torch.Generator(device=DEV).manual_seed(M + r)
    x, w = rand(M, K, seed=M), [rand(N, K, seed=M + 1 + i, scale=K ** -0.5) for i in range(sides)]
    a = [rand(L, r, K, seed=M + 5 + i, scale=K ** -0.5) for i in range(sides)]
    b = [torch.where(torch.rand(L, N, r, generator=g, device=DEV) < 0.5, -1.0, 1.0).to(BF) * 2.0 ** -120 * (1 + torch.rand(L, N, r, generator=g, device=DEV)).to(BF)
         for i in range(sides)]
    if how == "one":   # blocks of one adapter, the broken one's among them
        idx = torch.full((M,), 2, dtype=torch.int32, device=DEV)
        idx[:M // 3] = 1
    else:
        idx = (torch.arange(M, device=DEV) % (L + 1) - 1).int()
    return x, w, a, b, idx, torch.ones(L, device=DEV)


def call(x, w, a, b, idx, scale):
    if len(w) == 2:
        return mb.glu_lora(x, *w, a[0], b[0], a[1], b[1], idx, scale)
    return mb.linear_lora(x, *w, a[0], b[0], idx, scale)


# by rank and rows: the tensor cores of the pair with p of either kernel, those of single warps, rows of B by lanes, the join
SHAPES = [(1, 16), (20, 16), (20, 64), (100, 16), (100, 24), (300, 64), (333, 16), (700, 16), (700, 40), (1100, 128)]


@pytest.mark.parametrize("how", ["one", "several"])
@pytest.mark.parametrize("sides", [1, 2])
@pytest.mark.parametrize("M,r", SHAPES)
def test_p_beyond_bf16(M, r, sides, how):
    """p of 3.397e38 to 3.40e38 is finite in fp32 and infinite in bf16."""
    x, w, a, b, idx, scale = operands(M, r, sides, how)
    x[:, 0] = 1.0
    for t in a:
        t[2, r // 2] = 0
        t[2, r // 2, 0] = LARGEST
    scale[2] = 1.003   # 3.3997e38: fp32 ends at 3.4028e38
    got = call(x, w, a, b, idx, scale)
    assert torch.isfinite(got).all()
    if sides == 2:
        Q.assert_glu_lora(got, (x, *w, a[0], b[0], a[1], b[1], idx, scale))
    else:
        R.assert_bf16(got, *Q.adapted(x, w[0], a[0], b[0], idx, scale))


@pytest.mark.parametrize("how", ["one", "several"])
@pytest.mark.parametrize("M,r", SHAPES)
def test_infinite_p(M, r, how):
    """One infinite p and a B without zeros: the row is infinite with the signs of p and B, and no
    other row changes."""
    x, w, a, b, idx, scale = operands(M, r, 1, how)
    x[:, 0] = torch.where(torch.arange(M, device=DEV) % 2 == 0, 1.0, -1.0)
    scale[2] = 4.0
    for t in (w[0], a[0]):
        t[..., 0] = 0
    plain = call(x, w, a, b, idx, scale)
    a[0][2, r - 1] = 0
    a[0][2, r - 1, 0] = LARGEST   # four times that overflows
    got = call(x, w, a, b, idx, scale)
    hit = idx == 2
    assert torch.equal(got[~hit], plain[~hit])
    want = torch.where(x[hit, :1] > 0, 1.0, -1.0) * torch.sign(b[0][2, :, r - 1].float())[None, :]
    assert torch.isinf(got[hit]).all() and torch.equal(torch.sign(got[hit].float()), want)


@pytest.mark.parametrize("how", ["one", "several"])
@pytest.mark.parametrize("sides", [1, 2])
@pytest.mark.parametrize("M,r", SHAPES)
def test_an_infinite_element_of_b(M, r, sides, how):
    """It reaches the column that it belongs to, of its adapter's rows, which is not finite then; and
    an infinite p with two projections reaches its own rows."""
    x, w, a, b, idx, scale = operands(M, r, sides, how)
    for i in range(sides):
        b[i] = rand(*b[i].shape, seed=M + 20 + i, scale=r ** -0.5)
    plain = call(x, w, a, b, idx, scale)
    hit = idx == 2
    b[-1][2, 77, r - 1] = float("inf")
    got = call(x, w, a, b, idx, scale)
    assert not torch.isfinite(got[hit][:, 77]).any()
    got[:, 77] = plain[:, 77]
    assert torch.equal(got, plain)
    b[-1][2, 77, r - 1] = 1
    x[:, 0], scale[2] = 1.0, 4.0
    for t in (*w, *a):
        t[..., 0] = 0
    plain = call(x, w, a, b, idx, scale)
    a[-1][2, 0, 0] = LARGEST
    got = call(x, w, a, b, idx, scale)
    assert not torch.isfinite(got[hit]).any() and torch.equal(got[~hit], plain[~hit])
