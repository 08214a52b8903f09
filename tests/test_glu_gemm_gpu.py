"""glu_gemm and glu_gemm_backward against the definitions in 64 bits: sizes
around the tiles' edges, strides and alignments, g and u handed out, subsets of
the gradients, differences, streams and graphs."""
import pytest
import torch

import dense_ref as R
import memory_bound_glu_gb300 as mb

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def rand(*shape, seed=0, scale=1.0, pad=0, off=0):
    """bf16 normal values; pad: extra columns behind each row, off: first column of the view."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    t = (torch.randn(*shape[:-1], shape[-1] + pad + off, generator=g, device=DEV) * scale).to(BF)
    return t[..., off:off + shape[-1]]


def operands(M, N, K, seed=0, pad=0, off=0):
    return (rand(M, K, seed=seed, pad=pad, off=off), rand(N, K, seed=seed + 1, scale=K ** -0.5, pad=pad, off=off),
            rand(N, K, seed=seed + 2, scale=K ** -0.5, pad=pad, off=off))


def check_forward(h, gw, uw, mode="fused", gu=False, out=None):
    M, N = h.shape[0], gw.shape[0]
    buf = torch.full((M, 2 * N), float("nan"), device=DEV) if gu else None
    out = mb.glu_gemm(h, gw, uw, out=out, mode=mode, gu=buf)
    g, u, eg, eu = R.glu(h.double(), gw.double(), uw.double())
    if mode == "fused":
        R.assert_bf16(out, *R.glu_out(g, u, eg, eu), "out")
    else:
        # g, u and SiLU(g) round to bf16 too: 2^-8 of each more
        eg, eu = eg + R.EPS_BF16 * (g.abs() + eg), eu + R.EPS_BF16 * (u.abs() + eu)
        v, e = R.glu_out(g, u, eg, eu)
        R.assert_bf16(out, v, e + R.EPS_BF16 * (v.abs() + e), "out (hf)")
    if gu:
        for got, ref, err in ((buf[:, :N], g, eg), (buf[:, N:], u, eu)):
            assert ((got.double() - ref).abs() <= err + 2.0 ** -23 * ref.abs()).all()
    assert mb.read_device_error() == 0
    return out


@pytest.mark.parametrize("M", [65, 127, 128, 129, 255, 256, 257, 300, 700])
def test_rows_around_the_tiles(M):
    check_forward(*operands(M, 200, 136, seed=M))


@pytest.mark.parametrize("N", [1, 2, 31, 32, 33, 64, 127, 128, 129, 257, 1000])
def test_columns_around_the_tiles(N):
    check_forward(*operands(100, N, 72, seed=N), gu=True)


@pytest.mark.parametrize("K", [1, 7, 8, 16, 63, 64, 65, 128, 500, 2568])
def test_inner_dimension(K):
    check_forward(*operands(90, 136, K, seed=K))


@pytest.mark.parametrize("M,N,K,pad,variant", [(2000, 4801, 1104, 0, 11), (2001, 4864, 1099, 5, 11), (1000, 9728, 2048, 0, 11),
                                               (2000, 4800, 1100, 3, 12)])
def test_each_kernel(M, N, K, pad, variant):
    """Sizes that each of the kernels takes: CTA pairs (several rounds, ragged in
    every dimension), any alignment."""
    h, gw, uw = operands(M, N, K, seed=M, pad=pad)
    if variant == 12:
        h, gw, uw = h[:100], gw[:200], uw[:200]   # the slow kernel: a corner of it
    check_forward(h, gw, uw)
    assert mb.last_variant() == variant
    if variant != 12:
        check_forward(h, gw, uw, mode="hf", gu=True)


# tiles of 32 to 224 tokens and of 80, 96 and 128 outputs, several rounds of them, ragged
# in every dimension; (1100, ..) and (2100, ..) with 256 rows
@pytest.mark.parametrize("M,N,K", [(479, 520, 2048), (459, 1000, 152), (289, 2500, 352), (330, 2500, 1064), (160, 9729, 1000),
                                   (565, 2500, 1528), (333, 9728, 2560), (400, 9730, 2568), (66, 14336, 264), (1100, 2500, 136),
                                   (2100, 1300, 264), (17, 11008, 1096), (100, 10999, 2056), (130, 6999, 2056), (66, 13000, 1032),
                                   (333, 3300, 2056), (200, 300, 4096)])
@pytest.mark.parametrize("mode", ["fused", "hf"])
def test_tiles_of_tokens(M, N, K, mode):
    check_forward(*operands(M, N, K, seed=M), mode=mode)
    assert mb.last_variant() == 11


@pytest.mark.parametrize("mode", ["fused", "hf"])
@pytest.mark.parametrize("M", [1, 2, 16, 17, 31, 33, 40, 64])
@pytest.mark.parametrize("N,K", [(136, 264), (2500, 1000), (1, 8), (129, 4104)])
def test_few_rows(M, N, K, mode):
    ops = operands(M, N, K, seed=M)
    out = check_forward(*ops, mode=mode)
    assert (mb.last_variant() == 11) == (M > 16)
    if M <= 16:
        assert torch.equal(out, mb.glu_gemv(*ops, mode=mode))
    check_forward(*ops, mode=mode, gu=True)


@pytest.mark.parametrize("M", [17, 64])
def test_few_rows_of_any_alignment(M):
    ops = operands(M, 136, 264, seed=M, pad=1)
    assert torch.equal(check_forward(*ops), mb.glu_gemv(*ops))


@pytest.mark.parametrize("mode", ["fused", "hf"])
@pytest.mark.parametrize("pad,off", [(8, 0), (8, 8), (1, 0), (3, 2), (5, 1)])
def test_strides_and_alignment(mode, pad, off):
    h, gw, uw = operands(130, 96, 152, seed=pad + 10 * off, pad=pad, off=off)
    check_forward(h, gw, uw, mode=mode)


@pytest.mark.parametrize("M,N,K", [(130, 100, 64), (1100, 2500, 136)])
@pytest.mark.parametrize("pad", [0, 1, 8, 24])
def test_output_stride_and_what_lies_behind(pad, M, N, K):
    h, gw, uw = operands(M, N, K, seed=pad)
    whole = torch.full((M + 1, N + pad), 7.0, dtype=BF, device=DEV)
    check_forward(h, gw, uw, out=whole[:M, :N])
    assert (whole[:M, N:] == 7).all() and (whole[M] == 7).all()


def test_empty():
    h, gw, uw = operands(70, 24, 16)
    assert mb.glu_gemm(h[:0], gw, uw).shape == (0, 24)
    assert mb.glu_gemm(h, gw[:0], uw[:0]).shape == (70, 0)
    gu = torch.full((70, 48), 3.0, device=DEV)
    out = mb.glu_gemm(h[:, :0], gw[:, :0], uw[:, :0], gu=gu)
    assert (out == 0).all() and (gu == 0).all()


def test_outliers_and_nan_stay_in_their_row():
    h, gw, uw = operands(200, 136, 256, seed=4)
    base = mb.glu_gemm(h, gw, uw)
    h2 = h.clone()
    h2[77, 5] = float("nan")
    h2[100] = h2[100] * 1e30
    out = mb.glu_gemm(h2, gw, uw)
    rows = [i for i in range(200) if i not in (77, 100)]
    assert torch.equal(out[rows], base[rows]) and out[77].isnan().all()


def test_large_negative_gate():
    h, gw, uw = operands(80, 64, 64, seed=9)
    check_forward(h * 30, gw, uw)


def backward_reference(h, gw, uw, d):
    """The three gradients in 64 bits and their bounds before the last rounding."""
    h, gw, uw, d = (t.double() for t in (h, gw, uw, d))
    g, u, eg, eu = R.glu(h, gw, uw)
    dg, du = d * u * R.dsilu(g), d * R.silu(g)
    # |SiLU'| <= 1.1, |SiLU''| <= 0.5; dG and dU round to bf16
    edg = d.abs() * (0.5 * eg * (u.abs() + eu) + 1.1 * eu) + 2.0 ** -20 * (dg.abs() + d.abs() * u.abs() * 2.0 ** -3)
    edu = d.abs() * 1.1 * eg + 2.0 ** -20 * du.abs()
    edg, edu = edg + R.EPS_BF16 * (dg.abs() + edg), edu + R.EPS_BF16 * (du.abs() + edu)
    M, N = d.shape
    gh = dg @ gw + du @ uw
    egh = (edg + R.acc(2 * N) * dg.abs()) @ gw.abs() + (edu + R.acc(2 * N) * du.abs()) @ uw.abs()
    ggw, egw = dg.T @ h, (edg + R.acc(M) * dg.abs()).T @ h.abs()
    guw, euw = du.T @ h, (edu + R.acc(M) * du.abs()).T @ h.abs()
    return (gh, egh), (ggw, egw), (guw, euw)


def check_backward(h, gw, uw, d, gu=False, **kw):
    buf = None
    if gu:
        buf = torch.empty((h.shape[0], 2 * gw.shape[0]), device=DEV)
        mb.glu_gemm(h, gw, uw, gu=buf)
    got = mb.glu_gemm_backward(h, gw, uw, d, gu=buf, **kw)
    for name, x, (ref, err) in zip(("grad_h", "grad_gate", "grad_up"), got, backward_reference(h, gw, uw, d)):
        if x is not None:
            R.assert_bf16(x, ref, err, name)
            # the errors are independent: in the 2-norm two roundings of half a step at most
            rel = (x.double() - ref).norm() / ref.norm()
            assert rel <= 2 * R.EPS_BF16, (name, rel.item())
    assert mb.read_device_error() == 0
    return got


@pytest.mark.parametrize("gu", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (3, 40, 24), (65, 136, 72), (64, 64, 64), (128, 128, 256), (257, 264, 136),
                                   (300, 1000, 520), (33, 1, 9), (100, 77, 51), (70, 129, 257), (520, 56, 64),
                                   (2000, 4801, 1104)])
def test_backward_sizes(M, N, K, gu):
    h, gw, uw = operands(M, N, K, seed=M + N)
    check_backward(h, gw, uw, rand(M, N, seed=5), gu=gu)


@pytest.mark.parametrize("pad,off", [(8, 0), (8, 8), (1, 0), (3, 2)])
def test_backward_strides(pad, off):
    h, gw, uw = operands(100, 96, 88, seed=pad, pad=pad, off=off)
    d = rand(100, 96, seed=6, pad=pad, off=off)
    outs = [torch.full((n + 1, 88 + pad), 7.0, dtype=BF, device=DEV) for n in (100, 96, 96)]
    check_backward(h, gw, uw, d, grad_h=outs[0][:100, :88], grad_gate=outs[1][:96, :88], grad_up=outs[2][:96, :88])
    for t in outs:
        assert (t[-1] == 7).all() and (t[:, 88:] == 7).all()


def test_backward_subsets():
    h, gw, uw = operands(90, 72, 80)
    d = rand(90, 72, seed=8)
    whole = check_backward(h, gw, uw, d)
    a = mb.glu_gemm_backward(h, gw, uw, d, want_w=False)
    b = mb.glu_gemm_backward(h, gw, uw, d, want_h=False)
    assert a[1] is None and a[2] is None and b[0] is None
    assert torch.equal(a[0], whole[0]) and torch.equal(b[1], whole[1]) and torch.equal(b[2], whole[2])
    assert mb.glu_gemm_backward(h, gw, uw, d, want_h=False, want_w=False) == (None, None, None)


def test_backward_empty():
    h, gw, uw = operands(66, 24, 16)
    d = rand(66, 24)
    gh, gg, gu = mb.glu_gemm_backward(h[:0], gw, uw, d[:0])
    assert gh.shape == (0, 16) and (gg == 0).all() and (gu == 0).all()
    gh, gg, gu = mb.glu_gemm_backward(h, gw[:0], uw[:0], d[:, :0])
    assert (gh == 0).all() and gg.shape == (0, 16)


def test_autograd_follows_differences():
    """Central differences of <out, d> in 64 bits along random directions against the
    gradients that autograd returns: two bf16 roundings of each gradient element at most."""
    M, N, K = 80, 48, 40
    h, gw, uw = (t.clone().requires_grad_(True) for t in operands(M, N, K, seed=3))
    d = rand(M, N, seed=4)
    out = mb.DualWeightGlu.apply(h, gw, uw)
    assert torch.equal(out, mb.glu_gemm(h.detach(), gw.detach(), uw.detach()))
    grads = torch.autograd.grad(out, (h, gw, uw), d)
    refs = backward_reference(h.detach(), gw.detach(), uw.detach(), d)
    f = lambda *a: (R.silu(a[0] @ a[1].T) * (a[0] @ a[2].T) * d.double()).sum()  # noqa: E731
    base = [t.detach().double() for t in (h, gw, uw)]
    for i, (grad, (_, err)) in enumerate(zip(grads, refs)):
        v = torch.randn(base[i].shape, generator=torch.Generator(device=DEV).manual_seed(i), device=DEV, dtype=torch.float64)
        t = 1e-5
        plus, minus = list(base), list(base)
        plus[i], minus[i] = base[i] + t * v, base[i] - t * v
        diff = (f(*plus) - f(*minus)) / (2 * t)
        got = (grad.double() * v).sum()
        bound = ((err + R.EPS_BF16 * (grad.double().abs() + err)) * v.abs()).sum() + 1e-6 * diff.abs()
        assert (got - diff).abs() <= bound


def test_autograd_subsets_and_broadcast_gradient():
    h, gw, uw = operands(100, 64, 48, seed=11)
    for need in ((True, False, False), (False, True, False), (False, False, True)):
        leaves = [t.clone().requires_grad_(n) for t, n in zip((h, gw, uw), need)]
        mb.DualWeightGlu.apply(*leaves).float().sum().backward()   # the gradient of a sum is a broadcast
        want = backward_reference(h, gw, uw, torch.ones(100, 64, device=DEV, dtype=BF))
        for t, n, (ref, err) in zip(leaves, need, want):
            assert (t.grad is not None) == n
            if n:
                R.assert_bf16(t.grad, ref, err)
    col = [t.clone().requires_grad_(True) for t in (h, gw, uw)]
    out = mb.DualWeightGlu.apply(*col)
    (gh,) = torch.autograd.grad(out, col[0], torch.ones(1, 64, device=DEV, dtype=BF).expand(100, 64))
    R.assert_bf16(gh, *backward_reference(h, gw, uw, torch.ones(100, 64, device=DEV, dtype=BF))[0])


@pytest.mark.parametrize("M", [40, 100])
def test_a_second_derivative_is_an_error(M):
    """create_graph gives the first derivative; its own is refused, not taken as zero."""
    leaves = [t.requires_grad_(True) for t in operands(M, 64, 48, seed=11)]
    plain = torch.autograd.grad(mb.DualWeightGlu.apply(*leaves).float().square().sum(), leaves)
    first = torch.autograd.grad(mb.DualWeightGlu.apply(*leaves).float().square().sum(), leaves, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(plain, first))
    for g in first:
        with pytest.raises(RuntimeError):
            g.float().square().sum().backward(retain_graph=True)


def test_deterministic_and_rows_independent():
    h, gw, uw = operands(300, 264, 200, seed=12)
    a, b = mb.glu_gemm(h, gw, uw), mb.glu_gemm(h, gw, uw)
    assert torch.equal(a, b)
    perm = torch.randperm(300, generator=torch.Generator().manual_seed(0)).to(DEV)
    assert torch.equal(mb.glu_gemm(h[perm], gw, uw), a[perm])
    d = rand(300, 264, seed=13)
    for x, y in zip(mb.glu_gemm_backward(h, gw, uw, d), mb.glu_gemm_backward(h, gw, uw, d)):
        assert torch.equal(x, y)


def test_other_stream_and_graph():
    h, gw, uw = operands(200, 136, 128, seed=14)
    d = rand(200, 136, seed=15)
    want, grads = mb.glu_gemm(h, gw, uw), mb.glu_gemm_backward(h, gw, uw, d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = mb.glu_gemm(h, gw, uw, stream=s)
    got = mb.glu_gemm_backward(h, gw, uw, d, stream=s)
    s.synchronize()
    assert torch.equal(out, want) and all(torch.equal(x, y) for x, y in zip(got, grads))
    out.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mb.glu_gemm(h, gw, uw, out=out)
        got = mb.glu_gemm_backward(h, gw, uw, d)
    h2 = rand(200, 128, seed=99)
    keep = h.clone()
    h.copy_(h2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, mb.glu_gemm(h2, gw, uw))
    assert all(torch.equal(x, y) for x, y in zip(got, mb.glu_gemm_backward(h2, gw, uw, d)))
    h.copy_(keep)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_apply_without_gradients_keeps_nothing():
    h, gw, uw = operands(300, 520, 64, seed=20)
    want = mb.glu_gemm(h, gw, uw)
    leaves = [t.clone().requires_grad_(True) for t in (gw, uw)]
    with torch.no_grad():
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        out = mb.DualWeightGlu.apply(h, *leaves)
        assert torch.cuda.memory_allocated() - before < 300 * 520 * 8   # out, no g and u
    assert torch.equal(out, want) and not out.requires_grad
    assert torch.equal(mb.DualWeightGlu.apply(h, gw, uw), want)
    assert torch.equal(mb.DualWeightGlu.apply(h[:5], gw, uw), mb.glu_gemv(h[:5], gw, uw))
    assert mb.DualWeightGlu.apply(h, *leaves).requires_grad


def test_training_step_in_a_graph():
    """Forward and backward captured together, replayed on new values."""
    ops = operands(200, 136, 72, seed=21)
    d = rand(200, 136, seed=22)
    leaves = [t.clone().requires_grad_(True) for t in ops]

    def step():
        out = mb.DualWeightGlu.apply(*leaves)
        return (out.detach(), *torch.autograd.grad(out, leaves, d))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    new = operands(200, 136, 72, seed=23)
    with torch.no_grad():
        for t, n in zip(leaves, new):
            t.copy_(n)
    g.replay()
    torch.cuda.synchronize()
    want = step()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_same_tensor_twice_and_broadcast_rows():
    h, gw, _ = operands(130, 96, 96, seed=24)
    check_forward(h, gw, gw)
    check_forward(h, h[:96], h[:96])
    with pytest.raises(mb.MbgluError):
        mb.glu_gemm(h[:1].expand(130, 96), gw, gw)            # rows of stride 0
    with pytest.raises(mb.MbgluError):
        mb.DualWeightGlu.apply(h[:1].clone().requires_grad_(True).expand(130, 96), gw, gw)
    with pytest.raises(mb.MbgluError):
        mb.glu_gemm(h, gw, gw, out=h[:, :96])                 # in place
    with pytest.raises(ValueError):
        mb.glu_gemm(h.t(), gw[:, :1].expand(96, 130), gw[:, :1].expand(96, 130))


def test_operands_on_the_cpu_or_of_other_types_are_refused():
    h, gw, uw = operands(70, 32, 32)
    for bad in (gw.cpu(), gw.float(), gw[:, :31], gw[0]):
        with pytest.raises((TypeError, ValueError)):
            mb.glu_gemm(h, bad, uw)
    with pytest.raises((TypeError, ValueError)):
        mb.glu_gemm(h, gw, uw, gu=torch.zeros(70, 64, dtype=torch.bfloat16, device=DEV))
    with pytest.raises((TypeError, ValueError)):
        mb.glu_gemm_backward(h, gw, uw, rand(69, 32))
    with pytest.raises(ValueError):
        mb.glu_gemm_backward(h, gw, uw, rand(70, 32), workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    with pytest.raises(mb.MbgluError):
        mb.glu_gemm_backward(h, gw, uw, rand(70, 32), workspace=torch.zeros(256, dtype=torch.uint8, device=DEV))


def test_workspace_and_gu_used_again_by_the_next_step():
    """Training steps back to back through the same g/u buffer and workspace."""
    M, N, K = 300, 264, 136
    steps = [(operands(M, N, K, seed=30 + i), rand(M, N, seed=40 + i)) for i in range(4)]
    want = []
    for (h, gw, uw), d in steps:
        gu = torch.empty(M, 2 * N, device=DEV)
        mb.glu_gemm(h, gw, uw, gu=gu)
        want.append(mb.glu_gemm_backward(h, gw, uw, d, gu=gu))
        torch.cuda.synchronize()
    gu = torch.empty(M, 2 * N, device=DEV)
    ws = torch.empty(mb.glu_gemm_backward_workspace_bytes(M, N, K), dtype=torch.uint8, device=DEV)
    for _ in range(3):
        got = []
        for (h, gw, uw), d in steps:
            mb.glu_gemm(h, gw, uw, gu=gu)
            got.append(mb.glu_gemm_backward(h, gw, uw, d, gu=gu, workspace=ws))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for a, b in zip(got, want) for x, y in zip(a, b))


def far(t, odd=0):
    """t's values in rows so far apart that the last lies beyond 2^31 elements."""
    step = (2 ** 31 // (t.shape[0] - 1) + 64) // 64 * 64 + odd
    v = torch.empty((t.shape[0] - 1) * step + t.shape[1], dtype=t.dtype, device=DEV).as_strided(t.shape, (step, 1))
    assert (t.shape[0] - 1) * step > 2 ** 31 - 64
    return v.copy_(t)


@pytest.mark.parametrize("M,N,K,odd", [(200, 136, 72, 0), (1100, 2500, 136, 0), (90, 40, 24, 1)])
def test_offsets_beyond_32_bits(M, N, K, odd):
    h, gw, uw = (far(t, odd) for t in operands(M, N, K, seed=1))
    out, gu = far(torch.zeros(M, N, dtype=BF, device=DEV), odd), far(torch.zeros(M, 2 * N, device=DEV), odd)
    check_forward(h, gw, uw, out=out)
    mb.glu_gemm(h, gw, uw, gu=gu)
    d = far(rand(M, N, seed=5), odd)
    grads = [far(torch.zeros(n, K, dtype=BF, device=DEV), odd) for n in (M, N, N)]
    kw = dict(zip(("grad_h", "grad_gate", "grad_up"), grads))
    check_backward(h, gw, uw, d, **kw)
    first = [g.clone() for g in grads]
    mb.glu_gemm_backward(h, gw, uw, d, gu=gu, **kw)
    assert all(((a.double() - b.double()).norm() <= 4 * R.EPS_BF16 * a.double().norm()) for a, b in zip(first, grads))
    assert mb.read_device_error() == 0
