"""add_rmsnorm_fp8, quantize_weight_fp8, glu_fp8 and matmul_fp8 against the
definitions in 64 bits, alone and as the chain that a decode step runs."""
import pytest
import torch

import dense_ref as R
import memory_bound_glu_gb300 as mb

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
F8 = torch.float8_e4m3fn
SPLIT = (500, 2560, 8192)   # M, N, K of a product whose inner dimension is split between CTA pairs


def rand(*shape, seed=0, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV) * scale


def strided(t, pad, off=0):
    """t's values in a wider buffer: rows `pad` elements longer, from column `off`."""
    buf = torch.zeros((t.shape[0], t.shape[1] + pad + off), dtype=t.dtype, device=t.device)
    view = buf[:, off:off + t.shape[1]]
    view.copy_(t)
    return view


def activations(M, K, seed=0):
    return R.quantise_rows(rand(M, K, seed=seed).double())


def weight(N, K, seed=0):
    return R.quantise_blocks(rand(N, K, seed=seed, scale=K ** -0.5).double())


def wide_rows(a, s):
    return a.double() * R.spread_rows(s, a.shape[1])


def wide_blocks(w, s):
    return w.double() * R.spread_blocks(s, *w.shape)


def check_norm(x, r, w, eps=1e-6, **kw):
    want = (x.float() + r.float()).to(BF)
    q, s = mb.add_rmsnorm_fp8(x, r, w, eps, **kw)
    got = kw.get("residual_out", r)
    assert torch.equal(got, want)
    v = want.double()
    h = v / torch.sqrt((v * v).mean(1, keepdim=True) + eps) * (1 + w.double())
    # the statistic: a sum of K squares and its root, half the relative error; four more roundings
    K = x.shape[1]
    R.assert_e4m3(q, s, h, h.abs() * (R.acc(K) / 2 + 8 * 2.0 ** -24), "norm")
    return q, s


@pytest.mark.parametrize("M,K", [(1, 1), (1, 8), (1, 127), (2, 128), (3, 129), (1, 2560), (5, 2560), (4, 4096), (2, 5000),
                                 (3, 8192), (2, 8200), (1, 20000), (300, 640), (7, 136)])
def test_norm_sizes(M, K):
    check_norm(rand(M, K, seed=K).to(BF), rand(M, K, seed=K + 1, scale=3).to(BF), rand(K, seed=2, scale=0.1).to(BF))


@pytest.mark.parametrize("pad,off", [(8, 0), (16, 8), (1, 0), (3, 1)])
def test_norm_strides_and_separate_residual(pad, off):
    M, K = 9, 264
    x, r = rand(M, K, seed=1).to(BF), rand(M, K, seed=2).to(BF)
    w = rand(K, seed=3, scale=0.1).to(BF)
    ro = strided(torch.zeros_like(x), pad, off)
    q = strided(torch.zeros(M, K, device=DEV), pad, off).to(F8)
    qbuf = torch.zeros((M, K + pad + off), device=DEV).to(F8)
    q = qbuf[:, off:off + K]
    scale = torch.full((M, 5), 7.0, device=DEV)
    xs, rs = strided(x, pad, off), strided(r, pad, off)
    check_norm(xs, rs, w, residual_out=ro, q=q, scale=scale[:, :3])
    assert torch.equal(rs, r) and (scale[:, 3:] == 7).all()
    assert (qbuf[:, off + K:].float() == 0).all() and (qbuf[:, :off].float() == 0).all()
    # the same as the contiguous call
    q2, s2 = mb.add_rmsnorm_fp8(x, r.clone(), w, 1e-6)
    assert torch.equal(q2.float(), q.float()) and torch.equal(s2, scale[:, :3])


def test_norm_in_place_of_x():
    x, r = rand(4, 512, seed=1).to(BF), rand(4, 512, seed=2).to(BF)
    w = rand(512, seed=3, scale=0.1).to(BF)
    want = check_norm(x, r, w, residual_out=torch.empty_like(x))
    xx = x.clone()
    got = mb.add_rmsnorm_fp8(xx, r, w, 1e-6, residual_out=xx)
    assert torch.equal(got[0].float(), want[0].float()) and torch.equal(xx, (x.float() + r.float()).to(BF))


def test_norm_zeros_and_not_finite():
    x = torch.zeros(4, 384, dtype=BF, device=DEV)
    r = torch.zeros_like(x)
    x[1, 5] = float("nan")
    x[2, 130] = float("inf")
    x[3] = rand(384, seed=4).to(BF)
    w = torch.zeros(384, dtype=BF, device=DEV)
    q, s = mb.add_rmsnorm_fp8(x, r, w, 1e-6)
    assert (q[0].float() == 0).all() and (s[0] == 2.0 ** -126).all()
    assert s[1].isnan().all() and q[1].float().isnan().all()     # the statistic is NaN: so is the row
    assert s[2, 1].isnan() and q[2, 130].float().isnan()         # inf * 0
    assert q[3].float().isfinite().all() and s[3].isfinite().all()


@pytest.mark.parametrize("N,K", [(1, 1), (128, 128), (129, 130), (300, 1000), (56, 264)])
def test_quantise_weight(N, K):
    w = rand(N, K, seed=N).to(BF)
    w[: N // 2, : K // 2] *= 1e-3
    q, s = mb.quantize_weight_fp8(w)
    rq, rs = R.quantise_blocks(w.double())
    assert ((s.double() - rs.double()).abs() <= 2.0 ** -22 * rs.double()).all()
    ws = R.spread_blocks(s, N, K)
    d = (q.double() * ws - w.double()).abs()
    assert (d <= (R.EPS_E4M3 + 2.0 ** -20) * w.double().abs() + R.STEP_E4M3 * ws).all()
    z, zs = mb.quantize_weight_fp8(torch.zeros_like(w))
    assert (z.float() == 0).all() and (zs == 2.0 ** -126).all()


def check_matmul(a, sa, w, sw, **kw):
    A, W = wide_rows(a, sa), wide_blocks(w, sw)
    out = mb.matmul_fp8(a, sa, w, sw, **kw)
    K = a.shape[1]
    R.assert_bf16(out, A @ W.T, R.acc(K + 4 * R.blocks(K)) * (A.abs() @ W.abs().T), "matmul")
    assert mb.read_device_error() == 0
    return out


def check_glu(a, sa, g, sg, u, su, quant, **kw):
    A, G, U = wide_rows(a, sa), wide_blocks(g, sg), wide_blocks(u, su)
    K = a.shape[1]
    e = R.acc(K + 4 * R.blocks(K)) * A.abs()
    v, err = R.glu_out(A @ G.T, A @ U.T, e @ G.abs().T, e @ U.abs().T)
    got = mb.glu_fp8(a, sa, g, sg, u, su, out_dtype=F8 if quant else BF, **kw)
    if quant:
        R.assert_e4m3(*got, v, err, "glu")
    else:
        R.assert_bf16(got, v, err, "glu")
    assert mb.read_device_error() == 0
    return got


ROWS = [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 64, 65, 128, 129, 256, 257, 300]


@pytest.mark.parametrize("M", ROWS)
def test_matmul_rows(M):
    check_matmul(*activations(M, 272, seed=M), *weight(200, 272, seed=1))


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("quant", [False, True])
def test_glu_rows(M, quant):
    check_glu(*activations(M, 272, seed=M), *weight(200, 272, seed=1), *weight(200, 272, seed=2), quant)


# several tiles of tokens: every width of the few-row kernel's tile, ranges of the inner
# dimension, a last tile of one row
@pytest.mark.parametrize("M,N,K", [(33, 300, 2048), (97, 300, 2048), (129, 1000, 4096), (161, 4096, 1040), (200, 2560, 4096),
                                   (241, 2560, 2048), (333, 2560, 9728), (385, 1000, 4096), (512, 520, 2048), (769, 1000, 1040),
                                   (410, 520, 2656), (193, 4096, 2512), (374, 4096, 1616), (369, 2560, 4112), (208, 200, 4064)])
def test_tiles_of_tokens(M, N, K):
    a, g = activations(M, K, seed=K), weight(N, K, seed=N)
    check_matmul(*a, *g)
    assert mb.last_variant() == 16


@pytest.mark.parametrize("M,N,K", [(33, 300, 4096), (97, 1000, 2560), (160, 1000, 2064), (65, 2300, 1040), (333, 300, 4096),
                                   (513, 300, 4096), (769, 200, 2048), (49, 4100, 272),
                                   (479, 1000, 3248), (68, 11008, 2048), (274, 300, 2304)])
@pytest.mark.parametrize("quant", [False, True])
def test_gated_tiles_of_tokens(M, N, K, quant):
    a, g, u = activations(M, K, seed=K), weight(N, K, seed=N), weight(N, K, seed=N + 1)
    check_glu(*a, *g, *u, quant)
    assert mb.last_variant() == 16


@pytest.mark.parametrize("M,N,K", [(777, 2056, 128), (1100, 1501, 272), (1537, 1000, 400), (2100, 520, 16), (257, 9000, 144),
                                   (500, 2560, 8192), (1025, 2301, 8208)])
def test_pairs(M, N, K):
    check_matmul(*activations(M, K, seed=K), *weight(N, K, seed=N))
    assert mb.last_variant() == 15


@pytest.mark.parametrize("M,N,K", [(1100, 257, 400), (1500, 130, 128), (777, 392, 272), (513, 1000, 16), (300, 2100, 1040),
                                   (256, 9000, 144), (4097, 1, 272)])
@pytest.mark.parametrize("quant", [False, True])
def test_gated_pairs(M, N, K, quant):
    check_glu(*activations(M, K, seed=K), *weight(N, K, seed=N), *weight(N, K, seed=N + 1), quant)
    assert mb.last_variant() == 15


@pytest.mark.parametrize("M", [3, 20, 70])
@pytest.mark.parametrize("N,K", [(1, 16), (8, 1), (15, 128), (16, 144), (127, 256), (128, 130), (129, 384), (640, 48), (257, 1040),
                                 (72, 4112), (1100, 112)])
def test_columns_and_inner_dimension(M, N, K):
    a, g, u = activations(M, K, seed=K), weight(N, K, seed=N), weight(N, K, seed=N + 1)
    check_matmul(*a, *g)
    check_glu(*a, *g, *u, True)
    check_glu(*a, *g, *u, False)


@pytest.mark.parametrize("M", [4, 40, 150, 12300])
@pytest.mark.parametrize("pad,off", [(16, 0), (16, 16), (1, 0), (5, 3)])
def test_operand_strides(M, pad, off):
    K, N = 288, 136
    (a, sa), (g, sg), (u, su) = activations(M, K), weight(N, K, seed=1), weight(N, K, seed=2)
    a, g, u = (strided(t.view(torch.uint8), pad, off).view(F8) for t in (a, g, u))
    sa, sg, su = (strided(t, 2, 1) for t in (sa, sg, su))
    check_matmul(a, sa, g, sg)
    check_glu(a, sa, g, sg, u, su, True)


@pytest.mark.parametrize("M", [5, 40, 150, 12300])
@pytest.mark.parametrize("pad", [0, 1, 8, 24])
def test_what_lies_behind_the_outputs(M, pad):
    K, N = 160, 200
    a, g, u = activations(M, K), weight(N, K, seed=1), weight(N, K, seed=2)
    whole = torch.full((M + 1, N + pad), 7.0, dtype=BF, device=DEV)
    check_matmul(*a, *g, out=whole[:M, :N])
    assert (whole[M] == 7).all() and (whole[:, N:] == 7).all()
    q = torch.full((M + 1, N + pad), 2.0, device=DEV).to(F8)
    s = torch.full((M + 1, 2 + pad), 7.0, device=DEV)
    check_glu(*a, *g, *u, True, out=q[:M, :N], out_scale=s[:M, :2])
    assert (q[M].float() == 2).all() and (q[:, N:].float() == 2).all()
    assert (s[M] == 7).all() and (s[:, 2:] == 7).all()


@pytest.mark.parametrize("M", [1, 40])
def test_empty_and_zero(M):
    K, N = 256, 136
    (a, sa), (w, sw) = activations(M, K), weight(N, K)
    assert mb.matmul_fp8(a[:0], sa[:0], w, sw).shape == (0, N)
    assert mb.matmul_fp8(a, sa, w[:0], sw[:0]).shape == (M, 0)
    assert (mb.matmul_fp8(a[:, :0], sa[:, :0], w[:, :0], sw[:, :0]) == 0).all()
    q, s = mb.glu_fp8(a[:, :0], sa[:, :0], w[:, :0], sw[:, :0], w[:, :0], sw[:, :0], out_dtype=F8)
    assert (q.float() == 0).all() and (s == 2.0 ** -126).all()
    z = torch.zeros_like(a)
    q, s = mb.glu_fp8(z, sa, w, sw, w, sw, out_dtype=F8)
    assert (q.float() == 0).all() and (s == 2.0 ** -126).all()


@pytest.mark.parametrize("M", [3, 40, 150, 4100])
def test_scales_of_many_sizes_and_nan(M):
    """Scales over 60 binades, one infinite activation group, one NaN weight value."""
    K, N = 400, 264
    (a, sa), (w, sw) = activations(M, K), weight(N, K)
    gen = torch.Generator(device=DEV).manual_seed(5)
    sa = sa * torch.exp2(torch.randint(-30, 30, sa.shape, generator=gen, device=DEV).float())
    sw = sw * torch.exp2(torch.randint(-30, 30, sw.shape, generator=gen, device=DEV).float())
    base = check_matmul(a, sa, w, sw)
    w2 = w.clone()
    w2.view(torch.uint8)[130, 3] = 0x7F   # NaN
    out = mb.matmul_fp8(a, sa, w2, sw)
    cols = [i for i in range(N) if i != 130]
    assert out[:, 130].isnan().all() and torch.equal(out[:, cols], base[:, cols])
    sa2 = sa.clone()
    sa2[1, 2] = float("nan")
    out = mb.matmul_fp8(a, sa2, w, sw)
    assert out[1].isnan().all() and torch.equal(out[0], base[0]) and torch.equal(out[2:], base[2:])


@pytest.mark.parametrize("M", [1, 8, 48, 130, 4100])
def test_decode_chain(M):
    """norm -> gate and up -> down, as a decode step runs them, each against its
    definition on the operands that the one before gave; then the chain once more
    under a graph."""
    H, N = 384, 520
    x, r = rand(M, H, seed=1).to(BF), rand(M, H, seed=2).to(BF)
    nw = rand(H, seed=3, scale=0.1).to(BF)
    ws = [mb.quantize_weight_fp8((rand(*s, seed=i) * s[1] ** -0.5).to(BF)) for i, s in enumerate(((N, H), (N, H), (H, N)))]
    ro = torch.empty_like(r)
    q, s = check_norm(x, r, nw, residual_out=ro)
    q2, s2 = check_glu(q, s, *ws[0], *ws[1], True)
    y = check_matmul(q2, s2, *ws[2])

    def chain():
        q, s = mb.add_rmsnorm_fp8(x, r, nw, 1e-6, residual_out=ro)
        return mb.matmul_fp8(*mb.glu_fp8(q, s, *ws[0], *ws[1], out_dtype=F8), *ws[2])

    for _ in range(5):   # back to back, nothing waits between
        got = chain()
    assert torch.equal(got, y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = chain()
    for _ in range(2):
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, y)


def test_two_streams_with_their_own_workspaces():
    M, N, K = SPLIT
    assert mb.matmul_fp8_workspace_bytes(*SPLIT) > 0
    ops = [(*activations(M, K, seed=i), *weight(N, K, seed=i)) for i in (1, 2)]
    want = [mb.matmul_fp8(*o) for o in ops]
    streams = [torch.cuda.Stream() for _ in ops]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got = [mb.matmul_fp8(*o, stream=s) for o, s in zip(ops, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_rows_do_not_depend_on_their_place():
    for M in (16, 48, 300):
        a, sa = activations(M, 512, seed=3)
        w, u = weight(264, 512, seed=4), weight(264, 512, seed=5)
        perm = torch.randperm(M, generator=torch.Generator().manual_seed(0)).to(DEV)
        pa = a.view(torch.uint8)[perm].view(F8)
        assert torch.equal(mb.matmul_fp8(pa, sa[perm], *w), mb.matmul_fp8(a, sa, *w)[perm])
        x, y = mb.glu_fp8(pa, sa[perm], *w, *u, out_dtype=F8), mb.glu_fp8(a, sa, *w, *u, out_dtype=F8)
        assert torch.equal(x[0].float(), y[0].float()[perm]) and torch.equal(x[1], y[1][perm])


def test_weight_quantised_right_before_its_use():
    """The next call's kernel may copy its weight before its predecessor is waited for."""
    a, sa = activations(4, 2048)
    w = [(rand(2048, 2048, seed=i) * 2048 ** -0.5).to(BF) for i in range(6)]
    q, s = (torch.empty(2048, 2048, device=DEV).to(F8), torch.empty(16, 16, device=DEV))
    want = [mb.matmul_fp8(a, sa, *mb.quantize_weight_fp8(x)) for x in w]
    for _ in range(3):
        got = []
        for x in w:
            mb.quantize_weight_fp8(x, q=q, scale=s)
            got.append(mb.matmul_fp8(a, sa, q, s))
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_given_outputs_workspace_and_stream():
    M, N, K = SPLIT
    a, w, u = activations(M, K), weight(N, K, seed=1), weight(N, K, seed=2)
    want, (wq, ws) = mb.matmul_fp8(*a, *w), mb.glu_fp8(*a, *w, *u, out_dtype=F8)
    need = mb.matmul_fp8_workspace_bytes(M, N, K)
    assert need > 0
    out = torch.zeros(M, N, dtype=BF, device=DEV)
    q, s = torch.zeros(M, N, device=DEV).to(F8), torch.zeros(M, N // 128, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws1 = torch.empty(need, dtype=torch.uint8, device=DEV)
    assert mb.matmul_fp8(*a, *w, out=out, workspace=ws1, stream=side) is out
    r = mb.glu_fp8(*a, *w, *u, out=q, out_scale=s, out_dtype=F8, stream=side)
    side.synchronize()
    assert r[0] is q and r[1] is s
    assert torch.equal(out, want) and torch.equal(q.float(), wq.float()) and torch.equal(s, ws)
    with pytest.raises(mb.MbgluError):
        mb.matmul_fp8(*a, *w, workspace=ws1[: need - 256])
    with pytest.raises(ValueError):
        mb.glu_fp8(*a, *w, *u, out_scale=s)
    with pytest.raises((TypeError, ValueError)):
        mb.glu_fp8(*a, *w, *u, out=out, out_dtype=F8)
    with pytest.raises((TypeError, ValueError)):
        mb.matmul_fp8(a[0], a[1][:, :1], *w)
    with pytest.raises((TypeError, ValueError)):
        mb.add_rmsnorm_fp8(out, out, torch.zeros(N - 1, dtype=BF, device=DEV), 1e-6)


def test_launch_policies_agree():
    old = mb.get_launch_policy()
    ops = [(activations(m, 1024, seed=m), weight(400, 1024, seed=1), weight(400, 1024, seed=2)) for m in (3, 70, 200, 4100)]
    try:
        got = []
        for policy in (mb.POLICY_SERIAL, mb.POLICY_PDL, mb.POLICY_PREFETCH):
            mb.set_launch_policy(policy)
            got.append([(mb.matmul_fp8(*a, *w), *mb.glu_fp8(*a, *w, *u, out_dtype=F8)) for a, w, u in ops])
        for other in got[1:]:
            for x, y in zip(got[0], other):
                assert all(torch.equal(i.float(), j.float()) for i, j in zip(x, y))
    finally:
        mb.set_launch_policy(old)


def test_captured_calls_of_two_graphs_share_nothing():
    """Two graphs with calls that need workspaces, replayed at the same time."""
    M, N, K = SPLIT
    ops = [(*activations(M, K, seed=i), *weight(N, K, seed=i)) for i in (1, 2)]
    want = [mb.matmul_fp8(*o) for o in ops]
    graphs, outs = [], []
    for o in ops:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(mb.matmul_fp8(*o))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in ops]
    for _ in range(5):
        for x in outs:
            x.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, want))


@pytest.mark.parametrize("M", [1, 40, 150, 4100])
def test_buffers_used_again_by_the_next_step(M):
    """Steps back to back through the same q and scale buffers, each on other values:
    every kernel sees what the one before it wrote, not what an earlier one did."""
    H, N = 512, 640
    ws = [mb.quantize_weight_fp8((rand(*s, seed=i) * s[1] ** -0.5).to(BF)) for i, s in enumerate(((N, H), (N, H), (H, N)))]
    nw = rand(H, seed=3, scale=0.1).to(BF)
    xs = [rand(M, H, seed=10 + i, scale=4.0 ** (i - 3)).to(BF) for i in range(6)]
    r = rand(M, H, seed=9).to(BF)

    def step(x, bufs):
        q, s, q2, s2, ro, y = bufs
        mb.add_rmsnorm_fp8(x, r, nw, 1e-6, q=q, scale=s, residual_out=ro)
        mb.glu_fp8(q, s, *ws[0], *ws[1], out=q2, out_scale=s2, out_dtype=F8)
        return mb.matmul_fp8(q2, s2, *ws[2], out=y)

    def buffers():
        e = lambda *s: torch.empty(*s, device=DEV)   # noqa: E731
        return (e(M, H).to(F8), e(M, 4), e(M, N).to(F8), e(M, 5), e(M, H).to(BF), e(M, H).to(BF))

    want = []
    for x in xs:
        want.append(step(x, buffers()).clone())
        torch.cuda.synchronize()
    one = buffers()
    for _ in range(3):
        ys = [torch.empty(M, H, dtype=BF, device=DEV) for _ in xs]
        for x, y in zip(xs, ys):
            step(x, (*one[:5], y))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ys, want))
    # and within one graph
    ys = [torch.empty(M, H, dtype=BF, device=DEV) for _ in xs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for x, y in zip(xs, ys):
            step(x, (*one[:5], y))
    for _ in range(3):
        for y in ys:
            y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ys, want))


@pytest.mark.parametrize("K", [128, 130, 1000, 2567])
def test_one_row_needs_no_stride(K):
    """A single row has no row stride to be a multiple of anything."""
    pad = -K % 16
    a, sa = activations(1, K, seed=K)
    (g, sg), (u, su) = weight(200, K, seed=1), weight(200, K, seed=2)
    g, u = (strided(t.view(torch.uint8), pad).view(F8) for t in (g, u))
    check_matmul(a, sa, g, sg)
    assert mb.last_variant() == 16
    check_glu(a, sa, g, sg, u, su, True)
    assert mb.last_variant() == 16
    check_glu(a.expand(1, K), sa, g, sg, u, su, False)


def far(t, odd=0):
    """t's values in rows so far apart that the last lies beyond 2^31 elements."""
    step = (2 ** 31 // (t.shape[0] - 1) + 64) // 64 * 64 + odd
    raw = t.view(torch.uint8) if t.dtype == F8 else t
    v = torch.empty((t.shape[0] - 1) * step + t.shape[1], dtype=raw.dtype, device=DEV).as_strided(t.shape, (step, 1))
    assert (t.shape[0] - 1) * step > 2 ** 31 - 64
    return v.copy_(raw).view(t.dtype)


@pytest.mark.parametrize("M,N,K,odd", [(33, 300, 272, 0), (150, 136, 400, 0), (2100, 1000, 272, 0), (40, 72, 136, 1)])
def test_offsets_beyond_32_bits(M, N, K, odd):
    (a, sa), (g, sg), (u, su) = activations(M, K), weight(N, K, seed=1), weight(N, K, seed=2)
    a, sa, g, u = (far(t, odd) for t in (a, sa, g, u))
    check_matmul(a, sa, g, sg, out=far(torch.zeros(M, N, dtype=BF, device=DEV), odd))
    q, s = far(torch.zeros(M, N, device=DEV).to(F8), odd), far(torch.zeros(M, -(-N // 128), device=DEV), odd)
    check_glu(a, sa, g, sg, u, su, True, out=q, out_scale=s)
    check_glu(a, sa, g, sg, u, su, False, out=far(torch.zeros(M, N, dtype=BF, device=DEV), odd))
    x, r = far(rand(M, K, seed=3).to(BF), odd), far(rand(M, K, seed=4).to(BF), odd)
    q, s = far(torch.zeros(M, K, device=DEV).to(F8), odd), far(torch.zeros(M, -(-K // 128), device=DEV), odd)
    check_norm(x, r, rand(K, seed=5, scale=0.1).to(BF), q=q, scale=s, residual_out=far(torch.zeros(M, K, dtype=BF, device=DEV), odd))
    wq, ws = mb.quantize_weight_fp8(far(rand(N, K, seed=6).to(BF), odd), q=far(torch.zeros(N, K, device=DEV).to(F8), odd))
    rq, rs = mb.quantize_weight_fp8(rand(N, K, seed=6).to(BF))
    assert torch.equal(wq.float(), rq.float()) and torch.equal(ws, rs)
