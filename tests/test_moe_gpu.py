"""moe_glu against its definition in 64 bits: tokens, experts and top-k, sizes around
the tiles' edges, ties, unused experts, NaN and infinities, strides, workspaces used
again, streams and graphs."""
import pytest
import torch

import memory_bound_glu_gb300 as mb
import rows_ref as Q

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
FAST, SLOW = 21, 22


def rand(*shape, seed=0, scale=1.0, pad=0, off=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    t = (torch.randn(*shape[:-1], shape[-1] + pad + off, generator=g, device=DEV) * scale).to(BF)
    return t[..., off:off + shape[-1]]


def operands(T, E, N, K, seed=0, pad=0, off=0):
    kw = dict(pad=pad, off=off)
    return (rand(T, K, seed=seed, **kw), rand(E, K, seed=seed + 1, scale=K ** -0.5, **kw), rand(E, N, K, seed=seed + 2, scale=K ** -0.5, **kw),
            rand(E, N, K, seed=seed + 3, scale=K ** -0.5, **kw), rand(E, K, N, seed=seed + 4, scale=N ** -0.5, **kw))


def check(T, E, k, N, K, renormalize=True, variant=None, seed=0, **kw):
    args = operands(T, E, N, K, seed=seed, **kw)
    got = mb.moe_glu(*args, k, renormalize=renormalize)
    Q.assert_moe(got, *args, k, renormalize)
    assert variant is None or mb.last_variant() == variant
    assert mb.read_device_error() == 0
    return args, got


@pytest.mark.parametrize("T", [1, 2, 3, 8, 15, 16, 17, 31, 33, 48, 63, 64])
def test_tokens(T):
    check(T, 16, 4, 136, 200, seed=T)


@pytest.mark.parametrize("E,k", [(1, 1), (2, 1), (3, 3), (31, 2), (32, 8), (33, 5), (64, 16), (100, 7), (256, 8), (512, 10), (512, 16)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_experts(E, k, renormalize):
    check(5, E, k, 72, 136, renormalize, seed=E)
    check(40, E, k, 72, 136, renormalize, seed=E)


@pytest.mark.parametrize("N", [8, 16, 56, 64, 72, 120, 128, 136, 200, 776])
def test_inner_size(N):
    check(6, 9, 3, N, 264, seed=N, variant=FAST)
    check(33, 9, 3, N, 264, seed=N, variant=FAST)


@pytest.mark.parametrize("K", [8, 64, 72, 120, 128, 136, 1000, 2056])
def test_hidden_size(K):
    check(6, 9, 3, 136, K, seed=K, variant=FAST)
    check(33, 9, 3, 136, K, seed=K, variant=FAST)


@pytest.mark.parametrize("N,K", [(1, 1), (7, 33), (65, 130), (100, 77), (8, 63)])
def test_odd_sizes(N, K):
    check(5, 6, 2, N, K, seed=N, variant=SLOW)


# several pieces of a tile per block and several tiles per block
@pytest.mark.parametrize("T,E,k,N,K", [(1, 128, 8, 768, 2048), (4, 4, 2, 2752, 2048), (64, 40, 8, 520, 1032), (1, 2, 1, 11008, 4096), (64, 3, 2, 1000, 2056)])
def test_each_plan(T, E, k, N, K):
    check(T, E, k, N, K, seed=T, variant=FAST)


@pytest.mark.parametrize("pad,off", [(1, 0), (3, 1), (8, 0), (8, 8), (5, 3)])
def test_strides(pad, off):
    check(9, 7, 3, 136, 200, seed=pad, pad=pad, off=off, variant=FAST if pad % 8 == 0 and off % 8 == 0 else SLOW)


def test_gate_and_up_in_one_tensor():
    h, r, g, u, d = operands(12, 6, 136, 200, seed=7)
    both = torch.cat([g, u], 1)
    out = torch.full((12, 230), 7.0, dtype=BF, device=DEV)
    got = mb.moe_glu(h, r, both[:, :136], both[:, 136:], d, 3, out=out[:, 8:208])
    Q.assert_moe(got, h, r, g, u, d, 3, True)
    assert (out[:, :8] == 7).all() and (out[:, 208:] == 7).all()


@pytest.mark.parametrize("pad", [0, 1])
def test_ties_go_to_the_lowest_index(pad):
    h, r, g, u, d = operands(10, 40, 72, 136, seed=9, pad=pad)
    r[1::2] = r[0::2]   # every logit twice
    r[20:] = r[:20]     # and then four times
    h[4] = 0            # all equal, and of either sign of zero
    got = mb.moe_glu(h, r, g, u, d, 6)
    Q.assert_moe(got, h, r, g, u, d, 6, True)
    assert got[1][4].tolist() == [0, 1, 2, 3, 4, 5]


@pytest.mark.parametrize("T", [3, 50])
def test_every_token_one_expert_and_none_for_others(T):
    h, r, g, u, d = operands(T, 12, 136, 264, seed=10)
    h = h.abs()
    r[7] = 1.0
    r[3] = 0.5
    got = mb.moe_glu(h, r, g, u, d, 2)
    assert (got[1] == torch.tensor([7, 3], dtype=torch.int32, device=DEV)).all()
    Q.assert_moe(got, h, r, g, u, d, 2, True)


@pytest.mark.parametrize("pad", [0, 1])
def test_a_broken_token_reaches_itself_only(pad):
    args = list(operands(20, 12, 136, 264, seed=11, pad=pad))
    before = mb.moe_glu(*args, 3)
    args[0] = args[0].clone() if pad == 0 else args[0]
    args[0][4, 9], args[0][13] = float("nan"), float("inf")
    after = mb.moe_glu(*args, 3)
    keep = [i for i in range(20) if i not in (4, 13)]
    assert torch.equal(after[1][keep], before[1][keep]) and torch.equal(after[2][keep], before[2][keep])
    want = before[0][keep].double()
    # other experts may be read, which moves the borders between a sum's parts: two roundings
    assert ((after[0][keep].double() - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -12 * want.abs().max()).all()
    assert torch.isnan(after[2][4]).all() and torch.isnan(after[0][4]).all() and torch.isnan(after[0][13]).all()
    assert ((after[1] >= 0) & (after[1] < 12)).all()


@pytest.mark.parametrize("pad", [0, 1])
def test_a_broken_expert_reaches_its_own_tokens_only(pad):
    args = list(operands(30, 12, 136, 264, seed=12, pad=pad))
    before = mb.moe_glu(*args, 3)
    hit = (before[1] == 5).any(1)
    assert hit.any() and not hit.all()
    args[2][5], args[4][5] = float("nan"), float("inf")
    after = mb.moe_glu(*args, 3)
    assert torch.equal(after[0][~hit], before[0][~hit]) and not torch.isfinite(after[0][hit]).any()


def test_infinite_logits():
    h, r, g, u, d = operands(4, 8, 72, 136, seed=13)
    h = h.abs()
    r[2] = float("-inf")
    r[6] = float("-inf")
    got = mb.moe_glu(h, r, g, u, d, 7)
    keep = [0, 1, 3, 4, 5, 7]
    assert (got[1][:, 6] == 2).all() and (got[2][:, 6] == 0).all()
    want = mb.moe_glu(h, r[keep].contiguous(), g[keep].contiguous(), u[keep].contiguous(), d[keep].contiguous(), 6)
    assert torch.allclose(got[2][:, :6], want[2], rtol=1e-5, atol=0)


@pytest.mark.parametrize("pad", [0, 1])
def test_empty_sums(pad):
    h, r, g, u, d = operands(5, 6, 72, 136, seed=14, pad=pad)
    out, ids, w = mb.moe_glu(h, r, g[:, :0], u[:, :0], d[:, :, :0], 2)
    assert (out == 0).all() and torch.equal(ids.long(), Q.route(h, r, 2, True)[0])
    out, ids, w = mb.moe_glu(h[:0], r, g, u, d, 2)
    assert out.shape == (0, 136) and ids.shape == (0, 2)


def test_a_workspace_serves_many_calls():
    """One workspace for calls of several sizes in turn; its counters end at zero."""
    ws = mb.new_moe_workspace(64, 16, 4, 776, 1032)
    for i, (T, N, K) in enumerate([(64, 776, 1032), (1, 136, 200), (17, 776, 72), (64, 64, 1032), (2, 776, 1032)] * 2):
        args = operands(T, 16, N, K, seed=i)
        Q.assert_moe(mb.moe_glu(*args, 4, workspace=ws), *args, 4, True)
        assert (ws[:mb.MOE_COUNTER_BYTES] == 0).all()
        ws[mb.MOE_COUNTER_BYTES:] = 255


def test_the_same_call_gives_the_same_bits():
    for T in (1, 20, 64):
        args = operands(T, 30, 520, 1032, seed=T)
        ws = mb.new_moe_workspace(T, 30, 6, 520, 1032)
        first = mb.moe_glu(*args, 6, workspace=ws)
        for _ in range(5):
            again = mb.moe_glu(*args, 6, workspace=ws)
            assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_calls_on_two_streams():
    """Each stream with a workspace of its own."""
    a, b = operands(8, 30, 520, 1032, seed=1), operands(64, 30, 264, 1032, seed=2)
    wa, wb = mb.new_moe_workspace(8, 30, 4, 520, 1032), mb.new_moe_workspace(64, 30, 4, 264, 1032)
    want = mb.moe_glu(*a, 4), mb.moe_glu(*b, 4)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        x, y = mb.moe_glu(*a, 4, workspace=wa, stream=s1), mb.moe_glu(*b, 4, workspace=wb, stream=s2)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip((*x, *y), (*want[0], *want[1])))
    assert mb.read_device_error() == 0


@pytest.mark.parametrize("T,pad", [(1, 0), (40, 0), (6, 1)])
def test_graph_replays_with_new_tokens(T, pad):
    """A captured call routes anew at each replay."""
    h, r, g, u, d = operands(T, 20, 136, 264, seed=T, pad=pad)
    ws = mb.new_moe_workspace(T, 20, 4, 136, 264)
    out, ids, w = mb.moe_glu(h, r, g, u, d, 4, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        mb.moe_glu(h, r, g, u, d, 4, out=out, ids=ids, weights=w, workspace=ws)
        mb.moe_glu(h, r, g, u, d, 4, out=out, ids=ids, weights=w, workspace=ws)
    for i in range(4):
        h.copy_(rand(T, 264, seed=100 + i))
        graph.replay()
        Q.assert_moe((out, ids, w), h, r, g, u, d, 4, True)


def test_policies_agree():
    args = operands(9, 20, 136, 264, seed=15)
    got = []
    try:
        for p in (mb.POLICY_SERIAL, mb.POLICY_PDL, mb.POLICY_PREFETCH):
            mb.set_launch_policy(p)
            got.append(mb.moe_glu(*args, 4)[0])
    finally:
        mb.set_launch_policy(mb.POLICY_PREFETCH)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_offsets_beyond_32_bits():
    """Experts whose weights lie beyond 2^31 elements of the first."""
    E, N, K = 270, 2056, 4104
    h = rand(2, K, seed=1).abs()
    r = rand(E, K, seed=2, scale=K ** -0.5)
    r[269], r[1] = 1.0, 0.5
    g, u = (torch.zeros(E, N, K, dtype=BF, device=DEV) for _ in range(2))
    d = torch.zeros(E, K, N, dtype=BF, device=DEV)
    for i in (1, 269):
        g[i], u[i], d[i] = rand(N, K, seed=i, scale=K ** -0.5), rand(N, K, seed=i + 1, scale=K ** -0.5), rand(K, N, seed=i + 2, scale=N ** -0.5)
    got = mb.moe_glu(h, r, g, u, d, 2)
    assert got[1].tolist() == [[269, 1]] * 2
    Q.assert_moe(got, h, r, g, u, d, 2, True)


# as many tiles as half to all of the SMs: one per block, one token to 64
@pytest.mark.parametrize("T,E,k,N,K", [(1, 16, 8, 768, 520), (2, 4, 4, 1600, 264), (17, 4, 4, 1608, 264), (40, 4, 4, 2056, 136), (64, 2, 2, 4872, 72)])
def test_one_tile_per_block(T, E, k, N, K):
    check(T, E, k, N, K, seed=T, variant=FAST)


@pytest.mark.parametrize("T,E", [(1, 509), (1, 512), (2, 256), (2, 257), (4, 128), (5, 128), (16, 32), (64, 8), (64, 9), (64, 512)])
def test_who_chooses(T, E):
    """Around the number of logits up to which each block chooses for all tokens."""
    check(T, E, min(E, 5), 72, 136, renormalize=False, seed=T + E, variant=FAST)
