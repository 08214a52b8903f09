"""glu_lora and linear_lora against the definitions in 64 bits: sizes around the
tiles' edges, ranks, rows with and without adapters in any order, strides and
alignments, isolation of rows, streams, workspaces and graphs."""
import pytest
import torch

import dense_ref as R
import memory_bound_glu_gb300 as mb
import rows_ref as Q

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
FAST, SLOW = 19, 20


def rand(*shape, seed=0, scale=1.0, pad=0, off=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    t = (torch.randn(*shape[:-1], shape[-1] + pad + off, generator=g, device=DEV) * scale).to(BF)
    return t[..., off:off + shape[-1]]


def indices(M, L, seed, how="mixed"):
    """The rows' adapters: runs of one, every row its own, or mixed; some with none."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    if how == "runs":
        a = torch.arange(M, device=DEV) * 3 // max(M, 1) % max(L, 1)
    elif how == "own":
        a = torch.arange(M, device=DEV) % max(L, 1)
    else:
        a = torch.randint(-1, L, (M,), generator=g, device=DEV)
    return a.int()


def operands(M, N, K, r, L, seed=0, how="mixed", sides=2, pad=0, off=0):
    """(h, weights, adapters, indices, scales), in glu_lora's or linear_lora's order."""
    x = rand(M, K, seed=seed, pad=pad, off=off)
    w = [rand(N, K, seed=seed + 1 + i, scale=K ** -0.5, pad=pad, off=off) for i in range(sides)]
    ab = []
    for i in range(sides):
        ab += [rand(L, r, K, seed=seed + 5 + i, scale=K ** -0.5, pad=pad, off=off),
               rand(L, N, r, seed=seed + 9 + i, scale=(r or 1) ** -0.5, pad=pad, off=off)]
    scale = torch.rand(L, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV) * 2 - 0.5
    return (x, *w, *ab, indices(M, L, seed, how), scale)


def check(M, N, K, r, L, variant=None, mode="fused", sides=2, **kw):
    args = operands(M, N, K, r, L, sides=sides, **kw)
    if sides == 2:
        out = mb.glu_lora(*args, mode=mode)
        Q.assert_glu_lora(out, args, mode)
    else:
        out = mb.linear_lora(*args)
        R.assert_bf16(out, *Q.adapted(*args), "out")
    assert variant is None or mb.last_variant() == variant
    assert mb.read_device_error() == 0
    return args, out


@pytest.mark.parametrize("sides", [1, 2])
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 127, 129, 257, 300])
def test_rows(M, sides):
    check(M, 200, 136, 16, 5, seed=M, sides=sides)


@pytest.mark.parametrize("sides", [1, 2])
@pytest.mark.parametrize("N", [1, 2, 31, 33, 64, 127, 129, 255, 257, 1000])
def test_columns(N, sides):
    check(50, N, 72, 8, 3, seed=N, sides=sides)
    check(100, N, 72, 8, 3, seed=N, sides=sides, mode="hf")


@pytest.mark.parametrize("K", [1, 7, 8, 63, 64, 65, 128, 500, 2568])
def test_inner_dimension(K):
    check(20, 136, K, 16, 3, seed=K)
    check(90, 136, K, 16, 3, seed=K)
    check(20, 136, K, 16, 3, seed=K, sides=1)


@pytest.mark.parametrize("r", [1, 3, 8, 16, 24, 40, 64, 72, 128])
@pytest.mark.parametrize("M", [5, 100])
def test_ranks(r, M):
    check(M, 144, 96, r, 4, seed=r)
    check(M, 144, 96, r, 4, seed=r, sides=1)


@pytest.mark.parametrize("how", ["runs", "own", "mixed"])
@pytest.mark.parametrize("M,L", [(1, 1), (13, 64), (64, 64), (64, 1), (150, 200), (500, 2)])
def test_adapters_over_the_rows(M, L, how):
    check(M, 300, 264, 16, L, seed=M + L, how=how)
    check(M, 300, 264, 16, L, seed=M + L, how=how, sides=1)


# whole rounds of tiles, ranges of the inner dimension, several rows' tiles, ragged in every dimension
@pytest.mark.parametrize("M,N,K,r,sides", [(1, 2560, 9728, 16, 1), (8, 2560, 9728, 16, 1), (40, 1000, 4104, 24, 1), (8, 9728, 2560, 16, 2),
                                           (48, 9730, 1032, 16, 2), (333, 2504, 1000, 24, 2), (700, 2560, 2056, 32, 1),
                                           (479, 520, 2048, 64, 2), (2100, 1300, 264, 16, 2), (1500, 2561, 520, 40, 1)])
def test_each_plan(M, N, K, r, sides):
    check(M, N, K, r, 9, seed=M, sides=sides, variant=FAST, how="runs")
    check(M, N, K, r, 9, seed=M + 1, sides=sides, mode="hf")


@pytest.mark.parametrize("pad,off", [(1, 0), (3, 1), (8, 0), (8, 8), (5, 3)])
def test_strides(pad, off):
    """Views into wider buffers; odd ones take the kernels for any alignment."""
    variant = FAST if pad % 8 == 0 and off % 8 == 0 else SLOW
    for sides in (1, 2):
        check(40, 130, 136, 16, 3, seed=pad, pad=pad, off=off, variant=variant, sides=sides)


def test_output_and_adapter_strides():
    h, gw, uw, ga, gb, ua, ub, idx, scale = operands(70, 200, 136, 16, 4, seed=3)
    big = torch.full((70, 333), 7.0, dtype=BF, device=DEV)
    # adapters that lie interleaved in one buffer
    both = torch.stack([ga, ua], 1)
    args = (h, gw, uw, both[:, 0], gb, both[:, 1], ub, idx, scale)
    mb.glu_lora(*args, out=big[:, 9:209])
    Q.assert_glu_lora(big[:, 9:209], args)
    assert (big[:, :9] == 7).all() and (big[:, 209:] == 7).all()


def test_no_scale_no_adapter():
    h, gw, uw, ga, gb, ua, ub, idx, scale = operands(33, 200, 136, 16, 4, seed=4)
    args = (h, gw, uw, ga, gb, ua, ub, idx, None)
    Q.assert_glu_lora(mb.glu_lora(*args), args)
    none = torch.full_like(idx, -1)
    args = (h, gw, uw, ga, gb, ua, ub, none, scale)
    Q.assert_glu_lora(mb.glu_lora(*args), args)
    for r, L in ((0, 4), (16, 0)):
        args = (h, gw, uw, ga[:L, :r], gb[:L, :, :r], ua[:L, :r], ub[:L, :, :r], idx if L else none, scale[:L])
        Q.assert_glu_lora(mb.glu_lora(*args), args)


@pytest.mark.parametrize("M", [20, 200])
def test_indices_out_of_range_are_none(M):
    h, w, a, b, idx, scale = operands(M, 100, 72, 8, 3, seed=5, sides=1)
    wild = idx.clone()
    wild[::4] = torch.tensor([3, 2 ** 31 - 1, -2 ** 31, -7], dtype=torch.int32, device=DEV).repeat(M)[:wild[::4].numel()]
    R.assert_bf16(mb.linear_lora(h, w, a, b, wild, scale), *Q.adapted(h, w, a, b, wild, scale))


@pytest.mark.parametrize("M", [24, 200])
@pytest.mark.parametrize("sides", [1, 2])
def test_a_broken_adapter_reaches_its_own_rows_only(M, sides):
    args = list(operands(M, 200, 136, 16, 5, seed=M, sides=sides))
    call = mb.glu_lora if sides == 2 else mb.linear_lora
    before = call(*args)
    broken = args[-2] == 2
    assert broken.any() and not broken.all()
    for i in range(1 + sides, len(args) - 2):
        args[i] = args[i].clone()
        args[i][2] = float("nan") if i % 2 else float("inf")
    after = call(*args)
    assert torch.equal(after[~broken], before[~broken])
    assert not torch.isfinite(after[broken]).any()


def test_rows_with_infinities_and_nan():
    args = list(operands(40, 200, 136, 16, 4, seed=8))
    before = mb.glu_lora(*args)
    args[0] = args[0].clone()
    args[0][3, 5], args[0][17] = float("nan"), float("inf")
    after = mb.glu_lora(*args)
    keep = torch.ones(40, dtype=torch.bool, device=DEV)
    keep[[3, 17]] = False
    assert torch.equal(after[keep], before[keep]) and torch.isnan(after[3]).all()


def test_the_same_call_gives_the_same_bits():
    for M in (8, 64, 333):
        args = operands(M, 1300, 1032, 24, 30, seed=M)
        ws = torch.empty(mb.glu_lora_workspace_bytes(M, 1300, 1032, 30, 24), dtype=torch.uint8, device=DEV)
        first = mb.glu_lora(*args, workspace=ws)
        ws.fill_(255)   # what a call finds there is of no account
        assert torch.equal(first, mb.glu_lora(*args, workspace=ws))


def test_calls_on_two_streams():
    a, b = operands(64, 2504, 1000, 16, 40, seed=1), operands(300, 2504, 1000, 16, 40, seed=2)
    want = mb.glu_lora(*a), mb.glu_lora(*b)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        x, y = mb.glu_lora(*a, stream=s1), mb.glu_lora(*b, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(x, want[0]) and torch.equal(y, want[1])


@pytest.mark.parametrize("M", [4, 150])
def test_graph_replays_with_new_indices(M):
    """A captured call reads its inputs anew at each replay."""
    x, w, a, b, idx, scale = operands(M, 520, 264, 16, 7, seed=6, sides=1)
    out = torch.empty(M, 520, dtype=BF, device=DEV)
    ws = torch.empty(max(1, mb.linear_lora_workspace_bytes(M, 520, 264, 7, 16)), dtype=torch.uint8, device=DEV)
    mb.linear_lora(x, w, a, b, idx, scale, out=out, workspace=ws)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        mb.linear_lora(x, w, a, b, idx, scale, out=out, workspace=ws)
    for i in range(4):
        idx.copy_(indices(M, 7, 50 + i))
        scale.mul_(0.9)
        a.mul_(-1)
        g.replay()
        R.assert_bf16(out, *Q.adapted(x, w, a, b, idx, scale))


def test_policies_agree():
    args = operands(48, 2504, 1000, 16, 40, seed=11)
    got = []
    try:
        for p in (mb.POLICY_SERIAL, mb.POLICY_PDL, mb.POLICY_PREFETCH):
            mb.set_launch_policy(p)
            for _ in range(3):
                out = mb.glu_lora(*args)
            got.append(out)
    finally:
        mb.set_launch_policy(mb.POLICY_PREFETCH)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_offsets_beyond_32_bits():
    """Adapters whose elements lie beyond 2^31 of the first."""
    L, r, N, K = 70, 128, 8, 1 << 18
    x, w = rand(3, K, seed=1), rand(N, K, seed=2, scale=K ** -0.5)
    a = torch.zeros(L, r, K, dtype=BF, device=DEV)
    a[69] = rand(r, K, seed=3, scale=K ** -0.5)
    b = rand(L, N, r, seed=4, scale=r ** -0.5)
    idx = torch.tensor([69, -1, 69], dtype=torch.int32, device=DEV)
    y, e = Q.adapted(x, w, a[69:], b[69:], idx - 69, None)
    R.assert_bf16(mb.linear_lora(x, w, a, b, idx), y, e)


@pytest.mark.parametrize("sides", [1, 2])
@pytest.mark.parametrize("r", [8, 24, 32, 56, 64, 120, 128])
@pytest.mark.parametrize("M,N,K", [(2, 300, 264), (16, 700, 1032), (50, 2500, 520)])
def test_a_decode_batch_of_each_rank(M, N, K, r, sides):
    check(M, N, K, r, 64, seed=M + r, how="own", sides=sides, variant=FAST)


# p beside the products and in a kernel of its own: both sides of the bounds on rows, rank and columns
@pytest.mark.parametrize("sides", [1, 2])
@pytest.mark.parametrize("M,N,K,r", [(3, 300, 520, 16), (24, 520, 1032, 16), (64, 2500, 2056, 8), (64, 300, 4104, 128), (65, 2500, 2056, 8),
                                     (66, 700, 4104, 72), (100, 1000, 2568, 40), (160, 1300, 4104, 32), (161, 1300, 4104, 32),
                                     (256, 2504, 1544, 8), (257, 264, 5128, 16), (320, 1300, 4104, 16), (321, 1300, 4104, 16)])
@pytest.mark.parametrize("how", ["own", "mixed"])
def test_a_large_decode_batch(M, N, K, r, sides, how):
    check(M, N, K, r, 48, seed=M + r, how=how, sides=sides, variant=FAST)


# tiles of 128 rows with one adapter, some and many; the inner dimension whole and in up to eight ranges
@pytest.mark.parametrize("sides", [1, 2])
@pytest.mark.parametrize("M,K,r,L,how", [(512, 72, 8, 3, "runs"), (600, 520, 128, 4, "runs"), (640, 1032, 40, 200, "mixed"),
                                         (1100, 2056, 64, 7, "runs"), (1100, 264, 24, 5, "mixed")])
def test_many_rows(M, K, r, L, how, sides):
    check(M, 264, K, r, L, seed=M, how=how, sides=sides, variant=FAST)


@pytest.mark.parametrize("M", [40, 100, 700])
def test_one_adapter_for_all_but_some_rows(M):
    """Runs of 32 rows of one adapter, and beside them blocks with single rows of another or of none."""
    for lone in (0, 31, 32, M - 1):
        args = list(operands(M, 264, 136, 24, 4, seed=M))
        args[-2] = torch.full((M,), 2, dtype=torch.int32, device=DEV)
        args[-2][lone] = 3 if lone % 2 else -1
        Q.assert_glu_lora(mb.glu_lora(*args), args)


def test_shared_memory_of_adapters():
    """One adapter under every index: a stride of zero between adapters."""
    x, w, a, b, idx, scale = operands(70, 200, 136, 16, 1, seed=3, sides=1)
    a, b = a.expand(5, -1, -1), b.expand(5, -1, -1)
    idx = indices(70, 5, 4)
    scale = scale.expand(5).contiguous()
    for M in (9, 70):
        R.assert_bf16(mb.linear_lora(x[:M], w, a, b, idx[:M], scale), *Q.adapted(x[:M], w, a, b, idx[:M], scale))
