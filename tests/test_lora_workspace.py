"""Workspaces of glu_lora and linear_lora: one that is made for the most rows serves fewer,
and one that holds p and no partial sums is taken too."""
import ctypes

import pytest
import torch

import dense_ref as R
import memory_bound_glu_gb300 as mb
import rows_ref as Q
from memory_bound_glu_gb300.binding import _Adapters

SIZES = {1: mb.linear_lora_workspace_bytes, 2: mb.glu_lora_workspace_bytes}


def least(sides, M, r):
    """The bytes that the header promises to be enough."""
    return 8 * sides * r * M + M // 8 + 2048


@pytest.mark.parametrize("sides", [1, 2])
@pytest.mark.parametrize("N,K,r", [(9728, 2560, 16), (2560, 9728, 16), (2504, 1000, 24), (300, 264, 128), (30000, 520, 32), (1, 8, 8)])
def test_more_rows_need_no_less(N, K, r, sides):
    sizes = [SIZES[sides](M, N, K, 30, r) for M in (*range(1, 700), *range(700, 20000, 97))]
    assert sizes == sorted(sizes)
    assert all(s >= least(sides, M, r) - 2048 for M, s in enumerate(sizes[:699], 1))


@pytest.mark.parametrize("sides", [1, 2])
@pytest.mark.parametrize("r", [8, 64])
def test_many_rows_need_room_for_p_alone(r, sides):
    """Partial sums of p are for as many blocks as there are SMs, whatever the rows: 30000 more
    rows need no more than their own p, its terms and entries of the table."""
    few, many = (SIZES[sides](M, 2560, 2560, 30, r) for M in (30000, 60000))
    assert many - few <= least(sides, 30000, r)


def test_less_than_p_is_refused():
    """Pointers are never dereferenced: the calls end in the host's checks."""
    x, w, u, a, b, i, o, ws = (0x7F0000000000 + j * (1 << 36) for j in range(8))
    q = _Adapters(a, 8 * 64, 64, b, 32 * 8, 8)
    for M in (1, 20, 1000):
        args = (M, 32, 64, 3, 8)
        assert mb.lib().linear_lora(x, 64, w, 64, ctypes.byref(q), i, None, o, 32, *args, ws, 8 * 8 * M - 1, None) == 2
        assert mb.lib().glu_lora(x, 64, w, 64, u, 64, ctypes.byref(q), ctypes.byref(q), i, None, o, 32, *args, 0, ws, 16 * 8 * M - 1, None) == 2


gpu = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def rand(*shape, seed=0, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(BF)


def operands(M, N, K, r, L, sides, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = [rand(N, K, seed=seed + 1 + i, scale=K ** -0.5) for i in range(sides)]
    ab = []
    for i in range(sides):
        ab += [rand(L, r, K, seed=seed + 5 + i, scale=K ** -0.5), rand(L, N, r, seed=seed + 9 + i, scale=r ** -0.5)]
    return rand(M, K, seed=seed), w, ab, torch.randint(-1, L, (M,), generator=g, device=DEV).int(), torch.rand(L, generator=g, device=DEV) + 0.5


def check(x, w, ab, idx, scale, **kw):
    if len(w) == 2:
        Q.assert_glu_lora(mb.glu_lora(x, *w, *ab, idx, scale, **kw), (x, *w, *ab, idx, scale))
    else:
        R.assert_bf16(mb.linear_lora(x, *w, *ab, idx, scale, **kw), *Q.adapted(x, *w, *ab, idx, scale))
    assert mb.last_variant() == 19


# products that are cut along the inner dimension where there is room, and whole ones; p beside
# the products, from either kernel of its own, and formed by each block
@gpu
@pytest.mark.parametrize("M,N,K,r,sides", [(1, 264, 520, 16, 1), (8, 2560, 9728, 16, 1), (48, 9728, 2560, 16, 2), (50, 2500, 520, 64, 2), (64, 300, 4104, 128, 1),
                                           (160, 1300, 4104, 32, 2), (333, 2504, 1000, 24, 2), (600, 520, 2056, 40, 1), (1100, 1300, 2056, 64, 2)])
def test_a_small_workspace(M, N, K, r, sides):
    """From what the header promises to be enough up to all; nothing behind the given bytes is written."""
    args = operands(M, N, K, r, 20, sides, M)
    small, large = least(sides, M, r), SIZES[sides](M, N, K, 20, r)
    for size in (small, (3 * small + large) // 4, (small + large) // 2, large - 1, large):
        buffer = torch.full((size + 4096,), 170, dtype=torch.uint8, device=DEV)
        check(*args, workspace=buffer[:size])
        assert (buffer[size:] == 170).all()
    assert mb.read_device_error() == 0


@gpu
@pytest.mark.parametrize("N,K,r,sides", [(2560, 2056, 16, 1), (1304, 1032, 16, 2), (520, 1032, 64, 2)])
def test_one_workspace_for_all_rows(N, K, r, sides):
    """A buffer that a server made for its largest batch."""
    x, w, ab, idx, scale = operands(700, N, K, r, 20, sides, N)
    workspace = torch.empty(SIZES[sides](700, N, K, 20, r), dtype=torch.uint8, device=DEV)
    for M in (700, 1, 8, 255, 33, 512, 64, 320, 2, 130):
        check(x[:M], w, ab, idx[:M], scale, workspace=workspace)
    assert mb.read_device_error() == 0


@gpu
def test_a_small_workspace_in_a_graph():
    x, w, ab, idx, scale = operands(48, 2560, 1032, 16, 20, 2, 1)
    workspace = torch.empty(least(2, 48, 16), dtype=torch.uint8, device=DEV)
    out = mb.glu_lora(x, *w, *ab, idx, scale, workspace=workspace)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        mb.glu_lora(x, *w, *ab, idx, scale, out=out, workspace=workspace)
    for i in range(3):
        x.copy_(rand(48, 1032, seed=50 + i))
        workspace.fill_(255)
        graph.replay()
        Q.assert_glu_lora(out, (x, *w, *ab, idx, scale))


@gpu
@pytest.mark.parametrize("M,N,K,r,pad", [(1, 264, 520, 16, 0), (8, 2560, 2056, 16, 0), (48, 2504, 264, 64, 0), (300, 264, 136, 24, 0), (700, 520, 264, 40, 0),
                                         (20, 136, 72, 8, 1)])
def test_the_counters_of_an_expert_layer_stay(M, N, K, r, pad):
    """One buffer for adapters' calls and an expert layer's in turn, as a decode loop has it."""
    E, k, n, T = 20, 3, 136, min(M, 64)
    x, w, ab, idx, scale = operands(M, N, K, r, 20, 2, M)
    if pad:   # odd strides: the kernels for any alignment
        x = torch.nn.functional.pad(x, (0, 1))[:, :K]
    layer = rand(E, K, seed=1, scale=K ** -0.5), rand(E, n, K, seed=2, scale=K ** -0.5), rand(E, n, K, seed=3, scale=K ** -0.5), rand(E, K, n, seed=4, scale=n ** -0.5)
    size = max(mb.glu_lora_workspace_bytes(M, N, K, 20, r), mb.linear_lora_workspace_bytes(M, N, K, 20, r), mb.moe_glu_workspace_bytes(T, E, k, n, K))
    workspace = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    counters = workspace[:mb.MOE_COUNTER_BYTES].zero_()
    for _ in range(2):
        Q.assert_glu_lora(mb.glu_lora(x, *w, *ab, idx, scale, workspace=workspace), (x, *w, *ab, idx, scale))
        assert (counters == 0).all()
        R.assert_bf16(mb.linear_lora(x, w[0], *ab[:2], idx, scale, workspace=workspace), *Q.adapted(x, w[0], *ab[:2], idx, scale))
        assert (counters == 0).all()
        Q.assert_moe(mb.moe_glu(x[:T], *layer, k, workspace=workspace), x[:T], *layer, k, True)
        assert (counters == 0).all()
    assert mb.read_device_error() == 0
