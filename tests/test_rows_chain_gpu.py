"""A decode step's feed-forward blocks in a row, as a server runs them: the norm, gated
projections and down projection with adapters, and an expert layer on what comes out;
eagerly, in a CUDA graph with new tokens and adapters, and beside the framework's own
calls."""
import pytest
import torch

import dense_ref as R
import memory_bound_glu_gb300 as mb
import rows_ref as Q

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def rand(*shape, seed=0, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(BF)


class Layer:
    def __init__(self, K=264, N=520, r=16, L=6, E=20, n=136, seed=0):
        self.r, self.L, self.k = r, L, 4
        self.gate, self.up = (rand(N, K, seed=seed + i, scale=K ** -0.5) for i in range(2))
        self.down = rand(K, N, seed=seed + 2, scale=N ** -0.5)
        self.ab = [rand(L, r, K, seed=seed + 3, scale=K ** -0.5), rand(L, N, r, seed=seed + 4, scale=r ** -0.5),
                   rand(L, r, K, seed=seed + 5, scale=K ** -0.5), rand(L, N, r, seed=seed + 6, scale=r ** -0.5)]
        self.ab_down = [rand(L, r, N, seed=seed + 7, scale=N ** -0.5), rand(L, K, r, seed=seed + 8, scale=r ** -0.5)]
        self.scale = torch.rand(L, device=DEV) + 0.5
        self.router = rand(E, K, seed=seed + 9, scale=K ** -0.5)
        self.experts = [rand(E, n, K, seed=seed + 10, scale=K ** -0.5), rand(E, n, K, seed=seed + 11, scale=K ** -0.5),
                        rand(E, K, n, seed=seed + 12, scale=n ** -0.5)]
        self.ws = mb.new_moe_workspace(64, E, min(E, self.k), n, K)

    def step(self, x, adapter):
        act = mb.glu_lora(x, self.gate, self.up, *self.ab, adapter, self.scale)
        y = mb.linear_lora(act, self.down, *self.ab_down, adapter, self.scale)
        return act, y, mb.moe_glu(y, self.router, *self.experts, self.k, workspace=self.ws)

    def check(self, got, x, adapter):
        act, y, moe = got
        Q.assert_glu_lora(act, (x, self.gate, self.up, *self.ab, adapter, self.scale))
        R.assert_bf16(y, *Q.adapted(act, self.down, *self.ab_down, adapter, self.scale), "down")
        Q.assert_moe(moe, y, self.router, *self.experts, self.k, True)


def tokens(M, L, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return rand(M, 264, seed=seed), torch.randint(-1, L, (M,), generator=g, device=DEV).int()


@pytest.mark.parametrize("M", [1, 7, 64])
def test_step(M):
    layer = Layer(seed=M)
    for i in range(3):   # several steps back to back, checked afterwards
        x, adapter = tokens(M, layer.L, M + i)
        got = [layer.step(x, adapter) for _ in range(4)]
        layer.check(got[-1], x, adapter)
        assert all(torch.equal(a, b) for a, b in zip(got[0][:2], got[-1][:2])) and torch.equal(got[0][2][0], got[-1][2][0])
    assert mb.read_device_error() == 0


@pytest.mark.parametrize("M", [1, 20])
def test_step_in_a_graph(M):
    layer = Layer(seed=M)
    x, adapter = tokens(M, layer.L, 1)
    layer.step(x, adapter)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = layer.step(x, adapter)
        again = layer.step(x, adapter)
    for i in range(3):
        a, b = tokens(M, layer.L, 10 + i)
        x.copy_(a)
        adapter.copy_(b)
        graph.replay()
        layer.check(got, x, adapter)
        assert torch.equal(got[2][0], again[2][0])


def test_beside_the_frameworks_calls():
    """glu_lora without adapters is glu_gemm to one rounding, and an expert layer of one
    expert glu_gemv and the down projection; what ran before and after keeps its results."""
    layer = Layer(E=1, n=520)
    layer.k = 1
    x, adapter = tokens(40, layer.L, 3)
    plain = mb.glu_gemm(x, layer.gate, layer.up)
    none = torch.full_like(adapter, -1)
    out = mb.glu_lora(x, layer.gate, layer.up, *layer.ab, none, layer.scale)
    # sums in another order: 2 acc(K) of the products' magnitudes, then a rounding each
    g, u, eg, eu = R.glu(x.double(), layer.gate.double(), layer.up.double())
    v, e = R.glu_out(g, u, eg, eu)
    assert ((out.double() - plain.double()).abs() <= 2 * (e + R.EPS_BF16 * (v.abs() + e))).all()
    w, ids, weights = mb.moe_glu(x, layer.router, *layer.experts, 1, workspace=layer.ws)
    assert (ids == 0).all() and (weights == 1).all()
    Q.assert_moe((w, ids, weights), x, layer.router, *layer.experts, 1, True)
    assert torch.equal(mb.glu_gemm(x, layer.gate, layer.up), plain)
