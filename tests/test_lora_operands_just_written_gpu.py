"""Operands of glu_lora and linear_lora that the kernel right before a call writes: under every
launch policy the call uses the new ones, with p in a kernel of its own, beside the products and
formed by each block, and back to back with other calls on the same workspace."""
import pytest
import torch

import memory_bound_glu_gb300 as mb

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def rand(*shape, seed=0, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(BF)


@pytest.fixture(params=[mb.POLICY_SERIAL, mb.POLICY_PDL, mb.POLICY_PREFETCH])
def policy(request):
    old = mb.get_launch_policy()
    mb.set_launch_policy(request.param)
    yield
    mb.set_launch_policy(old)


@pytest.mark.parametrize("M,N,K,r,sides,small", [(1, 9728, 2560, 16, 2, False), (8, 2560, 9728, 16, 1, False), (8, 2560, 9728, 16, 1, True),
                                                 (48, 9728, 2560, 16, 2, False), (48, 9728, 2560, 16, 2, True), (200, 2504, 1000, 24, 2, False),
                                                 (700, 1304, 1032, 40, 2, False), (700, 1304, 1032, 40, 1, True)])
def test_new_operands_are_used(policy, M, N, K, r, sides, small):
    L = 12
    x, idx = rand(M, K, seed=1), (torch.arange(M, device=DEV) * L // max(M, L)).int()
    w = [rand(N, K, seed=2 + i, scale=K ** -0.5) for i in range(sides)]
    ab = [t for i in range(sides) for t in (rand(L, r, K, seed=5 + i, scale=K ** -0.5), rand(L, N, r, seed=8 + i, scale=r ** -0.5))]
    size = (mb.glu_lora_workspace_bytes if sides == 2 else mb.linear_lora_workspace_bytes)(M, N, K, L, r)
    ws = torch.empty(8 * sides * r * M + M // 8 + 2048 if small else size, dtype=torch.uint8, device=DEV)

    def call():
        return mb.glu_lora(x, *w, *ab, idx, workspace=ws) if sides == 2 else mb.linear_lora(x, *w, *ab, idx, workspace=ws)

    # each operand to other values and back by exclusive or, one kernel each; the last one written differs
    words = [t.view(torch.int16) for t in (x, *w, *ab)] + [idx]
    flips = [v ^ rand(*t.shape, seed=20 + i, scale=K ** -0.5).view(torch.int16) for i, (v, t) in enumerate(zip(words, (x, *w, *ab)))]
    flips.append(idx ^ (L - 1 - idx))
    for last in range(len(words)):
        order = [i for i in range(len(words)) if i != last] + [last]

        def turn():
            for i in order:
                words[i].bitwise_xor_(flips[i])

        want = []
        for _ in range(2):
            want.append(call())
            torch.cuda.synchronize()
            turn()
            torch.cuda.synchronize()
        assert not torch.equal(*want)
        got = []
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(4):
                got.append((call(), call()))   # twice: the second right behind the first
                turn()
        for _ in range(2):
            graph.replay()
            torch.cuda.synchronize()
            for i, pair in enumerate(got):
                assert all(torch.equal(g, want[i % 2]) for g in pair)
    assert mb.read_device_error() == 0
