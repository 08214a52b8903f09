"""Weights that the kernel right before a call writes: under every launch policy the
call multiplies with the new ones, its early weight copies included."""
import pytest
import torch

import memory_bound_glu_gb300 as mb

pytestmark = pytest.mark.gpu
DEV = "cuda"


def bf16_weights(N, K):
    return [(torch.randn(N, K, device=DEV) / K ** 0.5).bfloat16() for _ in range(2)]


@pytest.fixture(params=[mb.POLICY_SERIAL, mb.POLICY_PDL, mb.POLICY_PREFETCH])
def policy(request):
    old = mb.get_launch_policy()
    mb.set_launch_policy(request.param)
    yield
    mb.set_launch_policy(old)


@pytest.mark.parametrize("op,M,N,K", [("matmul_fp8", 1, 256, 1024), ("matmul_fp8", 8, 2560, 9728), ("matmul_fp8", 300, 1000, 4096),
                                      ("glu_fp8", 1, 9728, 2560), ("glu_fp8", 40, 1000, 2560), ("glu_gemv", 1, 9728, 2560),
                                      ("glu_gemv", 8, 1000, 2560), ("glu_gemv", 40, 2560, 2560), ("glu_gemm", 40, 2560, 2560),
                                      ("glu_gemm", 333, 1000, 1000)])
def test_new_weights_are_used(policy, op, M, N, K):
    torch.manual_seed(0)
    if op.endswith("fp8"):
        (g, gs), (u, us) = (mb.quantize_weight_fp8(w) for w in bf16_weights(N, K))
        other = [mb.quantize_weight_fp8(w)[0] for w in bf16_weights(N, K)]
        a, sa = torch.randn(M, K, device=DEV).to(mb.E4M3), torch.rand(M, -(-K // 128), device=DEV)
        words = torch.uint8
        call = (lambda: mb.matmul_fp8(a, sa, g, gs)) if op == "matmul_fp8" else (lambda: mb.glu_fp8(a, sa, g, gs, u, us))
    else:
        (g, u), other = bf16_weights(N, K), bf16_weights(N, K)
        h = torch.randn(M, K, device=DEV).bfloat16()
        words = torch.int16
        call = lambda: getattr(mb, op)(h, g, u)  # noqa: E731
    now = [w.view(words) for w in (g, u)]
    flip = [w ^ o.view(words) for w, o in zip(now, other)]

    def turn():   # to the other weights and back
        for w, f in zip(now, flip):
            w.bitwise_xor_(f)

    want = []
    for _ in range(2):
        want.append(call())
        torch.cuda.synchronize()
        turn()
        torch.cuda.synchronize()
    assert not torch.equal(*want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = []
        for _ in range(6):
            captured.append(call())
            turn()
    for _ in range(10):
        eager = []
        for _ in range(6):
            eager.append(call())
            turn()
        graph.replay()
        for got in (eager, captured):
            assert all(torch.equal(x, want[i & 1]) for i, x in enumerate(got))
