"""moe_glu where the activation is finite in fp32 and beyond bf16's largest number."""
import pytest
import torch

import memory_bound_glu_gb300 as mb

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.mark.parametrize("pad", [0, 1])   # the one kernel, and those for any alignment
@pytest.mark.parametrize("T,E,k,N,K", [(1, 4, 2, 72, 136), (9, 6, 3, 72, 136), (64, 12, 4, 776, 264)])
def test_activation_beyond_bf16(T, E, k, N, K, pad):
    def z(*shape):
        return torch.zeros(*shape[:-1], shape[-1] + pad, dtype=BF, device=DEV)[..., :shape[-1]]

    h, router, gate, up, down = z(T, K), z(E, K), z(E, N, K), z(E, N, K), z(E, K, N)
    router[:, 2] = torch.randn(E, device=DEV).to(BF)
    h[:, 2] = torch.randn(T, device=DEV).to(BF)
    h[:, :2] = 2.0 ** 32
    gate[:, :, 0] = 2.0 ** 32                       # g = 2^64, whose SiLU is itself
    up[:, :, 0], up[:, :, 1] = 2.0 ** 32, -2.0 ** 22   # u = 2^64 (1 - 2^-10): g u = 2^128 (1 - 2^-10)
    down[:, :, N // 2] = 2.0 ** -120
    out, ids, weights = mb.moe_glu(h, router, gate, up, down, k)
    assert mb.last_variant() == (21 if pad == 0 else 22)
    # 256 (1 - 2^-10), which bf16 rounds to 256; the weights' sum is off by less than 2^-16
    assert (out == 256).all()
