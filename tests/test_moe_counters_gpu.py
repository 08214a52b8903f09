"""moe_glu on a workspace whose counters are not zero, as a call leaves them whose wait gave
up: it reports an error, reads and writes nothing out of bounds and ends, and the workspace
serves again once its counters are zeroed."""
import pytest
import torch

import memory_bound_glu_gb300 as mb
import rows_ref as Q

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
TIMEOUT = 8


def rand(*shape, seed=0, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(BF)


def operands(T, E, N, K):
    return (rand(T, K, seed=1), rand(E, K, seed=2, scale=K ** -0.5), rand(E, N, K, seed=3, scale=K ** -0.5),
            rand(E, N, K, seed=4, scale=K ** -0.5), rand(E, K, N, seed=5, scale=N ** -0.5))


# each block chooses for all tokens, and blocks choose for tokens of their own
@pytest.mark.parametrize("T,E", [(1, 20), (4, 20), (40, 20), (64, 100)])
def test_counters_that_are_not_zero(T, E):
    args, k = operands(T, E, 136, 264), 3
    ws = mb.new_moe_workspace(T, E, k, 136, 264)
    Q.assert_moe(mb.moe_glu(*args, k, workspace=ws), *args, k, True)
    counters = ws[:mb.MOE_COUNTER_BYTES].view(torch.int32)
    for value in (1000, 0x3f800000, -2 ** 31):   # more arrivals than blocks, a float's bits, what a failed call leaves
        counters.fill_(value)
        for _ in range(2):
            mb.moe_glu(*args, k, workspace=ws)
            assert mb.read_device_error() == TIMEOUT
            assert (counters[:6] != 0).all()
        counters.zero_()
        Q.assert_moe(mb.moe_glu(*args, k, workspace=ws), *args, k, True)
        assert mb.read_device_error() == 0 and (counters == 0).all()


@pytest.mark.parametrize("T,E", [(40, 20), (64, 100)])
def test_the_choices_counter(T, E):
    """The barrier between the blocks' choices, by itself; the workspace holds no indices there."""
    args, k = operands(T, E, 136, 264), 3
    ws = mb.new_moe_workspace(T, E, k, 136, 264)
    for rest in (0, 255, 127):
        ws[mb.MOE_COUNTER_BYTES:] = rest
        counters = ws[:mb.MOE_COUNTER_BYTES].view(torch.int32)
        counters.zero_()
        counters[5] = 1000
        mb.moe_glu(*args, k, workspace=ws)
        assert mb.read_device_error() == TIMEOUT
        counters.zero_()
        Q.assert_moe(mb.moe_glu(*args, k, workspace=ws), *args, k, True)


def test_other_calls_are_not_affected():
    """A failed call on one workspace, then calls on another and on none."""
    args = operands(8, 20, 136, 264)
    bad, good = (mb.new_moe_workspace(8, 20, 3, 136, 264) for _ in range(2))
    bad[:4] = 255
    bad[3] = 1   # 0x01ffffff arrivals
    mb.moe_glu(*args, 3, workspace=bad)
    assert mb.read_device_error() == TIMEOUT
    Q.assert_moe(mb.moe_glu(*args, 3, workspace=good), *args, 3, True)
    Q.assert_moe(mb.moe_glu(*args, 3), *args, 3, True)
    assert mb.read_device_error() == 0


# several pieces of a tile per block, and one tile per block; each barrier by itself: after the gated
# products, after the activation (the first of them only), after the down products, and the exit
@pytest.mark.parametrize("T,E,k,N,K,counter", [(40, 20, 3, 136, 264, 1), (40, 20, 3, 136, 264, 2), (40, 20, 3, 136, 264, 3), (40, 20, 3, 136, 264, 4),
                                               (1, 16, 8, 768, 520, 1), (1, 16, 8, 768, 520, 3), (1, 16, 8, 768, 520, 4)])
def test_each_counter(T, E, k, N, K, counter):
    """All roles of all blocks leave together."""
    args = operands(T, E, N, K)
    ws = mb.new_moe_workspace(T, E, k, N, K)
    counters = ws[:mb.MOE_COUNTER_BYTES].view(torch.int32)
    counters[counter] = 1000
    mb.moe_glu(*args, k, workspace=ws)
    assert mb.read_device_error() == TIMEOUT
    counters.zero_()
    Q.assert_moe(mb.moe_glu(*args, k, workspace=ws), *args, k, True)
    assert mb.read_device_error() == 0 and (counters == 0).all()
